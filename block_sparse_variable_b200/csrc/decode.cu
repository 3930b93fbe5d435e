// decode.cu -- attention of a few query tokens per sequence over a cache.
//
// Math: out = softmax(scale Q K^T + mask) V and its log-sum-exp, in one pass
// over the keys with a running maximum and sum; the mask is none, causal
// (aligned to the end of the cache) or the ancestor bits of a draft tree.
//
// What bounds it: every key and value is read once for the few rows of a kv
// head's group, so memory does.  A block is four warps; each takes 16 of a
// chunk's 64 tokens through its own ring of cp.async stages and its own
// running maximum, so that nothing in the loop waits for another warp; the
// four states are joined at the end of a segment.  Products are 16 x 8 x 16
// warp matrix instructions: 16 query rows are the tile.
#include <cuda_runtime.h>

#include "cache.h"
#include "cp_async.cuh"
#include "decode_plan.cuh"
#include "launch.cuh"
#include "pack16.cuh"

namespace bsa {
namespace {

constexpr int kThreads = 128, kWarps = 4;
constexpr int kChunk = 64;   // tokens of a step, 16 a warp
constexpr int kTile = 16;    // query rows of a tile
constexpr int kStages = 3;
// Query rows of a kv head's group, in the mean, up to which this kernel is
// taken; above, the tensor core kernel with 128-row tiles.  (16 sequences of
// 2048 to 16384 tokens, 8 kv heads: 16 rows 113 us here; 20 rows, two tiles,
// 202 here and 121 there; 32 rows 206 and 120.  One sequence of 16384 tokens,
// 20 rows: 37 and 35; of 1500 tokens: 18.6 and 19.4.)  The mean decides for a
// mixed batch too: 128 sequences of 4096 tokens, 4 heads a group, 12 rows in the
// mean, 127 of them with a single token and one with 256: 409 us here, 368 there;
// one with 64: 334 and 347; all with one: 318 and 327.
constexpr int kFewRows = 16;

template <int D>
struct Smem {
  static constexpr int kRow = D * 2;                      // bytes of a token row
  static constexpr int kHalf = 16 * kRow;                 // K or V of a warp's 16 tokens
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kRing = kStages * kStage;          // of one warp
  static constexpr int kMl = kWarps * kRing;              // [warps][rows][2] floats
  static constexpr int kBlk = kMl + kWarps * kTile * 8;   // [warps][32] ids
  static constexpr int kU = kBlk + kWarps * 64;           // [warps][stages] first token of a stage
  static constexpr int kBytes = kU + kWarps * kStages * 4;
  static_assert(kWarps * kTile * D * 4 <= kWarps * kRing, "the states are joined in the ring's memory");
};

__device__ __forceinline__ void ldm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// columns [4 c, 4 c + 4) of one output row, and its lse: row x of the head
// group's rows from token t0 on; o unnormalised, m in log2 units
template <typename T>
__device__ __forceinline__ void write_row(const DecodeProblem &p, int64_t tok0, int b, int hh, int t0, int x, int c,
                                          float4 o, float m, float l) {
  const int y = div_gg(p, x), t = t0 + y, h = hh * p.gg + x - y * p.gg;
  const bool some = l > 0.f || l != l;
  const float inv = some ? 1.f / l : 0.f;
  uint2 w;
  w.x = Pack2<T>::pack(o.x * inv, o.y * inv);
  w.y = Pack2<T>::pack(o.z * inv, o.w * inv);
  T *dst = static_cast<T *>(p.out) + b * p.o_sb + (tok0 + t) * p.o_st + int64_t(h) * p.o_sh;
  reinterpret_cast<uint2 *>(dst)[c] = w;
  if (c == 0 && p.lse)
    p.lse[b * p.l_sb + (tok0 + t) * p.l_st + int64_t(h) * p.l_sh] =
        some ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// mask of one (row, kv token) pair of the last qlen tokens
template <int kMask>  // 0 none, 1 causal, 2 tree
__device__ __forceinline__ bool seen(const DecodeProblem &p, const int64_t *bits, int t, int node) {
  if constexpr (kMask == 1) return node <= t;
  if constexpr (kMask == 2) {
    if (node < 0) return true;
    if ((node >> 6) >= p.tree_words) return false;
    return (bits[node >> 6] >> (node & 63)) & 1;
  }
  return true;
}

template <int D, typename T, int kMask>
__global__ void __launch_bounds__(kThreads, D == 128 ? 2 : 4) k_decode(const DecodeProblem p) {
  using S = Smem<D>;
  constexpr int kLanes = D / 8;            // 16-byte pieces of a row
  constexpr int kPer = 16 * kLanes / 32;   // cp.async a lane for 16 rows
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_wait();
  griddep_launch_next();
  uint32_t flags = 0;
  __shared__ DecScratch<kThreads> scratch;
  const DecStart st = dec_start<kThreads>(p, scratch, flags);
  const uint32_t ring = smem_u32(smem) + uint32_t(warp * S::kRing);
  float *s_o = reinterpret_cast<float *>(smem);
  float2 *s_ml = reinterpret_cast<float2 *>(smem + S::kMl);
  uint16_t *s_blk = reinterpret_cast<uint16_t *>(smem + S::kBlk) + warp * 32;
  int *s_u = reinterpret_cast<int *>(smem + S::kU) + warp * kStages;
  DecodeJoin join{};

  DecCursor cursor = cursor_begin(st), here;
  DecBatch d;
  DecSeg seg;
  while (cursor_next(p, st, cursor, d, seg, here)) {
    const int b = here.b, hh = seg.hh, tile = seg.tile, cs = seg.cs, ce = seg.ce;
    const int h2 = hh / (p.H / p.N2);
    const DecRows v = dec_rows(p, d, tile);
    const int qbase = d.kv.kvlen - d.q.qlen;  // kv token of draft node 0

    // ---- the first stages, then Q while they fly
    DecWalk w = walk_begin(p, b, hh, v.irow, here.qoff);
    int cu, cpg, nu = -1, npg = 0;
    walk_fetch(p, d, b, w, cs & ~31, ce, s_blk, lane, cu, cpg);
    const int sub = lane / kLanes, col = lane % kLanes;
    auto issue = [&](int x) {
      if (x < ce) {
        if ((x & 31) == 0 && x != (cs & ~31)) { cu = nu; cpg = npg; }
        const int u0 = __shfl_sync(0xffffffffu, cu, x & 31), pg = __shfl_sync(0xffffffffu, cpg, x & 31);
        const int s = x % kStages;
        if (lane == 0) s_u[s] = u0;
        if (u0 >= 0) {
          const int u = u0 + 16 * warp, left = d.kv.kvlen - u;
          const T *k = static_cast<const T *>(p.k) + kv_off(p.kv, p.k_sb, p.k_sh, p.k_st, d.kv, b, h2, u, pg);
          const T *vv = static_cast<const T *>(p.v) + kv_off(p.kv, p.v_sb, p.v_sh, p.v_st, d.kv, b, h2, u, pg);
          const uint32_t at = ring + uint32_t(s * S::kStage);
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int r = sub + i * (32 / kLanes);
            const bool in = r < left;
            const uint32_t dst = at + uint32_t(r * S::kRow + ((col ^ (r & 7)) << 4));
            cp_async16(dst, in ? k + int64_t(r) * p.k_st + col * 8 : static_cast<const T *>(p.k), in);
            cp_async16(dst + S::kHalf, in ? vv + int64_t(r) * p.v_st + col * 8 : static_cast<const T *>(p.v), in);
          }
        }
        if ((x & 31) == 16 || (x == cs && (x & 31) > 16))
          walk_fetch(p, d, b, w, (x & ~31) + 32, ce, s_blk, lane, nu, npg);
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(cs + i);

    // rows lane / 4 and lane / 4 + 8 of the tile
    uint32_t qf[D / 16][4];
    int tq[2];
    const int64_t *bits[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = (lane >> 2) + 8 * half, x = v.first + min(r, v.rows - 1);
      const int y = div_gg(p, x), t = v.t0 + y, h = hh * p.gg + x - y * p.gg;
      const int64_t qb = p.cu_q ? 0 : b;
      const T *q = static_cast<const T *>(p.q) + qb * p.q_sb + (d.q.tok0 + t) * p.q_st + int64_t(h) * p.q_sh;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t *src = reinterpret_cast<const uint32_t *>(q + ks * 16) + (lane & 3);
        qf[ks][half] = __ldg(src);
        qf[ks][half + 2] = __ldg(src + 4);
      }
      tq[half] = t;
      bits[half] = kMask == 2 ? p.tree + qb * p.t_sb + (d.q.tok0 + t) * p.t_st : nullptr;
    }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int x = cs; x < ce; ++x) {
      cp_wait<kStages - 2>();
      __syncwarp();
      issue(x + kStages - 1);
      const int s = x % kStages;
      const int u0 = s_u[s];
      const int u = u0 + 16 * warp;
      if (u0 < 0 || u >= d.kv.kvlen) continue;  // the whole warp
      const uint32_t kS = ring + uint32_t(s * S::kStage), vS = kS + S::kHalf;
      float sc[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[i][j] = 0.f;
      {
        const int r = (lane & 7) + ((lane >> 4) << 3);  // kv row of this lane's address
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t kf[4];
          ldm4(kS + uint32_t(r * S::kRow + (((2 * ks + ((lane >> 3) & 1)) ^ (r & 7)) << 4)), kf);
          mma16<T>(sc[0], qf[ks], kf[0], kf[1]);
          mma16<T>(sc[1], qf[ks], kf[2], kf[3]);
        }
      }
      const bool edge = u + 16 > d.kv.kvlen || (kMask != 0 && u + 16 > qbase);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sc[i][j] *= p.scale_log2;
          if (edge) {
            const int uu = u + 8 * i + 2 * (lane & 3) + (j & 1);
            if (uu >= d.kv.kvlen || !seen<kMask>(p, bits[j >> 1], tq[j >> 1], uu - qbase)) sc[i][j] = -INFINITY;
          }
        }
      uint32_t pf[4];
      float alpha[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = fmaxf(fmaxf(sc[0][2 * h], sc[0][2 * h + 1]), fmaxf(sc[1][2 * h], sc[1][2 * h + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[h], mx);
        const float ref = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: every weight is 0
        alpha[h] = ex2(m[h] - ref);
        m[h] = mn;
        const float e0 = ex2(sc[0][2 * h] - ref), e1 = ex2(sc[0][2 * h + 1] - ref);
        const float e2 = ex2(sc[1][2 * h] - ref), e3 = ex2(sc[1][2 * h + 1] - ref);
        l[h] = l[h] * alpha[h] + ((e0 + e1) + (e2 + e3));
        // the weights are rounded to the inputs' type for the product, as in
        // the forward pass; their sum is not
        pf[h] = Pack2<T>::pack(e0, e1);
        pf[h + 2] = Pack2<T>::pack(e2, e3);
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= alpha[0];
          o[i][1] *= alpha[0];
          o[i][2] *= alpha[1];
          o[i][3] *= alpha[1];
        }
      }
      {
        const int r = lane & 15;  // kv row of this lane's address
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t vf[4];
          ldm4t(vS + uint32_t(r * S::kRow + (((2 * i + (lane >> 4)) ^ (r & 7)) << 4)), vf);
          mma16<T>(o[2 * i], pf, vf[0], vf[1]);
          mma16<T>(o[2 * i + 1], pf, vf[2], vf[3]);
        }
      }
    }
    cp_wait<0>();
    flags |= w.flags;

    // ---- join the four warps' states in the ring's memory
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = (lane >> 2) + 8 * h;
      if ((lane & 3) == 0) s_ml[warp * kTile + r] = make_float2(m[h], l[h]);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2 *>(s_o + (warp * kTile + r) * D + i * 8 + 2 * (lane & 3)) =
            make_float2(o[i][2 * h], o[i][2 * h + 1]);
    }
    __syncthreads();
    const bool whole = cs == 0 && ce == d.chunks;
    const int slot = here.pos == st.lo ? 2 * int(blockIdx.x) : 2 * int(blockIdx.x) + 1;
    for (int i = tid; i < v.rows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), c = i % (D / 4);
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int ww = 0; ww < kWarps; ++ww) mm = fmaxf(mm, s_ml[ww * kTile + r].x);
      const float ref = mm == -INFINITY ? 0.f : mm;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int ww = 0; ww < kWarps; ++ww) {
        const float2 ml = s_ml[ww * kTile + r];
        const float f = ex2(ml.x - ref);
        const float4 x = *reinterpret_cast<const float4 *>(s_o + (ww * kTile + r) * D + c * 4);
        ll += ml.y * f;
        acc.x += x.x * f;
        acc.y += x.y * f;
        acc.z += x.z * f;
        acc.w += x.w * f;
      }
      if (whole) {
        write_row<T>(p, d.q.tok0, p.cu_q ? 0 : b, hh, v.t0, v.first + r, c, acc, mm, ll);
      } else {
        reinterpret_cast<float4 *>(p.part_o + (int64_t(slot) * kTile + r) * D)[c] = acc;
        if (c == 0) reinterpret_cast<float2 *>(p.part_ml)[int64_t(slot) * kTile + r] = make_float2(mm, ll);
      }
    }
    __syncthreads();
    if (cs == 0 && !whole) join = dec_join(p, st, here, d, seg, v, slot);
  }
  __shared__ uint32_t s_flags;
  if (tid == 0) s_flags = 0;
  __syncthreads();
  if (flags) atomicOr(&s_flags, flags);
  __syncthreads();
  if (tid == 0) {
    p.join[blockIdx.x] = join;
    p.flags[blockIdx.x] = s_flags;
  }
}

// the attention blocks' flags into the status word, by one block
template <int kN>
__device__ void join_flags(const DecodeProblem &p) {
  __shared__ uint32_t s_flags;
  if (threadIdx.x == 0) s_flags = 0;
  __syncthreads();
  uint32_t f = 0;
  for (int i = threadIdx.x; i < p.grid; i += kN) f |= p.flags[i];
  if (f) atomicOr(&s_flags, f);
  __syncthreads();
  if (threadIdx.x < kStWords) p.status[threadIdx.x] = threadIdx.x == kStFlags ? s_flags : 0;
}

// Joins the parts of the unit that attention block blockIdx.x began and did
// not finish.  A warp takes a row, or, where the block has more warps than
// rows, every wpr-th part of it; a part's state and output are requested
// together, four parts at a time.
template <int D, typename T, int kJoinWarps>
__global__ void __launch_bounds__(32 * kJoinWarps) k_decode_join(const DecodeProblem p) {
  __shared__ float s_o[kJoinWarps][D], s_m[kJoinWarps], s_l[kJoinWarps];
  griddep_wait();
  griddep_launch_next();
  const DecodeJoin j = p.join[blockIdx.x];
  if (blockIdx.x == 0) join_flags<32 * kJoinWarps>(p);
  const int rows = j.rows;  // at most kJoinWarps
  if (j.parts == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int wpr = 1;
  while (2 * wpr * rows <= kJoinWarps) wpr *= 2;
  const int r = warp / wpr, phase = warp % wpr;
  constexpr int kC = D / 32, kBatch = 4;
  float m = -INFINITY, l = 0.f, acc[kC];
#pragma unroll
  for (int c = 0; c < kC; ++c) acc[c] = 0.f;
  if (r < rows) {
    // part 0 in slot0, part i at the beginning of the i-th group of blocks after this one's
    for (int i0 = phase; i0 < j.parts; i0 += wpr * kBatch) {
      float2 ml[kBatch];
      float o[kBatch][kC];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * wpr;
        if (i < j.parts) {
          const int64_t at = int64_t(i == 0 ? j.slot0 : 2 * (int(blockIdx.x) + i * p.group)) * p.TR + r;
          ml[k] = reinterpret_cast<const float2 *>(p.part_ml)[at];
          const float *src = p.part_o + at * D + lane * kC;
          if constexpr (kC == 4) {
            const float4 y = *reinterpret_cast<const float4 *>(src);
            o[k][0] = y.x; o[k][1] = y.y; o[k][2] = y.z; o[k][3] = y.w;
          } else {
            const float2 y = *reinterpret_cast<const float2 *>(src);
            o[k][0] = y.x; o[k][1] = y.y;
          }
        } else {
          ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
          for (int c = 0; c < kC; ++c) o[k][c] = 0.f;
        }
      }
      float mn = m;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) mn = fmaxf(mn, ml[k].x);
      const float ref = mn == -INFINITY ? 0.f : mn, f0 = ex2(m - ref);
      l *= f0;
#pragma unroll
      for (int c = 0; c < kC; ++c) acc[c] *= f0;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float f = ex2(ml[k].x - ref);
        l += ml[k].y * f;
#pragma unroll
        for (int c = 0; c < kC; ++c) acc[c] += o[k][c] * f;
      }
      m = mn;
    }
  }
  if (wpr > 1) {  // the same for every warp of the block
#pragma unroll
    for (int c = 0; c < kC; ++c) s_o[warp][lane * kC + c] = acc[c];
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
    __syncthreads();
    if (phase != 0) return;
    for (int w = 1; w < wpr; ++w) {
      const float mw = s_m[warp + w], mn = fmaxf(m, mw);
      const float ref = mn == -INFINITY ? 0.f : mn, f0 = ex2(m - ref), f1 = ex2(mw - ref);
      l = l * f0 + s_l[warp + w] * f1;
#pragma unroll
      for (int c = 0; c < kC; ++c) acc[c] = acc[c] * f0 + s_o[warp + w][lane * kC + c] * f1;
      m = mn;
    }
  }
  if (r >= rows) return;
  if constexpr (D == 128) {
    write_row<T>(p, j.tok0, j.b, j.hh, j.t0, j.first + r, lane, make_float4(acc[0], acc[1], acc[2], acc[3]), m, l);
  } else {
    const float a = __shfl_down_sync(0xffffffffu, acc[0], 1), c = __shfl_down_sync(0xffffffffu, acc[1], 1);
    if ((lane & 1) == 0)
      write_row<T>(p, j.tok0, j.b, j.hh, j.t0, j.first + r, lane / 2, make_float4(acc[0], acc[1], a, c), m, l);
  }
}

// The same for the parts of 128-row tiles, which hold four columns of all rows
// side by side: eight rows a block, a thread four columns of one.
template <int D, typename T>
__global__ void __launch_bounds__(2 * D) k_decode_join_tiles(const DecodeProblem p) {
  griddep_wait();
  griddep_launch_next();
  const DecodeJoin j = p.join[blockIdx.x];
  if (blockIdx.x == 0 && blockIdx.y == 0) join_flags<2 * D>(p);
  const int r = int(blockIdx.y) * 8 + int(threadIdx.x & 7), c = int(threadIdx.x >> 3);
  if (j.parts == 0 || r >= j.rows) return;
  constexpr int kBatch = 4;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < j.parts; i0 += kBatch) {
    float2 ml[kBatch];
    float4 o[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k;
      ml[k] = make_float2(-INFINITY, 0.f);
      o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < j.parts) {
        const int64_t at = i == 0 ? j.slot0 : 2 * (int(blockIdx.x) + i * p.group);
        ml[k] = reinterpret_cast<const float2 *>(p.part_ml)[at * p.TR + r];
        o[k] = reinterpret_cast<const float4 *>(p.part_o)[(at * (D / 4) + c) * p.TR + r];
      }
    }
    float mn = m;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) mn = fmaxf(mn, ml[k].x);
    const float ref = mn == -INFINITY ? 0.f : mn, f0 = ex2(m - ref);
    l *= f0;
    acc.x *= f0; acc.y *= f0; acc.z *= f0; acc.w *= f0;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float f = ex2(ml[k].x - ref);
      l += ml[k].y * f;
      acc.x += o[k].x * f; acc.y += o[k].y * f; acc.z += o[k].z * f; acc.w += o[k].w * f;
    }
    m = mn;
  }
  write_row<T>(p, j.tok0, j.b, j.hh, j.t0, j.first + r, c, acc, m, l);
}

template <int D, typename T>
cudaError_t launch_join(const DecodeProblem &p, cudaStream_t s) {
  // few rows: one block a unit, so that its warps can share the parts of a row
  if (p.TR == kTile) return launch_dep(k_decode_join<D, T, kTile>, dim3(unsigned(p.grid)), dim3(32 * kTile), 0, s, p);
  return launch_dep(k_decode_join_tiles<D, T>, dim3(unsigned(p.grid), unsigned(p.TR / 8)), dim3(2 * D), 0, s, p);
}

template <int D, typename T, int kMask>
cudaError_t launch(const DecodeProblem &p, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(k_decode<D, T, kMask>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Smem<D>::kBytes);
  if (e != cudaSuccess) return e;
  e = launch_dep(k_decode<D, T, kMask>, dim3(unsigned(p.grid)), dim3(kThreads), Smem<D>::kBytes, s, p);
  if (e != cudaSuccess) return e;
  return launch_join<D, T>(p, s);
}

template <int D, typename T>
cudaError_t launch_mask(const DecodeProblem &p, cudaStream_t s) {
  if (p.tree) return launch<D, T, 2>(p, s);
  return p.causal ? launch<D, T, 1>(p, s) : launch<D, T, 0>(p, s);
}

}  // namespace

bool decode_plan(DecodeProblem &p) {
  const int64_t tokens = p.q_layout == BSA_LAYOUT_BNSD ? p.Sq : (p.Tq + p.B - 1) / p.B;  // the mean
  const bool few = tokens * p.gg <= kFewRows;
  if (few) {
    p.TR = kTile;
    p.chunk = kChunk;
    p.group = 1;
    p.grid = num_sms() * (p.D == 128 ? 2 : 4);
  } else {
    decode_tc_plan(p);
  }
  auto log2 = [](int64_t x) { int n = 0; while ((int64_t(1) << n) < x) ++n; return n; };
  p.tr_sh = log2(p.TR);
  p.chunk_sh = log2(p.chunk);
  p.bq_sh = log2(p.BQ);
  p.bkv_sh = log2(p.kv.BKV);
  p.tpb = int32_t((int64_t(p.BQ) * p.gg + p.TR - 1) >> p.tr_sh);
  p.gg_inv = p.gg == 1 ? 0u : uint32_t(((int64_t(1) << 32) + p.gg - 1) / p.gg);
  // chunks of all units, at most: as dec_batch counts them, for the longest cache
  const int64_t all = p.q_layout == BSA_LAYOUT_BNSD ? p.Sq * p.B : p.Tq;
  const int64_t tiles = ((all * p.gg) >> p.tr_sh) + (p.index ? (all >> p.bq_sh) + p.B : p.B) + int64_t(p.group) * p.B;
  const int64_t kv = p.kv.layout == BSA_LAYOUT_TND ? p.kv.Tkv : p.kv.Skv, nk = (kv + p.kv.BKV - 1) >> p.bkv_sh;
  const int64_t some = p.index ? (p.W < nk ? p.W : nk) << (p.bkv_sh - p.chunk_sh) : (kv + p.chunk - 1) >> p.chunk_sh;
  const int64_t chunks = some > 0 ? some : 1;
  return p.gg < 65536 - 256 && double(tiles) * double(p.H) * double(chunks) < 4.0e9;
}

cudaError_t launch_decode(const DecodeProblem &p, cudaStream_t s) {
  if (p.TR != kTile) {
    cudaError_t e = launch_decode_tc(p, s);
    if (e != cudaSuccess) return e;
    if (p.dtype == BSA_BF16)
      return p.D == 64 ? launch_join<64, __nv_bfloat16>(p, s) : launch_join<128, __nv_bfloat16>(p, s);
    return p.D == 64 ? launch_join<64, __half>(p, s) : launch_join<128, __half>(p, s);
  }
  if (p.dtype == BSA_BF16)
    return p.D == 64 ? launch_mask<64, __nv_bfloat16>(p, s) : launch_mask<128, __nv_bfloat16>(p, s);
  return p.D == 64 ? launch_mask<64, __half>(p, s) : launch_mask<128, __half>(p, s);
}

}  // namespace bsa
