// decode_tc.cu -- tcgen05 form of the few-token attention for tiles of 128
// query rows (draft trees and chains: tokens times the heads of a group).
//
// Math, division of the work and joining of parts: decode.cu, decode_plan.cuh.
// The pipeline is the forward pass's: one block per SM, TMA loads of 128-token
// chunks of K and V through three-stage rings (warps 8 and 10), S = Q K^T and
// O += P V issued by warps 11 and 9, two softmax warpgroups on the two column
// halves of S with a reference maximum that moves only when a half-row sum
// passes 2^8.  Here the rows of a tile are gathered (any number of heads and
// tokens) by the softmax threads.  Only warp 8 walks the index and the block
// table: it publishes the chunks of a segment 32 at a time in shared memory,
// and the other warps read them there (a walk of their own cost the softmax
// threads 40 registers, spilled).  A chunk that reaches the masked tokens or
// the end of the cache gets a 64-bit visibility word per row and half.
//
// Bound by memory up to about 128 rows of a kv head, by the tensor pipe and
// the exponentials above.
#include <cuda.h>
#include <cuda_runtime.h>

#include "cache.h"
#include "decode_plan.cuh"
#include "launch.cuh"
#include "pack16.cuh"
#include "sm100.cuh"
#include "tc_common.h"
#include "tc_device.cuh"

namespace bsa {
namespace {

using namespace sm100;

constexpr int kTile = 128, kChunk = 128;
constexpr int kThreads = 384;
constexpr int kSoftmaxThreads = 256;
constexpr int kStages = 3;
constexpr int kSBufs = 3;
constexpr int kKWarp = 8, kPvWarp = 9, kVWarp = 10, kSWarp = 11;
constexpr int kCols = 64;  // kv columns of a softmax thread
constexpr float kRescaleSum = 256.0f;
constexpr int kMostGroup = 8;  // larger groups leave more SMs without a group
constexpr int kReaders = 11;  // warps that read the chunk lists

// up to 32 chunks of a segment, those that hold tokens
struct ChunkList {
  int n, last;  // last: the segment ends with this list
  int u[32], page[32];
};

enum : int {
  kBarQFull = 0,    // one arrival per softmax thread
  kBarKFull = 1,    // + K stage
  kBarKEmpty = 4,   // + K stage
  kBarVFull = 7,    // + V stage
  kBarVEmpty = 10,  // + V stage
  kBarSFull = 13,   // + S buffer
  kBarPFull = 16,   // + S buffer (one arrival per softmax thread)
  kBarPVDone = 19,  // + (chunk index & 1)
  kBarXchg = 21,    // + row quarter
  kBarDrain = 25,
  kBarSFree = 26,   // + S buffer
  kBarDrainS = 29,
  kBarQEmpty = 30,  // the segment's last S has read Q
  kBarListFull = 31,   // + list buffer
  kBarListEmpty = 33,  // + list buffer (one arrival per reading warp)
  kNumBars = 35
};

template <int D>
struct Layout {
  static constexpr int kBox = 128 * 128;  // 128 rows of 64 columns
  static constexpr int kTileBytes = D / 64 * kBox;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + kTileBytes;
  static constexpr int kV = kK + kStages * kTileBytes;
  static constexpr int kBars = kV + kStages * kTileBytes;
  static constexpr int kFlags = kBars + kNumBars * 8;     // [2][8 softmax warps] u32
  static constexpr int kXsum = kFlags + 2 * 8 * 4;        // [2][128] half-row sums
  static constexpr int kLists = kXsum + 2 * 128 * 4;      // [2] ChunkList
  static constexpr int kBlk = kLists + 2 * int(sizeof(ChunkList));  // [32] ints of the walking warp
  static constexpr int kTmemPtr = kBlk + 128;
  static constexpr int kAbort = kTmemPtr + 4;
  static constexpr int kBytes = kAbort + 4;
  static_assert(kXsum % 8 == 0 && sizeof(DecScratch<kThreads>) <= 1024, "the plan's scratch");
  static_assert(kBytes <= 232448, "shared memory budget");
};

// 64 consecutive draft nodes from node n0 on (negative: context, seen) of a
// row of ancestor bits
__device__ __forceinline__ uint64_t tree_bits(const DecodeProblem &p, const int64_t *bits, int n0) {
  auto word = [&](int w) { return w < p.tree_words ? uint64_t(bits[w]) : 0ull; };
  if (n0 <= -64) return ~0ull;
  if (n0 < 0) return (word(0) << -n0) | ((1ull << -n0) - 1ull);
  const int s = n0 & 63;
  return s ? (word(n0 >> 6) >> s) | (word((n0 >> 6) + 1) << (64 - s)) : word(n0 >> 6);
}
__device__ __forceinline__ uint64_t low_bits(int64_t n) { return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1ull; }

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    k_decode_tc(const DecodeProblem p, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v) {
  using L = Layout<D>;
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  extern __shared__ unsigned char smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_wait();
  griddep_launch_next();
  uint32_t *status = p.flags + blockIdx.x;  // this block's flags
  const uint32_t base = smem_u32(smem_raw);
  uint32_t len_flags = 0;
  // (the row sums' memory serves as scratch here; nothing is in static shared
  // memory, so that the tiles start at the 1024-byte aligned window)
  const DecStart st = dec_start<kThreads>(p, *reinterpret_cast<DecScratch<kThreads> *>(smem_raw + L::kXsum), len_flags);
  if (tid == 0) {
    *status = base & 1023u ? BSA_FLAG_INTERNAL : 0u;  // swizzled tiles need a 1024-byte aligned base
    p.join[blockIdx.x] = DecodeJoin{};
    __threadfence();
  }
  __syncthreads();
  if (len_flags) atomicOr(status, len_flags);
  if ((base & 1023u) || st.lo >= st.hi) return;  // the whole block
  const uint32_t sQ = base + L::kQ, sK = base + L::kK, sV = base + L::kV;
  auto bar = [&](int i) { return base + L::kBars + 8u * uint32_t(i); };
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem_raw + L::kTmemPtr);
  volatile int *abort = reinterpret_cast<volatile int *>(smem_raw + L::kAbort);
  volatile ChunkList *lists = reinterpret_cast<volatile ChunkList *>(smem_raw + L::kLists);

  if (tid == 0) {
    mbar_init(bar(kBarQFull), kSoftmaxThreads);
    mbar_init(bar(kBarQEmpty), 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(kBarKFull + s), 1);
      mbar_init(bar(kBarKEmpty + s), 1);
      mbar_init(bar(kBarVFull + s), 1);
      mbar_init(bar(kBarVEmpty + s), 1);
    }
    for (int b = 0; b < kSBufs; ++b) {
      mbar_init(bar(kBarSFull + b), 1);
      mbar_init(bar(kBarPFull + b), kSoftmaxThreads);
      mbar_init(bar(kBarSFree + b), 1);
    }
    mbar_init(bar(kBarPVDone), 1);
    mbar_init(bar(kBarPVDone + 1), 1);
    for (int q = 0; q < 4; ++q) mbar_init(bar(kBarXchg + q), kSoftmaxThreads / 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarListFull + i), 1);
      mbar_init(bar(kBarListEmpty + i), kReaders);
    }
    mbar_init(bar(kBarDrain), 1);
    mbar_init(bar(kBarDrainS), 1);
    *abort = 0;
    fence_barrier_init();
  }
  if (warp == kPvWarp) {
    tmem_alloc(base + L::kTmemPtr, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS0 = tmem, tO = tmem + uint32_t(kSBufs) * 128u;

  DecCursor cursor = cursor_begin(st), here{};
  DecBatch d{};
  DecSeg seg{};
  uint32_t kv_it = 0;
  bool ok = true;

  uint32_t list_it = 0;
  // f(first token, page) for every chunk of the segment, by a reading warp
  auto each_chunk = [&](auto &&f) {
    for (bool last = false; ok && !last; ++list_it) {
      const int i = int(list_it & 1u);
      if (!(ok = wait_warp(bar(kBarListFull + i), (list_it >> 1) & 1u, abort, status))) break;
      const int n = lists[i].n;
      last = lists[i].last;
      for (int c = 0; c < n && ok; ++c) f(lists[i].u[c], lists[i].page[c]);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarListEmpty + i));
    }
  };

  if (warp == kKWarp || warp == kVWarp) {
    // ----------------------------------------------------- TMA producers
    const bool is_k = warp == kKWarp;
    const CUtensorMap *map = is_k ? &map_k : &map_v;
    if (lane == 0) tma_prefetch_desc(map);
    const uint32_t ring = is_k ? sK : sV;
    const int full0 = is_k ? kBarKFull : kBarVFull, empty0 = is_k ? kBarKEmpty : kBarVEmpty;
    int armed[kStages] = {-1, -1, -1};
    uint32_t flags = 0;
    auto load = [&](int u, int pg, int h2) {
      const int s = int(kv_it % kStages);
      const uint32_t ph = (kv_it / kStages) & 1u;
      if (!(ok = wait_warp(bar(empty0 + s), ph ^ 1u, abort, status))) return;
      if (lane == 0) {
        int row, last;  // tile coordinates: (0, row, 0, h2, last)
        if (p.kv.table) { row = u % p.kv.page_size; last = pg; }
        else if (p.kv.cu_kv) { row = int(d.kv.tok0) + u; last = 0; }
        else { row = u; last = here.b; }
        mbar_expect_tx(bar(full0 + s), L::kTileBytes);
        tma_load_5d(ring + s * L::kTileBytes, map, bar(full0 + s), 0, row, 0, h2, last);
      }
      armed[s] = int(ph);
      ++kv_it;
    };
    while (ok && cursor_next(p, st, cursor, d, seg, here)) {
      const int h2 = seg.hh / (p.H / p.N2);
      if (is_k) {
        DecWalk w = walk_begin(p, here.b, seg.hh, dec_rows(p, d, seg.tile).irow, here.qoff);
        int *blk = reinterpret_cast<int *>(smem_raw + L::kBlk);
        for (int x = seg.cs & ~31; x < seg.ce && ok; x += 32, ++list_it) {
          int u, pg;
          walk_fetch(p, d, here.b, w, x, seg.ce, blk, lane, u, pg);
          const uint32_t some = __ballot_sync(0xffffffffu, u >= 0 && x + lane >= seg.cs);
          const int n = __popc(some), i = int(list_it & 1u);
          if (!(ok = wait_warp(bar(kBarListEmpty + i), ((list_it >> 1) & 1u) ^ 1u, abort, status))) break;
          if (some >> lane & 1u) {
            const int at = __popc(some & ((1u << lane) - 1u));
            lists[i].u[at] = u;
            lists[i].page[at] = pg;
          }
          if (lane == 0) {
            lists[i].n = n;
            lists[i].last = x + 32 >= seg.ce;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarListFull + i));
          for (int c = 0; c < n && ok; ++c) load(lists[i].u[c], lists[i].page[c], h2);
        }
        flags |= w.flags;
      } else {
        each_chunk([&](int u, int pg) { load(u, pg, h2); });
      }
    }
    if (*abort && lane == 0) {  // let every copy already issued land before the block exits
      for (int s = 0; s < kStages; ++s)
        if (armed[s] >= 0) drain_wait(bar(full0 + s), uint32_t(armed[s]));
    }
    if (is_k && flags) atomicOr(status, flags);
    __syncwarp();
  } else if (warp == kPvWarp || warp == kSWarp) {
    // -------------------------------------------------------- MMA issuers
    constexpr uint32_t idS = idesc_f16(BF16, 128, 128, false, false);
    constexpr uint32_t idPV = idesc_f16(BF16, 128, D, false, true);
    const uint64_t dQ = sw128_desc(sQ, 16, 1024);
    const uint64_t dK = sw128_desc(sK, 16, 1024);
    const uint64_t dV = sw128_desc(sV, L::kBox, 1024);
    auto kstep = [](int kk) { return uint64_t((kk >> 2) * (L::kBox >> 4) + (kk & 3) * 2); };
    // P of the first 64 kv columns in TMEM columns [0, 32) of the S buffer, of the next 64 in [64, 96)
    auto pcol = [](int kk) { return uint32_t(64 * (kk >> 2) + 8 * (kk & 3)); };
    const bool is_s = warp == kSWarp;
    uint32_t q_it = 0;
    while (ok && cursor_next(p, st, cursor, d, seg, here)) {
      if (is_s) {
        // Q is written for every segment, whether or not it has a chunk
        if (!(ok = wait_warp(bar(kBarQFull), q_it & 1u, abort, status))) break;
        ++q_it;
        each_chunk([&](int, int) {
          const uint32_t t = kv_it;
          const int b = int(t % kSBufs), sg = int(t % kStages);
          if (t >= uint32_t(kSBufs) && !(ok = wait_warp(bar(kBarSFree + b), (t / kSBufs - 1) & 1u, abort, status)))
            return;
          if (!(ok = wait_warp(bar(kBarKFull + sg), (t / kStages) & 1u, abort, status))) return;
          tc_fence_after();
          const uint32_t da = tS0 + uint32_t(b) * 128u;
          const uint64_t ka = dK + uint64_t(sg * (L::kTileBytes >> 4));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) mma_ss_e(da, dQ + kstep(kk), ka + kstep(kk), idS, kk > 0 ? 1u : 0u);
          mma_commit_e(bar(kBarSFull + b));
          mma_commit_e(bar(kBarKEmpty + sg));
          ++kv_it;
        });
        if (!ok) break;
        mma_commit_e(bar(kBarQEmpty));
      } else {
        uint32_t acc = 0;
        each_chunk([&](int, int) {
          const uint32_t t = kv_it;
          const int b = int(t % kSBufs), sg = int(t % kStages);
          if (!(ok = wait_warp(bar(kBarVFull + sg), (t / kStages) & 1u, abort, status))) return;
          if (!(ok = wait_warp(bar(kBarPFull + b), (t / kSBufs) & 1u, abort, status))) return;
          tc_fence_after();
          const uint32_t pa = tS0 + uint32_t(b) * 128u;
          const uint64_t vd = dV + uint64_t(sg * (L::kTileBytes >> 4));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            mma_ts_e(tO, pa + pcol(kk), vd + uint64_t(kk * 128), idPV, acc);
            acc = 1;
          }
          mma_commit_e(bar(kBarPVDone + int(t & 1u)));
          mma_commit_e(bar(kBarVEmpty + sg));
          mma_commit_e(bar(kBarSFree + b));
          ++kv_it;
        });
      }
    }
    if (*abort) {  // let issued MMAs finish before TMEM is freed
      const int dr = is_s ? kBarDrainS : kBarDrain;
      mma_commit_e(bar(dr));
      if (lane == 0) drain_wait(bar(dr), 0);
    }
    __syncwarp();
  } else {
    // --------------------------------------------- softmax warpgroups
    const int wg = warp >> 2;
    const int r = tid & 127;  // tile row = TMEM lane
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    volatile uint32_t *xflags = reinterpret_cast<volatile uint32_t *>(smem_raw + L::kFlags);
    float *xsum = reinterpret_cast<float *>(smem_raw + L::kXsum);
    uint32_t x_it = 0, seg_n = 0;
    auto rendezvous = [&]() {  // the warps that hold the same 32 rows (bounded)
      mbar_arrive(bar(kBarXchg + (warp & 3)));
      ok = wait_warp(bar(kBarXchg + (warp & 3)), x_it & 1u, abort, status);
      ++x_it;
      return ok;
    };
    while (ok && cursor_next(p, st, cursor, d, seg, here)) {
      const DecRows v = dec_rows(p, d, seg.tile);
      const int64_t qb = p.cu_q ? 0 : here.b;
      const int kvlen = d.kv.kvlen, qbase = kvlen - d.q.qlen;
      const int xr = v.first + min(r, v.rows - 1);
      const int tq = v.t0 + xr / p.gg;
      // ---- the Q tile, once the segment before has read its own
      if (!(ok = wait_warp(bar(kBarQEmpty), (seg_n & 1u) ^ 1u, abort, status))) break;
      {
        constexpr int kPieces = D / 8;  // 16-byte pieces of a row
        for (int i = tid; i < kTile * kPieces; i += kSoftmaxThreads) {
          const int rr = i / kPieces, c = i % kPieces;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (rr < v.rows) {
            const int y = v.first + rr, t = v.t0 + y / p.gg, h = seg.hh * p.gg + y % p.gg;
            const T *q = static_cast<const T *>(p.q) + qb * p.q_sb + (d.q.tok0 + t) * p.q_st + int64_t(h) * p.q_sh;
            x = __ldg(reinterpret_cast<const uint4 *>(q) + c);
          }
          // 128-byte swizzle: the 16-byte piece within a row of 128 bytes xor the row
          *reinterpret_cast<uint4 *>(smem_raw + L::kQ + (c >> 3) * L::kBox + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) = x;
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(kBarQFull));
      }
      const int64_t *bits = p.tree ? p.tree + qb * p.t_sb + (d.q.tok0 + tq) * p.t_st : nullptr;
      // the columns [u, u + 64) that the row sees
      auto visible = [&](int u) {
        uint64_t m = low_bits(int64_t(kvlen) - u);
        if (p.tree) m &= tree_bits(p, bits, u - qbase);
        else if (p.causal) m &= low_bits(int64_t(tq) + qbase - u + 1);
        return m;
      };
      const int edge_from = (p.tree || p.causal) ? qbase : kvlen;  // first token that some row may not see
      float m = -INFINITY, l = 0.f;
      int n = 0;
      each_chunk([&](const int u0c, int) {
        const int b = int(kv_it % kSBufs);
        if (!(ok = wait_warp(bar(kBarSFull + b), (kv_it / kSBufs) & 1u, abort, status))) return;
        tc_fence_after();
        const uint32_t tS = tS0 + uint32_t(b) * 128u + lane_off;
        const int valid_all = kvlen - u0c;
        if (valid_all < 128) {
          // rows past the used length may hold anything: their weights are 0,
          // and their V is made 0 as well before P is published
          const int sg = int(kv_it % kStages);
          if (!(ok = wait_warp(bar(kBarVFull + sg), (kv_it / kStages) & 1u, abort, status))) return;
          uint4 *vt = reinterpret_cast<uint4 *>(smem_raw + L::kV + sg * L::kTileBytes);
          const int per_half = (128 - valid_all) * 8;
          for (int w = tid; w < per_half * (D / 64); w += kSoftmaxThreads) {
            const int h = w / per_half, x = w % per_half;
            vt[h * (L::kBox / 16) + valid_all * 8 + x] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        const bool edge = u0c + kChunk > edge_from;
        uint32_t x[kCols];
        tmem_ld_cols<kCols>(tS + uint32_t(kCols * wg), x);
        tmem_wait_ld();
        if (edge) {
          const uint64_t vis = visible(u0c + kCols * wg);
          const uint32_t lo = uint32_t(vis), hi = uint32_t(vis >> 32);
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            if (!((c < 32 ? lo : hi) & (1u << (c & 31)))) x[c] = __float_as_uint(-INFINITY);
        }
        float ps[2] = {0.f, 0.f};
        uint32_t pk[kCols / 2];
        auto exps = [&](float mm) {
          ps[0] = ps[1] = 0.f;
#pragma unroll
          for (int c = 0; c < kCols; c += 2) {
            const float e0 = ex2(fmaf(__uint_as_float(x[c]), p.scale_log2, -mm));
            const float e1 = ex2(fmaf(__uint_as_float(x[c + 1]), p.scale_log2, -mm));
            ps[(c >> 1) & 1] += e0 + e1;
            pk[c >> 1] = Pack2<T>::pack(e0, e1);
          }
        };
        // a row that has seen nothing yet keeps m = -inf and asks for a reference
        const bool first = m == -INFINITY;
        if (!first) exps(m);
        uint32_t any = 1;
        if (n > 0) {
          const uint32_t need = __any_sync(0xffffffffu, first || !(ps[0] + ps[1] <= kRescaleSum)) ? 1u : 0u;
          if (lane == 0) xflags[(kv_it & 1u) * 8 + warp] = need;
          if (!rendezvous()) return;
          any = xflags[(kv_it & 1u) * 8 + (warp & 3)] | xflags[(kv_it & 1u) * 8 + 4 + (warp & 3)];
        }
        float alpha = 1.f;
        const bool grow = any != 0u;
        if (grow) {
          float pm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < kCols; ++c) pm[c & 3] = fmaxf(pm[c & 3], __uint_as_float(x[c]));
          float cm = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
          // the other group's columns are still S in TMEM
          const uint64_t vo = edge ? visible(u0c + kCols * (wg ^ 1)) : ~0ull;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t y[kCols / 2];
            tmem_ld_cols<kCols / 2>(tS + uint32_t(kCols * (wg ^ 1) + (kCols / 2) * h), y);
            tmem_wait_ld();
            const uint32_t vy = uint32_t(vo >> (32 * h));
#pragma unroll
            for (int c = 0; c < kCols / 2; ++c)
              if (vy & (1u << c)) cm = fmaxf(cm, __uint_as_float(y[c]));
          }
          if (!rendezvous()) return;  // nobody overwrites S with P before every thread has read it
          const float m_new = fmaxf(m, cm * p.scale_log2);
          alpha = first ? 1.f : ex2(m - m_new);
          m = m_new;
          exps(m > -INFINITY ? m : 0.f);  // nothing visible yet: every weight is 0
        }
        tmem_st_cols<kCols / 2>(tS + uint32_t(kCols * wg), pk);
        l = l * alpha + (ps[0] + ps[1]);
        if (grow && n > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          // O may be rescaled once every earlier product has landed
          const uint32_t t = kv_it - 1;
          if (!(ok = wait_warp(bar(kBarPVDone + int(t & 1u)), (t / 2) & 1u, abort, status))) return;
          tc_fence_after();
          const uint32_t col = tO + lane_off + uint32_t(wg * (D / 2));
          uint32_t o[D / 2];
          tmem_ld_cols<D / 2>(col, o);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < D / 2; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
          tmem_st_cols<D / 2>(col, o);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(kBarPFull + b));
        ++n;
        ++kv_it;
      });
      if (!ok) break;
      // ---- epilogue: the finished rows, or this block's part of them
      if (n > 0) {
        const uint32_t t = kv_it - 1;
        if (!(ok = wait_warp(bar(kBarPVDone + int(t & 1u)), (t / 2) & 1u, abort, status))) break;
        tc_fence_after();
      }
      // the partner has read the last segment's sums: it has met this warp
      // since, in the first chunk or here
      if (n == 0 && !rendezvous()) break;
      xsum[wg * 128 + r] = l;
      if (!rendezvous()) break;
      const float lsum = xsum[r] + xsum[128 + r];
      const bool whole = seg.cs == 0 && seg.ce == d.chunks;
      const int slot = here.pos == st.lo ? 2 * int(blockIdx.x) : 2 * int(blockIdx.x) + 1;
      uint32_t o[D / 2];
      if (n > 0) {
        tmem_ld_cols<D / 2>(tO + lane_off + uint32_t(wg * (D / 2)), o);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int c = 0; c < D / 2; ++c) o[c] = 0u;
      }
      if (r < v.rows) {
        const int h = seg.hh * p.gg + xr % p.gg;
        if (whole) {
          const float inv = lsum > 0.f || lsum != lsum ? 1.f / lsum : 0.f;
          T *dst = static_cast<T *>(p.out) + qb * p.o_sb + (d.q.tok0 + tq) * p.o_st + int64_t(h) * p.o_sh + wg * (D / 2);
#pragma unroll
          for (int c8 = 0; c8 < D / 16; ++c8) {
            uint4 w;
            w.x = Pack2<T>::pack(__uint_as_float(o[8 * c8]) * inv, __uint_as_float(o[8 * c8 + 1]) * inv);
            w.y = Pack2<T>::pack(__uint_as_float(o[8 * c8 + 2]) * inv, __uint_as_float(o[8 * c8 + 3]) * inv);
            w.z = Pack2<T>::pack(__uint_as_float(o[8 * c8 + 4]) * inv, __uint_as_float(o[8 * c8 + 5]) * inv);
            w.w = Pack2<T>::pack(__uint_as_float(o[8 * c8 + 6]) * inv, __uint_as_float(o[8 * c8 + 7]) * inv);
            reinterpret_cast<uint4 *>(dst)[c8] = w;
          }
          if (wg == 0 && p.lse)
            p.lse[qb * p.l_sb + (d.q.tok0 + tq) * p.l_st + int64_t(h) * p.l_sh] =
                lsum > 0.f || lsum != lsum ? (m + __log2f(lsum)) * 0.6931471805599453f : -INFINITY;
        } else {
          float4 *dst = reinterpret_cast<float4 *>(p.part_o + (int64_t(slot) * kTile + r) * D + wg * (D / 2));
#pragma unroll
          for (int c4 = 0; c4 < D / 8; ++c4)
            dst[c4] = make_float4(__uint_as_float(o[4 * c4]), __uint_as_float(o[4 * c4 + 1]),
                                  __uint_as_float(o[4 * c4 + 2]), __uint_as_float(o[4 * c4 + 3]));
          if (wg == 0) reinterpret_cast<float2 *>(p.part_ml)[int64_t(slot) * kTile + r] = make_float2(m, lsum);
        }
      }
      if (tid == 0 && seg.cs == 0 && !whole) p.join[blockIdx.x] = dec_join(p, st, here, d, seg, v, slot);
      tc_fence_before();
      ++seg_n;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kPvWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool BF16>
cudaError_t launch(const DecodeProblem &p, const CUtensorMap &k, const CUtensorMap &v, cudaStream_t s) {
  // at least 120 KB, so that one block (the owner of all TMEM columns) is on an SM
  const int smem = Layout<D>::kBytes > 120 * 1024 ? Layout<D>::kBytes : 120 * 1024;
  cudaError_t e = cudaFuncSetAttribute(k_decode_tc<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_dep(k_decode_tc<D, BF16>, dim3(unsigned(p.grid)), dim3(kThreads), size_t(smem), s, p, k, v);
}

}  // namespace

void decode_tc_plan(DecodeProblem &p) {
  p.TR = kTile;
  p.chunk = kChunk;
  // as many blocks side by side as a sequence of the mean number of tokens
  // has tiles (sparse: tiles of one query block, which share an index row)
  const int64_t tokens = p.q_layout == BSA_LAYOUT_BNSD ? p.Sq : (p.Tq + p.B - 1) / p.B;
  const int64_t rows = (p.index && tokens > p.BQ ? p.BQ : tokens) * p.gg;
  const int64_t tiles = (rows + kTile - 1) / kTile;
  p.group = int32_t(tiles < kMostGroup ? tiles : kMostGroup);
  p.grid = num_sms() / p.group * p.group;
}

cudaError_t launch_decode_tc(const DecodeProblem &p, cudaStream_t s) {
  auto some = [](int64_t n) { return n > 0 ? n : int64_t(1); };  // maps of empty caches, never read
  Problem t{};
  t.dtype = p.dtype; t.D = p.D; t.N2 = p.N2; t.B = p.B;
  t.kv_layout = p.kv.layout; t.page_size = p.kv.page_size; t.num_pages = int32_t(some(p.kv.num_pages));
  t.Tkv = some(p.kv.Tkv); t.Skv = some(p.kv.Skv);
  t.k = p.k; t.k_sb = p.k_sb; t.k_sh = p.k_sh; t.k_st = p.k_st;
  t.v = p.v; t.v_sb = p.v_sb; t.v_sh = p.v_sh; t.v_st = p.v_st;
  CUtensorMap k, v;
  cudaError_t e = make_kv_maps(t, k, v);
  if (e != cudaSuccess) return e;
  if (p.dtype == BSA_BF16) return p.D == 64 ? launch<64, true>(p, k, v, s) : launch<128, true>(p, k, v, s);
  return p.D == 64 ? launch<64, false>(p, k, v, s) : launch<128, false>(p, k, v, s);
}

}  // namespace bsa
