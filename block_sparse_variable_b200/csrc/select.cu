// select.cu -- the block index from scores of query blocks against block means.
//
// Math: for index head hi, query block i and kv block j of one sequence
//     s(hi,i,j) = (sum of the block's query rows over the heads of hi) . means[b,h2,j]
// and the row keeps the W blocks of the highest s (ties: the lower id),
// forced blocks first, written in ascending order and padded with 0xFFFF.
// The outcome is a set of whole numbers, so scores are 64-bit: two blocks
// whose scores differ in the 10th digit are ordered by their scores and not
// by the order of a sum.
//
// Three kernels: sums of the query rows (memory bound: reads q once), scores
// (reads the means once per row that L2 does not serve), choice (a warp per
// index row).
#include <cuda_runtime.h>

#include "cache.h"
#include "launch.cuh"
#include "pack16.cuh"

namespace bsa {
namespace {

constexpr int kThreads = 256;
constexpr uint64_t kForced = ~0ull;  // above every score
constexpr uint64_t kNan = 1;         // below every number

// A 16-bit value as a double times 2^-896, by moving its fp32 bits: the
// mantissa has at most 10 bits, so all of it stays in the high word, and
// subnormals and zeros come out exact.  Conversions to 64 bits run at a
// fraction of the rate of the multiply-adds they feed; this is two integer
// operations.  Infinities and NaN come out as numbers: callers look for them.
__device__ __forceinline__ double scaled64(float f) {
  const uint32_t x = __float_as_uint(f);
  return __hiloint2double(int((x & 0x80000000u) | ((x >> 3) & 0x0fffffffu)), 0);
}
constexpr double kTwo512 = 0x1p512, kTwo704 = 0x1p704, kTwoM896 = 0x1p-896;

template <typename T>
struct Abs2;
template <>
struct Abs2<__nv_bfloat16> {
  using V = __nv_bfloat162;
};
template <>
struct Abs2<__half> {
  using V = __half2;
};
// running maximum of |x| of both halves, NaN kept
template <typename T>
__device__ __forceinline__ uint32_t max_abs(uint32_t m, uint32_t x) {
  using V = typename Abs2<T>::V;
  V a = *reinterpret_cast<V *>(&m), b = *reinterpret_cast<V *>(&x);
  V r = __hmax2_nan(a, __habs2(b));
  return *reinterpret_cast<uint32_t *>(&r);
}
template <typename T>
__device__ __forceinline__ bool not_finite(uint32_t m) {
  const float2 f = Pack2<T>::unpack(m);
  return !(f.x < INFINITY) || !(f.y < INFINITY);
}

struct Row {
  int b, i, qlen;  // b < 0: no such row
  int64_t q0;
};

// the batch and query block of global index row r, by the whole block
__device__ Row find_row(const SelectProblem &p, int r) {
  __shared__ int s_warp[kThreads / 32];
  __shared__ Row s_row;
  uint32_t ignore = 0;
  if (!p.cu_q) return {r / p.R, r % p.R, int(p.Sq), 0};
  const int tid = threadIdx.x, lane = tid & 31;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += (q_batch(p.cu_q, p.Sq, p.Tq, b, ignore).qlen + p.BQ - 1) / p.BQ;
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) s_warp[tid >> 5] = inc;
  if (tid == 0) s_row.b = -1;
  __syncthreads();
  int before = inc - mine;
  for (int w = 0; w < (tid >> 5); ++w) before += s_warp[w];
  if (r >= before && r < before + mine) {
    for (int b = b0; b < b1; ++b) {
      const QBatch qb = q_batch(p.cu_q, p.Sq, p.Tq, b, ignore);
      const int nq = (qb.qlen + p.BQ - 1) / p.BQ;
      if (r < before + nq) {
        s_row = {b, r - before, qb.qlen, qb.tok0};
        break;
      }
      before += nq;
    }
  }
  __syncthreads();
  return s_row;
}

__device__ void check_inputs(const SelectProblem &p) {
  __shared__ uint32_t sflags;
  __shared__ unsigned long long rows;
  if (threadIdx.x == 0) { sflags = 0; rows = 0; }
  __syncthreads();
  uint32_t f = 0;
  unsigned long long n = 0;
  for (int b = threadIdx.x; b < p.B; b += kThreads) {
    if (kv_batch(p.kv, b, f).kvlen > int64_t(p.NB) * p.BKV) f |= BSA_FLAG_BAD_SEQLEN;
    n += (q_batch(p.cu_q, p.Sq, p.Tq, b, f).qlen + p.BQ - 1) / p.BQ;
  }
  if (f) atomicOr(&sflags, f);
  atomicAdd(&rows, n);
  __syncthreads();
  if (threadIdx.x < kStWords) {
    uint32_t v = sflags;
    if (p.cu_q && rows > (unsigned long long)p.R) v |= BSA_FLAG_BAD_INDEX;
    p.status[threadIdx.x] = threadIdx.x == kStFlags ? v : 0;
  }
}

// one block per (index row, index head)
template <int D, typename T>
__global__ void __launch_bounds__(kThreads) k_query_sums(const SelectProblem p) {
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes, kLoads = 8;
  __shared__ double red[kThreads / 32][D];
  griddep_wait();
  griddep_launch_next();
  if (blockIdx.x == 0) return check_inputs(p);
  const int id = int(blockIdx.x) - 1;
  const int hi = id % p.Hidx, r = id / p.Hidx;
  const Row row = find_row(p, r);
  if (row.b < 0) {
    if (hi == 0 && threadIdx.x == 0) p.row_nk[r] = -1;
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = row.i * p.BQ, nt = min(p.BQ, row.qlen - t0);
  if (hi == 0 && tid == 0) {
    uint32_t ignore = 0;
    const int kvlen = kv_batch(p.kv, row.b, ignore).kvlen;
    int64_t nk = min((kvlen + p.BKV - 1) / p.BKV, p.NB);
    if (p.causal) {  // the blocks that the query block's last row sees
      const int64_t end = int64_t(t0) + nt - 1 + kvlen - row.qlen;
      const int64_t see = end < 0 ? 0 : end / p.BKV + 1;
      nk = see < nk ? see : nk;
    }
    p.row_nk[r] = int(nk);
    p.row_batch[r] = row.b;
  }
  const int gg = p.N1 / p.Hidx, col = tid % kLanes, rl = tid / kLanes;
  const T *q = static_cast<const T *>(p.q) + int64_t(row.b) * p.q_sb * (p.cu_q ? 0 : 1) +
               (row.q0 + t0) * p.q_st + int64_t(hi) * gg * p.q_sh + col * 8;
  double acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0;
  uint32_t big = 0;
  for (int g = 0; g < gg; ++g) {
    const T *qh = q + int64_t(g) * p.q_sh;
    for (int t = rl; t < nt; t += kRows * kLoads) {
      uint4 x[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int tt = t + i * kRows;
        x[i] = tt < nt ? __ldg(reinterpret_cast<const uint4 *>(qh + int64_t(tt) * p.q_st)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 f = Pack2<T>::unpack(w[c]);
          big = max_abs<T>(big, w[c]);
          acc[2 * c] += scaled64(f.x);
          acc[2 * c + 1] += scaled64(f.y);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = acc[i] * kTwo704 * kTwo704;  // to q * 2^512
  if (not_finite<T>(big)) {  // rare: once more with conversions that keep infinities and NaN
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0;
    for (int g = 0; g < gg; ++g)
      for (int t = rl; t < nt; t += kRows) {
        const uint32_t *x = reinterpret_cast<const uint32_t *>(q + int64_t(g) * p.q_sh + int64_t(t) * p.q_st);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 f = Pack2<T>::unpack(x[c]);
          acc[2 * c] += double(f.x);
          acc[2 * c + 1] += double(f.y);
        }
      }
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] *= kTwo512;
  }
#pragma unroll
  for (int o = kLanes; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
  if (lane < kLanes)
#pragma unroll
    for (int i = 0; i < 8; ++i) red[warp][col * 8 + i] = acc[i];
  __syncthreads();
  if (tid < D) {
    double a = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) a += red[w][tid];
    p.qsum[(int64_t(hi) * p.Rg + r) * D + tid] = a;
  }
}

__device__ __forceinline__ uint64_t order_bits(double s) {
  if (s != s) return kNan;
  const uint64_t x = uint64_t(__double_as_longlong(s + 0.0));  // -0 and 0 tie
  return x >> 63 ? ~x : x | (1ull << 63);
}

// scores of kScoreBlocks kv blocks against one index row: eight lanes a block
constexpr int kScoreBlocks = 128;
template <int D, typename T>
__global__ void __launch_bounds__(kThreads) k_scores(const SelectProblem p, int chunks) {
  constexpr int kC = D / 64;  // 16-byte pieces a lane holds of a mean
  griddep_wait();
  griddep_launch_next();
  int64_t id = blockIdx.x;
  const int chunk = int(id % chunks);
  id /= chunks;
  const int hi = int(id % p.Hidx), r = int(id / p.Hidx);
  const int nk = p.row_nk[r], j0 = chunk * kScoreBlocks;
  if (j0 >= nk) return;
  const int b = p.row_batch[r], lane = threadIdx.x & 7, grp = threadIdx.x >> 3;
  const int h2 = hi / (p.Hidx / p.N2);
  const double *qs = p.qsum + (int64_t(hi) * p.Rg + r) * D;
  double q[kC][8];
#pragma unroll
  for (int c = 0; c < kC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) q[c][i] = qs[(c * 8 + lane) * 8 + i];
  const T *m = static_cast<const T *>(p.means) + int64_t(b) * p.m_sb + int64_t(h2) * p.m_sh + lane * 8;
  uint64_t *keys = p.keys + (int64_t(hi) * p.Rg + r) * p.NB;
#pragma unroll
  for (int jj = 0; jj < kScoreBlocks; jj += kThreads / 8) {
    const int j = j0 + jj + grp;
    const bool in = j < nk;
    uint4 x[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c)
      x[c] = in ? __ldg(reinterpret_cast<const uint4 *>(m + int64_t(j) * p.m_st + c * 64)) : make_uint4(0, 0, 0, 0);
    double s = 0.0;
    uint32_t big = 0;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = Pack2<T>::unpack(w[i]);
        big = max_abs<T>(big, w[i]);
        s = fma(q[c][2 * i], scaled64(f.x), s);
        s = fma(q[c][2 * i + 1], scaled64(f.y), s);
      }
    }
    if (not_finite<T>(big)) {
      s = 0.0;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = Pack2<T>::unpack(w[i]);
          s += q[c][2 * i] * (double(f.x) * kTwoM896) + q[c][2 * i + 1] * (double(f.y) * kTwoM896);
        }
      }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (in && lane == 0) keys[j] = j < p.sink || j >= nk - p.local ? kForced : order_bits(s);
  }
}

// One warp per (index row, index head).  The W-th highest key is found bit by
// bit from the top, each step a count of the keys at or above a candidate;
// a candidate with exactly W of them ends the search.  kKeys keys a lane stay
// in registers (0: they are read again each step).
constexpr int kChooseWarps = 4;
template <int kKeys>
__global__ void __launch_bounds__(32 * kChooseWarps) k_choose(const SelectProblem p) {
  griddep_wait();
  griddep_launch_next();
  const int lane = threadIdx.x & 31;
  const int64_t id = int64_t(blockIdx.x) * kChooseWarps + (threadIdx.x >> 5);
  if (id >= int64_t(p.Rg) * p.Hidx) return;
  const int hi = int(id % p.Hidx), r = int(id / p.Hidx);
  const int nk = p.row_nk[r];
  if (nk < 0) return;
  uint16_t *out;
  if (p.cu_q) out = p.index + int64_t(hi) * p.ix_s0 + int64_t(r) * p.ix_s1;
  else out = p.index + int64_t(r / p.R) * p.ix_s0 + int64_t(hi) * p.ix_s1 + int64_t(r % p.R) * p.ix_s2;
  const int W = p.W;
  if (nk <= W) {
    for (int w = lane; w < W; w += 32) out[w] = w < nk ? uint16_t(w) : kNoBlock;
    return;
  }
  const uint64_t *keys = p.keys + (int64_t(hi) * p.Rg + r) * p.NB;
  uint64_t k[kKeys > 0 ? kKeys : 1];
  if constexpr (kKeys > 0) {
#pragma unroll
    for (int i = 0; i < kKeys; ++i) k[i] = i * 32 + lane < nk ? keys[i * 32 + lane] : 0;
  }
  auto count = [&](uint64_t t) {  // keys at or above t (t > 0)
    int n = 0;
    if constexpr (kKeys > 0) {
#pragma unroll
      for (int i = 0; i < kKeys; ++i) n += k[i] >= t;
    } else {
      for (int j = lane; j < nk; j += 32) n += keys[j] >= t;
    }
    return int(__reduce_add_sync(0xffffffffu, n));
  };
  uint64_t thr = 0;
  bool exact = false;
  for (int bit = 63; bit >= 0 && !exact; --bit) {
    const uint64_t cand = thr | (1ull << bit);
    const int n = count(cand);
    if (n >= W) thr = cand;
    exact = n == W;
  }
  // all above the threshold, and the first `ties` of those at it
  int ties = exact ? W : W - (thr == ~0ull ? 0 : count(thr + 1));
  int at = 0;
  auto emit = [&](int j, uint64_t key) {
    const bool eq = key == thr && key != 0;
    const uint32_t m_eq = __ballot_sync(0xffffffffu, eq);
    const uint32_t below = (1u << lane) - 1u;
    const bool take = key > thr || (eq && (exact || __popc(m_eq & below) < ties));
    if (!exact) ties -= min(ties, __popc(m_eq));
    const uint32_t m = __ballot_sync(0xffffffffu, take);
    if (take) out[at + __popc(m & below)] = uint16_t(j);
    at += __popc(m);
  };
  if constexpr (kKeys > 0) {
#pragma unroll
    for (int i = 0; i < kKeys; ++i) emit(i * 32 + lane, k[i]);
  } else {
    for (int j = 0; j < nk; j += 32) emit(j + lane, j + lane < nk ? keys[j + lane] : 0);
  }
}

template <int D, typename T>
cudaError_t launch(const SelectProblem &p, cudaStream_t s) {
  cudaError_t e = launch_dep(k_query_sums<D, T>, dim3(unsigned(1 + int64_t(p.Rg) * p.Hidx)), dim3(kThreads), 0, s, p);
  if (e != cudaSuccess) return e;
  const int chunks = (p.NB + kScoreBlocks - 1) / kScoreBlocks;
  e = launch_dep(k_scores<D, T>, dim3(unsigned(int64_t(p.Rg) * p.Hidx * chunks)), dim3(kThreads), 0, s, p, chunks);
  if (e != cudaSuccess) return e;
  const dim3 grid(unsigned((int64_t(p.Rg) * p.Hidx + kChooseWarps - 1) / kChooseWarps)), block(32 * kChooseWarps);
  if (p.NB <= 256) return launch_dep(k_choose<8>, grid, block, 0, s, p);
  if (p.NB <= 1024) return launch_dep(k_choose<32>, grid, block, 0, s, p);
  return launch_dep(k_choose<0>, grid, block, 0, s, p);
}

}  // namespace

cudaError_t launch_select_blocks(const SelectProblem &p, cudaStream_t s) {
  if (p.dtype == BSA_BF16)
    return p.D == 64 ? launch<64, __nv_bfloat16>(p, s) : launch<128, __nv_bfloat16>(p, s);
  return p.D == 64 ? launch<64, __half>(p, s) : launch<128, __half>(p, s);
}

}  // namespace bsa
