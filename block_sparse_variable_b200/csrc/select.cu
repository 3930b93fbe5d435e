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
// Prompts (many query rows): k_query_sums reads q once (memory bound),
// k_scores_tile multiplies 16 index rows by 128 block means (64-bit multiply-add
// bound), k_choose picks, a warp or a block per index row.  A few tokens per
// sequence: k_scores_few sums the rows itself and streams the means (memory
// bound), then k_choose.
#include <cuda_runtime.h>

#include "cache.h"
#include "cp_async.cuh"
#include "launch.cuh"
#include "pack16.cuh"

namespace bsa {
namespace {

constexpr int kThreads = 256;
constexpr int kFewTokens = 64;  // query rows of an index row, in the mean, for the short path
constexpr uint64_t kForced = ~0ull;  // above every score
constexpr uint32_t kNan16x2 = 0x7fff7fffu;  // two NaN of either type
constexpr uint64_t kNan = 1;         // below every number

// The two 16-bit values of a word as doubles times 2^-896, by moving their
// fp32 bits: the mantissa has at most 10 bits, so all of it stays in the high
// word, and subnormals and zeros come out exact.  Conversions to 64 bits run at
// a fraction of the rate of the additions they feed; this is two or three
// integer operations.  Infinities and NaN come out as numbers: callers look for
// them.
__device__ __forceinline__ double scaled_bits(int fp32_bits) {  // arithmetic shift: the sign stays on top
  return __hiloint2double((fp32_bits >> 3) & int(0x8fffffffu), 0);
}
template <typename T>
__device__ __forceinline__ double2 scaled64(uint32_t w) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    return make_double2(__hiloint2double((int(w << 16) >> 3) & int(0x8fffffffu), 0),
                        __hiloint2double((int(w) >> 3) & int(0x8fffe000u), 0));
  } else {
    const float2 f = Pack2<T>::unpack(w);
    return make_double2(scaled_bits(__float_as_int(f.x)), scaled_bits(__float_as_int(f.y)));
  }
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

// the next row of the same call, by one thread or many alike
__device__ __forceinline__ Row next_row(const SelectProblem &p, Row w, int r) {
  if (!p.cu_q) return {r / p.R, r % p.R, int(p.Sq), 0};
  if (++w.i * p.BQ < w.qlen) return w;
  uint32_t ignore = 0;
  while (++w.b < p.B) {
    const QBatch qb = q_batch(p.cu_q, p.Sq, p.Tq, w.b, ignore);
    if (qb.qlen > 0) return {w.b, 0, qb.qlen, qb.tok0};
  }
  return {-1, 0, 0, 0};
}

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
  // index rows that no query block has
  if (p.cu_q)
    for (int64_t r = int64_t(rows) + threadIdx.x; r < p.Rg; r += kThreads) p.row_nk[r] = -1;
}

// blocks that index row `row` may choose from
__device__ __forceinline__ int candidates(const SelectProblem &p, const Row &row) {
  uint32_t ignore = 0;
  const int kvlen = kv_batch(p.kv, row.b, ignore).kvlen;
  int64_t nk = min((kvlen + p.BKV - 1) / p.BKV, p.NB);
  if (p.causal) {  // those that the query block's last row sees
    const int64_t end = int64_t(min((row.i + 1) * int64_t(p.BQ), int64_t(row.qlen))) - 1 + kvlen - row.qlen;
    const int64_t see = end < 0 ? 0 : end / p.BKV + 1;
    nk = see < nk ? see : nk;
  }
  return int(nk);
}

__device__ __forceinline__ uint4 load16(const void *p) {
  uint4 x;  // volatile: a batch of loads is issued before the first is used
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(p));
  return x;
}

// adds eight 16-bit values, scaled by 2^-896
template <typename T>
__device__ __forceinline__ void add8(const uint4 &x, double (&acc)[8], uint32_t &big) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const double2 f = scaled64<T>(w[c]);
    big = max_abs<T>(big, w[c]);
    acc[2 * c] += f.x;
    acc[2 * c + 1] += f.y;
  }
}

// The sum over the block's warps, times 2^512 of q's scale, as element tid < D
// of the row (the others get 0).  nt tokens of gg heads from q on; called by
// the whole block with its threads' sums.
template <int D, typename T>
__device__ __forceinline__ double row_sum(const SelectProblem &p, const T *q, int nt, int gg, double (&acc)[8],
                                          uint32_t big, double (&red)[kThreads / 32][D]) {
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, col = tid % kLanes;
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = acc[i] * kTwo704 * kTwo704;  // to q * 2^512
  if (not_finite<T>(big)) {  // rare: once more with conversions that keep infinities and NaN
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0;
    for (int g = 0; g < gg; ++g)
      for (int t = tid / kLanes; t < nt; t += kRows) {
        const uint32_t *x =
            reinterpret_cast<const uint32_t *>(q + int64_t(g) * p.q_sh + int64_t(t) * p.q_st + col * 8);
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
  double a = 0.0;
  if (tid < D) {
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) a += red[w][tid];
  }
  return a;
}

// first query row of (row, index head)
template <typename T>
__device__ __forceinline__ const T *q_of(const SelectProblem &p, const Row &row, int hi) {
  return static_cast<const T *>(p.q) + (p.cu_q ? 0 : int64_t(row.b) * p.q_sb) +
         (row.q0 + int64_t(row.i) * p.BQ) * p.q_st + int64_t(hi) * (p.N1 / p.Hidx) * p.q_sh;
}

// a place in the sequence of steps of k_query_sums: 128 tokens of one head
struct SumStep {
  int64_t item;
  int r, hi, g, t;
  Row row;  // b < 0: past the last query block
};
__device__ __forceinline__ int row_tokens(const SelectProblem &p, const Row &w) { return min(p.BQ, w.qlen - w.i * p.BQ); }
__device__ __forceinline__ bool step_next(const SelectProblem &p, SumStep &s, int64_t end) {  // true: the item is done
  if ((s.t += 128) < row_tokens(p, s.row)) return false;
  s.t = 0;
  if (++s.g < p.N1 / p.Hidx) return false;
  s.g = 0;
  ++s.item;
  if (++s.hi >= p.Hidx) {
    s.hi = 0;
    ++s.r;
    if (s.item < end) s.row = next_row(p, s.row, s.r);
  }
  return true;
}

// Sums of the query rows of (index row, index head) items, a run of items per
// block.  Each of the eight warps takes 16 of a step's 128 tokens through its
// own ring of cp.async stages (with the loads in registers, those of the next
// step beside this one's sums spilled).
template <int D, typename T>
struct SumSmem {
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kStage = 16 * D * 2;
  static constexpr int kRed = kThreads / 32 * kStages * kStage;  // [warps][D] doubles
  static constexpr int kBytes = kRed + kThreads / 32 * D * 8;
};
template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 2) k_query_sums(const SelectProblem p) {
  using S = SumSmem<D, T>;
  constexpr int kLanes = D / 8, kSub = 32 / kLanes, kLoads = 16 / kSub;  // pieces of a row, rows a load, loads a step
  extern __shared__ __align__(128) unsigned char smem[];
  double(&red)[kThreads / 32][D] = *reinterpret_cast<double(*)[kThreads / 32][D]>(smem + S::kRed);
  griddep_wait();
  griddep_launch_next();
  if (blockIdx.x == 0) return check_inputs(p);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, col = lane % kLanes, sub = lane / kLanes;
  const int64_t items = int64_t(p.Rg) * p.Hidx, blocks = int64_t(gridDim.x) - 1, c = int64_t(blockIdx.x) - 1;
  const int64_t lo = items * c / blocks, end = items * (c + 1) / blocks;
  if (lo >= end) return;
  SumStep at{lo, int(lo / p.Hidx), int(lo % p.Hidx), 0, 0, {}};
  at.row = find_row(p, at.r);
  SumStep ahead = at;
  const uint32_t ring = smem_u32(smem) + uint32_t(warp * S::kStages * S::kStage + lane * 16);
  auto issue = [&](int s) {
    if (ahead.item < end && ahead.row.b >= 0) {
      const int t0 = ahead.t + 16 * warp, left = row_tokens(p, ahead.row) - t0;
      const T *q = q_of<T>(p, ahead.row, ahead.hi) + int64_t(ahead.g) * p.q_sh + int64_t(t0 + sub) * p.q_st + col * 8;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const bool in = sub + i * kSub < left;  // else zeros, and nothing is read
        cp_async16(ring + uint32_t(s * S::kStage + i * 512), in ? q + int64_t(i * kSub) * p.q_st : static_cast<const T *>(p.q), in);
      }
      step_next(p, ahead, end);
    }
    cp_commit();
  };
#pragma unroll 1
  for (int s = 0; s < S::kStages - 1; ++s) issue(s);
  double acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0;
  uint32_t big = 0;
  int s = 0;
  while (at.item < end && at.row.b >= 0) {
    cp_wait<S::kStages - 2>();  // this lane's own copies: it reads no others
    const unsigned char *src = smem + warp * S::kStages * S::kStage + s * S::kStage + lane * 16;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) add8<T>(*reinterpret_cast<const uint4 *>(src + i * 512), acc, big);
    s = s + 1 == S::kStages ? 0 : s + 1;
    issue(s + S::kStages - 2 >= S::kStages ? s - 2 : s + S::kStages - 2);
    const SumStep now = at;
    if (step_next(p, at, end)) {
      if (now.hi == 0 && tid == 0) {
        p.row_nk[now.r] = candidates(p, now.row);
        p.row_batch[now.r] = now.row.b;
      }
      const T *q = q_of<T>(p, now.row, now.hi);
      const double a = row_sum<D, T>(p, q, row_tokens(p, now.row), p.N1 / p.Hidx, acc,
                                     __syncthreads_or(not_finite<T>(big)) ? kNan16x2 : 0u, red);
      if (tid < D) p.qsum[(int64_t(now.hi) * p.Rg + now.r) * D + tid] = a;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0.0;
      big = 0;
    }
  }
  cp_wait<0>();
}

__device__ __forceinline__ uint64_t order_bits(double s) {
  if (s != s) return kNan;
  const uint64_t x = uint64_t(__double_as_longlong(s + 0.0));  // -0 and 0 tie
  return x >> 63 ? ~x : x | (1ull << 63);
}

// one 16-byte piece of a mean against 8 elements of a row sum
template <typename T>
__device__ __forceinline__ void dot8(const uint4 &x, const double (&q)[8], double &s, uint32_t &big) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const double2 f = scaled64<T>(w[i]);
    big = max_abs<T>(big, w[i]);
    s = fma(q[2 * i], f.x, s);
    s = fma(q[2 * i + 1], f.y, s);
  }
}
// the same with conversions that keep infinities and NaN
template <typename T>
__device__ __forceinline__ double dot8_slow(const uint4 &x, const double (&q)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Pack2<T>::unpack(w[i]);
    s += q[2 * i] * (double(f.x) * kTwoM896) + q[2 * i + 1] * (double(f.y) * kTwoM896);
  }
  return s;
}

// A few query rows per sequence.  The runs of 128 kv blocks of all (index row,
// index head) units form one line, ordered by row and head, and each thread
// block takes an equal part of it: it sums the query rows of a unit and scores
// its runs, eight lanes a kv block.  The means of a unit's first run are
// requested before its query rows, those of the next run before this one's
// products.
constexpr int kFewRun = 128;
struct FewStart {
  uint32_t lo, hi, rem;  // this block's part of the line; its first run within batch b
  int b, r;              // r: index rows before batch b
};
template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 2) k_scores_few(const SelectProblem p) {
  constexpr int kC = D / 64;                     // 16-byte pieces a lane holds of a mean
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
  constexpr int kJ = kFewRun / (kThreads / 8);   // kv blocks of a run per group of eight lanes
  __shared__ double red[kThreads / 32][D], s_q[D];
  __shared__ uint32_t s_work[kThreads / 32];
  __shared__ int s_rows[kThreads / 32];
  __shared__ FewStart s_start;
  griddep_wait();
  griddep_launch_next();
  if (blockIdx.x == 0) return check_inputs(p);
  const int tid = threadIdx.x, gg = p.N1 / p.Hidx;
  uint32_t ignore = 0;
  // runs of one unit and units of batch b
  auto batch = [&](int b, QBatch &q, int &nq, uint32_t &runs) {
    q = q_batch(p.cu_q, p.Sq, p.Tq, b, ignore);
    nq = (q.qlen + p.BQ - 1) / p.BQ;
    const int nk = min((kv_batch(p.kv, b, ignore).kvlen + p.BKV - 1) / p.BKV, p.NB);
    runs = uint32_t(max(1, (nk + kFewRun - 1) / kFewRun));
    return uint32_t(nq) * uint32_t(p.Hidx) * runs;
  };
  {
    const int lane = tid & 31, warp = tid >> 5, per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    uint32_t work = 0, runs;
    int rows = 0, nq;
    QBatch q;
    for (int b = b0; b < b1; ++b) {
      work += batch(b, q, nq, runs);
      rows += nq;
    }
    uint32_t iw = work;
    int ir = rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, iw, o);
      const int y = __shfl_up_sync(0xffffffffu, ir, o);
      if (lane >= o) iw += x, ir += y;
    }
    if (lane == 31) s_work[warp] = iw, s_rows[warp] = ir;
    if (tid == 0) s_start = {0, 0, 0, p.B, 0};
    __syncthreads();
    uint32_t total = 0, bw = iw - work;
    int br = ir - rows;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) bw += s_work[w], br += s_rows[w];
      total += s_work[w];
    }
    const uint32_t blocks = gridDim.x - 1, c = blockIdx.x - 1, each = total / blocks, extra = total % blocks;
    const uint32_t lo = c * each + min(c, extra), hi = lo + each + (c < extra ? 1u : 0u);
    if (lo < hi && lo >= bw && lo - bw < work)
      for (int b = b0; b < b1; ++b) {
        const uint32_t n = batch(b, q, nq, runs);
        if (lo - bw < n) {
          s_start = {lo, hi, lo - bw, b, br};
          break;
        }
        bw += n;
        br += nq;
      }
    __syncthreads();
  }
  FewStart at = s_start;
  const int lane = tid & 7, grp = tid >> 3;
  while (at.lo < at.hi && at.b < p.B) {
    Row row{at.b, 0, 0, 0};
    int nq;
    uint32_t runs;
    QBatch qb;
    const uint32_t n = batch(at.b, qb, nq, runs);
    if (at.rem >= n) {
      at.rem -= n;
      at.r += nq;
      ++at.b;
      continue;
    }
    const uint32_t unit = at.rem / runs, rs = at.rem % runs, re = min(runs, rs + (at.hi - at.lo));
    const int hi = int(unit % uint32_t(p.Hidx));
    row.i = int(unit / uint32_t(p.Hidx));
    row.qlen = qb.qlen;
    row.q0 = qb.tok0;
    const int r = at.r + row.i;
    at.rem += re - rs;
    at.lo += re - rs;
    if (r >= p.Rg) continue;  // fewer index rows than the lengths need
    const int nk = candidates(p, row);
    if (tid == 0 && hi == 0 && rs == 0) p.row_nk[r] = nk;
    const int h2 = hi / (p.Hidx / p.N2), j_end = min(nk, int(re) * kFewRun);
    const T *m = static_cast<const T *>(p.means) + int64_t(row.b) * p.m_sb + int64_t(h2) * p.m_sh + lane * 8;
    uint4 x[kJ][kC];
    auto request = [&](int j0) {
#pragma unroll
      for (int k = 0; k < kJ; ++k) {
        const int j = j0 + k * (kThreads / 8) + grp;
#pragma unroll
        for (int c = 0; c < kC; ++c)
          x[k][c] = j < j_end ? load16(m + int64_t(j) * p.m_st + c * 64) : make_uint4(0, 0, 0, 0);
      }
    };
    int j0 = int(rs) * kFewRun;
    if (j0 >= j_end) continue;
    request(j0);
    {
      const T *q = q_of<T>(p, row, hi);
      const int nt = row_tokens(p, row), all = nt * gg, col = tid % kLanes;
      double acc[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0.0;
      uint32_t big = 0;
      for (int y = tid / kLanes; y < all; y += kRows)
        add8<T>(load16(q + int64_t(y % gg) * p.q_sh + int64_t(y / gg) * p.q_st + col * 8), acc, big);
      const double a = row_sum<D, T>(p, q, nt, gg, acc, __syncthreads_or(not_finite<T>(big)) ? kNan16x2 : 0u, red);
      if (tid < D) s_q[tid] = a;
      __syncthreads();
    }
    double q[kC][8];
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) q[c][i] = s_q[(c * 8 + lane) * 8 + i];
    uint64_t *keys = p.keys + (int64_t(hi) * p.Rg + r) * p.NB;
    for (; j0 < j_end; j0 += kFewRun) {
      double s[kJ];
#pragma unroll
      for (int k = 0; k < kJ; ++k) {
        uint32_t big = 0;
        s[k] = 0.0;
#pragma unroll
        for (int c = 0; c < kC; ++c) dot8<T>(x[k][c], q[c], s[k], big);
        if (not_finite<T>(big)) {
          s[k] = 0.0;
#pragma unroll
          for (int c = 0; c < kC; ++c) s[k] += dot8_slow<T>(x[k][c], q[c]);
        }
      }
      if (j0 + kFewRun < j_end) request(j0 + kFewRun);
#pragma unroll
      for (int k = 0; k < kJ; ++k) {
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
        const int j = j0 + k * (kThreads / 8) + grp;
        if (j < j_end && lane == 0) keys[j] = j < p.sink || j >= nk - p.local ? kForced : order_bits(s[k]);
      }
    }
  }
}

// 16 index rows of one head against 128 kv blocks: a thread two kv blocks and
// all rows.  The row sums are read from shared memory as broadcasts, two
// elements for four multiply-adds.  Rows of several sequences in a tile are
// done sequence by sequence.
constexpr int kTileRows = 16, kTileBlocks = 128, kTileThreads = 64;
template <int D, typename T>
__global__ void __launch_bounds__(kTileThreads) k_scores_tile(const SelectProblem p, int chunks) {
  __shared__ double2 s_q[kTileRows][D / 2];
  __shared__ int s_nk[kTileRows], s_b[kTileRows];
  griddep_wait();
  griddep_launch_next();
  int64_t id = blockIdx.x;
  const int j0 = int(id % chunks) * kTileBlocks;
  id /= chunks;
  const int hi = int(id % p.Hidx), r0 = int(id / p.Hidx) * kTileRows, tid = threadIdx.x;
  if (tid < kTileRows) {
    const int nk = r0 + tid < p.Rg ? p.row_nk[r0 + tid] : -1;
    s_nk[tid] = nk;
    s_b[tid] = nk < 0 ? -1 : p.row_batch[r0 + tid];
  }
  __syncthreads();
  int most = -1;
#pragma unroll
  for (int i = 0; i < kTileRows; ++i) most = max(most, s_nk[i]);
  if (j0 >= most) return;
  const double2 *qs = reinterpret_cast<const double2 *>(p.qsum + (int64_t(hi) * p.Rg + r0) * D);
#pragma unroll
  for (int k = 0; k < kTileRows * (D / 2) / kTileThreads; ++k) {
    const int i = tid + k * kTileThreads;
    s_q[i / (D / 2)][i % (D / 2)] = s_nk[i / (D / 2)] >= 0 ? qs[i] : make_double2(0.0, 0.0);
  }
  __syncthreads();
  const int h2 = hi / (p.Hidx / p.N2);
  for (int first = 0; first < kTileRows;) {
    const int b = s_b[first];
    int end = first + 1, nk = s_nk[first];
    for (; end < kTileRows && s_b[end] == b; ++end) nk = max(nk, s_nk[end]);
    const int ja = j0 + tid, jb = ja + kTileThreads;
    if (b >= 0 && (ja & ~31) < nk) {  // whole warps
      const T *m = static_cast<const T *>(p.means) + int64_t(b) * p.m_sb + int64_t(h2) * p.m_sh;
      const T *ma = m + int64_t(min(ja, nk - 1)) * p.m_st, *mb = m + int64_t(min(jb, nk - 1)) * p.m_st;
      double sa[kTileRows], sb[kTileRows];
#pragma unroll
      for (int i = 0; i < kTileRows; ++i) sa[i] = sb[i] = 0.0;
      uint32_t big = 0;
      uint4 xa = __ldg(reinterpret_cast<const uint4 *>(ma)), xb = __ldg(reinterpret_cast<const uint4 *>(mb));
#pragma unroll 1
      for (int d = 0; d < D; d += 8) {
        const uint32_t wa[4] = {xa.x, xa.y, xa.z, xa.w}, wb[4] = {xb.x, xb.y, xb.z, xb.w};
        if (d + 8 < D) {
          xa = __ldg(reinterpret_cast<const uint4 *>(ma + d + 8));
          xb = __ldg(reinterpret_cast<const uint4 *>(mb + d + 8));
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          big = max_abs<T>(max_abs<T>(big, wa[c]), wb[c]);
          const double2 fa = scaled64<T>(wa[c]), fb = scaled64<T>(wb[c]);
#pragma unroll
          for (int i = 0; i < kTileRows; ++i) {
            const double2 q = s_q[i][d / 2 + c];
            sa[i] = fma(q.x, fa.x, sa[i]);
            sb[i] = fma(q.x, fb.x, sb[i]);
            sa[i] = fma(q.y, fa.y, sa[i]);
            sb[i] = fma(q.y, fb.y, sb[i]);
          }
        }
      }
      if (not_finite<T>(big)) {  // rare: again with conversions that keep infinities and NaN
#pragma unroll 1
        for (int i = 0; i < kTileRows; ++i) {
          double a = 0.0, c = 0.0;
#pragma unroll 1
          for (int d = 0; d < D; ++d) {
            const double2 q2 = s_q[i][d / 2];
            const double q = d & 1 ? q2.y : q2.x;
            a += q * (double(float(ma[d])) * kTwoM896);
            c += q * (double(float(mb[d])) * kTwoM896);
          }
#pragma unroll
          for (int k = 0; k < kTileRows; ++k)
            if (k == i) sa[k] = a, sb[k] = c;
        }
      }
#pragma unroll
      for (int i = 0; i < kTileRows; ++i) {
        if (i < first || i >= end) continue;
        const int n = s_nk[i];
        uint64_t *keys = p.keys + (int64_t(hi) * p.Rg + r0 + i) * p.NB;
        if (ja < n) keys[ja] = ja < p.sink || ja >= n - p.local ? kForced : order_bits(sa[i]);
        if (jb < n) keys[jb] = jb < p.sink || jb >= n - p.local ? kForced : order_bits(sb[i]);
      }
    }
    first = end;
  }
}

// kWarps warps per (index row, index head).  The W-th highest key is found bit
// by bit from the first bit in which the keys differ, each step a count of the
// keys at or above a candidate; a candidate with exactly as many as are wanted
// ends the search.  Forced blocks are set aside first.  kKeys keys a thread
// stay in registers (0: they are read again each step).
template <int kKeys, int kWarps>
__global__ void __launch_bounds__(kWarps == 1 ? 128 : 32 * kWarps) k_choose(const SelectProblem p) {
  constexpr int kSpan = 32 * kWarps;
  __shared__ int s_n[2][kWarps];
  __shared__ uint64_t s_and[kWarps], s_or[kWarps];
  griddep_wait();
  griddep_launch_next();
  const int tid = threadIdx.x % kSpan, lane = tid & 31, warp = tid >> 5;
  const int64_t id = int64_t(blockIdx.x) * (blockDim.x / kSpan) + threadIdx.x / kSpan;
  if (id >= int64_t(p.Rg) * p.Hidx) return;  // whole warps; with several, whole blocks
  const int hi = int(id % p.Hidx), r = int(id / p.Hidx);
  const int nk = p.row_nk[r];
  if (nk < 0) return;
  uint16_t *out;
  if (p.cu_q) out = p.index + int64_t(hi) * p.ix_s0 + int64_t(r) * p.ix_s1;
  else out = p.index + int64_t(r / p.R) * p.ix_s0 + int64_t(hi) * p.ix_s1 + int64_t(r % p.R) * p.ix_s2;
  const int W = p.W;
  if (nk <= W) {
    for (int w = tid; w < W; w += kSpan) out[w] = w < nk ? uint16_t(w) : kNoBlock;
    return;
  }
  const uint64_t *keys = p.keys + (int64_t(hi) * p.Rg + r) * p.NB;
  uint64_t k[kKeys > 0 ? kKeys : 1];
  if constexpr (kKeys > 0) {
#pragma unroll
    for (int i = 0; i < kKeys; ++i) k[i] = i * kSpan + tid < nk ? keys[i * kSpan + tid] : 0;
  }
  // f(block, key) for this thread's blocks
  auto each = [&](auto &&f) {
    if constexpr (kKeys > 0) {
#pragma unroll
      for (int i = 0; i < kKeys; ++i) f(i * kSpan + tid, k[i]);
    } else {
      for (int j = tid; j < nk; j += kSpan) f(j, keys[j]);
    }
  };
  int flip = 0;
  auto sum = [&](int n) {  // over the warps of the row
    n = int(__reduce_add_sync(0xffffffffu, unsigned(n)));
    if constexpr (kWarps > 1) {
      if (lane == 0) s_n[flip][warp] = n;
      __syncthreads();
      n = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) n += s_n[flip][w];
      flip ^= 1;  // the next sum writes the other words
    }
    return n;
  };
  int forced = 0;
  uint64_t all = ~0ull, any = 0;
  each([&](int j, uint64_t x) {
    if (x == kForced) ++forced;
    else if (x != 0) all &= x, any |= x;
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all &= __shfl_xor_sync(0xffffffffu, all, o);
    any |= __shfl_xor_sync(0xffffffffu, any, o);
  }
  if constexpr (kWarps > 1) {
    if (lane == 0) s_and[warp] = all, s_or[warp] = any;  // read after the sum's barrier
  }
  forced = sum(forced);
  if constexpr (kWarps > 1) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) all &= s_and[w], any |= s_or[w];
  }
  const int want = W - forced;  // of the others
  uint64_t thr = kForced;       // want <= 0: the first W of the forced
  int ties = W;
  bool exact = false;
  if (want > 0) {
    const uint64_t diff = all ^ any;
    const int top = diff ? 63 - __clzll((long long)diff) : -1;
    thr = top < 0 ? any : top == 63 ? 0 : any >> (top + 1) << (top + 1);
    for (int bit = top; bit >= 0 && !exact; --bit) {
      const uint64_t cand = thr | (1ull << bit);
      int n = 0;
      each([&](int j, uint64_t x) { n += x >= cand && x != kForced; });
      n = sum(n);
      if (n >= want) thr = cand;
      exact = n == want;
    }
    int n = 0;
    each([&](int j, uint64_t x) { n += x > thr && x != kForced; });
    ties = want - sum(n);
  }
  // all above the threshold and the first `ties` at it, in ascending order
  int at = 0;
  auto emit = [&](int j, uint64_t x) {
    const bool over = x > thr, eq = x == thr && x != 0;
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t m_eq = __ballot_sync(0xffffffffu, eq);
    int eq_before = 0, eq_all = __popc(m_eq);
    if constexpr (kWarps > 1) {
      if (lane == 0) s_n[0][warp] = eq_all;
      __syncthreads();
      eq_all = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) eq_before += s_n[0][w];
        eq_all += s_n[0][w];
      }
    }
    const bool take = over || (eq && eq_before + __popc(m_eq & below) < ties);
    ties -= min(max(ties, 0), eq_all);
    const uint32_t m = __ballot_sync(0xffffffffu, take);
    int before = 0, n = __popc(m);
    if constexpr (kWarps > 1) {
      if (lane == 0) s_n[1][warp] = n;
      __syncthreads();
      n = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_n[1][w];
        n += s_n[1][w];
      }
    }
    if (take) out[at + before + __popc(m & below)] = uint16_t(j);
    at += n;
  };
  if constexpr (kWarps > 1) __syncthreads();  // the last sum's words have been read
  if constexpr (kKeys > 0) {
#pragma unroll
    for (int i = 0; i < kKeys; ++i) emit(i * kSpan + tid, k[i]);
  } else {
    for (int j = 0; j < nk; j += kSpan) emit(j + tid, j + tid < nk ? keys[j + tid] : 0);
  }
}

template <int D, typename T>
cudaError_t launch(const SelectProblem &p, cudaStream_t s) {
  const int64_t items = int64_t(p.Rg) * p.Hidx;
  cudaError_t e;
  // few query rows per index row, in the mean: their sums are a matter of
  // latency, and an index row has its means to itself
  const int64_t tokens = p.cu_q ? p.Tq : p.Sq * p.B;
  if (tokens * (p.N1 / p.Hidx) <= int64_t(p.Rg) * kFewTokens) {
    const int64_t runs = items * (p.NB > 0 ? (p.NB + kFewRun - 1) / kFewRun : 1), wave = int64_t(num_sms()) * 2;
    e = launch_dep(k_scores_few<D, T>, dim3(unsigned(1 + (runs < wave ? runs : wave))), dim3(kThreads), 0, s, p);
    if (e != cudaSuccess) return e;
  } else {
    const int64_t blocks = int64_t(num_sms()) * 2;
    e = cudaFuncSetAttribute(k_query_sums<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, SumSmem<D, T>::kBytes);
    if (e != cudaSuccess) return e;
    e = launch_dep(k_query_sums<D, T>, dim3(unsigned(1 + (items < blocks ? items : blocks))), dim3(kThreads),
                   SumSmem<D, T>::kBytes, s, p);
    if (e != cudaSuccess) return e;
    const int chunks = (p.NB + kTileBlocks - 1) / kTileBlocks;
    const int64_t tiles = (int64_t(p.Rg) + kTileRows - 1) / kTileRows;
    if (chunks > 0) {
      e = launch_dep(k_scores_tile<D, T>, dim3(unsigned(tiles * p.Hidx * chunks)), dim3(kTileThreads), 0, s, p, chunks);
      if (e != cudaSuccess) return e;
    }
  }
  // up to 256 blocks a warp a row; above, eight warps, whose steps are short
  if (p.NB <= 256) return launch_dep(k_choose<8, 1>, dim3(unsigned((items + 3) / 4)), dim3(128), 0, s, p);
  if (p.NB <= 1024) return launch_dep(k_choose<4, 8>, dim3(unsigned(items)), dim3(256), 0, s, p);
  return launch_dep(k_choose<0, 8>, dim3(unsigned(items)), dim3(256), 0, s, p);
}

}  // namespace

cudaError_t launch_select_blocks(const SelectProblem &p, cudaStream_t s) {
  if (p.dtype == BSA_BF16)
    return p.D == 64 ? launch<64, __nv_bfloat16>(p, s) : launch<128, __nv_bfloat16>(p, s);
  return p.D == 64 ? launch<64, __half>(p, s) : launch<128, __half>(p, s);
}

}  // namespace bsa
