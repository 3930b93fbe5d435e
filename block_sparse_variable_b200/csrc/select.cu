// select.cu -- the block index from scores of query blocks against block means.
//
// Math: for index head hi, query block i and kv block j of one sequence
//     s(hi,i,j) = (sum of the block's query rows over the heads of hi) . means[b,h2,j]
// and the row keeps the W blocks of the highest s (ties: the lower id),
// forced blocks first, written in ascending order and padded with 0xFFFF.
//
// The outcome is a set of whole numbers, so it must be that of exact scores: two
// blocks whose scores differ in the 10th digit are ordered by their scores and
// not by the order of a sum.  Scores are first computed in 32 bits with a bound
// on their error.  With tau the W-th highest of them and e the bound for the
// row, a block above tau + 2 e is one of the W best and one below tau - 2 e is
// not; nearly always that leaves no other block than the W-th itself, and the
// row is done.  Else the blocks in between are scored again in 64 bits.  (With
// all scores in 64 bits the conversions and additions bound the kernels: 45 us
// for the query sums and 27 us for the scores of a 32768-token prompt of 24
// heads, 41 us for one token of 64 sequences.)
//
// Error of a score: an element of the row sum Q is a sum of n values in chains of
// at most `depth` fp32 additions, the product with m one of at most kDotDepth.
// By Cauchy-Schwarz, over the rows and over the elements,
//     |s32 - s| <= 2^-24 |m| (depth sqrt(n) |q|_F + kDotDepth |Q|)
// with |.| the Euclidean norms, |q|_F that of all n x D query elements.  (With
// maxima in the place of norms, and plain chains, the bound was fifty times as
// wide and half of the rows were scored twice.)
//
// Prompts (many query rows): k_query_sums reads q once (memory bound),
// k_scores_tile multiplies 16 index rows by 128 block means.  A few tokens per
// sequence: k_scores_few sums the rows itself and streams the means (memory
// bound).  Then k_choose (a warp per index row) and k_choose_again, or for long
// rows k_choose_wide (a block per index row), pick.
#include <cuda_runtime.h>

#include "cache.h"
#include "cp_async.cuh"
#include "f32x2.cuh"
#include "launch.cuh"
#include "line.h"
#include "pack16.cuh"

namespace bsa {
namespace {

constexpr int kThreads = 256;
constexpr float kStep = 0x1p-24f;  // half a step of fp32, relative

// the additions that an element of a score goes through: 16 products in a chain,
// then the sums of four such, two halves and eight lanes at most
constexpr int kDotDepth = 24;
// squares below the normal numbers count as this much of a norm per element
constexpr float kTinyNorm = 0x1p-74f;

__device__ __forceinline__ float2 zero2() { return make_float2(0.f, 0.f); }

// a score as a whole number of the same order; NaN below every number
__device__ __forceinline__ uint32_t order32(float s) {
  if (s != s) return 1;
  const uint32_t x = __float_as_uint(s + 0.f);  // -0 and 0 tie
  return x >> 31 ? ~x : x | 0x80000000u;
}
__device__ __forceinline__ float value32(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k); }
__device__ __forceinline__ uint64_t order64(double s) {
  if (s != s) return 1;
  const uint64_t x = uint64_t(__double_as_longlong(s + 0.0));
  return x >> 63 ? ~x : x | (1ull << 63);
}
constexpr uint64_t kTaken = ~0ull;  // above every score

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

// the batch and query block of global index row r, by the whole block (sums of
// rows stop at a number that no row has: overlapping sequences can have more)
__device__ Row find_row(const SelectProblem &p, int r) {
  __shared__ uint32_t s_warp[kThreads / 32];
  __shared__ Row s_row;
  uint32_t ignore = 0;
  if (!p.cu_q) return {r / p.R, r % p.R, int(p.Sq), 0};
  const int tid = threadIdx.x, lane = tid & 31;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  uint32_t mine = 0;
  for (int b = b0; b < b1; ++b) mine = rows_add(mine, uint32_t((q_batch(p.cu_q, p.Sq, p.Tq, b, ignore).qlen + p.BQ - 1) / p.BQ));
  uint32_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc = rows_add(inc, x);
  }
  uint32_t before = __shfl_up_sync(0xffffffffu, inc, 1);
  if (lane == 0) before = 0;
  if (lane == 31) s_warp[tid >> 5] = inc;
  if (tid == 0) s_row.b = -1;
  __syncthreads();
  for (int w = 0; w < (tid >> 5); ++w) before = rows_add(before, s_warp[w]);
  if (uint32_t(r) >= before && uint32_t(r) - before < mine) {
    for (int b = b0; b < b1; ++b) {
      const QBatch qb = q_batch(p.cu_q, p.Sq, p.Tq, b, ignore);
      const uint32_t nq = uint32_t((qb.qlen + p.BQ - 1) / p.BQ);
      if (uint32_t(r) - before < nq) {
        s_row = {b, r - int(before), qb.qlen, qb.tok0};
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
    if (threadIdx.x == 0) *p.again_count = 0;
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

// first query row of (row, index head)
template <typename T>
__device__ __forceinline__ const T *q_of(const SelectProblem &p, const Row &row, int hi) {
  return static_cast<const T *>(p.q) + (p.cu_q ? 0 : int64_t(row.b) * p.q_sb) +
         (row.q0 + int64_t(row.i) * p.BQ) * p.q_st + int64_t(hi) * (p.N1 / p.Hidx) * p.q_sh;
}

// a place in the sequence of steps of k_query_sums: 128 tokens of one head
struct SumStep {
  uint32_t item;
  int r, hi, g, t;
  Row row;  // b < 0: past the last query block
};
__device__ __forceinline__ int row_tokens(const SelectProblem &p, const Row &w) { return min(p.BQ, w.qlen - w.i * p.BQ); }
__device__ __forceinline__ bool step_next(const SelectProblem &p, SumStep &s, uint32_t end) {  // true: the item is done
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

// sum over the block's warps of one row's elements: element tid < D (the
// others get 0), and the squares that its threads summed
template <int D>
struct SumRed {
  float v[kThreads / 32][D];
  float sq[kThreads / 32];
};
static_assert(kThreads / 32 == 8, "the sum of eight warps is a tree");
template <int D>
__device__ __forceinline__ float row_sum(float2 (&acc)[4], float2 sq2, SumRed<D> &red, float &squares) {
  constexpr int kLanes = D / 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
#pragma unroll
  for (int o = kLanes; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[i].x += __shfl_xor_sync(0xffffffffu, acc[i].x, o);
      acc[i].y += __shfl_xor_sync(0xffffffffu, acc[i].y, o);
    }
  if (lane < kLanes)
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<float2 *>(&red.v[warp][lane * 8 + 2 * i]) = acc[i];
  float sq = sq2.x + sq2.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
  if (lane == 0) red.sq[warp] = sq;
  __syncthreads();
  float a = 0.f;
  if (tid < D)
    a = ((red.v[0][tid] + red.v[1][tid]) + (red.v[2][tid] + red.v[3][tid])) +
        ((red.v[4][tid] + red.v[5][tid]) + (red.v[6][tid] + red.v[7][tid]));
  squares = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) squares += red.sq[w];
  return a;
}
// the first term of a row's bound, over n query rows; chain: additions of a
// thread (and 8 more to the whole sum; adding zeros rounds nothing)
template <int D>
__device__ __forceinline__ float sum_bound(int chain, int n, float squares) {
  return kStep * float(min(chain + 8, n)) * sqrtf(float(n)) * (sqrtf(squares) + float(n) * float(D) * kTinyNorm);
}

// Sums of the query rows of (index row, index head) items, a run of items per
// block.  Each of the eight warps takes 16 of a step's 128 tokens through its
// own ring of cp.async stages.
template <int D>
struct SumSmem {
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kStage = 16 * D * 2;
  static constexpr int kRed = kThreads / 32 * kStages * kStage;  // two, in turn
  static constexpr int kBytes = kRed + 2 * int(sizeof(SumRed<D>));
};
template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 2) k_query_sums(const SelectProblem p) {
  using S = SumSmem<D>;
  constexpr int kLanes = D / 8, kSub = 32 / kLanes, kLoads = 16 / kSub;  // pieces of a row, rows a load, loads a step
  extern __shared__ __align__(128) unsigned char smem[];
  SumRed<D> *red = reinterpret_cast<SumRed<D> *>(smem + S::kRed);
  griddep_wait();
  griddep_launch_next();
  if (blockIdx.x == 0) return check_inputs(p);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, col = lane % kLanes, sub = lane / kLanes;
  // (32 bits, which the host has checked: a 64-bit division takes some 500 clocks)
  const uint32_t items = uint32_t(p.Rg) * uint32_t(p.Hidx), blocks = gridDim.x - 1, c = blockIdx.x - 1;
  const uint32_t each = items / blocks, extra = items % blocks;
  const uint32_t lo = c * each + min(c, extra), end = lo + each + (c < extra ? 1u : 0u);
  if (lo >= end) return;
  SumStep at{lo, int(lo / uint32_t(p.Hidx)), int(lo % uint32_t(p.Hidx)), 0, 0, {}};
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
  float2 acc[4], sq = zero2();
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = zero2();
  int s = 0, chain = 0, turn = 0;
  while (at.item < end && at.row.b >= 0) {
    cp_wait<S::kStages - 2>();  // this lane's own copies: it reads no others
    const unsigned char *src = smem + warp * S::kStages * S::kStage + s * S::kStage + lane * 16;
    uint4 x[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) x[i] = *reinterpret_cast<const uint4 *>(src + i * 512);
#pragma unroll
    for (int c = 0; c < 4; ++c) {  // a tree over the step's rows, then one addition
      float2 v[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        v[i] = Pack2<T>::unpack(reinterpret_cast<const uint32_t *>(&x[i])[c]);
        sq = fma2(v[i], v[i], sq);
      }
#pragma unroll
      for (int o = 1; o < kLoads; o <<= 1)
#pragma unroll
        for (int i = 0; i < kLoads; i += 2 * o) v[i] = add2(v[i], v[i + o]);
      acc[c] = add2(acc[c], v[0]);
    }
    ++chain;
    s = s + 1 == S::kStages ? 0 : s + 1;
    issue(s + S::kStages - 2 >= S::kStages ? s - 2 : s + S::kStages - 2);
    const SumStep now = at;
    if (step_next(p, at, end)) {
      float squares;
      const float a = row_sum<D>(acc, sq, red[turn], squares);
      const int64_t row = int64_t(now.hi) * p.Rg + now.r;
      if (tid < D) p.qsum[row * D + tid] = a;
      if (tid == 0) {
        p.bound[row] = sum_bound<D>(chain, row_tokens(p, now.row) * (p.N1 / p.Hidx), squares);
        if (now.hi == 0) {
          p.row_nk[now.r] = candidates(p, now.row);
          p.row_batch[now.r] = now.row.b;
          p.row_block[now.r] = now.row.i;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = zero2();
      sq = zero2();
      chain = 0;
      turn ^= 1;
    }
  }
  cp_wait<0>();
}

// a score and the square of its mean's norm
__device__ __forceinline__ uint64_t score_key(float s, float2 sq) {
  return uint64_t(order32(s)) << 32 | __float_as_uint(sq.x + sq.y);
}

// A few query rows per sequence.  The runs of 128 kv blocks of all (index row,
// index head) units form one line, ordered by row and head, with a place more
// at the start of each unit for what its query rows cost, and each thread block
// takes an equal part of it.  It sums the query rows of a unit and scores its
// runs, eight lanes a kv block; the means come through a ring of cp.async
// stages, across units, each lane copying what it reads itself.
constexpr int kFewRun = 128;

// a place on the line
struct FewAt {
  uint32_t left;               // places to the end of this thread block's part
  int b, r0, i, hi, pos;       // batch, index rows before it, row within it, head, place in the unit
  int nq, runs, qlen;          // of the batch
  int64_t tok0;
  int nk;                      // of the row
};
// query blocks of batch b and runs of its units (the causal mask shortens rows, not the line)
__device__ __forceinline__ void few_batch(const SelectProblem &p, int b, int &nq, int &runs, int &qlen, int64_t &tok0) {
  uint32_t ignore = 0;
  const QBatch q = q_batch(p.cu_q, p.Sq, p.Tq, b, ignore);
  const int nk = min((kv_batch(p.kv, b, ignore).kvlen + p.BKV - 1) / p.BKV, p.NB);
  nq = (q.qlen + p.BQ - 1) / p.BQ;
  runs = (nk + kFewRun - 1) / kFewRun;
  qlen = q.qlen;
  tok0 = q.tok0;
}
__device__ __forceinline__ Row few_row(const FewAt &a) { return {a.b, a.i, a.qlen, a.tok0}; }
// to the next unit
__device__ __forceinline__ void few_unit(const SelectProblem &p, FewAt &a) {
  a.pos = 0;
  if (++a.hi < p.Hidx) return;
  a.hi = 0;
  if (++a.i >= a.nq) {
    a.i = 0;
    do {
      a.r0 += a.nq;
      if (++a.b >= p.B) { a.left = 0; return; }
      few_batch(p, a.b, a.nq, a.runs, a.qlen, a.tok0);
    } while (a.nq == 0);
  }
  a.nk = a.left > 0 && a.r0 + a.i < p.Rg ? candidates(p, few_row(a)) : 0;
}
__device__ __forceinline__ void few_step(const SelectProblem &p, FewAt &a) {
  --a.left;
  if (++a.pos > a.runs) few_unit(p, a);
}
// to the next place that holds a run; false at the end; `begin` is called where
// a unit begins
template <typename F>
__device__ __forceinline__ bool few_settle(const SelectProblem &p, FewAt &a, F &&begin) {
  while (a.left > 0) {
    if (a.r0 + a.i < p.Rg) {  // else fewer index rows than the lengths need
      if (a.pos == 0) begin();
      else if ((a.pos - 1) * kFewRun < a.nk) return true;
    }
    few_step(p, a);
  }
  return false;
}

template <int D>
struct FewSmem {
  static constexpr int kC = D / 64;             // 16-byte pieces a lane holds of a mean
  static constexpr int kJ = kFewRun / (kThreads / 8);  // kv blocks of a run per group of eight lanes
  static constexpr int kStages = 3;
  static constexpr int kStage = kC * kJ * kThreads * 16;
  static constexpr int kRed = kStages * kStage;
  static constexpr int kQ = kRed + int(sizeof(SumRed<D>));
  static constexpr int kBytes = kQ + D * 4;
};
template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 2) k_scores_few(const SelectProblem p) {
  using S = FewSmem<D>;
  constexpr int kC = S::kC, kJ = S::kJ, kLanes = D / 8, kRows = kThreads / kLanes;
  extern __shared__ __align__(128) unsigned char smem[];
  SumRed<D> &red = *reinterpret_cast<SumRed<D> *>(smem + S::kRed);
  float *s_q = reinterpret_cast<float *>(smem + S::kQ);
  __shared__ uint32_t s_work[kThreads / 32], s_rows[kThreads / 32];
  __shared__ FewAt s_at;
  griddep_wait();
  griddep_launch_next();
  if (blockIdx.x == 0) return check_inputs(p);
  const int tid = threadIdx.x, gg = p.N1 / p.Hidx;
  {
    const int lane = tid & 31, warp = tid >> 5, per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    uint32_t work = 0, rows = 0;
    int nq, runs, qlen;
    int64_t tok0;
    auto places = [&](int b) {  // of the batch's units
      few_batch(p, b, nq, runs, qlen, tok0);
      return line_places(uint64_t(uint32_t(nq) * uint32_t(p.Hidx)) * uint32_t(runs + 1));
    };
    for (int b = b0; b < b1; ++b) {
      work = line_add(work, places(b));
      rows = rows_add(rows, uint32_t(nq));
    }
    uint32_t iw = work, ir = rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, iw, o), y = __shfl_up_sync(0xffffffffu, ir, o);
      if (lane >= o) iw = line_add(iw, x), ir = rows_add(ir, y);
    }
    uint32_t bw = __shfl_up_sync(0xffffffffu, iw, 1), br = __shfl_up_sync(0xffffffffu, ir, 1);
    if (lane == 0) bw = br = 0;
    if (lane == 31) s_work[warp] = iw, s_rows[warp] = ir;
    if (tid == 0) s_at.left = 0;
    __syncthreads();
    uint32_t total = 0, wr = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w == warp) bw = line_add(total, bw), br = rows_add(wr, br);
      total = line_add(total, s_work[w]);
      wr = rows_add(wr, s_rows[w]);
    }
    // The units of the rows that the index has come first: lengths that need
    // more rows, or overlapping ones that pass 32 bits, lose the others.
    total = min(total, line_places(uint64_t(uint32_t(p.Rg) * uint32_t(p.Hidx)) * uint32_t((p.NB + kFewRun - 1) / kFewRun + 1)));
    const LinePart part = line_part(total, gridDim.x - 1, blockIdx.x - 1);
    const uint32_t lo = part.lo, n = part.hi - part.lo;
    if (n > 0 && lo >= bw && lo - bw < work)
      for (int b = b0; b < b1; ++b) {
        const uint32_t here = places(b);
        if (lo - bw < here) {
          const uint32_t unit = (lo - bw) / uint32_t(runs + 1);
          FewAt a{n, b, int(br), int(unit / uint32_t(p.Hidx)), int(unit % uint32_t(p.Hidx)),
                  int((lo - bw) % uint32_t(runs + 1)), nq, runs, qlen, tok0, 0};
          if (a.r0 + a.i < p.Rg) a.nk = candidates(p, few_row(a));
          s_at = a;
          break;
        }
        bw += here;
        br = rows_add(br, uint32_t(nq));
      }
    __syncthreads();
  }
  FewAt at = s_at, ahead = at;
  const int lane = tid & 7, grp = tid >> 3, per_group = p.Hidx / p.N2;
  const uint32_t ring = smem_u32(smem) + uint32_t(tid * 16);
  auto issue = [&](int s) {
    if (few_settle(p, ahead, [] {})) {
      const int j0 = (ahead.pos - 1) * kFewRun + grp;
      const T *m = static_cast<const T *>(p.means) + int64_t(ahead.b) * p.m_sb +
                   int64_t(ahead.hi / per_group) * p.m_sh + int64_t(j0) * p.m_st + lane * 8;
#pragma unroll
      for (int k = 0; k < kJ; ++k) {
        const bool in = j0 + k * (kThreads / 8) < ahead.nk;
        const T *src = in ? m + int64_t(k * (kThreads / 8)) * p.m_st : static_cast<const T *>(p.means);
#pragma unroll
        for (int c = 0; c < kC; ++c)
          cp_async16(ring + uint32_t(s * S::kStage + (k * kC + c) * kThreads * 16), in ? src + c * 64 : src, in);
      }
      few_step(p, ahead);
    }
    cp_commit();
  };
#pragma unroll 1
  for (int s = 0; s < S::kStages - 1; ++s) issue(s);
  float2 q[kC][4];
  uint64_t *keys = nullptr;
  bool fresh = true;  // the row sum of the unit is still to be made
  int s = 0;
  auto begin = [&]() {
    fresh = true;
    if (tid == 0 && at.hi == 0) {
      p.row_nk[at.r0 + at.i] = at.nk;
      p.row_batch[at.r0 + at.i] = at.b;
      p.row_block[at.r0 + at.i] = at.i;
    }
  };
  while (few_settle(p, at, begin)) {
    if (fresh) {
      fresh = false;
      const Row row = few_row(at);
      const T *src = q_of<T>(p, row, at.hi);
      const int all = row_tokens(p, row) * gg, col = tid % kLanes;
      float2 acc[4], sq = zero2();
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = zero2();
#pragma unroll 4
      for (int y = tid / kLanes; y < all; y += kRows) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(src + int64_t(y % gg) * p.q_sh + int64_t(y / gg) * p.q_st + col * 8));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 v = Pack2<T>::unpack(w[c]);
          acc[c] = add2(acc[c], v);
          sq = fma2(v, v, sq);
        }
      }
      float squares;
      const float a = row_sum<D>(acc, sq, red, squares);
      const int64_t at_row = int64_t(at.hi) * p.Rg + at.r0 + at.i;
      if (tid < D) s_q[tid] = a;
      if (at.pos == 1) {  // one thread block has the unit's first run
        if (tid < D) p.qsum[at_row * D + tid] = a;
        if (tid == 0) p.bound[at_row] = sum_bound<D>((all + kRows - 1) / kRows, all, squares);
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) q[c][i] = *reinterpret_cast<const float2 *>(s_q + (c * 8 + lane) * 8 + 2 * i);
      keys = p.keys + at_row * p.NB;
    }
    cp_wait<S::kStages - 2>();  // this lane's own copies
    // lane i of the eight ends with the i-th of four scores and four squares
    float v[2 * kJ];
#pragma unroll
    for (int k = 0; k < kJ; ++k) {
      float2 dot = zero2(), sq = zero2();
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const uint4 x = *reinterpret_cast<const uint4 *>(smem + s * S::kStage + ((k * kC + c) * kThreads + tid) * 16);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = Pack2<T>::unpack(w[i]);
          dot = fma2(q[c][i], f, dot);
          sq = fma2(f, f, sq);
        }
      }
      v[k] = dot.x + dot.y;
      v[kJ + k] = sq.x + sq.y;
    }
    s = s + 1 == S::kStages ? 0 : s + 1;
    issue(s + S::kStages - 2 >= S::kStages ? s - 2 : s + S::kStages - 2);
    static_assert(kJ == 4, "eight values over eight lanes");
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < o; ++i) {
        const float keep = lane & o ? v[i + o] : v[i], give = lane & o ? v[i] : v[i + o];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    const float squares = __shfl_down_sync(0xffffffffu, v[0], 4);
    const int j = (at.pos - 1) * kFewRun + lane * (kThreads / 8) + grp;
    if (lane < kJ && j < at.nk) keys[j] = score_key(v[0], make_float2(squares, 0.f));
    few_step(p, at);
  }
  cp_wait<0>();
}

// 16 index rows of one head against 128 kv blocks: a thread two kv blocks and
// eight rows.  The means are brought to shared memory first (rows padded by 16
// bytes: eight neighbouring blocks in different banks), the row sums are read
// as broadcasts, four elements for eight multiply-adds.  Rows of several
// sequences in a tile are done sequence by sequence.
constexpr int kTileRows = 16, kTileBlocks = 128, kTileThreads = 128, kMyRows = 8;
template <int D>
struct TileSmem {
  static constexpr int kPitch = D * 2 + 16;
  static constexpr int kQ = kTileBlocks * kPitch;
  static constexpr int kBytes = kQ + kTileRows * D * 4;
};
template <int D, typename T>
__global__ void __launch_bounds__(kTileThreads, 4) k_scores_tile(const SelectProblem p, int chunks) {
  using S = TileSmem<D>;
  extern __shared__ __align__(128) unsigned char smem[];
  float4(*s_q)[D / 4] = reinterpret_cast<float4(*)[D / 4]>(smem + S::kQ);
  __shared__ int s_nk[kTileRows], s_b[kTileRows];
  griddep_wait();
  griddep_launch_next();
  const uint32_t id = blockIdx.x / uint32_t(chunks);
  const int j0 = int(blockIdx.x - id * uint32_t(chunks)) * kTileBlocks;
  const int hi = int(id % uint32_t(p.Hidx)), r0 = int(id / uint32_t(p.Hidx)) * kTileRows, tid = threadIdx.x;
  const float4 *qs = reinterpret_cast<const float4 *>(p.qsum + (int64_t(hi) * p.Rg + r0) * D);
#pragma unroll
  for (int k = 0; k < kTileRows * (D / 4) / kTileThreads; ++k) {
    const int i = tid + k * kTileThreads;
    const bool in = r0 + i / (D / 4) < p.Rg;  // (a row of no query block holds anything: nothing uses it)
    cp_async16(smem_u32(&s_q[i / (D / 4)][i % (D / 4)]), in ? qs + i : qs, in);
  }
  cp_commit();
  if (tid < kTileRows) {
    const bool in = r0 + tid < p.Rg;
    const int nk = in ? p.row_nk[r0 + tid] : -1, b = in ? p.row_batch[r0 + tid] : -1;
    s_nk[tid] = nk;
    s_b[tid] = nk < 0 ? -1 : b;
  }
  __syncthreads();
  int most = -1;
#pragma unroll
  for (int i = 0; i < kTileRows; ++i) most = max(most, s_nk[i]);
  if (j0 >= most) return cp_wait<0>();
  const int h2 = hi / (p.Hidx / p.N2), jt = tid & 63, row0 = tid >> 6 << 3;
  for (int first = 0; first < kTileRows;) {
    const int b = s_b[first];
    int end = first + 1, nk = s_nk[first];
    for (; end < kTileRows && s_b[end] == b; ++end) nk = max(nk, s_nk[end]);
    if (b >= 0 && j0 < nk) {
      const T *m = static_cast<const T *>(p.means) + int64_t(b) * p.m_sb + int64_t(h2) * p.m_sh + int64_t(j0) * p.m_st;
      constexpr int kLanes = D / 8, kLoads = kTileBlocks * kLanes / kTileThreads;
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int i = tid + k * kTileThreads, j = i / kLanes, c = i % kLanes;
        const bool in = j0 + j < nk;
        cp_async16(smem_u32(smem) + uint32_t(j * S::kPitch + c * 16),
                   in ? m + int64_t(j) * p.m_st + c * 8 : static_cast<const T *>(p.means), in);
      }
      cp_commit();
      cp_wait<0>();
      __syncthreads();
      if (j0 + (jt & ~31) < nk && row0 < end && row0 + kMyRows > first) {  // whole warps
        const unsigned char *ma = smem + jt * S::kPitch, *mb = ma + 64 * S::kPitch;
        float2 sa[kMyRows], sb[kMyRows];
#pragma unroll
        for (int i = 0; i < kMyRows; ++i) sa[i] = sb[i] = zero2();
        float2 sq_a = zero2(), sq_b = zero2();
#pragma unroll 1
        for (int d0 = 0; d0 < D; d0 += 32) {  // chains of 16 products
          float2 ta[kMyRows], tb[kMyRows];
#pragma unroll
          for (int i = 0; i < kMyRows; ++i) ta[i] = tb[i] = zero2();
#pragma unroll
          for (int d = d0; d < d0 + 32; d += 8) {
            const uint4 xa = *reinterpret_cast<const uint4 *>(ma + d * 2), xb = *reinterpret_cast<const uint4 *>(mb + d * 2);
            const uint32_t wa[4] = {xa.x, xa.y, xa.z, xa.w}, wb[4] = {xb.x, xb.y, xb.z, xb.w};
#pragma unroll
            for (int c = 0; c < 4; c += 2) {
              const float2 a0 = Pack2<T>::unpack(wa[c]), a1 = Pack2<T>::unpack(wa[c + 1]);
              const float2 b0 = Pack2<T>::unpack(wb[c]), b1 = Pack2<T>::unpack(wb[c + 1]);
              sq_a = fma2(a1, a1, fma2(a0, a0, sq_a));
              sq_b = fma2(b1, b1, fma2(b0, b0, sq_b));
#pragma unroll
              for (int i = 0; i < kMyRows; ++i) {
                const float4 q = s_q[row0 + i][d / 4 + c / 2];
                const float2 q0 = {q.x, q.y}, q1 = {q.z, q.w};
                ta[i] = fma2(q1, a1, fma2(q0, a0, ta[i]));
                tb[i] = fma2(q1, b1, fma2(q0, b0, tb[i]));
              }
            }
          }
#pragma unroll
          for (int i = 0; i < kMyRows; ++i) {
            sa[i] = add2(sa[i], ta[i]);
            sb[i] = add2(sb[i], tb[i]);
          }
        }
        const int ja = j0 + jt, jb = ja + 64;
#pragma unroll
        for (int i = 0; i < kMyRows; ++i) {
          const int row = row0 + i;
          if (row < first || row >= end) continue;
          const int n = s_nk[row];
          uint64_t *keys = p.keys + (int64_t(hi) * p.Rg + r0 + row) * p.NB;
          if (ja < n) keys[ja] = score_key(sa[i].x + sa[i].y, sq_a);
          if (jb < n) keys[jb] = score_key(sb[i].x + sb[i].y, sq_b);
        }
      }
      __syncthreads();  // before the next sequence's means
    }
    first = end;
  }
  cp_wait<0>();
}

// ------------------------------------------------------------------- choice
// of a row that is scored again: all its query rows in flight at once (512 of
// them took 256 threads 12 us)
constexpr int kChooseThreads = 1024, kChooseWarps = 32;

static_assert(kChooseWarps == 32, "a lane a warp");
struct ChooseRed {
  uint32_t a[2][kChooseWarps], b[kChooseWarps];
};
// sum over the block; `turn` alternates the words, so that one barrier a sum is enough
__device__ __forceinline__ uint32_t block_sum(ChooseRed &red, int &turn, uint32_t n) {
  n = __reduce_add_sync(0xffffffffu, n);
  if ((threadIdx.x & 31) == 0) red.a[turn][threadIdx.x >> 5] = n;
  __syncthreads();
  n = __reduce_add_sync(0xffffffffu, red.a[turn][threadIdx.x & 31]);
  turn ^= 1;
  return n;
}
// the ids whose flag is set, in order: kChooseThreads blocks a turn
__device__ __forceinline__ void emit(ChooseRed &red, int &turn, bool take, int j, uint16_t *out, int &at) {
  const uint32_t m = __ballot_sync(0xffffffffu, take);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) red.a[turn][warp] = uint32_t(__popc(m));
  __syncthreads();
  const uint32_t n = red.a[turn][lane];
  const int before = int(__reduce_add_sync(0xffffffffu, lane < warp ? n : 0u)), all = int(__reduce_add_sync(0xffffffffu, n));
  turn ^= 1;
  if (take) out[at + before + __popc(m & ((1u << lane) - 1u))] = uint16_t(j);
  at += all;
}

// The `want`-th largest of the keys of some threads: each(f) calls f(key) for
// the keys of this thread, sum(n) adds over the threads, value(key) is a float
// that grows with it.  Brackets the key between thresholds with at least and
// with fewer than `want` keys at or above, and stops at one with `want`.  Two
// steps of three go where the counts say, taken as falling exponentially, as
// they do in the tail of many distributions (8 steps for 61 of 1000 normal
// values; 21 with straight lines, 15 halving), the third half way.  least, most:
// of all keys.  Returns the threshold (which may lie between keys).
template <typename K, typename F, typename S, typename V>
__device__ __forceinline__ K nth_key(K least, K most, uint32_t total, uint32_t want, F &&each, S &&sum, V &&value) {
  K lo = least, hi = most;  // at least `want` keys >= lo; keys > hi are not wanted
  uint32_t n_lo = total, n_hi = 0;
#pragma unroll 1
  for (int step = 0; lo < hi && n_lo != want; ++step) {
    K mid = lo + (hi - lo) / 2 + 1;
    if (step % 3 != 2) {
      const float a = value(lo), top = __log2f(float(n_lo));
      const float f = __fdividef(top - __log2f(float(want)), top - __log2f(float(n_hi) + 0.5f));
      const K at = value.inverse(a + f * (value(hi) - a));
      if (at > lo && at <= hi) mid = at;
    }
    uint32_t n = 0;
    each([&](K x) { n += x >= mid ? 1u : 0u; });
    n = sum(n);
    if (n >= want) lo = mid, n_lo = n;
    else hi = mid - 1, n_hi = n;
  }
  return lo;
}
struct Value32 {
  __device__ float operator()(uint32_t k) const { return value32(k); }
  __device__ uint32_t inverse(float v) const { return order32(v); }
};
struct Value64 {  // interpolates on the keys themselves
  __device__ float operator()(uint64_t k) const { return float(k); }
  __device__ uint64_t inverse(float v) const { return v < 1.8e19f ? uint64_t(v) : ~0ull; }
};

__device__ __forceinline__ uint16_t *index_row(const SelectProblem &p, int r, int hi) {
  if (p.cu_q) return p.index + int64_t(hi) * p.ix_s0 + int64_t(r) * p.ix_s1;
  return p.index + int64_t(r / p.R) * p.ix_s0 + int64_t(hi) * p.ix_s1 + int64_t(r % p.R) * p.ix_s2;
}

// Two 16-bit values as doubles times 2^-kDown, by moving their bits: sign,
// exponent and mantissa go to the top of a double's high word, so subnormals
// and zeros come out exact too.  (A conversion to 64 bits costs several times
// the addition that it feeds: 28 us for a row of 512 query rows against 8.)
// Infinities and NaN come out as numbers: `sticky` looks for them.
template <typename T>
struct Bits;
template <>
struct Bits<__nv_bfloat16> {
  using V = __nv_bfloat162;
  static constexpr int kShift = 3, kMask = int(0x8fffe000u);
  static constexpr double kUp = 0x1p448;  // kUp^2 = 1 / 2^-896
};
template <>
struct Bits<__half> {
  using V = __half2;
  static constexpr int kShift = 6, kMask = int(0x81fffc00u);
  static constexpr double kUp = 0x1p504;
};
template <typename T>
__device__ __forceinline__ double2 scaled64(uint32_t w) {  // arithmetic shifts: the sign stays on top
  return make_double2(__hiloint2double((int(w << 16) >> Bits<T>::kShift) & Bits<T>::kMask, 0),
                      __hiloint2double((int(w) >> Bits<T>::kShift) & Bits<T>::kMask, 0));
}
// m + 0 x: NaN from then on in each half that meets an infinity or a NaN
template <typename T>
__device__ __forceinline__ uint32_t sticky(uint32_t m, uint32_t x) {
  using V = typename Bits<T>::V;
  const uint32_t zero = 0;
  const V r = __hfma2(*reinterpret_cast<const V *>(&x), *reinterpret_cast<const V *>(&zero), *reinterpret_cast<V *>(&m));
  return *reinterpret_cast<const uint32_t *>(&r);
}

constexpr int kClose = 256;  // as many of them as are ranked in shared memory
struct ChooseClose {
  uint64_t key[kClose];
  uint16_t id[kClose];
  bool take[kClose];
};
// A row with 64-bit scores for the blocks whose 32-bit keys lie in [lo, up]:
// those above are taken, those below are not.
template <int D, typename T>
__device__ __forceinline__ void choose_again(const SelectProblem &p, const SelectAgain &a) {
  constexpr int kLanes = D / 8, kRows = kChooseThreads / kLanes, kLoads = 4;
  __shared__ double s_red[kChooseWarps][D], s_q[D];
  __shared__ ChooseClose close;
  __shared__ ChooseRed red;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gg = p.N1 / p.Hidx;
  const int r = a.r, hi = a.hi, nk = a.nk;
  const uint32_t lo = a.lo, up = a.up;
  uint16_t *out = index_row(p, r, hi);
  const uint32_t first = tid < nk ? uint32_t(p.keys[(int64_t(hi) * p.Rg + r) * p.NB + tid] >> 32) : 0u;
  uint32_t ignore = 0;
  Row row{a.b, a.i, 0, 0};
  const QBatch qb = q_batch(p.cu_q, p.Sq, p.Tq, row.b, ignore);
  row.qlen = qb.qlen;
  row.q0 = qb.tok0;
  {
    const int nt = row_tokens(p, row), col = tid % kLanes;
    double acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0;
    uint32_t big = 0;
    const T *q = q_of<T>(p, row, hi) + col * 8;
    const int all = nt * gg;
    auto load = [&](int y) {
      return y < all ? __ldg(reinterpret_cast<const uint4 *>(q + int64_t(y % gg) * p.q_sh + int64_t(y / gg) * p.q_st))
                     : make_uint4(0, 0, 0, 0);
    };
#pragma unroll 1
    for (int y = tid / kLanes; y < all; y += kRows * kLoads) {
      uint4 x[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) x[i] = load(y + i * kRows);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const double2 f = scaled64<T>(w[c]);
          big = sticky<T>(big, w[c]);
          acc[2 * c] += f.x;
          acc[2 * c + 1] += f.y;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = acc[i] * Bits<T>::kUp * Bits<T>::kUp;
    const float2 bad = Pack2<T>::unpack(big);
    if (bad.x != bad.x || bad.y != bad.y) {  // rare: once more with conversions that keep infinities and NaN
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0.0;
#pragma unroll 1
      for (int y = tid / kLanes; y < all; y += kRows) {
        const uint4 x1 = load(y);
        const uint32_t w[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 f = Pack2<T>::unpack(w[c]);
          acc[2 * c] += double(f.x);
          acc[2 * c + 1] += double(f.y);
        }
      }
    }
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    if (lane < kLanes)
#pragma unroll
      for (int i = 0; i < 8; ++i) s_red[warp][lane * 8 + i] = acc[i];
    __syncthreads();
    if (tid < D) {
      double a = 0.0;
#pragma unroll 8
      for (int w = 0; w < kChooseWarps; ++w) a += s_red[w][tid];
      s_q[tid] = a;
    }
  }
  const T *m = static_cast<const T *>(p.means) + int64_t(row.b) * p.m_sb + int64_t(hi / (p.Hidx / p.N2)) * p.m_sh;
  auto score = [&](int j) {  // by a warp
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) s += s_q[lane + 32 * i] * double(float(m[int64_t(j) * p.m_st + lane + 32 * i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return order64(s);
  };
  uint64_t *keys = p.keys + (int64_t(hi) * p.Rg + r) * p.NB;
  auto taken = [&](int j, uint32_t k) { return j < p.sink || j >= nk - p.local || k > up; };
  // (a thread's first key has been requested before the query rows)
  auto key32 = [&](int j) { return j < kChooseThreads ? first : j < nk ? uint32_t(keys[j] >> 32) : 0u; };
  int turn = 0;
  uint32_t n_taken = 0, n_close = 0;
  for (int j = tid; j < nk; j += kChooseThreads) {
    const uint32_t k = key32(j);
    if (taken(j, k)) ++n_taken;
    else if (k >= lo) ++n_close;
  }
  n_taken = block_sum(red, turn, n_taken);
  n_close = block_sum(red, turn, n_close);
  const uint32_t want = uint32_t(p.W) - n_taken;
  int at = 0;
  if (n_close <= uint32_t(kClose)) {
    // the usual case: a handful, ranked by comparing each with all
    for (int j0 = 0; j0 < nk; j0 += kChooseThreads) {
      const int j = j0 + tid;
      const uint32_t k = key32(j);
      emit(red, turn, j < nk && k >= lo && !taken(j, k), j, close.id, at);
    }
    __syncthreads();
    for (uint32_t i = warp; i < n_close; i += kChooseWarps) {
      const uint64_t k = score(close.id[i]);
      if (lane == 0) close.key[i] = k;
    }
    __syncthreads();
    for (uint32_t i = tid; i < n_close; i += kChooseThreads) {
      const uint64_t mine = close.key[i];
      uint32_t ahead = 0;
      for (uint32_t k = 0; k < n_close; ++k) ahead += close.key[k] > mine || (close.key[k] == mine && k < i) ? 1u : 0u;
      close.take[i] = ahead < want;
    }
    __syncthreads();
    at = 0;
    uint32_t seen = 0;
    for (int j0 = 0; j0 < nk; j0 += kChooseThreads) {
      const int j = j0 + tid;
      const uint32_t k = key32(j);
      const bool in = j < nk && taken(j, k), near = j < nk && !in && k >= lo;
      const uint32_t mask = __ballot_sync(0xffffffffu, near);
      if (lane == 0) red.b[warp] = uint32_t(__popc(mask));
      __syncthreads();
      const uint32_t n = red.b[lane];
      const uint32_t before = seen + __reduce_add_sync(0xffffffffu, lane < warp ? n : 0u);
      seen += __reduce_add_sync(0xffffffffu, n);
      emit(red, turn, in || (near && close.take[before + __popc(mask & ((1u << lane) - 1u))]), j, out, at);
    }
    return;
  }
  // many, as with equal means: the 64-bit keys in the workspace, and a search
  for (int j = tid; j < nk; j += kChooseThreads) {
    const uint32_t k = uint32_t(keys[j] >> 32);
    if (taken(j, k)) keys[j] = kTaken;
    else if (k < lo) keys[j] = 0;
  }
  __syncthreads();
  for (int j = warp; j < nk; j += kChooseWarps) {
    const uint64_t k = keys[j];
    if (k == 0 || k == kTaken) continue;  // the whole warp
    const uint64_t s = score(j);
    __syncwarp();
    if (lane == 0) keys[j] = s;
  }
  __syncthreads();
  auto each = [&](auto &&f) {
    for (int j = tid; j < nk; j += kChooseThreads) {
      const uint64_t k = keys[j];
      if (k != 0 && k != kTaken) f(k);
    }
  };
  const uint64_t thr = nth_key<uint64_t>(1, kTaken - 1, n_close, want, each, [&](uint32_t x) { return block_sum(red, turn, x); }, Value64{});
  uint32_t n = 0;
  each([&](uint64_t k) { n += k > thr ? 1u : 0u; });
  uint32_t ties = want - block_sum(red, turn, n);  // of the first at the threshold
  for (int j0 = 0; j0 < nk; j0 += kChooseThreads) {
    const int j = j0 + tid;
    const uint64_t k = j < nk ? keys[j] : 0;
    const bool eq = k != 0 && k == thr;
    const uint32_t m_eq = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) red.b[warp] = uint32_t(__popc(m_eq));
    __syncthreads();
    const uint32_t each_n = red.b[lane], before = __reduce_add_sync(0xffffffffu, lane < warp ? each_n : 0u);
    const uint32_t all = __reduce_add_sync(0xffffffffu, each_n);
    emit(red, turn, k > thr || (eq && before + __popc(m_eq & ((1u << lane) - 1u)) < ties), j, out, at);
    ties -= min(ties, all);
  }
}

// the rows that k_choose listed (in an order that does not matter)
template <int D, typename T>
__global__ void __launch_bounds__(kChooseThreads) k_choose_again(const SelectProblem p) {
  griddep_wait();
  griddep_launch_next();
  // (a grid has at most as many blocks as the list has room: the first entry
  // is read together with their number)
  SelectAgain a = p.again[blockIdx.x];
  const uint32_t n = *p.again_count;
  for (uint32_t i = blockIdx.x; i < n;) {
    choose_again<D, T>(p, a);
    __syncthreads();
    if ((i += gridDim.x) < n) a = p.again[i];
  }
}

// what a row chooses: false when that needs no scores and is written
struct Choice {
  uint16_t *out;
  int nk, b, i, sink, local;
  uint32_t want;  // of the blocks that are not forced
  int64_t row;
};
__device__ __forceinline__ bool choice_begin(const SelectProblem &p, int r, int hi, int tid, int threads, Choice &c) {
  c.nk = p.row_nk[r];
  c.b = p.row_batch[r];
  c.i = p.row_block[r];
  if (c.nk < 0) return false;
  c.out = index_row(p, r, hi);
  const int W = p.W;
  if (c.nk <= W) {
    for (int w = tid; w < W; w += threads) c.out[w] = w < c.nk ? uint16_t(w) : kNoBlock;
    return false;
  }
  c.sink = int(min(p.sink, int64_t(c.nk)));
  c.local = int(min(p.local, int64_t(c.nk - c.sink)));
  if (c.sink + c.local >= W) {  // the first W of the forced
    for (int w = tid; w < W; w += threads) c.out[w] = uint16_t(w < c.sink ? w : c.nk - c.local + (w - c.sink));
    return false;
  }
  c.want = uint32_t(W - c.sink - c.local);
  c.row = int64_t(hi) * p.Rg + r;
  return true;
}
// keys between which 32-bit scores do not decide, around the last one wanted.
// q2, m2: squares of the row sum's norm and of the largest mean's.  False: no
// bound, as something is not finite or a product may have overflowed.
template <int D>
__device__ __forceinline__ bool close_keys(const SelectProblem &p, const Choice &c, uint32_t tau, float q2, float m2,
                                           uint32_t &lo, uint32_t &up) {
  // 2 %: the sums of the bound itself, and its products in fp32
  const float t = value32(tau), norm_m = sqrtf(m2) + float(D) * kTinyNorm, norm_q = sqrtf(q2) + float(D) * kTinyNorm;
  const float err = 1.02f * norm_m * (p.bound[c.row] + kStep * float(kDotDepth) * norm_q) + 0x1p-120f;
  const float reach = 2.f * err + fabsf(t) * 0x1p-21f;
  const bool sure = reach < 1e37f && norm_q * norm_m < 1e37f && tau > 1;
  lo = sure ? order32(t - reach) : 0u;
  up = sure ? order32(t + reach) : ~0u;
  return sure;
}

// Many rows: a warp per (index row, index head), kKeys keys a lane in
// registers; rows that are too close go to the list of k_choose_again.
template <int D, typename T, int kKeys>
__global__ void __launch_bounds__(128) k_choose(const SelectProblem p) {
  griddep_wait();
  griddep_launch_next();
  const int lane = threadIdx.x & 31;
  const uint32_t id = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (id >= uint32_t(p.Rg) * uint32_t(p.Hidx)) return;
  const int r = int(id / uint32_t(p.Hidx)), hi = int(id - uint32_t(r) * uint32_t(p.Hidx));
  Choice c;
  if (!choice_begin(p, r, hi, lane, 32, c)) return;
  const uint64_t *keys = p.keys + c.row * p.NB;
  uint32_t key[kKeys], big = 0;
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {  // 0: forced, or no block
    const int j = i * 32 + lane;
    const uint64_t k = j >= c.sink && j < c.nk - c.local ? keys[j] : 0;
    key[i] = uint32_t(k >> 32);
    big = max(big, uint32_t(k));
  }
  float q2 = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const float q = p.qsum[c.row * D + lane + 32 * i];
    q2 = fmaf(q, q, q2);
  }
  auto each = [&](auto &&f) {  // (no threshold is as low as 0)
#pragma unroll
    for (int i = 0; i < kKeys; ++i) f(key[i]);
  };
  uint32_t least = ~0u, most = 0, n = 0;
  each([&](uint32_t k) { least = min(least, k - 1), most = max(most, k), n += k != 0 ? 1u : 0u; });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) q2 += __shfl_xor_sync(0xffffffffu, q2, o);
  least = __reduce_min_sync(0xffffffffu, least) + 1;
  most = __reduce_max_sync(0xffffffffu, most);
  big = __reduce_max_sync(0xffffffffu, big);
  auto total = [](uint32_t x) { return __reduce_add_sync(0xffffffffu, x); };
  const uint32_t thr = nth_key<uint32_t>(least, most, total(n), c.want, each, total, Value32{});
  uint32_t tau = ~0u;  // the lowest key at or above it
  each([&](uint32_t k) {
    if (k >= thr) tau = min(tau, k);
  });
  tau = __reduce_min_sync(0xffffffffu, tau);
  uint32_t lo, up;
  const bool sure = close_keys<D>(p, c, tau, q2, __uint_as_float(big), lo, up);
  n = 0;
  each([&](uint32_t k) { n += k >= lo ? 1u : 0u; });
  if (!sure || total(n) != c.want) {
    if (lane == 0) p.again[atomicAdd(p.again_count, 1u)] = {r, hi, c.nk, c.b, c.i, lo, up};
    return;
  }
  int at = 0;
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    const int j = i * 32 + lane;
    if (i * 32 >= c.nk) break;
    const bool take = j < c.nk && (j < c.sink || j >= c.nk - c.local || key[i] >= lo);
    const uint32_t m = __ballot_sync(0xffffffffu, take);
    if (take) c.out[at + __popc(m & ((1u << lane) - 1u))] = uint16_t(j);
    at += __popc(m);
  }
}

// Long rows: a block per (index row, index head), which reads the keys in every
// step and also scores again where it has to.
template <int D, typename T>
__global__ void __launch_bounds__(kChooseThreads) k_choose_wide(const SelectProblem p) {
  __shared__ ChooseRed red;
  __shared__ uint32_t s_least[kChooseWarps], s_most[kChooseWarps], s_big[kChooseWarps];
  __shared__ float s_q2[kChooseWarps];
  griddep_wait();
  griddep_launch_next();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hi = int(blockIdx.x % unsigned(p.Hidx)), r = int(blockIdx.x / unsigned(p.Hidx));
  Choice c;
  if (!choice_begin(p, r, hi, tid, kChooseThreads, c)) return;
  const uint64_t *keys = p.keys + c.row * p.NB;
  uint32_t big = 0;
  auto read = [&](int j) {  // 0: forced, or no block
    const uint64_t k = j >= c.sink && j < c.nk - c.local ? keys[j] : 0;
    big = max(big, uint32_t(k));
    return uint32_t(k >> 32);
  };
  const float q = tid < D ? p.qsum[c.row * D + tid] : 0.f;
  auto each = [&](auto &&f) {
#pragma unroll 4
    for (int j = tid; j < c.nk; j += kChooseThreads) {
      const uint32_t k = read(j);
      if (k) f(k);
    }
  };
  uint32_t least = ~0u, most = 0, n = 0;
  each([&](uint32_t k) { least = min(least, k), most = max(most, k), ++n; });
  float q2 = q * q;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) q2 += __shfl_xor_sync(0xffffffffu, q2, o);
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  big = __reduce_max_sync(0xffffffffu, big);
  if (lane == 0) s_least[warp] = least, s_most[warp] = most, s_big[warp] = big, s_q2[warp] = q2;
  int turn = 0;
  n = block_sum(red, turn, n);
  q2 = 0.f;
#pragma unroll
  for (int w = 0; w < kChooseWarps; ++w) q2 += s_q2[w];
  least = __reduce_min_sync(0xffffffffu, s_least[lane]);
  most = __reduce_max_sync(0xffffffffu, s_most[lane]);
  big = __reduce_max_sync(0xffffffffu, s_big[lane]);
  auto total = [&](uint32_t x) { return block_sum(red, turn, x); };
  const uint32_t thr = nth_key<uint32_t>(least, most, n, c.want, each, total, Value32{});
  uint32_t tau = ~0u;  // the lowest key at or above it
  each([&](uint32_t k) {
    if (k >= thr) tau = min(tau, k);
  });
  tau = __reduce_min_sync(0xffffffffu, tau);
  __syncthreads();
  if (lane == 0) s_least[warp] = tau;
  __syncthreads();
  tau = __reduce_min_sync(0xffffffffu, s_least[lane]);
  uint32_t lo, up;
  const bool sure = close_keys<D>(p, c, tau, q2, __uint_as_float(big), lo, up);
  n = 0;
  each([&](uint32_t k) { n += k >= lo ? 1u : 0u; });
  if (!sure || total(n) != c.want) return choose_again<D, T>(p, {r, hi, c.nk, c.b, c.i, lo, up});
  int at = 0;
  for (int j0 = 0; j0 < c.nk; j0 += kChooseThreads) {
    const int j = j0 + tid;
    emit(red, turn, j < c.nk && (j < c.sink || j >= c.nk - c.local || read(j) >= lo), j, c.out, at);
  }
}

template <int D, typename T>
cudaError_t launch(const SelectProblem &p, cudaStream_t s) {
  const int64_t items = int64_t(p.Rg) * p.Hidx;
  cudaError_t e;
  // two blocks an SM, the first of them for the lengths: one more than that
  // would begin when another has ended (3 us later here)
  const int64_t wave = int64_t(num_sms()) * 2 - 1;
  // Up to two query blocks per sequence, in the mean: rows hardly share their
  // block means, so each streams its own, and their sums are a matter of
  // latency.  (32 sequences of 4096 to 16384 tokens, 32 heads, one 128-token
  // block: 34 to 41 us against 78 to 119 by tiles; two blocks 46 to 60 against
  // 65 to 90; three 58 to 79 against 64 to 76; four 70 to 93 against 63 to 79.)
  // Longer query blocks cost the first kernel more, as every thread block that
  // streams a part of a row sums its queries: one block of 1024 tokens of 8 and 32
  // sequences before 16384, 85 against 87 and 121 against 142; two of 8 sequences
  // 134 against 98.
  if (p.Rg <= 2 * int64_t(p.B)) {
    const int64_t runs = items * (p.NB > 0 ? (p.NB + kFewRun - 1) / kFewRun : 1);
    e = cudaFuncSetAttribute(k_scores_few<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, FewSmem<D>::kBytes);
    if (e != cudaSuccess) return e;
    e = launch_dep(k_scores_few<D, T>, dim3(unsigned(1 + (runs < wave ? runs : wave))), dim3(kThreads),
                   FewSmem<D>::kBytes, s, p);
    if (e != cudaSuccess) return e;
  } else {
    e = cudaFuncSetAttribute(k_query_sums<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, SumSmem<D>::kBytes);
    if (e != cudaSuccess) return e;
    e = launch_dep(k_query_sums<D, T>, dim3(unsigned(1 + (items < wave ? items : wave))), dim3(kThreads),
                   SumSmem<D>::kBytes, s, p);
    if (e != cudaSuccess) return e;
    const int chunks = (p.NB + kTileBlocks - 1) / kTileBlocks;
    const int64_t tiles = (int64_t(p.Rg) + kTileRows - 1) / kTileRows;
    if (chunks > 0) {
      e = cudaFuncSetAttribute(k_scores_tile<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, TileSmem<D>::kBytes);
      if (e != cudaSuccess) return e;
      e = launch_dep(k_scores_tile<D, T>, dim3(unsigned(tiles * p.Hidx * chunks)), dim3(kTileThreads),
                     TileSmem<D>::kBytes, s, p, chunks);
      if (e != cudaSuccess) return e;
    }
  }
  if (items == 0) return cudaSuccess;  // the lengths have been checked
  // Up to 1024 blocks a row's keys fit a warp's registers, and no step of its
  // search waits for a barrier: the whole call takes 48 us against 74 for 64
  // single tokens before 1024 blocks, and 82 against 317 for a 32768-token
  // prompt of 24 heads.  Up to 256, eight registers do: 68 us for that prompt.
  // The room of the means decides, not the blocks that a row has (256 there in
  // all three), which only the device knows.
  if (p.NB > 1024) return launch_dep(k_choose_wide<D, T>, dim3(unsigned(items)), dim3(kChooseThreads), 0, s, p);
  const dim3 grid(unsigned((items + 3) / 4));
  e = p.NB <= 256 ? launch_dep(k_choose<D, T, 8>, grid, dim3(128), 0, s, p)
                  : launch_dep(k_choose<D, T, 32>, grid, dim3(128), 0, s, p);
  if (e != cudaSuccess) return e;
  const int64_t blocks = num_sms();
  return launch_dep(k_choose_again<D, T>, dim3(unsigned(items < blocks ? items : blocks)), dim3(kChooseThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_select_blocks(const SelectProblem &p, cudaStream_t s) {
  if (p.dtype == BSA_BF16)
    return p.D == 64 ? launch<64, __nv_bfloat16>(p, s) : launch<128, __nv_bfloat16>(p, s);
  return p.D == 64 ? launch<64, __half>(p, s) : launch<128, __half>(p, s);
}

}  // namespace bsa
