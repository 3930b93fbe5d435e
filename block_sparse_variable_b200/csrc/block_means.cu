// block_means.cu -- means of the keys of every kv block of a cache.
//
// Math: means[b,h,j,:] = (1/n_j) sum k[b,u,h,:] over the tokens u of block j
// that exist (u < kvlen_b, valid page).  One pass over the keys: memory
// bound, one addition per element read, summed in fp32 and rounded once.
//
// One 256-thread block per (sequence, kv head, kv block): 16 bytes a thread,
// D / 8 threads a row, the rows of a 128-row chunk (one page at most) all
// requested before the first is used.  From first_kv on (an append touches
// the last block or two of each sequence) a sequence gets a few blocks of
// threads that stride over its kv blocks instead of one for every kv block
// it could have.
#include <cuda_runtime.h>

#include "cache.h"
#include "launch.cuh"
#include "pack16.cuh"

namespace bsa {
namespace {

constexpr int kThreads = 256;

// Lengths and page table entries that the blocks to be written cover; one
// block of the grid reads them for the status word.
__device__ void check_inputs(const MeansProblem &p) {
  __shared__ uint32_t sflags;
  if (threadIdx.x == 0) sflags = 0;
  __syncthreads();
  uint32_t f = 0;
  for (int b = threadIdx.x; b < p.kv.B; b += kThreads) {
    const KvBatch kb = kv_batch(p.kv, b, f);
    if (p.first_kv && p.first_kv[b] < 0) f |= BSA_FLAG_BAD_SEQLEN;
    if (kb.kvlen > int64_t(p.NB) * p.kv.BKV) f |= BSA_FLAG_BAD_SEQLEN;
  }
  if (p.kv.table) {
    for (int b = 0; b < p.kv.B; ++b) {
      uint32_t g = 0;
      const KvBatch kb = kv_batch(p.kv, b, g);
      const int first = p.first_kv ? max(p.first_kv[b], 0) / p.kv.BKV * p.kv.BKV : 0;
      for (int64_t u = int64_t(first) / p.kv.page_size + threadIdx.x; u * p.kv.page_size < kb.kvlen; u += kThreads) {
        const int pg = p.kv.table[int64_t(b) * p.kv.bt_s0 + u];
        if (pg < 0 || pg >= p.kv.num_pages) f |= BSA_FLAG_BAD_PAGE;
      }
    }
  }
  if (f) atomicOr(&sflags, f);
  __syncthreads();
  if (threadIdx.x < kStWords) p.status[threadIdx.x] = threadIdx.x == kStFlags ? sflags : 0;
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) k_block_means(const MeansProblem p, int slots) {
  constexpr int kLanes = D / 8;                  // threads of a row, 16 bytes each
  constexpr int kRows = kThreads / kLanes;       // rows in flight per load
  constexpr int kLoads = 128 / kRows;            // loads of a 128-row chunk
  __shared__ float red[kThreads / 32][D];
  griddep_wait();
  griddep_launch_next();
  if (blockIdx.x == 0) return check_inputs(p);
  int64_t id = int64_t(blockIdx.x) - 1;
  // heads fastest: blocks that run together read neighbouring rows
  const int h = int(id % p.kv.N2);
  id /= p.kv.N2;
  const int slot = int(id % slots), b = int(id / slots);
  uint32_t ignore = 0;
  const KvBatch kb = kv_batch(p.kv, b, ignore);
  const int BKV = p.kv.BKV;
  const int j0 = p.first_kv ? max(p.first_kv[b], 0) / BKV : 0;
  const int nk = min((kb.kvlen + BKV - 1) / BKV, p.NB);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int col = tid % kLanes, row = tid / kLanes;
  const T *k = static_cast<const T *>(p.k);
  for (int j = j0 + slot; j < nk; j += slots) {
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    int n = 0;
    const int u_end = min(kb.kvlen - j * BKV, BKV) + j * BKV;
    for (int u0 = j * BKV; u0 < u_end; u0 += 128) {
      const int pg = kv_page_of(p.kv, b, u0);
      if (pg < 0) continue;
      const int here = min(u_end - u0, 128);
      n += here;
      const T *src = k + kv_off(p.kv, p.k_sb, p.k_sh, p.k_st, kb, b, h, u0, pg) + col * 8;
      uint4 x[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = row + i * kRows;
        x[i] = r < here ? __ldg(reinterpret_cast<const uint4 *>(src + int64_t(r) * p.k_st)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 f = Pack2<T>::unpack(w[c]);
          acc[2 * c] += f.x;
          acc[2 * c + 1] += f.y;
        }
      }
    }
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    if (lane < kLanes)
#pragma unroll
      for (int i = 0; i < 8; ++i) red[warp][col * 8 + i] = acc[i];
    __syncthreads();
    if (tid < D / 2) {
      float a = 0.f, c = 0.f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        a += red[w][2 * tid];
        c += red[w][2 * tid + 1];
      }
      const float d = n > 0 ? float(n) : 1.f;  // every page bad: zeros
      T *dst = static_cast<T *>(p.means) + int64_t(b) * p.m_sb + int64_t(h) * p.m_sh + int64_t(j) * p.m_st;
      reinterpret_cast<uint32_t *>(dst)[tid] = Pack2<T>::pack(a / d, c / d);
    }
    __syncthreads();
  }
}

template <int D, typename T>
cudaError_t launch(const MeansProblem &p, cudaStream_t s) {
  // a whole pass gives every kv block its own thread block; from first_kv on
  // about eight thread blocks per SM walk the kv blocks there are
  int64_t slots = p.NB;
  if (p.first_kv) {
    const int64_t want = (int64_t(num_sms()) * 8 + int64_t(p.kv.B) * p.kv.N2 - 1) / (int64_t(p.kv.B) * p.kv.N2);
    slots = want < p.NB ? want : p.NB;
  }
  const int64_t grid = 1 + int64_t(p.kv.B) * p.kv.N2 * slots;
  return launch_dep(k_block_means<D, T>, dim3(unsigned(grid)), dim3(kThreads), 0, s, p, int(slots));
}

}  // namespace

cudaError_t launch_block_means(const MeansProblem &p, cudaStream_t s) {
  if (p.dtype == BSA_BF16)
    return p.D == 64 ? launch<64, __nv_bfloat16>(p, s) : launch<128, __nv_bfloat16>(p, s);
  return p.D == 64 ? launch<64, __half>(p, s) : launch<128, __half>(p, s);
}

}  // namespace bsa
