// block_means.cu -- means of the keys of every kv block of a cache.
//
// Math: means[b,h,j,:] = (1/n_j) sum k[b,u,h,:] over the tokens u of block j
// that exist (u < kvlen_b, valid page).  One pass over the keys: memory
// bound, one addition per element read, summed in fp32 and rounded once.
//
// One or eight warps per (sequence, kv head, kv block): 16 bytes a thread, D / 8
// threads a row, up to 16 loads of a thread requested before the first is used.
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
    // a thread takes kRun consecutive entries of a sequence, so that the loads
    // of many sequences are in flight together
    constexpr int kRun = 16;
    const int runs = (p.kv.max_pages + kRun - 1) / kRun;
    for (int64_t id = threadIdx.x; id < int64_t(p.kv.B) * runs; id += kThreads) {
      const int b = int(id / runs), run = int(id % runs);
      uint32_t ignore = 0;
      const KvBatch kb = kv_batch(p.kv, b, ignore);
      const int covered = int(min(int64_t(kb.kvlen), int64_t(p.NB) * p.kv.BKV));  // by blocks that are written
      const int used = (covered + p.kv.page_size - 1) / p.kv.page_size;
      const int first = p.first_kv ? max(p.first_kv[b], 0) / p.kv.BKV * p.kv.BKV / p.kv.page_size : 0;
      const int x0 = first + run * kRun, n = min(kRun, used - x0);
      const int32_t *row = p.kv.table + int64_t(b) * p.kv.bt_s0 + x0;
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const int pg = i < n ? row[i] : 0;
        if (i < n && (pg < 0 || pg >= p.kv.num_pages)) f |= BSA_FLAG_BAD_PAGE;
      }
    }
  }
  if (f) atomicOr(&sflags, f);
  __syncthreads();
  if (threadIdx.x < kStWords) p.status[threadIdx.x] = threadIdx.x == kStFlags ? sflags : 0;
}

// volatile: the loads of a batch are issued before the first is used
__device__ __forceinline__ uint4 load16(const void *p) {
  uint4 x;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(p));
  return x;
}

// kWarps warps share the rows of one kv block of one head
template <int D, typename T, int kWarps>
__global__ void __launch_bounds__(kThreads) k_block_means(const MeansProblem p, int slots) {
  constexpr int kLanes = D / 8;                       // threads of a row, 16 bytes each
  constexpr int kRows = kWarps * 32 / kLanes;         // rows of one load
  constexpr int kAll = 128 / kRows;                   // loads of a 128-row chunk
  constexpr int kLoads = kAll < 16 ? kAll : 16;       // in flight together
  __shared__ float red[kThreads / 32][D];
  griddep_wait();
  griddep_launch_next();
  if (blockIdx.x == 0) return check_inputs(p);
  const int tid = threadIdx.x % (32 * kWarps), lane = tid & 31, warp = tid >> 5;
  const int64_t all = int64_t(p.kv.B) * slots * p.kv.N2;
  int64_t id = (int64_t(blockIdx.x) - 1) * (kThreads / 32 / kWarps) + threadIdx.x / (32 * kWarps);
  if (id >= all) return;  // whole warps; with kWarps == 8 whole blocks
  // heads fastest: warps that run together read neighbouring rows
  const int h = int(id % p.kv.N2);
  id /= p.kv.N2;
  const int slot = int(id % slots), b = int(id / slots);
  uint32_t ignore = 0;
  const KvBatch kb = kv_batch(p.kv, b, ignore);
  const int BKV = p.kv.BKV;
  const int j0 = p.first_kv ? max(p.first_kv[b], 0) / BKV : 0;
  const int nk = min((kb.kvlen + BKV - 1) / BKV, p.NB);
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
#pragma unroll 1
      for (int i0 = 0; i0 < kAll; i0 += kLoads) {
        if (i0 * kRows >= here) break;
        uint4 x[kLoads];
        const T *at = src + int64_t(row + i0 * kRows) * p.k_st;
        if (here == 128) {
#pragma unroll
          for (int i = 0; i < kLoads; ++i) x[i] = load16(at + int64_t(i * kRows) * p.k_st);
        } else {
#pragma unroll
          for (int i = 0; i < kLoads; ++i)
            x[i] = row + (i0 + i) * kRows < here ? load16(at + int64_t(i * kRows) * p.k_st) : make_uint4(0, 0, 0, 0);
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
    }
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    const float d = n > 0 ? float(n) : 1.f;  // every page bad: zeros
    T *dst = static_cast<T *>(p.means) + int64_t(b) * p.m_sb + int64_t(h) * p.m_sh + int64_t(j) * p.m_st;
    if constexpr (kWarps == 1) {
      if (lane < kLanes)
        reinterpret_cast<uint4 *>(dst)[col] =
            make_uint4(Pack2<T>::pack(acc[0] / d, acc[1] / d), Pack2<T>::pack(acc[2] / d, acc[3] / d),
                       Pack2<T>::pack(acc[4] / d, acc[5] / d), Pack2<T>::pack(acc[6] / d, acc[7] / d));
    } else {
      if (lane < kLanes)
#pragma unroll
        for (int i = 0; i < 8; ++i) red[warp][col * 8 + i] = acc[i];
      __syncthreads();
      if (tid < D / 2) {
        float a = 0.f, c = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          a += red[w][2 * tid];
          c += red[w][2 * tid + 1];
        }
        reinterpret_cast<uint32_t *>(dst)[tid] = Pack2<T>::pack(a / d, c / d);
      }
      __syncthreads();
    }
  }
}

template <int D, typename T>
cudaError_t launch(const MeansProblem &p, cudaStream_t s) {
  const int64_t pairs = int64_t(p.kv.B) * p.kv.N2, wide = int64_t(num_sms()) * 8;
  // A whole pass gives every kv block a warp (no barrier, 8 KB of loads in
  // flight a warp) once there are eight for each SM; fewer blocks than that,
  // and an append's, get eight warps each, for their latency.  (One against
  // eight warps, D = 128, blocks of 128 tokens: 512 blocks 8.3 and 6.3 us, 1024
  // 11 and 10, 2048 14 and 16.5, 32768 159 and 180; blocks of 1024 tokens: 512
  // 44 and 24, 2048 81 and 83.)  An append's thread blocks stride over the kv
  // blocks that there are.
  if (!p.first_kv && pairs * p.NB >= wide) {
    const int64_t grid = 1 + (pairs * p.NB + kThreads / 32 - 1) / (kThreads / 32);
    return launch_dep(k_block_means<D, T, 1>, dim3(unsigned(grid)), dim3(kThreads), 0, s, p, int(p.NB));
  }
  int64_t slots = p.NB;
  if (p.first_kv) {
    const int64_t want = (wide + pairs - 1) / pairs;
    slots = want < p.NB ? want : p.NB;
  }
  return launch_dep(k_block_means<D, T, 8>, dim3(unsigned(1 + pairs * slots)), dim3(kThreads), 0, s, p, int(slots));
}

}  // namespace

cudaError_t launch_block_means(const MeansProblem &p, cudaStream_t s) {
  if (p.dtype == BSA_BF16)
    return p.D == 64 ? launch<64, __nv_bfloat16>(p, s) : launch<128, __nv_bfloat16>(p, s);
  return p.D == 64 ? launch<64, __half>(p, s) : launch<128, __half>(p, s);
}

}  // namespace bsa
