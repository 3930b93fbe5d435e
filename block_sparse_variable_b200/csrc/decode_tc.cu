// decode_tc.cu -- tcgen05 form of the few-token attention for tiles of 128
// query rows (draft trees and chains: tokens times the heads of a group).
//
// Math, division of the work and joining of parts: decode.cu, decode_plan.cuh.
//
// One block per SM.  TMA loads of 128-token chunks of K and V through
// three-stage rings (warps 8 and 10); S = Q K^T issued by warp 11, up to three
// chunks ahead, O += P V by warp 9; two softmax warpgroups that take the chunks
// in turn, a thread a whole row of 128 scores.  O is one accumulator, so a row's
// weights have one reference maximum: the group of a chunk passes it on, as soon
// as it has it, to the group of the next, which may move it again before its own
// weights (a move, to a score more than 2^8 above, rescales O and is rare).
// TMEM: three S / P buffers and O, all 512 columns at D = 128.
//
// Measured on the way (kernel, 768 rows over 16384 .. 32768 tokens): two groups
// on the column halves of one chunk, as in the forward pass, 211 us; an output
// for each group and two S buffers, whose chain S - softmax - P V - S is 4000
// clocks long, 164 to 185 us (the products of 64 columns of S take the tensor
// pipe as long as those of 128).
//
// The rows of a tile are gathered (any number of heads and tokens): the first
// segment's by the softmax threads, the next one's by the warp that issues the
// scores, once those of the segment before are done (by the softmax threads,
// before their epilogue: 113 us instead of 88 for 19 sequences of 2560 tokens
// with 33 nodes and an index row per head, four segments a block).
// Only warp 8, which runs ahead, follows the division of the work and walks
// the index and the block table: it publishes segments and their chunks, 32 at
// a time, in shared memory.  (Under a loaded memory system a dependent load
// costs 2000 to 3000 clocks; with every warp following the plan by itself a
// change of segments took 38000.)  A chunk that reaches the masked tokens or
// the end of the cache gets 64-bit visibility words per row.
//
// Bound by memory up to about 128 rows of a kv head, by the tensor pipe and
// the exponentials above.
#include <cuda.h>
#include <cuda_runtime.h>

#include "cache.h"
#include "cp_async.cuh"
#include "decode_plan.cuh"
#include "f32x2.cuh"
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
constexpr int kKWarp = 8, kPvWarp = 9, kVWarp = 10, kSWarp = 11;
// a row's reference maximum moves once a score passes it by 2^8: weights stay
// below 2^8, and the output is rarely rescaled
constexpr float kSlack = 8.0f;
// blocks side by side; 16 for 16 tiles are no faster (2 x 256 tokens of 8 heads
// before 8192: 82 us one by one, 73 to 74 by four, eight or sixteen; 64 sequences
// of 65 tokens before 8192: 822 one by one, 748 by the rule below).  The mean
// number of tokens decides, which a batch of unequal ones pays for: 63 single
// tokens and a sequence of 4096 before 8192 take 1080 us by the rule and 712 one by
// one, with a sequence of 1024 357 and 276.
constexpr int kMostGroup = 8;
constexpr int kReaders = 11;  // warps that read the chunk lists

// a segment as the reading warps need it
struct SegInfo {
  int b, tok0;            // BNSD sequence (0 when packed), first query row
  int kv_b, kv_tok0, h2;  // where K and V are
  int kvlen, qlen;
  int hh, t0, first, rows;  // decode_plan.cuh: DecSeg, DecRows
  int slot;               // of the workspace; -1: the unit is finished here
};
// up to 32 chunks of a segment, those that hold tokens
struct ChunkList {
  int n, last;  // last: the segment ends with this list; n < 0: no more segments
  int u[32], page[32];
  SegInfo seg;
};

enum : int {
  kBarQFull = 0,       // the first segment's Q: one arrival per softmax thread
  kBarQEmpty = 1,      // the segment's last S has read Q
  kBarKFull = 2,       // + K stage
  kBarKEmpty = 5,      // + K stage
  kBarVFull = 8,       // + V stage
  kBarVEmpty = 11,     // + V stage
  kBarSFull = 14,      // + S buffer
  kBarPFull = 17,      // + 2 S buffer + half (one arrival per warp of the chunk's group)
  kBarSFree = 23,      // + S buffer: the product that read its P is done
  kBarPVDone = 26,     // + chunk & 1
  kBarODone = 28,      // the segment's products are in O (segments with a chunk)
  kBarRef = 29,        // + 4 group + row quarter: the reference after the group's chunk is known
  kBarXchg = 37,       // + row quarter: rendezvous of the warps on the same 32 rows
  kBarListFull = 41,   // + list buffer
  kBarListEmpty = 43,  // + list buffer (one arrival per reading warp)
  kBarDrain = 45,
  kBarDrainS = 46,
  kNumBars = 47
};

template <int D>
struct Layout {
  static constexpr int kBox = 128 * 128;  // 128 rows of 64 columns
  static constexpr int kTileBytes = D / 64 * kBox;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + kTileBytes;
  static constexpr int kV = kK + kStages * kTileBytes;
  static constexpr int kBars = kV + kStages * kTileBytes;
  static constexpr int kRef = kBars + kNumBars * 8;       // [2 groups][128] reference maxima
  static constexpr int kSum = kRef + 2 * 128 * 4;         // [2 groups][128] sums
  static constexpr int kLists = kSum + 2 * 128 * 4;       // [2] ChunkList
  static constexpr int kTmemPtr = kLists + 2 * int(sizeof(ChunkList));
  static constexpr int kAbort = kTmemPtr + 4;
  static constexpr int kBytes = kAbort + 4;
  static_assert(kRef % 8 == 0 && sizeof(DecScratch<kThreads>) <= 2048, "the plan's scratch");
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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
  uint32_t *status = p.flags + blockIdx.x;  // this block's flags
  const uint32_t base = smem_u32(smem_raw);
  const bool aligned = (base & 1023u) == 0;  // swizzled tiles need a 1024-byte aligned base
  const uint32_t sQ = base + L::kQ, sK = base + L::kK, sV = base + L::kV;
  auto bar = [&](int i) { return base + L::kBars + 8u * uint32_t(i); };
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(smem_raw + L::kTmemPtr);
  volatile int *abort = reinterpret_cast<volatile int *>(smem_raw + L::kAbort);
  volatile ChunkList *lists = reinterpret_cast<volatile ChunkList *>(smem_raw + L::kLists);

  // what needs no data comes before the wait for the kernel before this one
  if (tid == 0) {
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
    for (int i = 0; i < kNumBars; ++i) {
      const bool list_empty = i == kBarListEmpty || i == kBarListEmpty + 1;
      const bool weights = i >= kBarPFull && i < kBarPFull + 6, xchg = i >= kBarXchg && i < kBarXchg + 4;
      mbar_init(bar(i), i == kBarQFull ? kSoftmaxThreads : xchg ? 64 : weights ? 4 : list_empty ? kReaders : 1);
    }
    *abort = 0;
    fence_barrier_init();
  }
  griddep_wait();
  // (tensor memory is none of what a block is placed by: taken before the wait,
  // it could be what a block of the kernel before this one still waits for)
  if (warp == kPvWarp && aligned) {
    tmem_alloc(base + L::kTmemPtr, 512);
    tmem_relinquish();
  }
  uint32_t len_flags = 0;
  // (the states' memory serves as scratch here; nothing is in static shared
  // memory, so that the tiles start at the aligned window)
  const DecStart st = dec_start<kThreads>(p, *reinterpret_cast<DecScratch<kThreads> *>(smem_raw + L::kRef), len_flags);
  if (tid == 0) {
    *status = aligned ? 0u : BSA_FLAG_INTERNAL;
    p.join[blockIdx.x] = DecodeJoin{};
    __threadfence();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (len_flags) atomicOr(status, len_flags);
  if (!aligned) return;  // the whole block
  griddep_launch_next();  // the next kernel's blocks find this one's tensor memory taken
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS0 = tmem, tO0 = tmem + 384u;

  uint32_t kv_it = 0, list_it = 0;
  bool ok = true;
  // the list that begins the next segment, or null at the end
  auto next_segment = [&]() -> const volatile ChunkList * {
    const int i = int(list_it & 1u);
    ok = ok && wait_warp(bar(kBarListFull + i), (list_it >> 1) & 1u, abort, status);
    return ok && lists[i].n >= 0 ? lists + i : nullptr;
  };
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

  // piece c of row rr of Q: 128-byte swizzle, the 16-byte piece within a row of
  // 128 bytes xor the row
  auto swizzled = [](int rr, int c) { return (c >> 3) * L::kBox + rr * 128 + (((c & 7) ^ (rr & 7)) << 4); };

  // registers: the softmax threads hold a row of 128 scores (256 x 216 + 128 x
  // 72 = the 384 x 168 of the launch)
  if (warp >= 8) {
    regs_dec<72>();
    if (warp == kKWarp || warp == kVWarp) {
      // --------------------------------------------------- TMA producers
      const bool is_k = warp == kKWarp;
      const CUtensorMap *map = is_k ? &map_k : &map_v;
      const uint32_t ring = is_k ? sK : sV;
      const int full0 = is_k ? kBarKFull : kBarVFull, empty0 = is_k ? kBarKEmpty : kBarVEmpty;
      int armed[kStages] = {-1, -1, -1};
      auto load = [&](int u, int pg, const volatile SegInfo &g) {
        const int s = int(kv_it % kStages);
        const uint32_t ph = (kv_it / kStages) & 1u;
        if (!(ok = wait_warp(bar(empty0 + s), ph ^ 1u, abort, status))) return;
        if (lane == 0) {
          int row, last;  // tile coordinates: (0, row, 0, h2, last)
          if (p.kv.table) { row = u % p.kv.page_size; last = pg; }
          else if (p.kv.cu_kv) { row = g.kv_tok0 + u; last = 0; }
          else { row = u; last = g.kv_b; }
          mbar_expect_tx(bar(full0 + s), L::kTileBytes);
          tma_load_5d(ring + s * L::kTileBytes, map, bar(full0 + s), 0, row, 0, g.h2, last);
        }
        armed[s] = int(ph);
        ++kv_it;
      };
      if (is_k) {
        uint32_t flags = 0;
        DecCursor cursor = cursor_begin(st), here;
        DecBatch d;
        DecSeg seg;
        while (ok && cursor_next(p, st, cursor, d, seg, here)) {
          const DecRows v = dec_rows(p, d, seg.tile);
          const bool whole = seg.cs == 0 && seg.ce == d.chunks;
          const int slot = here.pos == st.lo ? 2 * int(blockIdx.x) : 2 * int(blockIdx.x) + 1;
          if (lane == 0 && seg.cs == 0 && !whole) p.join[blockIdx.x] = dec_join(p, st, here, d, seg, v, slot);
          // the tile's query rows into L2, ahead of their gathering
          for (int r = lane; r < v.rows; r += 32) {
            const int y = v.first + r, z = div_gg(p, y);
            const T *q = static_cast<const T *>(p.q) + (p.cu_q ? 0 : here.b) * p.q_sb +
                         (d.q.tok0 + v.t0 + z) * p.q_st + int64_t(seg.hh * p.gg + y - z * p.gg) * p.q_sh;
            asm volatile("prefetch.global.L2 [%0];\n" ::"l"(q));
            asm volatile("prefetch.global.L2 [%0];\n" ::"l"(q + D - 8));
          }
          DecWalk w = walk_begin(p, here.b, seg.hh, v.irow, here.qoff);
          for (int x = seg.cs & ~31; x < seg.ce && ok; x += 32, ++list_it) {
            const int i = int(list_it & 1u);
            if (!(ok = wait_warp(bar(kBarListEmpty + i), ((list_it >> 1) & 1u) ^ 1u, abort, status))) break;
            volatile ChunkList &list = lists[i];
            int u, pg;
            // (the list's own memory serves for the ids)
            walk_fetch(p, d, here.b, w, x, seg.ce, reinterpret_cast<uint16_t *>(const_cast<int *>(list.u)), lane, u, pg);
            const uint32_t some = __ballot_sync(0xffffffffu, u >= 0 && x + lane >= seg.cs);
            const int n = __popc(some);
            if (some >> lane & 1u) {
              const int at = __popc(some & ((1u << lane) - 1u));
              list.u[at] = u;
              list.page[at] = pg;
            }
            if (lane == 0) {
              list.n = n;
              list.last = x + 32 >= seg.ce;
              volatile SegInfo &g = list.seg;
              g.b = p.cu_q ? 0 : here.b; g.tok0 = int(d.q.tok0);
              g.kv_b = here.b; g.kv_tok0 = int(d.kv.tok0); g.h2 = seg.hh / (p.H / p.N2);
              g.kvlen = d.kv.kvlen; g.qlen = d.q.qlen;
              g.hh = seg.hh; g.t0 = v.t0; g.first = v.first; g.rows = v.rows;
              g.slot = whole ? -1 : slot;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarListFull + i));
            for (int c = 0; c < n && ok; ++c) load(list.u[c], list.page[c], list.seg);
          }
          flags |= w.flags;
        }
        const int i = int(list_it & 1u);
        if (ok && (ok = wait_warp(bar(kBarListEmpty + i), ((list_it >> 1) & 1u) ^ 1u, abort, status))) {
          if (lane == 0) {
            lists[i].n = -1;
            mbar_arrive(bar(kBarListFull + i));
          }
        }
        if (flags) atomicOr(status, flags);
      } else {
        while (const volatile ChunkList *list = next_segment()) {
          SegInfo g{};
          g.kv_b = list->seg.kv_b; g.kv_tok0 = list->seg.kv_tok0; g.h2 = list->seg.h2;
          each_chunk([&](int u, int pg) { load(u, pg, g); });
        }
      }
      if (*abort && lane == 0) {  // let every copy already issued land before the block exits
        for (int s = 0; s < kStages; ++s)
          if (armed[s] >= 0) drain_wait(bar(full0 + s), uint32_t(armed[s]));
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------ MMA issuers
      constexpr uint32_t idS = idesc_f16(BF16, 128, 128, false, false);
      constexpr uint32_t idPV = idesc_f16(BF16, 128, D, false, true);
      const uint64_t dQ = sw128_desc(sQ, 16, 1024);
      const uint64_t dK = sw128_desc(sK, 16, 1024);
      const uint64_t dV = sw128_desc(sV, L::kBox, 1024);
      auto kstep = [](int kk) { return uint64_t((kk >> 2) * (L::kBox >> 4) + (kk & 3) * 2); };
      if (warp == kSWarp) {
        // Q of a segment but the first: while the softmax threads are busy with
        // the last chunks of the one before, whose products have read its Q
        auto gather_q = [&](const volatile SegInfo &g) {
          const int first = g.first, rows = g.rows, h0 = g.hh * p.gg;
          const T *q = static_cast<const T *>(p.q) + g.b * p.q_sb + (int64_t(g.tok0) + g.t0) * p.q_st;
          constexpr int kPieces = D / 8;  // 16-byte pieces of a row
          const int c = lane % kPieces;
#pragma unroll 4
          for (int rr = lane / kPieces; rr < kTile; rr += 32 / kPieces) {
            const int y = first + rr, z = div_gg(p, y);
            const bool in = rr < rows;
            cp_async16(sQ + uint32_t(swizzled(rr, c)),
                       in ? q + int64_t(z) * p.q_st + int64_t(h0 + y - z * p.gg) * p.q_sh + c * 8 : q, in);
          }
          cp_commit();
          cp_wait<0>();
          fence_proxy_async_smem();
          __syncwarp();
        };
        uint32_t q_it = 0;
        for (; const volatile ChunkList *list = next_segment(); ++q_it) {
          if (q_it == 0) {
            if (!(ok = wait_warp(bar(kBarQFull), 0u, abort, status))) break;
          } else {
            if (!(ok = wait_warp(bar(kBarQEmpty), (q_it - 1) & 1u, abort, status))) break;
            gather_q(list->seg);
          }
          each_chunk([&](int, int) {
            const uint32_t t = kv_it, buf = t % 3u;
            const int sg = int(t % kStages);
            if (t >= 3 && !(ok = wait_warp(bar(kBarSFree + buf), (t / 3 - 1) & 1u, abort, status))) return;
            if (!(ok = wait_warp(bar(kBarKFull + sg), (t / kStages) & 1u, abort, status))) return;
            tc_fence_after();
            const uint32_t da = tS0 + buf * 128u;
            const uint64_t ka = dK + uint64_t(sg * (L::kTileBytes >> 4));
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) mma_ss_e(da, dQ + kstep(kk), ka + kstep(kk), idS, kk > 0 ? 1u : 0u);
            mma_commit_e(bar(kBarSFull + buf));
            mma_commit_e(bar(kBarKEmpty + sg));
            ++kv_it;
          });
          if (!ok) break;
          mma_commit_e(bar(kBarQEmpty));
        }
      } else {
        while (next_segment()) {
          uint32_t on = 0;
          each_chunk([&](int, int) {
            const uint32_t t = kv_it, buf = t % 3u;
            const int sg = int(t % kStages);
            if (!(ok = wait_warp(bar(kBarVFull + sg), (t / kStages) & 1u, abort, status))) return;
#pragma unroll 1
            for (uint32_t h = 0; h < 2; ++h) {
              if (!(ok = wait_warp(bar(kBarPFull + 2 * buf + h), (t / 3) & 1u, abort, status))) return;
              tc_fence_after();
              const uint32_t pa = tS0 + buf * 128u + h * 32u;  // 16 kv rows of P are 8 columns, of V 2 KB
              const uint64_t vd = dV + uint64_t(sg * (L::kTileBytes >> 4)) + uint64_t(h * 512u);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                mma_ts_e(tO0, pa + uint32_t(8 * kk), vd + uint64_t(kk * 128), idPV, on);
                on = 1;
              }
            }
            mma_commit_e(bar(kBarPVDone + int(t & 1u)));
            mma_commit_e(bar(kBarVEmpty + sg));
            mma_commit_e(bar(kBarSFree + buf));
            ++kv_it;
          });
          if (!ok) break;
          if (on) mma_commit_e(bar(kBarODone));  // (a segment may have no chunk)
        }
      }
      if (*abort) {  // let issued MMAs finish before TMEM is freed
        const int dr = warp == kSWarp ? kBarDrainS : kBarDrain;
        mma_commit_e(bar(dr));
        if (lane == 0) drain_wait(bar(dr), 0);
      }
      __syncwarp();
    }
  } else {
    // --------------------------------------------- softmax warpgroups
    regs_inc<216>();
    const int wg = warp >> 2;
    const int r = tid & 127;  // tile row = TMEM lane
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tO = tO0 + lane_off;
    volatile float *s_ref = reinterpret_cast<volatile float *>(smem_raw + L::kRef);
    volatile float *s_sum = reinterpret_cast<volatile float *>(smem_raw + L::kSum);
    const int mine_bar = kBarRef + 4 * wg + (warp & 3), other_bar = kBarRef + 4 * (wg ^ 1) + (warp & 3);
    uint32_t x_it = 0, ended = 0, others = 0;  // others: chunks of the other group so far
    auto rendezvous = [&]() {  // the warps that hold the same 32 rows (bounded)
      mbar_arrive(bar(kBarXchg + (warp & 3)));
      ok = wait_warp(bar(kBarXchg + (warp & 3)), x_it & 1u, abort, status);
      ++x_it;
      return ok;
    };
    const volatile ChunkList *list = next_segment();
    if (list) {  // the first segment's Q; all loads of a thread in flight together
      const volatile SegInfo &g = list->seg;
      const int first = g.first, rows = g.rows, h0 = g.hh * p.gg;
      const T *q = static_cast<const T *>(p.q) + g.b * p.q_sb + (int64_t(g.tok0) + g.t0) * p.q_st;
      constexpr int kPieces = D / 8;
      constexpr int kRounds = kTile * kPieces / kSoftmaxThreads;
      const int c = tid % kPieces;
      uint4 x[kRounds];
#pragma unroll
      for (int i = 0; i < kRounds; ++i) {
        const int rr = tid / kPieces + i * (kSoftmaxThreads / kPieces), y = first + rr, z = div_gg(p, y);
        x[i] = make_uint4(0, 0, 0, 0);
        if (rr < rows)
          x[i] = __ldg(reinterpret_cast<const uint4 *>(q + int64_t(z) * p.q_st + int64_t(h0 + y - z * p.gg) * p.q_sh) + c);
      }
#pragma unroll
      for (int i = 0; i < kRounds; ++i)
        *reinterpret_cast<uint4 *>(smem_raw + L::kQ + swizzled(tid / kPieces + i * (kSoftmaxThreads / kPieces), c)) = x[i];
      fence_proxy_async_smem();
      mbar_arrive(bar(kBarQFull));
    }
    while (ok && list) {
      const volatile SegInfo &g = list->seg;  // read before the list is given back
      const int kvlen = g.kvlen, qbase = kvlen - g.qlen, qb = g.b, slot = g.slot;
      const bool live = r < g.rows;
      const int xr = g.first + min(r, g.rows - 1);
      const int z = div_gg(p, xr), tq = g.t0 + z, row = g.tok0 + tq, head = g.hh * p.gg + xr - z * p.gg;
      const int64_t *bits = p.tree ? p.tree + qb * p.t_sb + int64_t(row) * p.t_st : nullptr;
      // the columns [u, u + 64) that the row sees
      auto visible = [&](int u) {
        uint64_t m = low_bits(int64_t(kvlen) - u);
        if (p.tree) m &= tree_bits(p, bits, u - qbase);
        else if (p.causal) m &= low_bits(int64_t(tq) + qbase - u + 1);
        return m;
      };
      const int edge_from = (p.tree || p.causal) ? qbase : kvlen;  // first token that some row may not see
      // m: the reference after the last chunk that this thread knows of; l: the
      // sum of this group's weights against it
      float m = -INFINITY, l = 0.f;
      int n = 0;  // chunks of the segment so far
      // the reference as the other group has left it
      auto take_reference = [&]() {
        if (!(ok = wait_warp(bar(other_bar), (others - 1) & 1u, abort, status))) return;
        if (n > 0) {
          const float now = s_ref[(wg ^ 1) * 128 + r];
          if (now != m) {
            if (l != 0.f) l *= ex2(m - now);
            m = now;
          }
        }
      };
      each_chunk([&](const int u0c, int) {
        const uint32_t t = kv_it++, buf = t % 3u;
        if (int(t & 1u) != wg) {
          ++others;
          ++n;
          return;
        }
        if (!(ok = wait_warp(bar(kBarSFull + buf), (t / 3) & 1u, abort, status))) return;
        tc_fence_after();
        const uint32_t tS = tS0 + buf * 128u + lane_off;
        uint32_t x[128];
        tmem_ld_cols<128>(tS, x);
        const int valid_all = kvlen - u0c;
        if (valid_all < 128) {
          // rows past the used length may hold anything: their weights are 0,
          // and their V is made 0 as well before P is published
          const int sg = int(t % kStages);
          if (!(ok = wait_warp(bar(kBarVFull + sg), (t / kStages) & 1u, abort, status))) return;
          uint4 *vt = reinterpret_cast<uint4 *>(smem_raw + L::kV + sg * L::kTileBytes);
          const int per_half = (128 - valid_all) * 8;
          for (int w = r; w < per_half * (D / 64); w += 128) {
            const int h = w / per_half, y = w % per_half;
            vt[h * (L::kBox / 16) + valid_all * 8 + y] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tmem_wait_ld();
        if (u0c + kChunk > edge_from) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint64_t vis = visible(u0c + 64 * h);
            const uint32_t lo = uint32_t(vis), hi = uint32_t(vis >> 32);
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (!((c < 32 ? lo : hi) & (1u << (c & 31)))) x[64 * h + c] = __float_as_uint(-INFINITY);
          }
        }
        float pm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 128; c += 2)
          pm[(c >> 1) & 3] = max3(pm[(c >> 1) & 3], __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
        const float cm = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])) * p.scale_log2;
        if (others > 0) {
          take_reference();
          if (!ok) return;
        }
        const bool move = cm > m + kSlack;  // (true for a first finite maximum)
        const float before = m;
        if (move) m = cm;
        s_ref[wg * 128 + r] = m;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(mine_bar));
        if (__any_sync(0xffffffffu, move)) {
          const float alpha = move ? ex2(before - m) : 1.f;
          l *= alpha;
          if (n > 0) {  // every product before must be in O
            const uint32_t k = t - 1;
            if (!(ok = wait_warp(bar(kBarPVDone + int(k & 1u)), (k / 2) & 1u, abort, status))) return;
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < D / 32; ++j) {
              uint32_t o[32];
              tmem_ld32(tO + uint32_t(32 * j), o);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
              tmem_st32(tO + uint32_t(32 * j), o);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;  // nothing seen yet: every weight is 0
        float2 ps[2] = {{0.f, 0.f}, {0.f, 0.f}};
        const float2 sc = {p.scale_log2, p.scale_log2}, mm = {-ref, -ref};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 a = fma2(make_float2(__uint_as_float(x[32 * h + c]), __uint_as_float(x[32 * h + c + 1])), sc, mm);
            const float2 e = {ex2(a.x), ex2(a.y)};
            ps[(c >> 1) & 1] = add2(ps[(c >> 1) & 1], e);
            // rounded to the inputs' type for the product, as in the forward
            // pass (its sum is not): the product takes one type, and a second
            // one with the remainders would be half as much again for the
            // tensor pipe.  Outputs of 32-node trees differ from exact ones by
            // 0.0023 of their norm, of which the rounding of out makes 0.0017.
            pk[c >> 1] = Pack2<T>::pack(e.x, e.y);
          }
          tmem_st16(tS + uint32_t(16 * h), pk);  // the whole row of S is in registers
          if (h & 1) {  // the products of the first 64 tokens begin half way
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarPFull + 2 * int(buf) + (h >> 1)));
          }
        }
        l += (ps[0].x + ps[0].y) + (ps[1].x + ps[1].y);
        ++n;
      });
      if (!ok) break;
      // the other group's chunk may have been the last
      if (n > 0 && int((kv_it - 1) & 1u) != wg) take_reference();
      if (!ok) break;
      // ---- epilogue: the finished rows, or this block's part of them; group
      // w writes half of the columns, divided by both groups' sums
      if (n > 0) {
        if (!(ok = wait_warp(bar(kBarODone), ended & 1u, abort, status))) break;
        ++ended;
      }
      s_sum[wg * 128 + r] = l;
      if (!rendezvous()) break;
      tc_fence_after();
      const float lsum = s_sum[r] + s_sum[128 + r], mx = m;
      float o[D / 2];
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        uint32_t a[32];
        tmem_ld32(tO + uint32_t(wg * (D / 2) + 32 * h), a);
        tmem_wait_ld();
        // (no chunk, or nothing seen: there may be no output at all)
#pragma unroll
        for (int c = 0; c < 32; ++c) o[32 * h + c] = m != -INFINITY ? __uint_as_float(a[c]) : 0.f;
      }
      tc_fence_before();
      // the next segment's products write O, and the sums' memory is used again
      if (!rendezvous()) break;
      if (live) {
        if (slot < 0) {
          const bool some = lsum > 0.f || lsum != lsum;
          const float inv = some ? 1.f / lsum : 0.f;
          T *dst = static_cast<T *>(p.out) + qb * p.o_sb + int64_t(row) * p.o_st + int64_t(head) * p.o_sh + wg * (D / 2);
#pragma unroll
          for (int c8 = 0; c8 < D / 16; ++c8) {
            uint4 w;
            w.x = Pack2<T>::pack(o[8 * c8] * inv, o[8 * c8 + 1] * inv);
            w.y = Pack2<T>::pack(o[8 * c8 + 2] * inv, o[8 * c8 + 3] * inv);
            w.z = Pack2<T>::pack(o[8 * c8 + 4] * inv, o[8 * c8 + 5] * inv);
            w.w = Pack2<T>::pack(o[8 * c8 + 6] * inv, o[8 * c8 + 7] * inv);
            reinterpret_cast<uint4 *>(dst)[c8] = w;
          }
          if (wg == 0 && p.lse)
            p.lse[qb * p.l_sb + int64_t(row) * p.l_st + int64_t(head) * p.l_sh] =
                some ? (mx + log2f(lsum)) * 0.6931471805599453f : -INFINITY;
        } else {
          // four columns of all rows side by side: a warp's stores are contiguous
          float4 *dst = reinterpret_cast<float4 *>(p.part_o) + (int64_t(slot) * (D / 4) + wg * (D / 8)) * kTile + r;
#pragma unroll
          for (int c4 = 0; c4 < D / 8; ++c4)
            dst[c4 * kTile] = make_float4(o[4 * c4], o[4 * c4 + 1], o[4 * c4 + 2], o[4 * c4 + 3]);
          if (wg == 0) reinterpret_cast<float2 *>(p.part_ml)[int64_t(slot) * kTile + r] = make_float2(mx, lsum);
        }
      }
      list = next_segment();
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
