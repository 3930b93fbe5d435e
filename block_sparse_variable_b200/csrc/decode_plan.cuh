// decode_plan.cuh -- how the few-token attention is divided among the blocks
// of its grid, and the walk over the kv tokens of a unit.
//
// A unit is one tile of query rows (the heads of a kv head's group and the
// query tokens, token-major: they read the same keys) against the kv tokens
// it sees, cut into chunks.  The chunks of all units form one line, ordered
// by sequence, head, tile, and block c of G takes the c-th G-th of it: every
// block has the same number of chunks (within one).  A unit that lies within
// one block is finished there; the parts of one that does not go to the
// workspace and a second kernel joins them.  A block starts at most one part at
// its beginning and one at its end, hence two slots each.
// Where a head has several row tiles, `group` blocks side by side take the
// same chunks for as many tiles, at the same time: the keys and values that
// one of them brings in serve the others from L2 (32 query heads over 4 kv
// heads; 16 sequences of 4096 to 16384 tokens, 2 tiles: 134 us without groups,
// 107 with; 4 of 16384 to 32768, 3 tiles: 105 and 94; 6 tiles: 179 and 154).
// The line then holds the chunks of whole groups, and where a sequence has
// fewer tiles than the group, or a rest, the blocks without a tile pass over
// them: work is even among groups, within a group as the tiles allow.
#pragma once

#include <limits.h>

#include "cache.h"
#include "line.h"
#include "pack16.cuh"

namespace bsa {
namespace {

// Positions on the line are unsigned 32-bit numbers (line.h).  The host refuses
// sizes that could pass them; sequences that overlap, which the host cannot see,
// can: such a line is empty, and the call reports BAD_SEQLEN.
struct DecBatch {
  QBatch q;
  KvBatch kv;
  int nk;         // kv blocks (sparse)
  int tiles;      // row tiles per head
  int passes;     // turns of a group of blocks over them
  int chunks;     // chunks of a unit
  uint32_t work;  // chunks of all units of the batch
  uint32_t rows;  // index rows of the batch
};

__device__ __forceinline__ DecBatch dec_batch(const DecodeProblem &p, int b, uint32_t &flags) {
  DecBatch d;
  d.q = q_batch(p.cu_q, p.Sq, p.Tq, b, flags);
  d.kv = kv_batch(p.kv, b, flags);
  d.nk = (d.kv.kvlen + p.kv.BKV - 1) >> p.bkv_sh;
  const int up = p.TR - 1;
  if (p.index) {  // a tile's rows share an index row: tiles do not cross query blocks
    const int full = d.q.qlen >> p.bq_sh, rem = d.q.qlen & (p.BQ - 1);
    d.tiles = full * p.tpb + ((rem * p.gg + up) >> p.tr_sh);
    d.chunks = max(1, min(p.W, d.nk) << (p.bkv_sh - p.chunk_sh));
  } else {
    d.tiles = (d.q.qlen * p.gg + up) >> p.tr_sh;
    d.chunks = max(1, (d.kv.kvlen + p.chunk - 1) >> p.chunk_sh);
  }
  d.passes = p.group == 1 ? d.tiles : int(unsigned(d.tiles + p.group - 1) / unsigned(p.group));
  d.work = line_places(uint64_t(uint32_t(d.passes) * uint32_t(p.H)) * uint32_t(d.chunks));
  d.rows = uint32_t(d.q.qlen + p.BQ - 1) >> p.bq_sh;
  return d;
}

// where a block of the grid begins and how far it goes
struct DecStart {
  uint32_t lo, hi;        // this group's range
  uint32_t rem;           // first chunk within batch b
  uint32_t each, extra;   // chunks of a group; the first `extra` groups have one more
  int b;                  // batch of the first chunk
  uint32_t qoff;          // index rows of the batches before it
};

template <int kThreads>
struct DecScratch {
  uint32_t work[kThreads / 32], rows[kThreads / 32];
  DecStart start;
};

// by the whole block of kThreads threads; flags: contradictory lengths
template <int kThreads>
__device__ DecStart dec_start(const DecodeProblem &p, DecScratch<kThreads> &sh, uint32_t &flags) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  uint32_t work = 0, rows = 0;
  for (int b = b0; b < b1; ++b) {
    const DecBatch d = dec_batch(p, b, flags);
    work = line_add(work, d.work);
    rows = rows_add(rows, d.rows);
  }
  uint32_t iw = work, ir = rows;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, iw, o), y = __shfl_up_sync(0xffffffffu, ir, o);
    if (lane >= o) iw = line_add(iw, x), ir = rows_add(ir, y);
  }
  // (sums that stop cannot be taken apart again: what is before this thread is
  // what is up to its neighbour)
  uint32_t bw = __shfl_up_sync(0xffffffffu, iw, 1), br = __shfl_up_sync(0xffffffffu, ir, 1);
  if (lane == 0) bw = br = 0;
  if (lane == 31) sh.work[warp] = iw, sh.rows[warp] = ir;
  __syncthreads();
  uint32_t total = 0, wr = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) bw = line_add(total, bw), br = rows_add(wr, br);
    total = line_add(total, sh.work[w]);
    wr = rows_add(wr, sh.rows[w]);
  }
  if (total == kLineOver) {
    flags |= BSA_FLAG_BAD_SEQLEN;
    total = 0;
  }
  const LinePart part = line_part(total, gridDim.x / unsigned(p.group), blockIdx.x / unsigned(p.group));
  if (part.lo < part.hi) {
    if (part.lo >= bw && part.lo - bw < work) {
      uint32_t ignore = 0;
      for (int b = b0; b < b1; ++b) {
        const DecBatch d = dec_batch(p, b, ignore);
        if (part.lo - bw < d.work) {
          sh.start = {part.lo, part.hi, part.lo - bw, part.each, part.extra, b, br};
          break;
        }
        bw += d.work;
        br = rows_add(br, d.rows);
      }
    }
  } else if (tid == 0) {
    sh.start = {part.lo, part.lo, 0, part.each, part.extra, p.B, 0};
  }
  __syncthreads();
  return sh.start;
}

// a block's share of one unit
struct DecSeg {
  int hh, tile, cs, ce;  // head group, row tile, chunks [cs, ce)
};

// y / gg for y < 2^16: the rows of a tile
__device__ __forceinline__ int div_gg(const DecodeProblem &p, int y) {
  return p.gg == 1 ? y : int(__umulhi(unsigned(y), p.gg_inv));
}

// the query rows of a tile
struct DecRows {
  int t0, first, rows;  // row r: token t0 + (first + r) / gg, head hh * gg + (first + r) % gg
  int irow;             // query block within the batch (sparse)
};
__device__ __forceinline__ DecRows dec_rows(const DecodeProblem &p, const DecBatch &d, int tile) {
  DecRows v;
  if (p.index) {
    v.irow = tile / p.tpb;
    v.t0 = v.irow << p.bq_sh;
    int first = (tile - v.irow * p.tpb) << p.tr_sh;
    v.rows = min(p.TR, min(p.BQ, d.q.qlen - v.t0) * p.gg - first);
    const int t = first / p.gg;
    v.t0 += t;
    v.first = first - t * p.gg;
  } else {
    const int x = tile << p.tr_sh;
    v.irow = 0;
    v.t0 = x / p.gg;
    v.first = x - v.t0 * p.gg;
    v.rows = min(p.TR, d.q.qlen * p.gg - x);
  }
  return v;
}

// The chunks of a segment, 32 at a time, one a lane: lane i holds the first
// token of chunk base + i (-1: nothing there) and its page.  Sparse: chunk x
// is chunk x % cpb of the (x / cpb)-th accepted entry of the index row.
struct DecWalk {
  const uint16_t *row;  // index row, null when dense
  int slot, last;       // next slot to look at, highest accepted entry so far
  int taken;            // entries accepted so far
  uint32_t flags;
};

__device__ __forceinline__ DecWalk walk_begin(const DecodeProblem &p, int b, int hh, int irow, uint32_t qoff) {
  DecWalk w{nullptr, 0, -1, 0, 0};
  if (p.index) {
    // fewer index rows than the lengths need: such a row selects nothing
    const uint32_t row = qoff + uint32_t(irow);  // (both below 2^31)
    const bool have = p.cu_q ? row < uint32_t(p.R) : true;
    if (!have) { w.slot = p.W; w.flags = BSA_FLAG_BAD_INDEX; }
    w.row = p.cu_q ? p.index + int64_t(hh) * p.ix_s0 + (have ? int64_t(row) * p.ix_s1 : 0)
                   : p.index + int64_t(b) * p.ix_s0 + int64_t(hh) * p.ix_s1 + int64_t(irow) * p.ix_s2;
  }
  return w;
}

// accept entries up to number `until`, by a converged warp; entry number
// first + i goes to blk[i] (shared memory of the warp)
__device__ __forceinline__ void walk_accept(const DecodeProblem &p, int nk, DecWalk &w, int first, int until,
                                            uint16_t *blk, int lane) {
  while (w.taken < until && w.slot < p.W) {
    const int s = w.slot + lane;
    const int e = s < p.W ? int(w.row[s]) : int(kNoBlock);
    const bool used = e != int(kNoBlock), in = used && e < nk;
    int pre = in ? e : -1;  // inclusive maximum of the entries in range
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre = max(pre, x);
    }
    int before = __shfl_up_sync(0xffffffffu, pre, 1);
    before = max(lane ? before : -1, w.last);
    const bool take = in && e > before;
    const uint32_t m = __ballot_sync(0xffffffffu, take);
    const int room = until - w.taken, rank = __popc(m & ((1u << lane) - 1u));
    // slots past the last entry that is wanted are looked at again next time
    const bool keep = take && rank < room;
    const uint32_t kept = __ballot_sync(0xffffffffu, keep);
    const int n = __popc(kept);
    const int end = n == room ? 32 - __clz(kept) : 32;  // slots consumed
    if (keep && w.taken + rank >= first) blk[w.taken + rank - first] = uint16_t(e);
    if (__any_sync(0xffffffffu, lane < end && used && !take)) w.flags |= BSA_FLAG_BAD_INDEX;
    w.last = max(w.last, __shfl_sync(0xffffffffu, pre, end - 1));
    w.taken += n;
    w.slot += end;
  }
  __syncwarp();
}

// Chunks [x, x + 32) of the unit, one a lane; x is a multiple of 32, so that
// no entry is divided between two fetches.  blk: 32 ids in the warp's shared
// memory.
__device__ __forceinline__ void walk_fetch(const DecodeProblem &p, const DecBatch &d, int b, DecWalk &w, int x,
                                           int ce, uint16_t *blk, int lane, int &u, int &page) {
  u = -1;
  page = 0;
  if (p.index) {
    const int cpb_sh = p.bkv_sh - p.chunk_sh;  // 1 .. 16 chunks a block
    const int first = x >> cpb_sh;
    // the unit's last fetch reads the rest of the row, for its bad entries
    const int until = x + 32 >= d.chunks ? INT_MAX : (x + 32) >> cpb_sh;
    walk_accept(p, d.nk, w, first, until, blk, lane);
    const int e = (x + lane) >> cpb_sh;
    if (x + lane < ce && e < w.taken) u = (int(blk[e - first]) << p.bkv_sh) + (((x + lane) & ((1 << cpb_sh) - 1)) << p.chunk_sh);
    __syncwarp();
  } else if (x + lane < ce) {
    u = (x + lane) << p.chunk_sh;
  }
  if (u >= d.kv.kvlen) u = -1;
  if (u >= 0) {
    page = kv_page_of(p.kv, b, u);
    if (page < 0) { u = -1; w.flags |= BSA_FLAG_BAD_PAGE; }
  }
}

// A block's place on the line: the segment it is at.
struct DecCursor {
  uint32_t pos, rem;  // chunk of the line, chunk within the batch
  int b;
  uint32_t qoff;
};
__device__ __forceinline__ DecCursor cursor_begin(const DecStart &s) { return {s.lo, s.rem, s.b, s.qoff}; }
// the segment at the cursor, which is then moved past it; false at the end
__device__ __forceinline__ bool cursor_next(const DecodeProblem &p, const DecStart &s, DecCursor &c, DecBatch &d,
                                            DecSeg &g, DecCursor &at) {
  while (c.pos < s.hi && c.b < p.B) {
    uint32_t ignore = 0;
    d = dec_batch(p, c.b, ignore);
    if (c.rem >= d.work) {
      c.rem -= d.work;
      c.qoff = rows_add(c.qoff, d.rows);
      ++c.b;
      continue;
    }
    const uint32_t unit = c.rem / uint32_t(d.chunks);
    g.cs = int(c.rem - unit * uint32_t(d.chunks));
    g.ce = int(min(uint32_t(d.chunks), uint32_t(g.cs) + (s.hi - c.pos)));
    g.hh = int(unit / uint32_t(d.passes));
    g.tile = int(unit - uint32_t(g.hh) * uint32_t(d.passes));
    if (p.group > 1) g.tile = g.tile * p.group + int(blockIdx.x % unsigned(p.group));
    at = c;
    c.pos += uint32_t(g.ce - g.cs);
    c.rem += uint32_t(g.ce - g.cs);
    if (g.tile < d.tiles) return true;
  }
  return false;
}

// What the join kernel has to know of a unit that a segment of this block
// begins and does not finish.
__device__ __forceinline__ DecodeJoin dec_join(const DecodeProblem &p, const DecStart &st, const DecCursor &at,
                                               const DecBatch &d, const DecSeg &seg, const DecRows &v, int slot) {
  const int last = int(line_owner(st.each, st.extra, gridDim.x / unsigned(p.group), at.pos + uint32_t(d.chunks - 1)));
  return {d.q.tok0, p.cu_q ? 0 : at.b, seg.hh, v.t0, v.first, v.rows, last - int(blockIdx.x / unsigned(p.group)) + 1, slot};
}

}  // namespace
}  // namespace bsa
