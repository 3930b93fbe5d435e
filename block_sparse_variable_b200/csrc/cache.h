// cache.h -- the device-side description of the cache operators (block means,
// block selection, few-token attention), shared by their host entry points
// (cache_api.cu) and their kernels.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "bsa_internal.h"

namespace bsa {

// where the tokens of a kv cache are; tensors' strides are kept beside
struct KvWhere {
  int32_t layout, B, N2, BKV;
  int32_t page_size, max_pages, num_pages;
  int64_t Skv, Tkv;
  const int64_t *cu_kv;
  const int32_t *seqused;
  const int32_t *table;
  int64_t bt_s0;
};

struct MeansProblem {
  KvWhere kv;
  int32_t D, NB, dtype;
  const int32_t *first_kv;
  const void *k;
  int64_t k_sb, k_sh, k_st;
  void *means;
  int64_t m_sb, m_sh, m_st;
  uint32_t *status;
};

// an index row whose scores are too close for 32 bits
struct SelectAgain {
  int32_t r, hi, nk;
  int32_t b, i;     // sequence, query block within it
  uint32_t lo, up;  // keys between which blocks are scored again
};

struct SelectProblem {
  KvWhere kv;  // lengths only: no table, no cache
  int32_t q_layout, B, N1, N2, D, g, Hidx, BQ, BKV, NB, W, R, Rg, dtype, causal;
  int64_t Sq, Tq, sink, local;
  const int64_t *cu_q;
  const void *q;
  int64_t q_sb, q_sh, q_st;
  const void *means;
  int64_t m_sb, m_sh, m_st;
  uint16_t *index;
  int64_t ix_s0, ix_s1, ix_s2;
  uint32_t *status;
  int32_t *row_nk;     // [Rg] blocks that the index row may choose from, -1: no such row
  int32_t *row_batch, *row_block;  // [Rg] its sequence, and its query block there
  float *qsum;         // [Hidx][Rg][D] sums of the query rows of a row's block
  float *bound;        // [Hidx][Rg] what bounds their errors (select.cu)
  uint64_t *keys;      // [Hidx][Rg][NB] scores
  uint32_t *again_count;
  SelectAgain *again;  // [Hidx * Rg]
};

// a unit that a decode block begins and others finish: what the join kernel reads
struct DecodeJoin {
  int64_t tok0;          // first query row of the sequence
  int32_t b, hh;         // BNSD sequence (0 when packed), head group
  int32_t t0, first, rows;  // the tile's rows (decode_plan.cuh: DecRows)
  int32_t parts, slot0;  // parts == 0: nothing to join
};

struct DecodeProblem {
  KvWhere kv;
  int32_t q_layout, B, N1, N2, D, g, H, gg, BQ, W, R, dtype, causal;
  int32_t TR;         // query rows of a tile
  int32_t chunk;      // kv tokens of a work unit's step
  int32_t grid;       // blocks of the attention kernel
  int32_t tr_sh, chunk_sh, bq_sh, bkv_sh;  // base-2 logarithms
  int32_t tpb;        // tiles of a query block (sparse)
  uint32_t gg_inv;    // ceil(2^32 / gg), 0 for 1
  int32_t group;      // blocks that take the same chunks for different row tiles
  int32_t tree_words;
  int64_t Sq, Tq;
  float scale_log2;
  const int64_t *cu_q;
  const void *q, *k, *v;
  int64_t q_sb, q_sh, q_st, k_sb, k_sh, k_st, v_sb, v_sh, v_st;
  void *out;
  int64_t o_sb, o_sh, o_st;
  float *lse;
  int64_t l_sb, l_sh, l_st;
  const uint16_t *index;
  int64_t ix_s0, ix_s1, ix_s2;
  const int64_t *tree;
  int64_t t_sb, t_st;
  // workspace
  uint32_t *status;
  uint32_t *flags;    // [grid] each block's flags, joined into status[0]
  DecodeJoin *join;   // [grid]
  float *part_ml;     // [2 * grid][TR][2]  running maximum (log2 units) and sum
  float *part_o;      // [2 * grid][TR][D]  unnormalised output
};

cudaError_t launch_block_means(const MeansProblem &p, cudaStream_t s);
cudaError_t launch_select_blocks(const SelectProblem &p, cudaStream_t s);
cudaError_t launch_decode(const DecodeProblem &p, cudaStream_t s);
cudaError_t launch_decode_tc(const DecodeProblem &p, cudaStream_t s);
void decode_tc_plan(DecodeProblem &p);
// fills the tile, step and grid of a problem whose sizes are set; false: too
// large for one call
bool decode_plan(DecodeProblem &p);

#ifdef __CUDACC__
struct KvBatch {
  int32_t kvlen;
  int64_t tok0;
};

// used length and first token row of batch b; contradictory lengths count as 0
__device__ __forceinline__ KvBatch kv_batch(const KvWhere &kv, int b, uint32_t &flags) {
  int64_t st = kv.Skv, tok0 = 0;
  if (kv.cu_kv) {
    const int64_t a = kv.cu_kv[b], e = kv.cu_kv[b + 1];
    const bool bad = a < 0 || e < a || e > kv.Tkv;
    if (bad) flags |= BSA_FLAG_BAD_SEQLEN;
    st = bad ? 0 : e - a;
    tok0 = bad ? 0 : a;
  }
  int64_t len = st;
  if (kv.seqused) {
    len = kv.seqused[b];
    if (len < 0 || len > st) { flags |= BSA_FLAG_BAD_SEQLEN; len = 0; }
  }
  return {int32_t(len), tok0};
}

// page of kv token u, or -1 when the table entry names none (0 unless paged)
__device__ __forceinline__ int kv_page_of(const KvWhere &kv, int b, int u) {
  if (!kv.table) return 0;
  const int pg = kv.table[int64_t(b) * kv.bt_s0 + u / kv.page_size];
  return (pg < 0 || pg >= kv.num_pages) ? -1 : pg;
}

// element offset of kv token u (head h) given its page
__device__ __forceinline__ int64_t kv_off(const KvWhere &kv, int64_t sb, int64_t sh, int64_t st,
                                          const KvBatch &kb, int b, int h, int u, int page) {
  if (kv.table) return int64_t(page) * sb + int64_t(u % kv.page_size) * st + int64_t(h) * sh;
  return int64_t(b) * sb + (kb.tok0 + u) * st + int64_t(h) * sh;
}

struct QBatch {
  int32_t qlen;
  int64_t tok0;
};
__device__ __forceinline__ QBatch q_batch(const int64_t *cu_q, int64_t Sq, int64_t Tq, int b,
                                          uint32_t &flags) {
  if (!cu_q) return {int32_t(Sq), 0};
  const int64_t a = cu_q[b], e = cu_q[b + 1];
  if (a < 0 || e < a || e > Tq) { flags |= BSA_FLAG_BAD_SEQLEN; return {0, 0}; }
  return {int32_t(e - a), a};
}
#endif

}  // namespace bsa
