// cache_api.cu -- host side of the cache operators of the C ABI: block means,
// block selection and few-token attention.  Same two-phase form as the
// attention passes: every descriptor is validated on both calls, data values
// are checked on the device.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "args.h"
#include "cache.h"

namespace {

using namespace bsa;

constexpr int64_t kMaxLen = int64_t(1) << 30;  // kv or query tokens of one sequence
constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 2;

bool dtype16(int dt) { return dt == BSA_F16 || dt == BSA_BF16; }

// layouts and block shape of params, as the attention passes accept them
bsa_status check_params(const bsa_params &P) {
  const int ql = P.q_layout, kl = P.kv_layout;
  if (!((ql == BSA_LAYOUT_BNSD && kl == BSA_LAYOUT_BNSD) ||
        (ql == BSA_LAYOUT_TND && (kl == BSA_LAYOUT_TND || kl == BSA_LAYOUT_PA_BBND))))
    return BSA_ERR_PARAM_INVALID;
  if (!block_ok(P.block_shape[0]) || !block_ok(P.block_shape[1])) return BSA_ERR_PARAM_INVALID;
  if (P.mask_type != BSA_MASK_NONE && P.mask_type != BSA_MASK_CAUSAL) return BSA_ERR_PARAM_INVALID;
  return BSA_OK;
}

// Lengths of B kv sequences.  stored: rows of a BNSD cache (paged: ignored).
bsa_status kv_lengths(const bsa_tensor *cu_kv, const bsa_tensor *seqused, const bsa_params &P, int64_t B,
                      KvWhere &kv) {
  if (P.kv_layout == BSA_LAYOUT_TND) {
    if (!present(cu_kv)) return BSA_ERR_NULLPTR;
    if (!vec_ok(cu_kv, BSA_I64, B + 1)) return BSA_ERR_PARAM_INVALID;
    kv.cu_kv = static_cast<const int64_t *>(cu_kv->data);
  } else if (present(cu_kv)) {
    return BSA_ERR_PARAM_INVALID;
  }
  if (P.kv_layout == BSA_LAYOUT_PA_BBND && !present(seqused)) return BSA_ERR_NULLPTR;
  if (present(seqused)) {
    if (!vec_ok(seqused, BSA_I32, B)) return BSA_ERR_PARAM_INVALID;
    kv.seqused = static_cast<const int32_t *>(seqused->data);
  }
  kv.layout = P.kv_layout;
  kv.B = int32_t(B);
  kv.BKV = int32_t(P.block_shape[1]);
  return BSA_OK;
}

// A k or v cache of B sequences and N2 heads in params' layout, with its
// lengths and block table.
bsa_status kv_cache(const bsa_tensor *k, const bsa_tensor *cu_kv, const bsa_tensor *seqused, const bsa_tensor *bt,
                    const bsa_params &P, int64_t B, int64_t N2, KvWhere &kv) {
  bsa_status st = kv_lengths(cu_kv, seqused, P, B, kv);
  if (st != BSA_OK) return st;
  kv.N2 = int32_t(N2);
  if (P.kv_layout == BSA_LAYOUT_BNSD) {
    if (k->shape[0] != B || k->shape[1] != N2) return BSA_ERR_PARAM_INVALID;
    kv.Skv = k->shape[2];
    if (kv.Skv >= kMaxLen) return BSA_ERR_UNSUPPORTED;
  } else if (P.kv_layout == BSA_LAYOUT_TND) {
    if (k->shape[1] != N2) return BSA_ERR_PARAM_INVALID;
    kv.Tkv = k->shape[0];
    if (kv.Tkv >= kMaxLen) return BSA_ERR_UNSUPPORTED;
  } else {
    if (!present(bt)) return BSA_ERR_NULLPTR;
    if (k->shape[2] != N2) return BSA_ERR_PARAM_INVALID;
    const int64_t page = k->shape[1];
    if (page <= 0 || page % 128 != 0) return BSA_ERR_UNSUPPORTED;
    if (bt->ndim != 2 || bt->dtype != BSA_I32 || bt->shape[0] != B || bt->shape[1] < 1 ||
        (bt->shape[1] > 1 && bt->stride[1] != 1) || bt->stride[0] < 0 || !aligned_to(bt, 4))
      return BSA_ERR_PARAM_INVALID;
    if (k->shape[0] >= kMaxLen || page >= kMaxLen || bt->shape[1] >= kMaxLen / page) return BSA_ERR_UNSUPPORTED;
    kv.page_size = int32_t(page);
    kv.max_pages = int32_t(bt->shape[1]);
    kv.num_pages = int32_t(k->shape[0]);
    kv.table = static_cast<const int32_t *>(bt->data);
    kv.bt_s0 = bt->stride[0];
    kv.Skv = bt->shape[1] * page;
  }
  if (P.kv_layout != BSA_LAYOUT_PA_BBND && present(bt)) return BSA_ERR_PARAM_INVALID;
  return BSA_OK;
}

void kv_strides(const bsa_tensor *t, int layout, int64_t &sb, int64_t &sh, int64_t &st) {
  if (layout == BSA_LAYOUT_BNSD) { sb = t->stride[0]; sh = t->stride[1]; st = t->stride[2]; }
  else if (layout == BSA_LAYOUT_TND) { sb = 0; st = t->stride[0]; sh = t->stride[1]; }
  else { sb = t->stride[0]; st = t->stride[1]; sh = t->stride[2]; }
}

void q_strides(const bsa_tensor *t, int layout, int64_t &sb, int64_t &sh, int64_t &st) {
  if (layout == BSA_LAYOUT_BNSD) { sb = t->stride[0]; sh = t->stride[1]; st = t->stride[2]; }
  else { sb = 0; st = t->stride[0]; sh = t->stride[1]; }
}

// q of params' layout: batches, tokens and heads
bsa_status check_q(const bsa_tensor *q, const bsa_tensor *cu_q, const bsa_params &P, int64_t &B, int64_t &Sq,
                   int64_t &Tq, int64_t &N2, int64_t &D) {
  const int nd = P.q_layout == BSA_LAYOUT_BNSD ? 4 : 3;
  if (q->dtype == BSA_F8E4M3) return BSA_ERR_UNSUPPORTED;  // 16-bit inputs
  if (!dtype16(q->dtype)) return BSA_ERR_PARAM_INVALID;
  bsa_status st = check_values(q, nd, q->dtype);
  if (st != BSA_OK) return st;
  D = q->shape[nd - 1];
  const int64_t N1 = q->shape[1];
  N2 = P.num_kv_heads == 0 ? P.num_heads : P.num_kv_heads;
  if (P.num_heads != N1 || N2 <= 0 || N1 % N2 != 0) return BSA_ERR_PARAM_INVALID;
  if (D != 64 && D != 128) return BSA_ERR_UNSUPPORTED;
  if (P.q_layout == BSA_LAYOUT_BNSD) {
    if (present(cu_q)) return BSA_ERR_PARAM_INVALID;
    B = q->shape[0];
    Sq = q->shape[2];
    Tq = 0;
  } else {
    if (!present(cu_q)) return BSA_ERR_NULLPTR;
    if (cu_q->ndim != 1 || cu_q->shape[0] < 1) return BSA_ERR_PARAM_INVALID;
    B = cu_q->shape[0] - 1;
    if (!vec_ok(cu_q, BSA_I64, B + 1)) return BSA_ERR_PARAM_INVALID;
    Sq = 0;
    Tq = q->shape[0];
  }
  if (B >= kMaxLen || (Sq + Tq) * N1 >= kMaxLen || B * Sq >= kMaxLen) return BSA_ERR_UNSUPPORTED;
  return BSA_OK;
}

// an index of params' layout over B sequences: its heads, rows per sequence
// (BNSD) or in all (TND), and width
bsa_status check_index(const bsa_tensor *ix, const bsa_params &P, int64_t B, int64_t Sq, int64_t N1, int64_t N2,
                       int64_t &H, int64_t &R, int64_t &W) {
  if (ix->dtype != BSA_U16 || !aligned_to(ix, 2)) return BSA_ERR_PARAM_INVALID;
  if (P.q_layout == BSA_LAYOUT_BNSD) {
    if (ix->ndim != 4 || ix->shape[0] != B || ix->shape[2] != cdiv(Sq, P.block_shape[0]))
      return BSA_ERR_PARAM_INVALID;
  } else if (ix->ndim != 3) {
    return BSA_ERR_PARAM_INVALID;
  }
  const int n = ix->ndim;
  H = ix->shape[n - 3];
  R = ix->shape[n - 2];
  W = ix->shape[n - 1];
  if (H != N1 && H != N2) return BSA_ERR_PARAM_INVALID;
  if (W < 1 || W > 65535 || R < 0 || R >= kMaxLen || (W > 1 && ix->stride[n - 1] != 1)) return BSA_ERR_PARAM_INVALID;
  for (int i = 0; i < n - 1; ++i)
    if (ix->stride[i] < 0) return BSA_ERR_PARAM_INVALID;
  return BSA_OK;
}

bsa_status check_ws(uint64_t total, void *ws, size_t bytes) {
  if (!ws || bytes < total || reinterpret_cast<uintptr_t>(ws) % 256 != 0) return BSA_ERR_WORKSPACE;
  return BSA_OK;
}

uint64_t round256(uint64_t x) { return (x + 255) & ~uint64_t(255); }

// a call without work: its status word, where there is a workspace, reads 0
bsa_status finish_empty(void *ws, size_t bytes, void *stream) {
  if (check_ws(kStWords * 4, ws, bytes) != BSA_OK) return BSA_OK;
  return cudaMemsetAsync(ws, 0, kStWords * 4, static_cast<cudaStream_t>(stream)) == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

// ------------------------------------------------------------- block means
bsa_status prepare_means(const bsa_tensor *k, const bsa_tensor *cu_kv, const bsa_tensor *seqused,
                         const bsa_tensor *bt, const bsa_tensor *first, const bsa_params *prm,
                         const bsa_tensor *means, MeansProblem &p, uint64_t &bytes, bool &empty) {
  std::memset(&p, 0, sizeof(p));
  bytes = round256(kStWords * 4);
  empty = false;
  if (!prm || !present(k) || !present(means)) return BSA_ERR_NULLPTR;
  const bsa_params &P = *prm;
  bsa_status st = check_params(P);
  if (st != BSA_OK) return st;
  const int nd = P.kv_layout == BSA_LAYOUT_TND ? 3 : 4;
  if (k->dtype == BSA_F8E4M3) return BSA_ERR_UNSUPPORTED;
  if (!dtype16(k->dtype)) return BSA_ERR_PARAM_INVALID;
  if ((st = check_values(k, nd, k->dtype)) != BSA_OK) return st;
  if ((st = check_values(means, 4, k->dtype)) != BSA_OK) return st;
  const int64_t D = k->shape[nd - 1], N2 = P.num_kv_heads == 0 ? P.num_heads : P.num_kv_heads;
  if (N2 <= 0) return BSA_ERR_PARAM_INVALID;
  if (D != 64 && D != 128) return BSA_ERR_UNSUPPORTED;
  const int64_t B = means->shape[0], NB = means->shape[2];
  if (means->shape[1] != N2 || means->shape[3] != D) return BSA_ERR_PARAM_INVALID;
  if (B >= kMaxLen || NB > 65535) return BSA_ERR_UNSUPPORTED;  // block ids are 16-bit
  if ((st = kv_cache(k, cu_kv, seqused, bt, P, B, N2, p.kv)) != BSA_OK) return st;
  if (present(first)) {
    if (!vec_ok(first, BSA_I32, B)) return BSA_ERR_PARAM_INVALID;
    p.first_kv = static_cast<const int32_t *>(first->data);
  }
  if (B * N2 * (NB > 0 ? NB : 1) >= kMaxGrid) return BSA_ERR_UNSUPPORTED;
  empty = B == 0;
  p.D = int32_t(D);
  p.NB = int32_t(NB);
  p.dtype = k->dtype;
  p.k = k->data;
  kv_strides(k, P.kv_layout, p.k_sb, p.k_sh, p.k_st);
  p.means = means->data;
  p.m_sb = means->stride[0]; p.m_sh = means->stride[1]; p.m_st = means->stride[2];
  return BSA_OK;
}

// ---------------------------------------------------------- block selection
struct SelectRegions {
  bsa_ws_region status, row_nk, row_batch, row_block, qsum, bound, keys, again_count, again;
};

bsa_status prepare_select(const bsa_tensor *q, const bsa_tensor *means, const bsa_tensor *cu_q,
                          const bsa_tensor *cu_kv, const bsa_tensor *seqused, const bsa_params *prm, int64_t sink,
                          int64_t local, const bsa_tensor *index, SelectProblem &p, SelectRegions &L,
                          uint64_t &bytes, bool &empty) {
  std::memset(&p, 0, sizeof(p));
  std::memset(&L, 0, sizeof(L));
  bytes = 0;
  empty = false;
  if (!prm || !present(q) || !present(means) || !present(index)) return BSA_ERR_NULLPTR;
  const bsa_params &P = *prm;
  bsa_status st = check_params(P);
  if (st != BSA_OK) return st;
  int64_t B, Sq, Tq, N2, D;
  if ((st = check_q(q, cu_q, P, B, Sq, Tq, N2, D)) != BSA_OK) return st;
  if ((st = check_values(means, 4, q->dtype)) != BSA_OK) return st;
  const int64_t N1 = P.num_heads, NB = means->shape[2];
  if (means->shape[0] != B || means->shape[1] != N2 || means->shape[3] != D) return BSA_ERR_PARAM_INVALID;
  if (NB > 65535) return BSA_ERR_UNSUPPORTED;
  if (sink < 0 || local < 0) return BSA_ERR_PARAM_INVALID;
  int64_t H, R, W;
  if ((st = check_index(index, P, B, Sq, N1, N2, H, R, W)) != BSA_OK) return st;
  if ((st = kv_lengths(cu_kv, seqused, P, B, p.kv)) != BSA_OK) return st;
  // no cache here: the means say how many blocks there can be
  p.kv.N2 = int32_t(N2);
  p.kv.Skv = p.kv.seqused ? kMaxLen : NB * P.block_shape[1];
  p.kv.Tkv = kMaxLen;
  const int64_t Rg = P.q_layout == BSA_LAYOUT_BNSD ? B * R : R;
  const int64_t chunks = NB > 0 ? cdiv(NB, 128) : 1;
  if (Rg >= kMaxLen || H * Rg * chunks >= kMaxGrid) return BSA_ERR_UNSUPPORTED;
  empty = B == 0;
  p.q_layout = P.q_layout;
  p.B = int32_t(B); p.N1 = int32_t(N1); p.N2 = int32_t(N2); p.D = int32_t(D); p.g = int32_t(N1 / N2);
  p.Hidx = int32_t(H); p.BQ = int32_t(P.block_shape[0]); p.BKV = int32_t(P.block_shape[1]);
  p.NB = int32_t(NB); p.W = int32_t(W); p.R = int32_t(R); p.Rg = int32_t(Rg); p.dtype = q->dtype;
  p.causal = P.mask_type == BSA_MASK_CAUSAL;
  p.Sq = Sq; p.Tq = Tq; p.sink = sink; p.local = local;
  p.cu_q = present(cu_q) ? static_cast<const int64_t *>(cu_q->data) : nullptr;
  p.q = q->data;
  q_strides(q, P.q_layout, p.q_sb, p.q_sh, p.q_st);
  p.means = means->data;
  p.m_sb = means->stride[0]; p.m_sh = means->stride[1]; p.m_st = means->stride[2];
  p.index = static_cast<uint16_t *>(index->data);
  p.ix_s0 = index->stride[0]; p.ix_s1 = index->stride[1]; p.ix_s2 = index->stride[2];
  uint64_t cur = 0;
  place(cur, kStWords * 4, L.status);
  place(cur, uint64_t(Rg) * 4, L.row_nk);
  place(cur, uint64_t(Rg) * 4, L.row_batch);
  place(cur, uint64_t(Rg) * 4, L.row_block);
  place(cur, uint64_t(H) * Rg * D * 4, L.qsum);
  place(cur, uint64_t(H) * Rg * 4, L.bound);
  place(cur, uint64_t(H) * Rg * NB * 8, L.keys);
  place(cur, 4, L.again_count);
  place(cur, uint64_t(H) * Rg * sizeof(SelectAgain), L.again);
  bytes = round256(cur);
  return BSA_OK;
}

// ------------------------------------------------------- few-token attention
struct DecodeRegions {
  bsa_ws_region status, flags, join, part_ml, part_o;
};

bsa_status prepare_decode(const bsa_tensor *q, const bsa_tensor *k, const bsa_tensor *v, const bsa_tensor *index,
                          const bsa_tensor *tree, const bsa_tensor *cu_q, const bsa_tensor *cu_kv,
                          const bsa_tensor *seqused, const bsa_tensor *bt, const bsa_params *prm,
                          const bsa_tensor *out, const bsa_tensor *lse, DecodeProblem &p, DecodeRegions &L,
                          uint64_t &bytes, bool &empty) {
  std::memset(&p, 0, sizeof(p));
  std::memset(&L, 0, sizeof(L));
  bytes = 0;
  empty = false;
  if (!prm || !present(q) || !present(k) || !present(v) || !present(out)) return BSA_ERR_NULLPTR;
  const bsa_params &P = *prm;
  bsa_status st = check_params(P);
  if (st != BSA_OK) return st;
  int64_t B, Sq, Tq, N2, D;
  if ((st = check_q(q, cu_q, P, B, Sq, Tq, N2, D)) != BSA_OK) return st;
  const int qnd = q->ndim, knd = P.kv_layout == BSA_LAYOUT_TND ? 3 : 4, dt = q->dtype;
  if ((st = check_values(k, knd, dt)) != BSA_OK) return st;
  if ((st = check_values(v, knd, dt)) != BSA_OK) return st;
  if ((st = check_values(out, qnd, dt)) != BSA_OK) return st;
  if (!same_shape(k, v) || !same_shape(q, out) || k->shape[knd - 1] != D) return BSA_ERR_PARAM_INVALID;
  // the copies of k and v have no form for rows, heads or sequences that share
  // their memory
  for (int i = 0; i < knd - 1; ++i)
    if (k->shape[i] > 1 && (k->stride[i] == 0 || v->stride[i] == 0)) return BSA_ERR_UNSUPPORTED;
  if (!(P.scale >= 0.0) || std::isinf(P.scale)) return BSA_ERR_PARAM_INVALID;
  const int64_t N1 = P.num_heads;
  if ((st = kv_cache(k, cu_kv, seqused, bt, P, B, N2, p.kv)) != BSA_OK) return st;
  int64_t H = N2, R = 0, W = 0;
  if (present(index)) {
    if ((st = check_index(index, P, B, Sq, N1, N2, H, R, W)) != BSA_OK) return st;
    p.index = static_cast<const uint16_t *>(index->data);
    p.ix_s0 = index->stride[0]; p.ix_s1 = index->stride[1]; p.ix_s2 = index->stride[2];
  }
  if (present(tree)) {
    if (P.mask_type != BSA_MASK_NONE) return BSA_ERR_PARAM_INVALID;  // the bits are the whole mask
    const int n = qnd - 1;  // the tokens of q, then the words
    if (tree->dtype != BSA_I64 || tree->ndim != n || tree->shape[n - 1] < 1 || tree->shape[n - 1] >= kMaxLen / 64 ||
        (tree->shape[n - 1] > 1 && tree->stride[n - 1] != 1) || !aligned_to(tree, 8))
      return BSA_ERR_PARAM_INVALID;
    if (P.q_layout == BSA_LAYOUT_BNSD) {
      if (tree->shape[0] != B || tree->shape[1] != Sq || tree->shape[2] * 64 < Sq) return BSA_ERR_PARAM_INVALID;
      p.t_sb = tree->stride[0]; p.t_st = tree->stride[1];
    } else {
      if (tree->shape[0] != Tq) return BSA_ERR_PARAM_INVALID;
      p.t_st = tree->stride[0];
    }
    if (p.t_sb < 0 || p.t_st < 0) return BSA_ERR_PARAM_INVALID;
    p.tree = static_cast<const int64_t *>(tree->data);
    p.tree_words = int32_t(tree->shape[n - 1]);
  }
  if (P.return_lse) {
    if (!present(lse)) return BSA_ERR_NULLPTR;
    if (lse->dtype != BSA_F32 || lse->ndim != qnd - 1 || !aligned_to(lse, 4))
      return BSA_ERR_PARAM_INVALID;
    for (int i = 0; i < qnd - 1; ++i)
      if (lse->shape[i] != q->shape[i] || lse->stride[i] < 0) return BSA_ERR_PARAM_INVALID;
    p.lse = static_cast<float *>(lse->data);
    if (P.q_layout == BSA_LAYOUT_BNSD) { p.l_sb = lse->stride[0]; p.l_sh = lse->stride[1]; p.l_st = lse->stride[2]; }
    else { p.l_st = lse->stride[0]; p.l_sh = lse->stride[1]; }
  }
  empty = B == 0 || Sq + Tq == 0;
  p.q_layout = P.q_layout;
  p.B = int32_t(B); p.N1 = int32_t(N1); p.N2 = int32_t(N2); p.D = int32_t(D); p.g = int32_t(N1 / N2);
  p.H = int32_t(H); p.gg = int32_t(N1 / H); p.BQ = int32_t(P.block_shape[0]);
  p.W = int32_t(W); p.R = int32_t(R); p.dtype = dt;
  p.causal = P.mask_type == BSA_MASK_CAUSAL;
  p.Sq = Sq; p.Tq = Tq;
  const double scale = P.scale == 0.0 ? 1.0 / std::sqrt(double(D)) : P.scale;
  p.scale_log2 = float(scale * 1.4426950408889634);
  p.cu_q = present(cu_q) ? static_cast<const int64_t *>(cu_q->data) : nullptr;
  p.q = q->data; q_strides(q, P.q_layout, p.q_sb, p.q_sh, p.q_st);
  p.k = k->data; kv_strides(k, P.kv_layout, p.k_sb, p.k_sh, p.k_st);
  p.v = v->data; kv_strides(v, P.kv_layout, p.v_sb, p.v_sh, p.v_st);
  p.out = out->data; q_strides(out, P.q_layout, p.o_sb, p.o_sh, p.o_st);
  if (!empty && !decode_plan(p)) return BSA_ERR_UNSUPPORTED;
  uint64_t cur = 0;
  place(cur, kStWords * 4, L.status);
  place(cur, uint64_t(p.grid) * 4, L.flags);
  place(cur, uint64_t(p.grid) * sizeof(DecodeJoin), L.join);
  place(cur, uint64_t(p.grid) * 2 * p.TR * 8, L.part_ml);
  place(cur, uint64_t(p.grid) * 2 * p.TR * D * 4, L.part_o);
  bytes = round256(cur);
  return BSA_OK;
}

}  // namespace

extern "C" {

bsa_status bsa_block_means_get_workspace(const bsa_tensor *k, const bsa_tensor *cu_kv, const bsa_tensor *seqused,
                                         const bsa_tensor *bt, const bsa_tensor *first_kv,
                                         const bsa_params *params, const bsa_tensor *means,
                                         size_t *workspace_bytes) {
  if (!workspace_bytes) return BSA_ERR_NULLPTR;
  MeansProblem p;
  uint64_t bytes;
  bool empty;
  bsa_status st = prepare_means(k, cu_kv, seqused, bt, first_kv, params, means, p, bytes, empty);
  if (st == BSA_OK) *workspace_bytes = size_t(bytes);
  return st;
}

bsa_status bsa_block_means(const bsa_tensor *k, const bsa_tensor *cu_kv, const bsa_tensor *seqused,
                           const bsa_tensor *bt, const bsa_tensor *first_kv, const bsa_params *params,
                           const bsa_tensor *means, void *workspace, size_t workspace_bytes, void *stream) {
  MeansProblem p;
  uint64_t bytes;
  bool empty;
  bsa_status st = prepare_means(k, cu_kv, seqused, bt, first_kv, params, means, p, bytes, empty);
  if (st != BSA_OK) return st;
  if (empty) return finish_empty(workspace, workspace_bytes, stream);
  if ((st = check_ws(bytes, workspace, workspace_bytes)) != BSA_OK) return st;
  p.status = static_cast<uint32_t *>(workspace);
  return launch_block_means(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

bsa_status bsa_select_blocks_get_workspace(const bsa_tensor *q, const bsa_tensor *means, const bsa_tensor *cu_q,
                                           const bsa_tensor *cu_kv, const bsa_tensor *seqused,
                                           const bsa_params *params, int64_t sink_blocks, int64_t local_blocks,
                                           const bsa_tensor *index, size_t *workspace_bytes) {
  if (!workspace_bytes) return BSA_ERR_NULLPTR;
  SelectProblem p;
  SelectRegions L;
  uint64_t bytes;
  bool empty;
  bsa_status st = prepare_select(q, means, cu_q, cu_kv, seqused, params, sink_blocks, local_blocks, index, p, L,
                                 bytes, empty);
  if (st == BSA_OK) *workspace_bytes = size_t(bytes);
  return st;
}

bsa_status bsa_select_blocks(const bsa_tensor *q, const bsa_tensor *means, const bsa_tensor *cu_q,
                             const bsa_tensor *cu_kv, const bsa_tensor *seqused, const bsa_params *params,
                             int64_t sink_blocks, int64_t local_blocks, const bsa_tensor *index, void *workspace,
                             size_t workspace_bytes, void *stream) {
  SelectProblem p;
  SelectRegions L;
  uint64_t bytes;
  bool empty;
  bsa_status st = prepare_select(q, means, cu_q, cu_kv, seqused, params, sink_blocks, local_blocks, index, p, L,
                                 bytes, empty);
  if (st != BSA_OK) return st;
  if (empty) return finish_empty(workspace, workspace_bytes, stream);
  if ((st = check_ws(bytes, workspace, workspace_bytes)) != BSA_OK) return st;
  p.status = at<uint32_t>(workspace, L.status);
  p.row_nk = at<int32_t>(workspace, L.row_nk);
  p.row_batch = at<int32_t>(workspace, L.row_batch);
  p.row_block = at<int32_t>(workspace, L.row_block);
  p.qsum = at<float>(workspace, L.qsum);
  p.bound = at<float>(workspace, L.bound);
  p.keys = at<uint64_t>(workspace, L.keys);
  p.again_count = at<uint32_t>(workspace, L.again_count);
  p.again = at<SelectAgain>(workspace, L.again);
  return launch_select_blocks(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

bsa_status bsa_decode_get_workspace(const bsa_tensor *q, const bsa_tensor *k, const bsa_tensor *v,
                                    const bsa_tensor *index, const bsa_tensor *tree_mask, const bsa_tensor *cu_q,
                                    const bsa_tensor *cu_kv, const bsa_tensor *seqused, const bsa_tensor *bt,
                                    const bsa_params *params, const bsa_tensor *out, const bsa_tensor *lse,
                                    size_t *workspace_bytes) {
  if (!workspace_bytes) return BSA_ERR_NULLPTR;
  DecodeProblem p;
  DecodeRegions L;
  uint64_t bytes;
  bool empty;
  bsa_status st = prepare_decode(q, k, v, index, tree_mask, cu_q, cu_kv, seqused, bt, params, out, lse, p, L,
                                 bytes, empty);
  if (st == BSA_OK) *workspace_bytes = size_t(bytes);
  return st;
}

bsa_status bsa_decode(const bsa_tensor *q, const bsa_tensor *k, const bsa_tensor *v, const bsa_tensor *index,
                      const bsa_tensor *tree_mask, const bsa_tensor *cu_q, const bsa_tensor *cu_kv,
                      const bsa_tensor *seqused, const bsa_tensor *bt, const bsa_params *params,
                      const bsa_tensor *out, const bsa_tensor *lse, void *workspace, size_t workspace_bytes,
                      void *stream) {
  DecodeProblem p;
  DecodeRegions L;
  uint64_t bytes;
  bool empty;
  bsa_status st = prepare_decode(q, k, v, index, tree_mask, cu_q, cu_kv, seqused, bt, params, out, lse, p, L,
                                 bytes, empty);
  if (st != BSA_OK) return st;
  if (empty) return finish_empty(workspace, workspace_bytes, stream);
  if ((st = check_ws(bytes, workspace, workspace_bytes)) != BSA_OK) return st;
  p.status = at<uint32_t>(workspace, L.status);
  p.flags = at<uint32_t>(workspace, L.flags);
  p.join = at<DecodeJoin>(workspace, L.join);
  p.part_ml = at<float>(workspace, L.part_ml);
  p.part_o = at<float>(workspace, L.part_o);
  return launch_decode(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // extern "C"
