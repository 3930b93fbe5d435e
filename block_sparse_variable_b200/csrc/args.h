// args.h -- host-side descriptor checks shared by the C-ABI entry points
// (bsa_api.cu, cache_api.cu).
#pragma once

#include <stdint.h>

#include "bsa_internal.h"

namespace bsa {

inline bool present(const bsa_tensor *t) { return t != nullptr && t->data != nullptr; }

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool block_ok(int64_t x) { return x == 128 || x == 256 || x == 512 || x == 1024; }

// A dense-value tensor (q/k/v/out/...): given ndim, dtype, last stride 1, the
// other strides 16-byte multiples (8 16-bit or 16 8-bit elements) and a
// 16-byte-aligned base (16-byte vector loads and TMA boxes start on 16-byte
// boundaries).
inline bsa_status check_values(const bsa_tensor *t, int ndim, int dtype) {
  if (t->ndim != ndim || t->dtype != dtype) return BSA_ERR_PARAM_INVALID;
  if (t->stride[ndim - 1] != 1) return BSA_ERR_PARAM_INVALID;
  const int64_t per16 = dtype == BSA_F8E4M3 ? 16 : 8;
  for (int i = 0; i < ndim; ++i) {
    if (t->shape[i] < 0) return BSA_ERR_PARAM_INVALID;
    if (i < ndim - 1 && (t->stride[i] % per16 != 0 || t->stride[i] < 0)) return BSA_ERR_PARAM_INVALID;
  }
  if (reinterpret_cast<uintptr_t>(t->data) % 16 != 0) return BSA_ERR_PARAM_INVALID;
  return BSA_OK;
}

inline bool same_shape(const bsa_tensor *a, const bsa_tensor *b) {
  if (a->ndim != b->ndim || a->dtype != b->dtype) return false;
  for (int i = 0; i < a->ndim; ++i)
    if (a->shape[i] != b->shape[i]) return false;
  return true;
}

// whole numbers start at a multiple of their size: a load from elsewhere faults
inline bool aligned_to(const bsa_tensor *t, unsigned bytes) { return reinterpret_cast<uintptr_t>(t->data) % bytes == 0; }

inline bool vec_ok(const bsa_tensor *t, int dtype, int64_t n) {
  return t->ndim == 1 && t->dtype == dtype && t->shape[0] == n && (n <= 1 || t->stride[0] == 1) &&
         aligned_to(t, dtype == BSA_I64 ? 8 : 4);
}

inline uint64_t place(uint64_t &cur, uint64_t bytes, bsa_ws_region &r) {
  cur = (cur + 255) & ~uint64_t(255);
  r.offset = cur;
  r.bytes = bytes;
  cur += bytes;
  return r.offset;
}

template <typename T>
T *at(void *ws, const bsa_ws_region &r) {
  return r.bytes ? reinterpret_cast<T *>(static_cast<char *>(ws) + r.offset) : nullptr;
}

}  // namespace bsa
