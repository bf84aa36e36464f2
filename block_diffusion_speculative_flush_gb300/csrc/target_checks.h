// Argument checks of the target-side operators: what the host can see of a call
// is answered with a status and a message before any device work.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "dflash.h"
#include "ragged.h"

extern "C" int dflash__set_error(int code, const char* msg);

namespace dfl {

inline int rfail(int code, const char* call, const char* what) {
  char buf[256];
  snprintf(buf, sizeof buf, "%s: %s", call, what);
  return dflash__set_error(code, buf);
}
inline int rcheck(cudaError_t e, const char* call) {
  return e == cudaSuccess ? DFLASH_OK : rfail(DFLASH_ERR_CUDA, call, cudaGetErrorString(e));
}
inline int esize(int32_t dtype) { return dtype == DFLASH_DTYPE_F32 ? 4 : 2; }
inline bool pow2(int64_t x) { return x > 0 && (x & (x - 1)) == 0; }

inline int check_shape(const char* call, int32_t dtype, int32_t hkv, int32_t d) {
  if (dtype != DFLASH_DTYPE_F32 && dtype != DFLASH_DTYPE_BF16) return rfail(DFLASH_ERR_INVALID_ARG, call, "dtype");
  if (hkv < 1 || hkv > 1024) return rfail(DFLASH_ERR_SHAPE, call, "n_kv_heads outside 1..1024");
  if (dtype == DFLASH_DTYPE_BF16 ? (d != 64 && d != 128) : (d < 4 || d > 128 || d % 4))
    return rfail(DFLASH_ERR_SHAPE, call, "head_dim: bf16 64 or 128, fp32 a multiple of 4 up to 128");
  return DFLASH_OK;
}

// strides below 2^40 bytes keep every offset of 2^30 rows within 64 bits
inline bool stride_ok(int64_t s, int es) { return s >= 0 && (s * es) % 16 == 0 && s < ((int64_t)1 << 38); }

inline int check_heads(const char* call, const dflash_heads* h, int32_t dtype, int32_t heads, int32_t d, bool rows) {
  if (!h || (rows && !h->data)) return rfail(DFLASH_ERR_INVALID_ARG, call, "null rows");
  const int es = esize(dtype);
  if ((uintptr_t)h->data % 16 || !stride_ok(h->row_stride, es) || !stride_ok(h->head_stride, es))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "rows: 16-byte aligned base, strides multiples of 16 bytes");
  if ((heads > 1 && h->head_stride < d) || h->row_stride < d)
    return rfail(DFLASH_ERR_INVALID_ARG, call, "rows: strides shorter than a head");
  return DFLASH_OK;
}

inline int check_pages(const char* call, const dflash_kv_pages* p) {
  if (!p || !p->k || !p->v) return rfail(DFLASH_ERR_INVALID_ARG, call, "null pages");
  if (int rc = check_shape(call, p->dtype, p->n_kv_heads, p->head_dim)) return rc;
  if (p->page_size < 8 || p->page_size > 1024 || !pow2(p->page_size))
    return rfail(DFLASH_ERR_SHAPE, call, "page_size: a power of two in 8..1024");
  if (p->n_pages < 1 || p->n_pages > INT32_MAX) return rfail(DFLASH_ERR_SHAPE, call, "n_pages outside 1..2^31 - 1");
  const int es = esize(p->dtype);
  if ((uintptr_t)p->k % 16 || (uintptr_t)p->v % 16 || !stride_ok(p->page_stride, es) ||
      !stride_ok(p->slot_stride, es) || !stride_ok(p->head_stride, es))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "pages: 16-byte aligned bases, strides multiples of 16 bytes");
  if (p->slot_stride < p->head_dim || (p->n_kv_heads > 1 && p->head_stride < p->head_dim) ||
      (p->n_pages > 1 && p->page_stride < p->head_dim))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "pages: strides shorter than a head");
  return DFLASH_OK;
}

// Host bounds of the batch; the device fields only have to be there.
inline int check_ragged(const char* call, const dflash_ragged* b, const dflash_kv_pages* pages, bool pointers) {
  if (!b) return rfail(DFLASH_ERR_INVALID_ARG, call, "null batch");
  if (b->batch < 1 || b->batch > 32768) return rfail(DFLASH_ERR_INVALID_ARG, call, "batch outside 1..32768");
  if (b->total_rows < 0 || b->total_rows > (1 << 30) || b->max_rows < 1 || b->max_rows > (1 << 24))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "total_rows outside 0..2^30 or max_rows outside 1..2^24");
  if (pointers && !b->starts) return rfail(DFLASH_ERR_INVALID_ARG, call, "null starts");
  if (pages) {
    if (pointers && (!b->lens || !b->table)) return rfail(DFLASH_ERR_INVALID_ARG, call, "null lens or table");
    if (b->max_len < 1 || b->max_len > (1 << 30)) return rfail(DFLASH_ERR_INVALID_ARG, call, "max_len outside 1..2^30");
    if (b->table_width < 1 || b->table_stride < b->table_width)
      return rfail(DFLASH_ERR_INVALID_ARG, call, "table_width < 1 or table_stride below it");
  }
  return DFLASH_OK;
}

inline int check_attention(const char* call, const dflash_attention* a, bool pointers, bool rows) {
  if (!a) return rfail(DFLASH_ERR_INVALID_ARG, call, "null attention");
  if (int rc = check_shape(call, a->dtype, a->n_kv_heads, a->head_dim)) return rc;
  if (a->n_q_heads < 1 || a->n_q_heads % a->n_kv_heads || a->n_q_heads / a->n_kv_heads > 128)
    return rfail(DFLASH_ERR_SHAPE, call, "n_q_heads: a multiple of n_kv_heads, at most 128 per KV head");
  if ((a->causal != 0 && a->causal != 1) || a->window < 0 || a->window > (1 << 30))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "causal 0 or 1, window 0 or 1..2^30");
  // (the kernels work with scale log2(e); an infinite one makes NaN of a score of 0)
  if (!(a->scale > 0.f) || !std::isfinite(1.5f * a->scale))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "scale: > 0, 1.5 x scale finite");
  if (!pointers) return DFLASH_OK;
  if (int rc = check_heads(call, &a->q, a->dtype, a->n_q_heads, a->head_dim, rows)) return rc;
  if (int rc = check_heads(call, &a->out, a->dtype, a->n_q_heads, a->head_dim, rows)) return rc;
  if (rows && a->out.data == a->q.data) return rfail(DFLASH_ERR_INVALID_ARG, call, "out is q");
  return DFLASH_OK;
}

inline Ragged make_ragged(const dflash_ragged* b, const dflash_kv_pages* pages) {
  const int32_t max_rows = std::min(b->max_rows, std::max(b->total_rows, 1));
  int64_t max_len = max_rows;
  if (pages) max_len = std::min<int64_t>(b->max_len, (int64_t)b->table_width * pages->page_size);
  return Ragged{b->batch, b->total_rows, max_rows, (int32_t)max_len, b->starts,
                pages ? b->lens : nullptr, pages ? b->table : nullptr, b->table_stride, b->status};
}

}  // namespace dfl
