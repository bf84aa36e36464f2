// Argument checks of the 8-bit paged cache.
#pragma once

#include "kv8.h"
#include "target_checks.h"

namespace dfl {

inline int check_kv8_pages(const char* call, const dflash_kv8_pages* p) {
  if (!p || !p->k || !p->v || !p->k_scale || !p->v_scale) return rfail(DFLASH_ERR_INVALID_ARG, call, "null pages or scales");
  if (p->n_kv_heads < 1 || p->n_kv_heads > 1024) return rfail(DFLASH_ERR_SHAPE, call, "n_kv_heads outside 1..1024");
  if (p->head_dim < 16 || p->head_dim > 128 || p->head_dim % 16)
    return rfail(DFLASH_ERR_SHAPE, call, "head_dim: a multiple of 16 up to 128");
  if (p->page_size < 16 || p->page_size > 1024 || !pow2(p->page_size))
    return rfail(DFLASH_ERR_SHAPE, call, "page_size: a power of two in 16..1024");
  if (p->reserved != 0) return rfail(DFLASH_ERR_INVALID_ARG, call, "reserved: 0");
  if (p->n_pages < 1 || p->n_pages > INT32_MAX) return rfail(DFLASH_ERR_SHAPE, call, "n_pages outside 1..2^31 - 1");
  if ((uintptr_t)p->k % 16 || (uintptr_t)p->v % 16 || !stride_ok(p->page_stride, 1) || !stride_ok(p->slot_stride, 1) ||
      !stride_ok(p->head_stride, 1))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "pages: 16-byte aligned bases, strides multiples of 16");
  if (p->slot_stride < p->head_dim || (p->n_kv_heads > 1 && p->head_stride < p->head_dim) ||
      (p->n_pages > 1 && p->page_stride < p->head_dim))
    return rfail(DFLASH_ERR_INVALID_ARG, call, "pages: strides shorter than a head");
  const int64_t most = (int64_t)1 << 38;
  if ((uintptr_t)p->k_scale % 4 || (uintptr_t)p->v_scale % 4 || p->scale_page_stride < 1 || p->scale_head_stride < 1 ||
      p->scale_page_stride > most || p->scale_head_stride > most)
    return rfail(DFLASH_ERR_INVALID_ARG, call, "scales: 4-byte aligned, strides of at least 1");
  return DFLASH_OK;
}

inline int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

// What check_ragged and make_ragged look at: the page size.
inline dflash_kv_pages kv8_as_pages(const dflash_kv8_pages* p) {
  dflash_kv_pages l{};
  l.page_size = p->page_size;
  return l;
}

inline Kv8View kv8_view(const dflash_kv8_pages* p) {
  return Kv8View{(uint8_t*)p->k, (uint8_t*)p->v, p->k_scale, p->v_scale, p->page_stride, p->slot_stride, p->head_stride,
                 p->scale_page_stride, p->scale_head_stride, log2_of(p->page_size), (int32_t)p->n_pages};
}

}  // namespace dfl
