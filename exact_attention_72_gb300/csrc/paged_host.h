// Argument checks of the paged cache shared by its entry points.
#pragma once
#include <cstdint>

#include "attn.h"
#include "paged.cuh"

namespace gb300 {

inline bool is_aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// The kernels' form of a cache (strides in bytes), or why it is refused.
inline attn_status_t paged_cache_args(const attn_paged_cache_t* c, PagedCache* out) {
  if (!c || !c->k || !c->v || !is_aligned(c->k, 16) || !is_aligned(c->v, 16)) return ATTN_ERR_INVALID_ARG;
  if (c->type != ATTN_CACHE_BF16 && c->type != ATTN_CACHE_INT4) return ATTN_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->page_size < 1 || c->Hkv < 1 || c->d < 1) return ATTN_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128 && c->d != 256) return ATTN_ERR_UNSUPPORTED;
  if (c->page_size % 16) return ATTN_ERR_UNSUPPORTED;   // 16 neighbouring keys lie in one page
  const bool int4 = c->type == ATTN_CACHE_INT4;
  const int elt = int4 ? 1 : 2;
  // rows are read in 16-byte pieces; strides stay far inside 64 bits
  for (const long long s : {c->page_stride, c->token_stride, c->head_stride})
    if (s < 0 || s > (1LL << 40) || s * elt % 16) return ATTN_ERR_INVALID_ARG;
  out->k = static_cast<uint8_t*>(c->k);
  out->v = static_cast<uint8_t*>(c->v);
  out->page_b = c->page_stride * elt;
  out->token_b = c->token_stride * elt;
  out->head_b = c->head_stride * elt;
  out->k_sz = out->v_sz = nullptr;
  out->sz_page_b = out->sz_token_b = out->sz_head_b = 0;
  if (int4) {
    const int pairs = c->d / kInt4Group;   // (scale, zero) pairs of a row: one 4-, 8- or 16-byte copy
    if (!c->k_sz || !c->v_sz || !is_aligned(c->k_sz, 4 * pairs) || !is_aligned(c->v_sz, 4 * pairs))
      return ATTN_ERR_INVALID_ARG;
    for (const long long s : {c->sz_page_stride, c->sz_token_stride, c->sz_head_stride})
      if (s < 0 || s > (1LL << 40) || s % (2 * pairs)) return ATTN_ERR_INVALID_ARG;
    out->k_sz = static_cast<uint8_t*>(c->k_sz);
    out->v_sz = static_cast<uint8_t*>(c->v_sz);
    out->sz_page_b = c->sz_page_stride * 2;
    out->sz_token_b = c->sz_token_stride * 2;
    out->sz_head_b = c->sz_head_stride * 2;
  }
  out->num_pages = c->num_pages;
  out->page_size = c->page_size;
  out->Hkv = c->Hkv;
  return ATTN_OK;
}

}  // namespace gb300
