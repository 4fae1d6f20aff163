// The paged cache of 8-bit floating point as the kernels see it, and the host
// checks that its entry points share.
#pragma once
#include <cstdint>

#include "attn.h"
#include "attn_paged.h"

namespace attn {

struct PagedKV8 {
  PagedKV t;              // table, lengths, pages, heads (its own pointers and strides are not used)
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  long long s_page, s_token, s_head;   // of k and v, bytes
  long long c_page, c_token, c_head;   // of ks and vs, floats
};

// The largest e4m3 value, and the smallest scale of a row.
constexpr float kE4M3Top = 448.0f;
constexpr float kLeastScale = 0x1p-126f;

inline int paged8_check(const attn_paged_kv8* c, int B, PagedKV8& out) {
  if (!c || !c->k || !c->v || !c->k_scales || !c->v_scales) return ATTN_EINVAL;
  // what both kinds of cache have, checked by the other's rules (its strides stand in)
  attn_paged_kv h = {};
  h.k = c->k;
  h.v = c->v;
  h.page_table = c->page_table;
  h.seqlens_k = c->seqlens_k;
  h.stride_page = h.stride_token = h.stride_head = 8;
  h.table_stride = c->table_stride;
  h.max_pages = c->max_pages;
  h.num_pages = c->num_pages;
  h.page_size = c->page_size;
  h.num_kv_heads = c->num_kv_heads;
  h.head_dim = c->head_dim;
  if (!ptr_aligned(c->k_scales, 4) || !ptr_aligned(c->v_scales, 4)) return ATTN_EINVAL;
  for (long long s : {c->stride_page, c->stride_token, c->stride_head})
    if (s <= 0 || s % 16 != 0 || s >= (1LL << 39)) return ATTN_EINVAL;
  for (long long s : {c->scale_stride_page, c->scale_stride_token, c->scale_stride_head})
    if (s <= 0 || s >= (1LL << 39)) return ATTN_EINVAL;
  if (int rc = paged_check(&h, B, true, out.t)) return rc;
  out.k = static_cast<uint8_t*>(c->k);
  out.v = static_cast<uint8_t*>(c->v);
  out.ks = c->k_scales;
  out.vs = c->v_scales;
  out.s_page = c->stride_page;
  out.s_token = c->stride_token;
  out.s_head = c->stride_head;
  out.c_page = c->scale_stride_page;
  out.c_token = c->scale_stride_token;
  out.c_head = c->scale_stride_head;
  return ATTN_OK;
}

}  // namespace attn
