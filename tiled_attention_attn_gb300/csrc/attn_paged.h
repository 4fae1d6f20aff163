// The paged key/value cache as the kernels see it, and the host checks that
// its entry points share.
#pragma once
#include <cstdint>

#include "attn.h"
#include "attn_internal.h"

namespace attn {

struct PagedKV {
  uint16_t* k;
  uint16_t* v;
  const int* table;     // row b at table + b * table_stride
  const int* seqlens;   // (B)
  long long s_page, s_token, s_head;   // elements
  int table_stride, max_pages, num_pages, page_log2, hkv;
};

constexpr int kPagedMaxB = 65535;

// Softmax weights, which are at most 2^8 of the running maximum's (it lags by up
// to that), are held times 2^kLift for the second product; so are their sums l
// until the unit's end, where kDrop takes the factor out.  fp16 then keeps weights
// down to 2^-32 of the maximum (2^-25 as they are): 65,535 keys of 2^-25.2 each are
// 1.6e-3 of l, and were nothing in u.  bf16 has the range of fp32.
template <bool BF16>
constexpr int kLift = BF16 ? 0 : 7;
template <bool BF16>
constexpr float kDrop = BF16 ? 1.0f : 0x1p-7f;

inline bool ptr_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// Whether [a, a + na) and [b, b + nb) share bytes.
inline bool overlap(const void* a, unsigned long long na, const void* b, unsigned long long nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// Checks the host struct and fills `out`.  need_v: the values are used.
inline int paged_check(const attn_paged_kv* c, int B, bool need_v, PagedKV& out) {
  if (!c || !c->k || (need_v && !c->v) || !c->page_table || !c->seqlens_k) return ATTN_EINVAL;
  if (!ptr_aligned(c->k, 16) || (need_v && !ptr_aligned(c->v, 16))) return ATTN_EINVAL;
  if (B <= 0 || B > kPagedMaxB || c->num_kv_heads <= 0 || c->num_kv_heads > 65535 || c->num_pages <= 0) return ATTN_EINVAL;
  if (c->max_pages <= 0 || c->table_stride < c->max_pages || (c->fp16 != 0 && c->fp16 != 1)) return ATTN_EINVAL;
  for (long long s : {c->stride_page, c->stride_token, c->stride_head})
    if (s <= 0 || s % 8 != 0 || s >= (1LL << 39)) return ATTN_EINVAL;
  if (c->head_dim != 64 && c->head_dim != 128) return ATTN_EUNSUPPORTED;
  int lg = 4;
  while (lg <= 8 && (1 << lg) != c->page_size) ++lg;
  if (lg > 8) return ATTN_EUNSUPPORTED;
  if (static_cast<long long>(c->max_pages) << lg > (1LL << 30)) return ATTN_EINVAL;   // 32-bit key indices
  out.k = static_cast<uint16_t*>(c->k);
  out.v = static_cast<uint16_t*>(c->v);
  out.table = c->page_table;
  out.seqlens = c->seqlens_k;
  out.s_page = c->stride_page;
  out.s_token = c->stride_token;
  out.s_head = c->stride_head;
  out.table_stride = c->table_stride;
  out.max_pages = c->max_pages;
  out.num_pages = c->num_pages;
  out.page_log2 = lg;
  out.hkv = c->num_kv_heads;
  return ATTN_OK;
}

#if defined(__CUDACC__)
// A key count as it was read: 0 (and the error recorded) when out of range.
__device__ __forceinline__ int checked_len(const PagedKV& c, int n, int* err) {
  if (n < 0 || n > (c.max_pages << c.page_log2)) {
    atomicCAS(err, 0, ATTN_DEVERR_BAD_SEQLENS);
    return 0;
  }
  return n;
}
// Keys of sequence b.
__device__ __forceinline__ int paged_len(const PagedKV& c, int b, int* err) {
  return checked_len(c, __ldg(c.seqlens + b), err);
}
// Page i of sequence b, or -1 (and the error recorded) when it is not one.
__device__ __forceinline__ int paged_page(const PagedKV& c, int b, int i, int* err) {
  const int p = __ldg(c.table + static_cast<long long>(b) * c.table_stride + i);
  if (p < 0 || p >= c.num_pages) {
    atomicCAS(err, 0, ATTN_DEVERR_BAD_PAGE);
    return -1;
  }
  return p;
}
// First row and count of sequence b's new tokens: none (and the error
// recorded) when its offsets are decreasing or leave [0, total].
__device__ __forceinline__ int chunk_len(const int* cu, int b, int total, int& row, int* err) {
  const int a = __ldg(cu + b), e = __ldg(cu + b + 1);
  row = a;
  if (a < 0 || e < a || e > total) {
    atomicCAS(err, 0, ATTN_DEVERR_BAD_SEQLENS);
    return 0;
  }
  return e - a;
}
// New tokens and keys of sequence b: all three reads on their way before any
// is looked at.
__device__ __forceinline__ void chunk_and_keys(const PagedKV& c, const int* cu, int b, int total, int& q_len, int& row,
                                               int& k_len, int* err) {
  const int a = __ldg(cu + b), e = __ldg(cu + b + 1), n = __ldg(c.seqlens + b);
  row = a;
  q_len = e - a;
  if (a < 0 || e < a || e > total) {
    atomicCAS(err, 0, ATTN_DEVERR_BAD_SEQLENS);
    q_len = 0;
  }
  k_len = checked_len(c, n, err);
}
#endif

}  // namespace attn
