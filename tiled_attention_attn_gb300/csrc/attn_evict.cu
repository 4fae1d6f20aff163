// Eviction from a paged cache by accumulated attention weight
// (attn_cache_evict): per sequence and key/value head, the `recent` last keys
// and the heaviest of the others are kept, in order, and their rows moved to
// the front.
//
// Selection (evict_select_kernel, one block per sequence and head): the
// weights' bit patterns are mapped to unsigned integers of the same order, and
// the k-th largest is found digit by digit (8 bits, most significant first): a
// histogram of the digit over the keys that match the digits so far, then the
// digit whose count from above passes k.  Keys above it are kept, and the
// first of those equal to it, so that exactly k are; a prefix sum over the
// keys in order gives each kept key its place.
//
// Moving (evict_move_kernel): row s of the kept keys goes from key kept[s] >= s
// to key s.  A block owns a 64-byte column of the rows of one (sequence, head,
// K or V) and walks the rows in order, a batch at a time, every load of a batch
// before its stores: a store to key s can only meet loads of keys kept[s'] = s
// with s' <= s, which came in the same batch or an earlier one, so rows may
// move in place.  Bound by HBM: each kept row read and written once.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attn_paged.h"

namespace attn {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 4;   // rows in flight per thread

struct EvictParams {
  const float* weights;
  float* weights_out;
  int* kept;
  int* seqlens_out;
  PagedKV c;            // source
  const int* dst_table;
  int dst_stride, dst_max_pages;
  int weights_len, weights_out_len, budget, recent, d;
  int* err;
};

// Unsigned key of the same order as the float: NaNs largest.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  if (u == 0x80000000u) return 0x80000000u;   // -0 is 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Keys of sequence b, bounded by the weights' row too.
__device__ __forceinline__ int evict_len(const EvictParams& p, int b) {
  const int n = paged_len(p.c, b, p.err);
  if (n <= p.weights_len) return n;
  atomicCAS(p.err, 0, ATTN_DEVERR_BAD_SEQLENS);
  return 0;
}

// Inclusive prefix sum over the block; total in *sum.
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int* sum) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[w] = x;
  __syncthreads();
  if (w == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  x += w > 0 ? warp_sums[w - 1] : 0;
  *sum = warp_sums[31];
  __syncthreads();
  return x;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int hist[256];
  __shared__ int warp_sums[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int g = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int n = evict_len(p, b), m = min(n, p.budget);
  const long long row = static_cast<long long>(b) * p.c.hkv + g;
  const float* w = p.weights + row * p.weights_len;
  int* kept = p.kept + row * p.budget;
  if (g == 0 && tid == 0) p.seqlens_out[b] = m;
  for (int s = m + tid; s < p.budget; s += kSelThreads) kept[s] = -1;
  if (n <= p.budget) {
    for (int s = tid; s < n; s += kSelThreads) kept[s] = s;
    return;
  }
  const int cand = n - p.recent;       // keys that compete
  const int k = p.budget - p.recent;   // of which this many stay
  for (int s = tid; s < p.recent; s += kSelThreads) kept[k + s] = cand + s;
  if (k == 0) return;
  uint32_t prefix = 0;
  int need = k;   // still to take among the keys that match the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int j = tid; j < cand; j += kSelThreads) {
      const uint32_t u = order_key(__ldg(w + j));
      if ((u & mask) == prefix) atomicAdd(&hist[(u >> shift) & 255], 1);
    }
    __syncthreads();
    int sum;
    const int c = tid < 256 ? hist[255 - tid] : 0;   // from the largest digit down
    const int above = block_scan(c, warp_sums, &sum);
    if (tid < 256 && above >= need && above - c < need) {
      s_prefix = prefix | static_cast<uint32_t>(255 - tid) << shift;
      s_need = need - (above - c);
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    __syncthreads();
  }
  // keys above the threshold, and the first `need` of those equal to it
  int above0 = 0, equal0 = 0;
  for (int j0 = 0; j0 < cand; j0 += kSelThreads) {
    const int j = j0 + tid;
    const uint32_t u = j < cand ? order_key(__ldg(w + j)) : 0u;
    const int gt = j < cand && u > prefix, eq = j < cand && u == prefix;
    int n_gt, n_eq;
    const int a = above0 + block_scan(gt, warp_sums, &n_gt);
    const int e = equal0 + block_scan(eq, warp_sums, &n_eq);
    // a, e: keys above / equal up to and with this one
    if (gt || (eq && e <= need)) kept[a + min(e, need) - 1] = j;
    above0 += n_gt;
    equal0 += n_eq;
  }
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictParams p) {
  const int n_col = p.d / 32;   // 64-byte columns
  const int g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int n = evict_len(p, b), m = min(n, p.budget);
  const long long row = static_cast<long long>(b) * p.c.hkv + g;
  const int* kept = p.kept + row * p.budget;
  if (static_cast<int>(blockIdx.x) == 2 * n_col) {
    // the weights themselves, in the same order
    const float* w = p.weights + row * p.weights_len;
    float* out = p.weights_out + row * p.weights_out_len;
    for (int s0 = 0; s0 < m; s0 += kMoveThreads) {
      const int s = s0 + tid;
      const float x = s < m ? w[__ldg(kept + s)] : 0.0f;
      __syncthreads();
      if (s < m) out[s] = x;
    }
    __syncthreads();
    for (int s = m + tid; s < p.weights_out_len; s += kMoveThreads) out[s] = 0.0f;
    return;
  }
  const int which = blockIdx.x / n_col, col = blockIdx.x % n_col;
  uint16_t* base = (which == 0 ? p.c.k : p.c.v) + g * p.c.s_head + col * 32 + (tid & 3) * 8;
  const int pm = (1 << p.c.page_log2) - 1;
  constexpr int kRows = kMoveThreads / 4;
  const int* dst_row = p.dst_table + static_cast<long long>(b) * p.dst_stride;
  for (int s0 = 0; s0 < m; s0 += kRows * kMoveRows) {
    uint4 x[kMoveRows];
    uint16_t* to[kMoveRows];
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      to[u] = nullptr;
      const int s = s0 + u * kRows + (tid >> 2);
      if (s >= m) continue;
      const int j = __ldg(kept + s);
      const int from = paged_page(p.c, b, j >> p.c.page_log2, p.err);
      const int page = (s >> p.c.page_log2) < p.dst_max_pages ? __ldg(dst_row + (s >> p.c.page_log2)) : -1;
      if (page < 0 || page >= p.c.num_pages) atomicCAS(p.err, 0, ATTN_DEVERR_BAD_PAGE);
      else if (from >= 0 && !(from == page && j == s)) {
        x[u] = *reinterpret_cast<const uint4*>(base + from * p.c.s_page + (j & pm) * p.c.s_token);
        to[u] = base + page * p.c.s_page + (s & pm) * p.c.s_token;
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u)
      if (to[u]) *reinterpret_cast<uint4*>(to[u]) = x[u];
    __syncthreads();
  }
}

}  // namespace
}  // namespace attn

extern "C" int attn_cache_evict(const float* weights, int weights_len, int* kept, int* seqlens_out, float* weights_out,
                                int weights_out_len, int B, const attn_paged_kv* cache, const int* dst_page_table,
                                int dst_stride, int dst_max_pages, int budget, int recent, cudaStream_t stream) {
  using namespace attn;
  EvictParams p = {};
  if (int rc = paged_check(cache, B, true, p.c)) return rc;
  if (!weights || !kept || !seqlens_out || !weights_out || weights_len <= 0) return ATTN_EINVAL;
  for (const void* x : {static_cast<const void*>(weights), static_cast<const void*>(kept),
                        static_cast<const void*>(seqlens_out), static_cast<const void*>(weights_out)})
    if (!ptr_aligned(x, 4)) return ATTN_EINVAL;
  if (budget < 1 || recent < 0 || recent > budget || weights_out_len < budget || budget > (1 << 30)) return ATTN_EINVAL;
  if (seqlens_out == cache->seqlens_k || (weights_out == weights && weights_out_len != weights_len)) return ATTN_EINVAL;
  if (dst_page_table) {
    if (dst_max_pages <= 0 || dst_stride < dst_max_pages ||
        static_cast<long long>(dst_max_pages) * cache->page_size < std::min<long long>(
            budget, static_cast<long long>(cache->max_pages) * cache->page_size))
      return ATTN_EINVAL;
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ELAUNCH;
  DeviceInfo info;
  if (int rc = device_info(dev, info)) return rc;
  if (!info.supported) return ATTN_EUNSUPPORTED;
  p.weights = weights;
  p.weights_out = weights_out;
  p.kept = kept;
  p.seqlens_out = seqlens_out;
  p.dst_table = dst_page_table ? dst_page_table : cache->page_table;
  p.dst_stride = dst_page_table ? dst_stride : cache->table_stride;
  p.dst_max_pages = dst_page_table ? dst_max_pages : cache->max_pages;
  p.weights_len = weights_len;
  p.weights_out_len = weights_out_len;
  p.budget = budget;
  p.recent = recent;
  p.d = cache->head_dim;
  p.err = info.err_word;
  evict_select_kernel<<<dim3(p.c.hkv, B), kSelThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ELAUNCH;
  count_launch();
  evict_move_kernel<<<dim3(2 * p.d / 32 + 1, p.c.hkv, B), kMoveThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ELAUNCH;
  count_launch();
  return ATTN_OK;
}
