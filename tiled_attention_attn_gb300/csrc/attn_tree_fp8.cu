// Attention of single tokens and of trees of drafted tokens over a paged cache of
// 8-bit floating point (attn_tree_fp8).
//
// The plain form: a block per (token, query head), its warps take every fourth
// key, a lane d / 32 features; online softmax per warp, the warps joined at the
// end.  (K's and V's scales are applied to the score and to the weight.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "attn.h"
#include "attn_fp8.h"
#include "attn_turns.cuh"

namespace attn {
namespace tree {

struct Params {
  const uint16_t* q;
  uint16_t* o;
  float* lse;
  const int* cu;
  const long long* mask;
  PagedKV8 c;
  int* err;
  int B, Hq, total, max_tokens;
  float scale;
};

template <int E>
__device__ __forceinline__ void load_row(const uint8_t* p, float (&x)[E]) {
  const uint32_t u = E == 4 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u >> (8 * i)), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    x[i] = f.x;
    x[i + 1] = f.y;
  }
}

template <bool BF16, int D>
__global__ void __launch_bounds__(128) plain_kernel(const __grid_constant__ Params p) {
  constexpr int E = D / 32;
  __shared__ float s_m[4], s_l[4], s_o[4][D];
  const int row = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int b = row, i = 0, T = 1;
  if (p.cu) {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu + mid) <= row) lo = mid; else hi = mid;
    }
    b = lo;
    int first;
    T = chunk_len(p.cu, b, p.total, first, p.err);
    i = row - first;
    if (T > p.max_tokens) {
      atomicCAS(p.err, 0, ATTN_DEVERR_BAD_SEQLENS);
      return;
    }
    if (i < 0 || i >= T) return;
  }
  const int n = paged_len(p.c.t, b, p.err), g = h / (p.Hq / p.c.t.hkv);
  const unsigned long long bits = p.mask ? p.mask[row] : (2ull << i) - 1;
  float q[E], acc[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int x = 0; x < E; ++x) {
    const uint16_t w = p.q[(static_cast<long long>(row) * p.Hq + h) * D + lane * E + x];
    q[x] = BF16 ? __bfloat162float(__ushort_as_bfloat16(w)) : __half2float(__ushort_as_half(w));
    acc[x] = 0.0f;
  }
  for (int j = warp; j < n; j += 4) {
    const int place = j - (n - T);
    if (place >= 0 && !((bits >> place) & 1)) continue;
    const int page = paged_page(p.c.t, b, j >> p.c.t.page_log2, p.err);
    if (page < 0) continue;
    const int slot = j & ((1 << p.c.t.page_log2) - 1);
    const long long at = page * p.c.s_page + slot * p.c.s_token + g * p.c.s_head + lane * E;
    const long long sc = page * p.c.c_page + slot * p.c.c_token + g * p.c.c_head;
    float k[E], v[E], dot = 0.0f;
    load_row<E>(p.c.k + at, k);
    load_row<E>(p.c.v + at, v);
#pragma unroll
    for (int x = 0; x < E; ++x) dot = fmaf(q[x], k[x], dot);
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    const float s = dot * p.c.ks[sc] * p.scale, vs = p.c.vs[sc];
    const float mn = s > m || m == -INFINITY ? s : m;
    const float r = m == -INFINITY ? 0.0f : __expf(m - mn), w = s == -INFINITY ? 0.0f : __expf(s - mn);
    m = mn;
    l = l * r + w;
#pragma unroll
    for (int x = 0; x < E; ++x) acc[x] = acc[x] * r + w * vs * v[x];
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int x = 0; x < E; ++x) s_o[warp][lane * E + x] = acc[x];
  __syncthreads();
  const int f = threadIdx.x;
  if (f >= D) return;
  float M = -INFINITY, L = 0.0f, a = 0.0f;
  for (int w = 0; w < 4; ++w)
    if (s_l[w] != 0.0f) M = fmaxf(M, s_m[w]);
  for (int w = 0; w < 4; ++w) {
    if (s_l[w] == 0.0f) continue;
    const float r = __expf(s_m[w] - M);
    L += s_l[w] * r;
    a += s_o[w][f] * r;
  }
  const float y = L != 0.0f ? a / L : 0.0f;
  uint16_t* o = p.o + (static_cast<long long>(row) * p.Hq + h) * D + f;
  *o = BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(y)) : __half_as_ushort(__float2half_rn(y));
  if (f == 0) p.lse[static_cast<long long>(h) * p.total + row] = L != 0.0f ? M + logf(L) : -INFINITY;
}

}  // namespace tree
}  // namespace attn

extern "C" {

long long attn_fp8_workspace_bytes(int d) {
  if (d != 64 && d != 128) return ATTN_EUNSUPPORTED;
  return 256;
}

int attn_tree_fp8(const void* q, void* o, float* lse, int B, int Hq, int total, int max_tokens,
                  const attn_paged_kv8* cache, const int* cu_seqlens_or_null, const long long* tree_mask_or_null,
                  float scale, int fp16, void* workspace, long long workspace_bytes, cudaStream_t stream) {
  using namespace attn;
  tree::Params p = {};
  if (int rc = paged8_check(cache, B, p.c)) return rc;
  if (Hq <= 0 || Hq % p.c.t.hkv != 0 || total < 0 || (fp16 != 0 && fp16 != 1)) return ATTN_EINVAL;
  if (max_tokens < 1 || max_tokens > 64 || (!cu_seqlens_or_null && total != B)) return ATTN_EINVAL;
  if (total > 0 && (!q || !o || !lse)) return ATTN_EINVAL;
  if (!ptr_aligned(q, 16) || !ptr_aligned(o, 16) || !ptr_aligned(lse, 4) || !ptr_aligned(tree_mask_or_null, 8)) return ATTN_EINVAL;
  if (!std::isfinite(scale) || scale < 0.0f) return ATTN_EINVAL;
  if (static_cast<long long>(total) * Hq > (1LL << 31) - 1 || total > (1 << 30)) return ATTN_EINVAL;
  if (!workspace || !ptr_aligned(workspace, 256) || workspace_bytes < 256) return ATTN_EINVAL;
  const int d = cache->head_dim;
  const unsigned long long nq = 2ull * total * Hq * d;
  if (overlap(q, nq, o, nq)) return ATTN_EINVAL;
  if (total == 0) return ATTN_OK;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ELAUNCH;
  DeviceInfo info;
  if (int rc = device_info(dev, info)) return rc;
  if (!info.supported) return ATTN_EUNSUPPORTED;
  p.q = static_cast<const uint16_t*>(q);
  p.o = static_cast<uint16_t*>(o);
  p.lse = lse;
  p.cu = cu_seqlens_or_null;
  p.mask = tree_mask_or_null;
  p.err = info.err_word;
  p.B = B;
  p.Hq = Hq;
  p.total = total;
  p.max_tokens = max_tokens;
  p.scale = scale;
  const dim3 grid(total, Hq);
  if (d == 64) fp16 ? tree::plain_kernel<false, 64><<<grid, 128, 0, stream>>>(p) : tree::plain_kernel<true, 64><<<grid, 128, 0, stream>>>(p);
  else fp16 ? tree::plain_kernel<false, 128><<<grid, 128, 0, stream>>>(p) : tree::plain_kernel<true, 128><<<grid, 128, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ELAUNCH;
  count_launch();
  return ATTN_OK;
}

}  // extern "C"
