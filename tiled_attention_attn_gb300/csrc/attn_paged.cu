// Attention over a paged key/value cache (attn_fwd_paged, attn_decode_paged)
// and the accumulated attention weight of each key (attn_key_weights): host
// checks and the first, plain kernels: one warp per query row (or per key),
// the row's features spread over the lanes, fp32 throughout, keys one after
// another with the running maximum and sum of the softmax.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "attn_paged_launch.h"

namespace attn {
namespace {

constexpr int kWarps = 8;

template <bool BF16>
__device__ __forceinline__ float cvt(uint16_t x) {
  if constexpr (BF16) return __bfloat162float(__ushort_as_bfloat16(x));
  return __half2float(__ushort_as_half(x));
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// One warp per (sequence, key/value head, key).
template <int D, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) key_weights_kernel(const uint16_t* q, const float* lse, float* weights,
                                                                  int weights_len, PagedKV c, const int* cu, int Hq,
                                                                  int total, int causal, float scale, float decay,
                                                                  int* err) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, b = blockIdx.z, g = blockIdx.y;
  const int G = Hq / c.hkv;
  int len = paged_len(c, b, err);
  if (len > weights_len) {
    atomicCAS(err, 0, ATTN_DEVERR_BAD_SEQLENS);
    len = 0;
  }
  int first;
  const int n_q = chunk_len(cu, b, total, first, err);
  for (int j = blockIdx.x * kWarps + (threadIdx.x >> 5); j < len; j += gridDim.x * kWarps) {
    const int page = paged_page(c, b, j >> c.page_log2, err);
    if (page < 0) continue;
    const long long at = page * c.s_page + (j & ((1 << c.page_log2) - 1)) * c.s_token + g * c.s_head;
    float kv[E];
#pragma unroll
    for (int e = 0; e < E; ++e) kv[e] = cvt<BF16>(c.k[at + lane + 32 * e]) * scale;
    float sum = 0.0f;
    for (int i = causal ? max(0, j - (len - n_q)) : 0; i < n_q; ++i)
      for (int x = 0; x < G; ++x) {
        const int h = g * G + x;
        const float l = __ldg(lse + static_cast<long long>(h) * total + first + i);
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e)
          s = fmaf(kv[e], cvt<BF16>(q[(static_cast<long long>(first + i) * Hq + h) * D + lane + 32 * e]), s);
        s = warp_sum(s);
        if (l != -INFINITY) sum += expf(s - l);
      }
    float* w = weights + (static_cast<long long>(b) * c.hkv + g) * weights_len + j;
    if (lane == 0) *w = (decay != 0.0f ? *w * decay : 0.0f) + sum;
  }
}

int run(bool decode, const void* q, void* o, float* lse, int B, int Hq, int total, const attn_paged_kv* cache,
        const int* cu, int causal, float scale, void* ws, long long ws_bytes, cudaStream_t stream) {
  PagedKV c;
  if (int rc = paged_check(cache, B, true, c)) return rc;
  if (!q || !o || !lse || !ptr_aligned(q, 16) || !ptr_aligned(o, 16) || !ptr_aligned(lse, 4)) return ATTN_EINVAL;
  if (Hq <= 0 || Hq % c.hkv != 0 || total < 0 || (causal != 0 && causal != 1)) return ATTN_EINVAL;
  if (!std::isfinite(scale) || scale < 0.0f) return ATTN_EINVAL;
  if (static_cast<long long>(total) * Hq > (1LL << 31) - 1 || total > (1 << 30)) return ATTN_EINVAL;
  if (!ws || !ptr_aligned(ws, 256) || ws_bytes < 256) return ATTN_EINVAL;
  if (total == 0) return ATTN_OK;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ELAUNCH;
  DeviceInfo info;
  if (int rc = device_info(dev, info)) return rc;
  if (!info.supported) return ATTN_EUNSUPPORTED;
  const int d = cache->head_dim;
  if (ws_bytes < (decode ? paged_decode_workspace(info.sm_count, d) : paged_fwd_workspace(info.sm_count, d)))
    return ATTN_EINVAL;
  const bool bf16 = cache->fp16 == 0;
  if (decode)
    return paged_decode(q, o, lse, B, Hq, c, d, bf16, cache->page_size, scale, ws, info.sm_count, info.err_word, stream);
  return paged_fwd(q, o, lse, B, Hq, total, c, d, bf16, cache->page_size, cu, causal != 0, scale, ws, info.sm_count,
                   info.err_word, stream);
}

}  // namespace
}  // namespace attn

extern "C" {

long long attn_paged_workspace_bytes(int d, int decode) {
  if (d != 64 && d != 128) return ATTN_EUNSUPPORTED;
  if (decode != 0 && decode != 1) return ATTN_EINVAL;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ELAUNCH;
  attn::DeviceInfo info;
  if (int rc = attn::device_info(dev, info)) return rc;
  return decode ? attn::paged_decode_workspace(info.sm_count, d) : attn::paged_fwd_workspace(info.sm_count, d);
}

int attn_fwd_paged(const void* q, void* o, float* lse, int B, int Hq, int total_q, const attn_paged_kv* cache,
                   const int* cu_seqlens_q, int causal, float scale, void* workspace, long long workspace_bytes,
                   cudaStream_t stream) {
  if (!cu_seqlens_q) return ATTN_EINVAL;
  return attn::run(false, q, o, lse, B, Hq, total_q, cache, cu_seqlens_q, causal, scale, workspace, workspace_bytes,
                   stream);
}

int attn_decode_paged(const void* q, void* o, float* lse, int B, int Hq, const attn_paged_kv* cache, float scale,
                      void* workspace, long long workspace_bytes, cudaStream_t stream) {
  return attn::run(true, q, o, lse, B, Hq, B, cache, nullptr, 0, scale, workspace, workspace_bytes, stream);
}

int attn_key_weights(const void* q, const float* lse, float* weights, int weights_len, int B, int Hq, int total_q,
                     const attn_paged_kv* cache, const int* cu_seqlens_q, int causal, float scale, float decay,
                     cudaStream_t stream) {
  using namespace attn;
  PagedKV c;
  if (int rc = paged_check(cache, B, false, c)) return rc;
  if (!q || !lse || !weights || !cu_seqlens_q || !ptr_aligned(q, 16) || !ptr_aligned(lse, 4) || !ptr_aligned(weights, 4))
    return ATTN_EINVAL;
  if (Hq <= 0 || Hq % c.hkv != 0 || total_q < 0 || weights_len <= 0 || (causal != 0 && causal != 1)) return ATTN_EINVAL;
  if (!std::isfinite(scale) || scale < 0.0f || !std::isfinite(decay)) return ATTN_EINVAL;
  if (static_cast<long long>(total_q) * Hq > (1LL << 31) - 1 || total_q > (1 << 30)) return ATTN_EINVAL;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ELAUNCH;
  DeviceInfo info;
  if (int rc = device_info(dev, info)) return rc;
  if (!info.supported) return ATTN_EUNSUPPORTED;
  const dim3 grid(64, c.hkv, B);
  auto* qp = static_cast<const uint16_t*>(q);
#define ATTN_RUN(D, T)                                                                                            \
  key_weights_kernel<D, T><<<grid, kWarps * 32, 0, stream>>>(qp, lse, weights, weights_len, c, cu_seqlens_q, Hq, \
                                                             total_q, causal, scale, decay, info.err_word)
  if (cache->head_dim == 64) {
    if (cache->fp16 == 0) ATTN_RUN(64, true);
    else ATTN_RUN(64, false);
  } else {
    if (cache->fp16 == 0) ATTN_RUN(128, true);
    else ATTN_RUN(128, false);
  }
#undef ATTN_RUN
  if (cudaGetLastError() != cudaSuccess) return ATTN_ELAUNCH;
  count_launch();
  return ATTN_OK;
}

}  // extern "C"
