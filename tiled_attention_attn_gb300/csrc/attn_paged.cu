// Entry points of attention over a paged key/value cache (attn_fwd_paged,
// attn_decode_paged) and of the accumulated key weights (attn_key_weights):
// argument checks; the kernels are in attn_paged_fwd.cu, attn_paged_decode.cu
// and attn_paged_weights.cu.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "attn_paged_launch.h"

namespace attn {
namespace {

// The checks that the three share.  `total`: rows of q.
int check(const attn_paged_kv* cache, int B, bool need_v, const void* q, const float* lse, int Hq, int total,
          int causal, float scale, const void* ws, long long ws_bytes, PagedKV& c) {
  if (int rc = paged_check(cache, B, need_v, c)) return rc;
  if (Hq <= 0 || Hq % c.hkv != 0 || total < 0 || (causal != 0 && causal != 1)) return ATTN_EINVAL;
  if (total > 0 && (!q || !lse)) return ATTN_EINVAL;
  if (!ptr_aligned(q, 16) || !ptr_aligned(lse, 4)) return ATTN_EINVAL;
  if (!std::isfinite(scale) || scale < 0.0f) return ATTN_EINVAL;
  if (static_cast<long long>(total) * Hq > (1LL << 31) - 1 || total > (1 << 30)) return ATTN_EINVAL;
  if (!ws || !ptr_aligned(ws, 256) || ws_bytes < 256) return ATTN_EINVAL;
  return ATTN_OK;
}

int device(DeviceInfo& info) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ELAUNCH;
  if (int rc = device_info(dev, info)) return rc;
  return info.supported ? ATTN_OK : ATTN_EUNSUPPORTED;
}

}  // namespace
}  // namespace attn

extern "C" {

long long attn_paged_workspace_bytes(int d, int call) {
  using namespace attn;
  if (d != 64 && d != 128) return ATTN_EUNSUPPORTED;
  if (call < ATTN_PAGED_CHUNK || call > ATTN_PAGED_WEIGHTS) return ATTN_EINVAL;
  DeviceInfo info;
  if (int rc = device(info)) return rc;
  return call == ATTN_PAGED_CHUNK    ? paged_fwd_workspace(info.sm_count, d)
         : call == ATTN_PAGED_DECODE ? paged_decode_workspace(info.sm_count, d)
                                     : paged_weights_workspace(info.sm_count);
}

int attn_fwd_paged(const void* q, void* o, float* lse, int B, int Hq, int total_q, const attn_paged_kv* cache,
                   const int* cu_seqlens_q, int causal, float scale, void* workspace, long long workspace_bytes,
                   cudaStream_t stream) {
  using namespace attn;
  PagedKV c;
  if (int rc = check(cache, B, true, q, lse, Hq, total_q, causal, scale, workspace, workspace_bytes, c)) return rc;
  if (!cu_seqlens_q || (total_q > 0 && !o) || !ptr_aligned(o, 16)) return ATTN_EINVAL;
  if (total_q == 0) return ATTN_OK;
  DeviceInfo info;
  if (int rc = device(info)) return rc;
  if (workspace_bytes < paged_fwd_workspace(info.sm_count, cache->head_dim)) return ATTN_EINVAL;
  return paged_fwd(q, o, lse, B, Hq, total_q, c, cache->head_dim, cache->fp16 == 0, cache->page_size, cu_seqlens_q,
                   causal != 0, scale, workspace, info.sm_count, info.err_word, stream);
}

int attn_decode_paged(const void* q, void* o, float* lse, int B, int Hq, const attn_paged_kv* cache, float scale,
                      void* workspace, long long workspace_bytes, cudaStream_t stream) {
  using namespace attn;
  PagedKV c;
  if (int rc = check(cache, B, true, q, lse, Hq, B, 0, scale, workspace, workspace_bytes, c)) return rc;
  if (!o || !ptr_aligned(o, 16)) return ATTN_EINVAL;
  DeviceInfo info;
  if (int rc = device(info)) return rc;
  if (workspace_bytes < paged_decode_workspace(info.sm_count, cache->head_dim)) return ATTN_EINVAL;
  return paged_decode(q, o, lse, B, Hq, c, cache->head_dim, cache->fp16 == 0, cache->page_size, scale, workspace,
                      info.sm_count, info.err_word, stream);
}

int attn_key_weights(const void* q, const float* lse, float* weights, int weights_len, int B, int Hq, int total_q,
                     const attn_paged_kv* cache, const int* cu_seqlens_q, int causal, float scale, float decay,
                     void* workspace, long long workspace_bytes, cudaStream_t stream) {
  using namespace attn;
  PagedKV c;
  if (int rc = check(cache, B, false, q, lse, Hq, total_q, causal, scale, workspace, workspace_bytes, c)) return rc;
  // (below 2^-20 a left-out query's -kFar scale, in fp16, would come near exp2's range)
  if (scale != 0.0f && scale < 0x1p-20f) return ATTN_EINVAL;
  if (!weights || !cu_seqlens_q || !ptr_aligned(weights, 4) || weights_len <= 0 || !std::isfinite(decay)) return ATTN_EINVAL;
  DeviceInfo info;
  if (int rc = device(info)) return rc;
  if (workspace_bytes < paged_weights_workspace(info.sm_count)) return ATTN_EINVAL;
  // without queries the maps still need an address: the weights alone change
  const void* base = total_q > 0 ? q : cache->k;
  return paged_weights(base, lse, weights, weights_len, B, Hq, total_q, c, cache->head_dim, cache->fp16 == 0,
                       cache->page_size, cu_seqlens_q, causal != 0, scale, decay, workspace, info.sm_count,
                       info.err_word, stream);
}

}  // extern "C"
