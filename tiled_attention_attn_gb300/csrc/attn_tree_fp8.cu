// Entry points of the attention over paged caches of 8-bit floating point
// (attn_tree_fp8): argument checks; the kernels are in
// attn_tree_fp8_kernel.cuh and attn_tree_fp8_rows.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attn_paged_launch.h"
#include "attn_paged_line.cuh"
#include "attn_tree_fp8.h"

namespace attn {
namespace tree {
namespace {

size_t rec_bytes(int sms) { return (static_cast<size_t>(sms) * sizeof(int4) + 255) / 256 * 256; }
size_t ml_bytes(int sms) { return static_cast<size_t>(2 * sms) * kRowsPerUnit * sizeof(float2); }
long long workspace(int sms, int d) {
  return static_cast<long long>(rec_bytes(sms) + ml_bytes(sms) + static_cast<size_t>(2 * sms) * kRowsPerUnit * d * sizeof(float));
}

int device(DeviceInfo& info) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ELAUNCH;
  if (int rc = device_info(dev, info)) return rc;
  return info.supported ? ATTN_OK : ATTN_EUNSUPPORTED;
}

}  // namespace
}  // namespace tree
}  // namespace attn

extern "C" {

long long attn_fp8_workspace_bytes(int d) {
  using namespace attn;
  if (d != 64 && d != 128) return ATTN_EUNSUPPORTED;
  DeviceInfo info;
  if (int rc = tree::device(info)) return rc;
  return tree::workspace(info.sm_count, d);
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
  DeviceInfo info;
  if (int rc = tree::device(info)) return rc;
  const int sms = info.sm_count;
  if (workspace_bytes < tree::workspace(sms, d)) return ATTN_EINVAL;
  const int page = cache->page_size, box = std::min(page, tree::kKeys);
  for (int i = 0; i < 2; ++i)
    if (int rc = byte_map(i == 0 ? p.c.k : p.c.v, d, p.c.t.hkv, page, p.c.t.num_pages, p.c.s_head, p.c.s_token, p.c.s_page,
                          box, i == 0 || d == 128 ? d : 0, i == 0 ? p.tm_k : p.tm_v))
      return rc;
  char* ws = static_cast<char*>(workspace);
  p.rec = reinterpret_cast<int4*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + tree::rec_bytes(sms));
  p.part_o = reinterpret_cast<float*>(ws + tree::rec_bytes(sms) + tree::ml_bytes(sms));
  p.q = static_cast<const uint16_t*>(q);
  p.o = static_cast<uint16_t*>(o);
  p.lse = lse;
  p.cu = cu_seqlens_or_null;
  p.mask = tree_mask_or_null;
  p.err = info.err_word;
  p.timeout_ns = wait_timeout_ns();
  p.B = B;
  p.Hq = Hq;
  p.total = total;
  p.max_tokens = cu_seqlens_or_null ? max_tokens : 1;
  p.group = Hq / p.c.t.hkv;
  // Up to 8 columns (token, head) of a key/value head are a unit of the kernel that has
  // them as columns; more are rows, 128 to a unit, and the units of a head each read the
  // keys.  (8 sequences of 1,000 to 16,384 keys, 8 heads of 128: 8 columns 44.5 us against
  // 60 as rows, 16 columns 63 against 60.6; 16 sequences of 4 heads, 32 columns 60 against 36.)
  const long long cols = static_cast<long long>(p.max_tokens) * p.group;
  if (cols > (1 << 20)) return ATTN_EINVAL;
  const bool rows = cols > tree::kMostCols;
  const int unit = rows ? tree::kRowsPerUnit : tree::kMostCols;
  p.parts = static_cast<int>((cols + unit - 1) / unit);
  p.abreast = heads_abreast(p.c.t.hkv * p.parts, sms);
  p.cuts = (p.c.t.max_pages << p.c.t.page_log2) > tree::kMinSteps * (d == 64 && !rows ? 256 : 128);
  p.fp16 = fp16;
  p.inv_group = 1.0f / static_cast<float>(p.group);
  p.scale_log2 = scale * 1.4426950408889634f;
  const int most = static_cast<int>(std::min<long long>(cols, unit));
  cudaError_t e;
  if (rows) e = d == 64 ? tree::launch_rows_d64(p, most, sms, stream) : tree::launch_rows_d128(p, most, sms, stream);
  else e = d == 64 ? tree::launch_d64(p, most, sms, stream) : tree::launch_d128(p, most, sms, stream);
  return e == cudaSuccess ? ATTN_OK : ATTN_ELAUNCH;
}

}  // extern "C"
