// Launchers of the paged-cache kernels (arguments checked by the entry points).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "attn_paged.h"

namespace attn {

// 4-D TMA map over (d, H, L, N) of a 16-bit tensor whose features are
// contiguous, the other axes at the given strides (elements); box 64 x box_h x
// box_l x 1, 128-byte swizzle, fill 0.
int tile_map(const void* ptr, bool bf16, int d, int H, int L, int N, long long s_h, long long s_l, long long s_n,
             int box_h, int box_l, CUtensorMap& out);

long long paged_decode_workspace(int sms, int d);
int paged_decode(const void* q, void* o, float* lse, int B, int Hq, const PagedKV& c, int d, bool bf16, int page_size,
                 float scale, void* ws, int sms, int* err, cudaStream_t stream);

long long paged_fwd_workspace(int sms, int d);
int paged_fwd(const void* q, void* o, float* lse, int B, int Hq, int total, const PagedKV& c, int d, bool bf16,
              int page_size, const int* cu, bool causal, float scale, void* ws, int sms, int* err, cudaStream_t stream);

long long paged_weights_workspace(int sms);
int paged_weights(const void* q, const float* lse, float* weights, int weights_len, int B, int Hq, int total,
                  const PagedKV& c, int d, bool bf16, int page_size, const int* cu, bool causal, float scale,
                  float decay, void* ws, int sms, int* err, cudaStream_t stream);

}  // namespace attn
