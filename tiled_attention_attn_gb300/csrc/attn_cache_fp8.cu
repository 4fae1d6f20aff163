// Caches of 8-bit floating point: new tokens quantised as they are written to
// the pages, with the rotary embedding of their queries and keys
// (attn_cache_append_fp8), and keys and values read back in 16 bits
// (attn_cache_read_fp8).
//
// A row x (the features of one token and head) is held as e4m3 values v and one
// fp32 scale s, x ~ v s:
//   s = max(max |x| / 448, 2^-126),   v = e4m3(x / s), to nearest even;
// a row with an infinity or a NaN has s = NaN and v = 0.  Keys are turned in fp32 first and
// rounded once, to e4m3.  e4m3 being a floating type, v is off by at most 2^-4 of
// itself, or 2^-10 s below 2^-6 s.  The quotient is the IEEE one: a product with
// 1 / s is off by an ulp, which moves values that lie on a border between two
// e4m3 values, and rows whose largest is a power of two have many of those.
//
// Bound by HBM: q, k and v read once; q written in 16 bits, k and v in 8 and a
// scale per row.  A lane holds 16 features of a head as two 16-byte words that
// contain its pairs whole, 4 or 8 lanes a head, so the row's maximum is 2 or 3
// shuffles.  A warp takes a token (with few tokens a part of its heads), two heads
// in flight per lane and step.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attn.h"
#include "attn_fp8.h"
#include "attn_turns.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 64;   // head_dim <= 128

struct AppendParams {
  const uint16_t* x[3];   // q (or null), k, v
  long long s_token[3];   // heads of a token are contiguous
  uint16_t* q_out;
  int Hq;
  int rows, parts, B;
  int d, lg;              // log2 of the lanes per head
  int rot;
  float amplitude;
  const int* cu;
  const int* positions;
  PagedKV8 c;
  int* err;
  unsigned long long turns[kMaxPairs];
};

// The sequence that a packed row belongs to, its index there and the sequence's
// rows; false outside every sequence.
__device__ __forceinline__ bool find(const int* cu, int B, int total, int row, int& b, int& i, int& n, int* err) {
  int lo = 0, hi = B;   // largest b with cu[b] <= row
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= row) lo = mid; else hi = mid;
  }
  b = lo;
  int first;
  n = chunk_len(cu, b, total, first, err);
  i = row - first;
  return i >= 0 && i < n;
}

template <bool BF16, bool GPTJ>
__global__ void __launch_bounds__(kThreads, 3) append_kernel(const __grid_constant__ AppendParams p) {
  extern __shared__ float4 tables[];
  constexpr int U = 2;   // heads in flight
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lanes = 1 << p.lg, sub = lane >> p.lg, e = lane & (lanes - 1), per = 32 >> p.lg;
  const int groups = p.rot >> 4;
  const bool turns_here = e < groups;
  const int lo = !GPTJ && turns_here ? 8 * e : 16 * e;
  const int hi = !GPTJ && turns_here ? (p.rot >> 1) + 8 * e : lo + 8;
  float2* cs_tab = reinterpret_cast<float2*>(tables) + warp * (p.rot >> 1);
  if (blockIdx.x == 0) {
    // offsets that no row lookup meets
    int first;
    for (int b = threadIdx.x; b < p.B; b += kThreads) chunk_len(p.cu, b, p.rows, first, p.err);
  }
  const long long tasks = static_cast<long long>(p.rows) * p.parts;
  for (long long task = static_cast<long long>(blockIdx.x) * kWarps + warp; task < tasks;
       task += static_cast<long long>(gridDim.x) * kWarps) {
    const int row = static_cast<int>(task / p.parts), part = static_cast<int>(task - static_cast<long long>(row) * p.parts);
    int b, i, n;
    if (!find(p.cu, p.B, p.rows, row, b, i, n, p.err)) continue;
    const int key = paged_len(p.c.t, b, p.err) - n + i;
    if (key < 0) {
      if (lane == 0) atomicCAS(p.err, 0, ATTN_DEVERR_BAD_SEQLENS);
      continue;
    }
    const int page = paged_page(p.c.t, b, key >> p.c.t.page_log2, p.err);
    if (page < 0) continue;
    const int slot = key & ((1 << p.c.t.page_log2) - 1);
    const int pos = p.positions ? __ldg(p.positions + row) : key;
    __syncwarp();   // the table's readers of the token before
    for (int t = lane; t < p.rot >> 1; t += 32) {
      const float2 f = turned(p.turns[t], pos);
      cs_tab[(((t & 7) >> 1) * groups + (t >> 3)) * 2 + (t & 1)] = make_float2(f.x * p.amplitude, f.y * p.amplitude);
    }
    __syncwarp();
    float2 cs[8];
    if (turns_here) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float4 f = reinterpret_cast<const float4*>(cs_tab)[t * groups + e];
        cs[2 * t] = make_float2(f.x, f.y);
        cs[2 * t + 1] = make_float2(f.z, f.w);
      }
    }
#pragma unroll 1
    for (int k = 0; k < 3; ++k) {
      const int heads = k == 0 ? p.Hq : p.c.t.hkv;
      const uint16_t* x = p.x[k] + row * p.s_token[k];
      uint8_t* dst = (k == 1 ? p.c.k : p.c.v) + page * p.c.s_page + slot * p.c.s_token;
      float* scales = (k == 1 ? p.c.ks : p.c.vs) + page * p.c.c_page + slot * p.c.c_token;
      for (int h0 = part * per; h0 < heads; h0 += U * p.parts * per) {
        uint4 a[U], c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = h0 + u * p.parts * per + sub;
          a[u] = c[u] = make_uint4(0, 0, 0, 0);
          if (h < heads) {
            a[u] = *reinterpret_cast<const uint4*>(x + h * p.d + lo);
            c[u] = *reinterpret_cast<const uint4*>(x + h * p.d + hi);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = h0 + u * p.parts * per + sub;
          float z[16];
          widen<BF16>(a[u], c[u], z);
          if (turns_here && k < 2) turn<GPTJ>(z, cs, 1.0f);
          if (k == 0) {
            if (h < heads) {
              uint4 oa, ob;
              narrow<BF16>(z, oa, ob);
              uint16_t* y = p.q_out + (static_cast<long long>(row) * heads + h) * p.d;
              *reinterpret_cast<uint4*>(y + lo) = oa;
              *reinterpret_cast<uint4*>(y + hi) = ob;
            }
            continue;
          }
          // the row's largest magnitude, as bits: a NaN counts above infinity
          uint32_t top = 0;
#pragma unroll
          for (int t = 0; t < 16; ++t) top = max(top, __float_as_uint(z[t]) & 0x7fffffffu);
          for (int o = lanes >> 1; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
          const bool finite = top < 0x7f800000u;
          const float s = finite ? fmaxf(__uint_as_float(top) / kE4M3Top, kLeastScale) : __uint_as_float(0x7fffffffu);
          uint32_t w[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint32_t l = __nv_cvt_float2_to_fp8x2(make_float2(z[4 * t] / s, z[4 * t + 1] / s), __NV_SATFINITE, __NV_E4M3);
            const uint32_t r = __nv_cvt_float2_to_fp8x2(make_float2(z[4 * t + 2] / s, z[4 * t + 3] / s), __NV_SATFINITE, __NV_E4M3);
            w[t] = finite ? l | r << 16 : 0;
          }
          if (h < heads) {
            uint8_t* y = dst + h * p.c.s_head;
            *reinterpret_cast<uint2*>(y + lo) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint2*>(y + hi) = make_uint2(w[2], w[3]);
            if (e == 0) scales[h * p.c.c_head] = s;
          }
        }
      }
    }
  }
}

struct ReadParams {
  uint16_t* k;
  uint16_t* v;
  const int* cu;
  const int* starts;   // or null: 0
  int rows, parts, B;
  int d, lg;
  PagedKV8 c;
  int* err;
};

// 16 e4m3 values times s, rounded once to 16 bits.
template <bool BF16>
__device__ __forceinline__ void scaled(const uint4& x, float s, uint4& a, uint4& b) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
  float z[16];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u[t] >> (16 * i)), __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      z[4 * t + 2 * i] = f.x * s;
      z[4 * t + 2 * i + 1] = f.y * s;
    }
  }
  narrow<BF16>(z, a, b);
}

// A warp reads a row (token), or with few rows a part of its heads: 16 values per
// lane and load, keys and values of two steps in flight.
template <bool BF16>
__global__ void __launch_bounds__(kThreads, 4) read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int U = 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lanes = 1 << p.lg, sub = lane >> p.lg, e = lane & (lanes - 1), per = 32 >> p.lg, heads = p.c.t.hkv;
  if (blockIdx.x == 0) {
    int first;
    for (int b = threadIdx.x; b < p.B; b += kThreads) chunk_len(p.cu, b, p.rows, first, p.err);
  }
  const long long tasks = static_cast<long long>(p.rows) * p.parts;
  for (long long task = static_cast<long long>(blockIdx.x) * kWarps + warp; task < tasks;
       task += static_cast<long long>(gridDim.x) * kWarps) {
    const int row = static_cast<int>(task / p.parts), part = static_cast<int>(task - static_cast<long long>(row) * p.parts);
    int b, i, n;
    if (!find(p.cu, p.B, p.rows, row, b, i, n, p.err)) continue;
    const long long at = static_cast<long long>(i) + (p.starts ? __ldg(p.starts + b) : 0);
    if (at < 0 || at >= paged_len(p.c.t, b, p.err)) {
      if (lane == 0) atomicCAS(p.err, 0, ATTN_DEVERR_BAD_SEQLENS);
      continue;
    }
    const int key = static_cast<int>(at);
    const int page = paged_page(p.c.t, b, key >> p.c.t.page_log2, p.err);
    if (page < 0) continue;
    const int slot = key & ((1 << p.c.t.page_log2) - 1);
    const long long from = page * p.c.s_page + slot * p.c.s_token, scale = page * p.c.c_page + slot * p.c.c_token;
    const long long to = static_cast<long long>(row) * heads;
    for (int h0 = part * per; h0 < heads; h0 += U * p.parts * per) {
      uint4 x[U][2];
      float s[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * p.parts * per + sub;
        if (h < heads) {
          x[u][0] = *reinterpret_cast<const uint4*>(p.c.k + from + h * p.c.s_head + 16 * e);
          x[u][1] = *reinterpret_cast<const uint4*>(p.c.v + from + h * p.c.s_head + 16 * e);
          s[u][0] = p.c.ks[scale + h * p.c.c_head];
          s[u][1] = p.c.vs[scale + h * p.c.c_head];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * p.parts * per + sub;
        if (h >= heads) continue;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint4 a, c;
          scaled<BF16>(x[u][k], s[u][k], a, c);
          uint4* y = reinterpret_cast<uint4*>((k == 0 ? p.k : p.v) + (to + h) * p.d + 16 * e);
          y[0] = a;
          y[1] = c;
        }
      }
    }
  }
}

int device(DeviceInfo& info) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ELAUNCH;
  if (int rc = device_info(dev, info)) return rc;
  return info.supported ? ATTN_OK : ATTN_EUNSUPPORTED;
}

// Warps per row: one once the rows fill the GPU's warps, below that a row's heads
// are shared by up to 8.
int parts_of(int rows, int heads, int lg, int per_sm, int sms) {
  const long long slots = static_cast<long long>(per_sm) * kWarps * sms;
  const int per = 32 >> lg;
  return static_cast<int>(std::max<long long>(1, std::min<long long>({8, slots / std::max(rows, 1), (heads + per - 1) / per})));
}
int grid_of(int rows, int parts, int per_sm, int sms) {
  const long long tasks = static_cast<long long>(rows) * parts;
  return static_cast<int>(std::min<long long>((tasks + kWarps - 1) / kWarps, static_cast<long long>(per_sm) * sms));
}

}  // namespace
}  // namespace attn

extern "C" {

int attn_cache_append_fp8(const void* q, const void* k, const void* v, void* q_out, long long q_stride_token,
                          long long k_stride_token, long long v_stride_token, int B, int Hq, int total,
                          const attn_paged_kv8* cache, const int* cu_seqlens, int rot_dim, const double* freqs_or_null,
                          float amplitude, int interleaved, const int* positions_or_null, int fp16, cudaStream_t stream) {
  using namespace attn;
  AppendParams p = {};
  if (int rc = paged8_check(cache, B, p.c)) return rc;
  if (!cu_seqlens || total < 0 || (q == nullptr) != (q_out == nullptr) || (fp16 != 0 && fp16 != 1)) return ATTN_EINVAL;
  const int d = cache->head_dim, hkv = cache->num_kv_heads;
  if (q && (Hq <= 0 || Hq > 65535 || !freqs_or_null)) return ATTN_EINVAL;
  if (total == 0) return ATTN_OK;
  if (!k || !v) return ATTN_EINVAL;
  if (freqs_or_null) {
    if (rot_dim <= 0 || rot_dim > d || (rot_dim & 1) || !std::isfinite(amplitude)) return ATTN_EINVAL;
    if (interleaved != 0 && interleaved != 1) return ATTN_EINVAL;
    if (rot_dim % 16 != 0) return ATTN_EUNSUPPORTED;
    for (int i = 0; i < rot_dim / 2; ++i) {
      if (!std::isfinite(freqs_or_null[i])) return ATTN_EINVAL;
      p.turns[i] = turn_of(freqs_or_null[i]);
    }
    p.rot = rot_dim;
    p.amplitude = amplitude;
  }
  const void* base[3] = {q, k, v};
  const long long st[3] = {q_stride_token, k_stride_token, v_stride_token};
  const int heads[3] = {q ? Hq : 0, hkv, hkv};
  const bool same = q != nullptr && q == q_out;
  const unsigned long long nq = 2ull * total * heads[0] * d;
  for (int i = 0; i < 3; ++i) {
    if (heads[i] == 0) continue;
    if (!ptr_aligned(base[i], 16) || st[i] % 8 != 0 || st[i] < static_cast<long long>(heads[i]) * d || st[i] > (1LL << 40))
      return ATTN_EINVAL;
    if (q && !(i == 0 && same) && overlap(base[i], extent(total, st[i], heads[i], d, d), q_out, nq)) return ATTN_EINVAL;
    p.x[i] = static_cast<const uint16_t*>(base[i]);
    p.s_token[i] = st[i];
  }
  if (q && (!ptr_aligned(q_out, 16) || (same && q_stride_token != static_cast<long long>(Hq) * d))) return ATTN_EINVAL;
  DeviceInfo info;
  if (int rc = device(info)) return rc;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.Hq = heads[0];
  p.rows = total;
  p.B = B;
  p.d = d;
  p.lg = d == 128 ? 3 : 2;
  p.cu = cu_seqlens;
  p.positions = positions_or_null;
  p.err = info.err_word;
  constexpr int kPerSM = 3;
  p.parts = parts_of(total, std::max(p.Hq, hkv), p.lg, kPerSM, info.sm_count);
  const int grid = grid_of(total, p.parts, kPerSM, info.sm_count);
  const size_t smem = static_cast<size_t>(kWarps) * (p.rot / 2) * sizeof(float2);
  if (fp16 == 0) interleaved ? append_kernel<true, true><<<grid, kThreads, smem, stream>>>(p)
                             : append_kernel<true, false><<<grid, kThreads, smem, stream>>>(p);
  else interleaved ? append_kernel<false, true><<<grid, kThreads, smem, stream>>>(p)
                   : append_kernel<false, false><<<grid, kThreads, smem, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ELAUNCH;
  count_launch();
  return ATTN_OK;
}

int attn_cache_read_fp8(void* k, void* v, int B, int total, const attn_paged_kv8* cache, const int* cu_seqlens,
                        const int* starts_or_null, int fp16, cudaStream_t stream) {
  using namespace attn;
  ReadParams p = {};
  if (int rc = paged8_check(cache, B, p.c)) return rc;
  if (!cu_seqlens || total < 0 || (fp16 != 0 && fp16 != 1)) return ATTN_EINVAL;
  if (total == 0) return ATTN_OK;
  if (!k || !v || !ptr_aligned(k, 16) || !ptr_aligned(v, 16)) return ATTN_EINVAL;
  const int d = cache->head_dim, hkv = cache->num_kv_heads;
  const unsigned long long n = 2ull * total * hkv * d;
  if (overlap(k, n, v, n)) return ATTN_EINVAL;
  DeviceInfo info;
  if (int rc = device(info)) return rc;
  p.k = static_cast<uint16_t*>(k);
  p.v = static_cast<uint16_t*>(v);
  p.cu = cu_seqlens;
  p.starts = starts_or_null;
  p.rows = total;
  p.B = B;
  p.d = d;
  p.lg = d == 128 ? 3 : 2;
  p.err = info.err_word;
  constexpr int kPerSM = 4;
  p.parts = parts_of(total, hkv, p.lg, kPerSM, info.sm_count);
  const int grid = grid_of(total, p.parts, kPerSM, info.sm_count);
  if (fp16 == 0) read_kernel<true><<<grid, kThreads, 0, stream>>>(p);
  else read_kernel<false><<<grid, kThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ELAUNCH;
  count_launch();
  return ATTN_OK;
}

}  // extern "C"
