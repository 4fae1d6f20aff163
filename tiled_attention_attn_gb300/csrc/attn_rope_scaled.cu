// Rotary embedding with given frequencies (attn_rotary_scaled), and the append
// of new tokens to a paged cache with the rotation of their queries and keys
// (attn_cache_append).
//
// Pair p of a token at position t turns by a = t f_p:
//   A (x1 cos a - x2 sin a, x1 sin a + x2 cos a),
// its gradient by -a.  The angle: f_p / 2 pi is held as a 64-bit fixed-point
// fraction of a turn, t times it modulo 2^64 is the fraction that the pair has
// turned at position t (whole turns fall out of the product), and its top 32
// bits give sincospi's argument in [-1, 1) with an error of 2^-25, at any
// position.  An fp32 product t * f_p would be off by t f_p 2^-24 radians,
// 2^-7 at position 131072.
//
// Bound by HBM: x read once, y written once.  A block takes a few rows
// (tokens): it first forms the rows' (cos, sin) tables in shared memory, once
// for all heads, and their places in the cache, then moves 16-byte words (two
// per thread and item: the 8 pairs' members), several items in flight.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attn_paged.h"

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 8;      // rows per block
constexpr int kMaxPairs = 256;   // rot_dim <= 512

// One tensor of the call.  Rows of `heads` heads; dst is contiguous (place 0)
// or the key (1) or value (2) pages.
struct Seg {
  const uint16_t* src;
  uint16_t* dst;
  long long src_token, src_head;
  int heads, place, rotate;
  int per;    // items per head
  int items;  // heads * per
};

struct RopeParams {
  Seg seg[3];
  int n_seg, items;             // items per row, all segments
  unsigned long long rows;
  int rows_per_block, d, rot, gptj, in_place;
  float amplitude, sin_sign;    // sin_sign: -1 for the gradient
  const int* cu;                // packed rows, or null: rows of L per sequence
  int L, B, total;
  const int* offsets;
  const int* positions;
  int append;
  PagedKV cache;
  int* err;
  unsigned long long turns[kMaxPairs];   // f_p / 2 pi, fixed point
};

template <bool BF16>
__device__ __forceinline__ float2 unpack(uint32_t w) {
  if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack(float a, float b) {
  if constexpr (BF16) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __half2 r = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <bool BF16>
__device__ __forceinline__ float ld1(const uint16_t* p) {
  if constexpr (BF16) return __bfloat162float(__ushort_as_bfloat16(*p));
  return __half2float(__ushort_as_half(*p));
}
template <bool BF16>
__device__ __forceinline__ void st1(uint16_t* p, float x) {
  if constexpr (BF16) *p = __bfloat16_as_ushort(__float2bfloat16_rn(x));
  else *p = __half_as_ushort(__float2half_rn(x));
}

// A row's place: its rotary position and, appending, where its token lies in
// the pages (elements from the cache's base; negative: the row is skipped).
__device__ __forceinline__ void locate(const RopeParams& p, long long row, int& pos, long long& at) {
  at = 0;
  pos = 0;
  int b, i, n = 0;
  if (p.positions && !p.append) {
    pos = __ldg(p.positions + row);
    return;
  }
  if (p.cu == nullptr) {
    b = static_cast<int>(row / p.L);
    i = static_cast<int>(row - static_cast<long long>(b) * p.L);
  } else {
    int lo = 0, hi = p.B;   // largest b with cu[b] <= row
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu + mid) <= row) lo = mid; else hi = mid;
    }
    b = lo;
    int first;
    n = chunk_len(p.cu, b, p.total, first, p.err);
    if (row < first || row >= static_cast<long long>(first) + n) {
      at = -1;
      return;
    }
    i = static_cast<int>(row - first);
  }
  pos = i + (p.offsets ? __ldg(p.offsets + b) : 0);
  if (p.append) {
    const int len = paged_len(p.cache, b, p.err);
    const int key = len - n + i;
    at = -1;
    if (key < 0) {
      atomicCAS(p.err, 0, ATTN_DEVERR_BAD_SEQLENS);
      return;
    }
    pos = p.positions ? __ldg(p.positions + row) : key;
    const int page = paged_page(p.cache, b, key >> p.cache.page_log2, p.err);
    if (page < 0) return;
    at = page * p.cache.s_page + (key & ((1 << p.cache.page_log2) - 1)) * p.cache.s_token;
  }
}

// VEC: items are 8 pairs (two 16-byte words) or 8 copied features; else one
// pair or one feature.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ float2 cs[];   // [row][pair] (A cos, A sin)
  __shared__ int s_pos[kMaxRows];
  __shared__ long long s_at[kMaxRows];
  const int tid = threadIdx.x;
  const long long row0 = static_cast<long long>(blockIdx.x) * p.rows_per_block;
  const int nr = static_cast<int>(min(static_cast<long long>(p.rows_per_block), static_cast<long long>(p.rows) - row0));
  if (tid < nr) locate(p, row0 + tid, s_pos[tid], s_at[tid]);
  if (p.append && blockIdx.x == 0) {
    // offsets that no row lookup meets
    int first;
    for (int b = tid; b < p.B; b += kThreads) chunk_len(p.cu, b, p.total, first, p.err);
  }
  __syncthreads();
  const int half = p.rot >> 1;
  for (int e = tid; e < nr * half; e += kThreads) {
    const int r = e / half, i = e - r * half;
    const unsigned long long turn = p.turns[i] * static_cast<unsigned long long>(static_cast<long long>(s_pos[r]));
    float sn, c;
    sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f, &sn, &c);   // 2^-31
    cs[e] = make_float2(c * p.amplitude, sn * p.amplitude * p.sin_sign);
  }
  __syncthreads();

  const int n = nr * p.items;
  constexpr int U = VEC ? 4 : 1;   // items in flight per thread
  const int groups = VEC ? half / 8 : half;
  for (int base = tid; base < n; base += kThreads * U) {
    uint4 va[U], vb[U];
    float sa[U], sb[U];
    const uint16_t* src[U];
    uint16_t* dst[U];
    int row[U], g[U], oa[U], ob[U];   // g: pair group, or -1: copied
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int it = base + u * kThreads;
      src[u] = nullptr;
      if (it >= n) continue;
      const int r = it / p.items;
      int rem = it - r * p.items;
      const long long at = s_at[r];
      if (at < 0) continue;
      int k = 0;
      while (k + 1 < p.n_seg && rem >= p.seg[k].items) rem -= p.seg[k++].items;
      const Seg& s = p.seg[k];
      const int h = rem / s.per, e = rem - h * s.per;
      row[u] = r;
      src[u] = s.src + (row0 + r) * s.src_token + h * s.src_head;
      dst[u] = s.place == 0 ? s.dst + ((row0 + r) * s.heads + h) * p.d : s.dst + at + h * p.cache.s_head;
      g[u] = (s.rotate && e < groups) ? e : -1;
      if constexpr (VEC) {
        if (g[u] >= 0) {
          // GPT-NeoX pairs (8g + e, half + 8g + e); GPT-J pairs (16g + 2e, 16g + 2e + 1)
          oa[u] = p.gptj ? 16 * e : 8 * e;
          ob[u] = p.gptj ? 16 * e + 8 : half + 8 * e;
          vb[u] = *reinterpret_cast<const uint4*>(src[u] + ob[u]);
        } else {
          oa[u] = s.rotate ? p.rot + 8 * (e - groups) : 8 * e;
        }
        va[u] = *reinterpret_cast<const uint4*>(src[u] + oa[u]);
      } else {
        if (g[u] >= 0) {
          oa[u] = p.gptj ? 2 * e : e;
          ob[u] = p.gptj ? 2 * e + 1 : half + e;
          sb[u] = ld1<BF16>(src[u] + ob[u]);
        } else {
          oa[u] = s.rotate ? p.rot + (e - groups) : e;
        }
        sa[u] = ld1<BF16>(src[u] + oa[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (src[u] == nullptr) continue;
      if constexpr (VEC) {
        if (g[u] < 0) {
          *reinterpret_cast<uint4*>(dst[u] + oa[u]) = va[u];
          continue;
        }
        const float2* t = cs + row[u] * half + 8 * g[u];
        uint32_t a[4] = {va[u].x, va[u].y, va[u].z, va[u].w}, b[4] = {vb[u].x, vb[u].y, vb[u].z, vb[u].w};
        if (p.gptj) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = unpack<BF16>(a[e]), y = unpack<BF16>(b[e]);
            const float2 ta = t[e], tb = t[4 + e];
            a[e] = pack<BF16>(x.x * ta.x - x.y * ta.y, x.x * ta.y + x.y * ta.x);
            b[e] = pack<BF16>(y.x * tb.x - y.y * tb.y, y.x * tb.y + y.y * tb.x);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = unpack<BF16>(a[e]), y = unpack<BF16>(b[e]);
            const float2 t0 = t[2 * e], t1 = t[2 * e + 1];
            a[e] = pack<BF16>(x.x * t0.x - y.x * t0.y, x.y * t1.x - y.y * t1.y);
            b[e] = pack<BF16>(x.x * t0.y + y.x * t0.x, x.y * t1.y + y.y * t1.x);
          }
        }
        *reinterpret_cast<uint4*>(dst[u] + oa[u]) = make_uint4(a[0], a[1], a[2], a[3]);
        *reinterpret_cast<uint4*>(dst[u] + ob[u]) = make_uint4(b[0], b[1], b[2], b[3]);
      } else {
        if (g[u] < 0) {
          st1<BF16>(dst[u] + oa[u], sa[u]);
          continue;
        }
        const float2 t = cs[row[u] * half + g[u]];
        st1<BF16>(dst[u] + oa[u], sa[u] * t.x - sb[u] * t.y);
        st1<BF16>(dst[u] + ob[u], sa[u] * t.y + sb[u] * t.x);
      }
    }
  }
}

// Checks the rotation's arguments and fills the turn table.
int fill_turns(RopeParams& p, int rot_dim, int d, const double* freqs, float amplitude, int interleaved) {
  if (rot_dim <= 0 || rot_dim > d || (rot_dim & 1) || rot_dim > 2 * kMaxPairs || !freqs) return ATTN_EINVAL;
  if (!std::isfinite(amplitude) || (interleaved != 0 && interleaved != 1)) return ATTN_EINVAL;
  for (int i = 0; i < rot_dim / 2; ++i) {
    if (!std::isfinite(freqs[i])) return ATTN_EINVAL;
    const double t = freqs[i] * 0.15915494309189533577;   // 1 / (2 pi)
    const double f = t - std::floor(t);                   // [0, 1]
    p.turns[i] = f >= 1.0 ? 0ull : static_cast<unsigned long long>(f * 18446744073709551616.0);
  }
  p.rot = rot_dim;
  p.gptj = interleaved;
  p.amplitude = amplitude;
  return ATTN_OK;
}

int launch(RopeParams& p, bool vec, bool bf16, cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ELAUNCH;
  DeviceInfo info;
  if (int rc = device_info(dev, info)) return rc;
  if (!info.supported) return ATTN_EUNSUPPORTED;
  p.err = info.err_word;
  p.items = 0;
  const int group = vec ? 8 : 1;
  for (int k = 0; k < p.n_seg; ++k) {
    Seg& s = p.seg[k];
    // in place the features past rot_dim stay where they are
    s.per = s.rotate ? p.rot / 2 / group + (p.in_place && s.place == 0 ? 0 : (p.d - p.rot) / group) : p.d / group;
    s.items = s.heads * s.per;
    p.items += s.items;
  }
  // few rows: one per block, so that every SM takes part; many: up to 8
  p.rows_per_block = static_cast<int>(
      std::min<unsigned long long>(kMaxRows, std::max<unsigned long long>(1, p.rows / (4ull * info.sm_count))));
  const unsigned long long grid = (p.rows + p.rows_per_block - 1) / p.rows_per_block;
  if (grid > 0x7fffffffull) return ATTN_EINVAL;
  const size_t smem = static_cast<size_t>(p.rows_per_block) * (p.rot / 2) * sizeof(float2);
  const int g = static_cast<int>(grid);
  if (vec) {
    if (bf16) rope_kernel<true, true><<<g, kThreads, smem, stream>>>(p);
    else rope_kernel<false, true><<<g, kThreads, smem, stream>>>(p);
  } else {
    if (bf16) rope_kernel<true, false><<<g, kThreads, smem, stream>>>(p);
    else rope_kernel<false, false><<<g, kThreads, smem, stream>>>(p);
  }
  if (cudaGetLastError() != cudaSuccess) return ATTN_ELAUNCH;
  count_launch();
  return ATTN_OK;
}

// Whether [a, a + na) and [b, b + nb) share bytes.
bool overlap(const void* a, unsigned long long na, const void* b, unsigned long long nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}
// Bytes from the first to past the last element of a strided (rows, heads, d) tensor.
unsigned long long extent(unsigned long long rows, long long st, int heads, long long sh, int d) {
  return rows == 0 ? 0 : 2 * ((rows - 1) * st + (heads - 1) * sh + d);
}

}  // namespace
}  // namespace attn

extern "C" {

int attn_rotary_scaled(const void* x, void* y, int B, int L, int H, int d, int rot_dim, const double* freqs,
                       float amplitude, int interleaved, int inverse, long long x_stride_token,
                       long long x_stride_head, const int* cu_seqlens_or_null, int total,
                       const int* offsets_or_null, const int* positions_or_null, int fp16, cudaStream_t stream) {
  using namespace attn;
  if (!x || !y || B <= 0 || H <= 0 || d <= 0 || H > (1 << 20) || d > (1 << 16) || (fp16 != 0 && fp16 != 1) ||
      (inverse != 0 && inverse != 1))
    return ATTN_EINVAL;
  if (!ptr_aligned(x, 2) || !ptr_aligned(y, 2)) return ATTN_EINVAL;
  const bool packed = cu_seqlens_or_null != nullptr;
  if (packed ? total < 0 : L < 0) return ATTN_EINVAL;
  if (positions_or_null && (offsets_or_null || packed)) return ATTN_EINVAL;
  if (x_stride_head < d || x_stride_token < d || x_stride_head > (1LL << 40) || x_stride_token > (1LL << 40)) return ATTN_EINVAL;
  static thread_local RopeParams p;
  p = RopeParams{};
  p.d = d;
  if (int rc = fill_turns(p, rot_dim, d, freqs, amplitude, interleaved)) return rc;
  p.rows = packed ? static_cast<unsigned long long>(total) : static_cast<unsigned long long>(B) * L;
  if (p.rows > 0x7fffffffull || p.rows * H > (1ull << 40) / d) return ATTN_EINVAL;
  if (static_cast<long long>(H) * d > (1 << 26)) return ATTN_EINVAL;   // a block's items are 32-bit
  const bool same = x == y;
  if (same && (x_stride_head != d || x_stride_token != static_cast<long long>(H) * d)) return ATTN_EINVAL;
  if (!same && overlap(x, extent(p.rows, x_stride_token, H, x_stride_head, d), y, p.rows * H * d * 2))
    return ATTN_EINVAL;
  if (p.rows == 0) return ATTN_OK;
  p.in_place = same;
  p.sin_sign = inverse ? -1.0f : 1.0f;
  p.cu = cu_seqlens_or_null;
  p.L = L;
  p.B = B;
  p.total = total;
  p.offsets = offsets_or_null;
  p.positions = positions_or_null;
  p.n_seg = 1;
  p.seg[0] = Seg{static_cast<const uint16_t*>(x), static_cast<uint16_t*>(y), x_stride_token, x_stride_head, H, 0, 1, 0, 0};
  const bool vec = rot_dim % 16 == 0 && d % 8 == 0 && x_stride_token % 8 == 0 && x_stride_head % 8 == 0 &&
                   ptr_aligned(x, 16) && ptr_aligned(y, 16);
  return launch(p, vec, fp16 == 0, stream);
}

int attn_cache_append(const void* q, const void* k, const void* v, void* q_out, long long q_stride_token,
                      long long k_stride_token, long long v_stride_token, int B, int Hq, int total,
                      const attn_paged_kv* cache, const int* cu_seqlens, int rot_dim, const double* freqs_or_null,
                      float amplitude, int interleaved, const int* positions_or_null, cudaStream_t stream) {
  using namespace attn;
  static thread_local RopeParams p;
  p = RopeParams{};
  if (int rc = paged_check(cache, B, true, p.cache)) return rc;
  if (!cu_seqlens || total < 0 || (q == nullptr) != (q_out == nullptr)) return ATTN_EINVAL;
  const int d = cache->head_dim, hkv = cache->num_kv_heads;
  if (q && (Hq <= 0 || Hq > 65535 || !freqs_or_null)) return ATTN_EINVAL;
  if (total == 0) return ATTN_OK;
  if (!k || !v) return ATTN_EINVAL;
  p.d = d;
  if (freqs_or_null) {
    if (int rc = fill_turns(p, rot_dim, d, freqs_or_null, amplitude, interleaved)) return rc;
  }
  const void* base[3] = {q, k, v};
  const long long st[3] = {q_stride_token, k_stride_token, v_stride_token};
  const int heads[3] = {Hq, hkv, hkv};
  for (int i = q ? 0 : 1; i < 3; ++i) {
    if (!ptr_aligned(base[i], 16) || st[i] % 8 != 0 || st[i] < static_cast<long long>(heads[i]) * d || st[i] > (1LL << 40))
      return ATTN_EINVAL;
    Seg& s = p.seg[p.n_seg++];
    s.src = static_cast<const uint16_t*>(base[i]);
    s.dst = i == 0 ? static_cast<uint16_t*>(q_out) : i == 1 ? p.cache.k : p.cache.v;
    s.src_token = st[i];
    s.src_head = d;
    s.heads = heads[i];
    s.place = i;
    s.rotate = i < 2 && freqs_or_null != nullptr;
  }
  p.in_place = q != nullptr && q == q_out;
  if (q) {
    if (!ptr_aligned(q_out, 16) || (p.in_place && q_stride_token != static_cast<long long>(Hq) * d)) return ATTN_EINVAL;
    const unsigned long long nq = static_cast<unsigned long long>(total) * Hq * d * 2;
    for (int i = p.in_place ? 1 : 0; i < 3; ++i)
      if (overlap(base[i], extent(total, st[i], heads[i], d, d), q_out, nq)) return ATTN_EINVAL;
  }
  p.rows = total;
  p.sin_sign = 1.0f;
  p.cu = cu_seqlens;
  p.B = B;
  p.total = total;
  p.positions = positions_or_null;
  p.append = 1;
  return launch(p, !freqs_or_null || rot_dim % 16 == 0, cache->fp16 == 0, stream);
}

}  // extern "C"
