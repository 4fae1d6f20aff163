// Rotary embedding with given frequencies (attn_rotary_scaled), and the append
// of new tokens to a paged cache with the rotation of their queries and keys
// (attn_cache_append).
//
// Pair p of a token at position t turns by a = t f_p:
//   A (x1 cos a - x2 sin a, x1 sin a + x2 cos a),
// its gradient by -a.  The angle: f_p / 2 pi, formed in two doubles, is held as a
// 64-bit fixed-point fraction of a turn, t times it modulo 2^64 is the fraction
// that the pair has turned at position t (whole turns fall out of the product),
// and its top 32 bits give sincospi's argument in [-1, 1).  The fraction is off by
// t (2^-63 + |f_p| 2^-105) turns, 2^-32 at position 2^31 (for |f_p| up to 2^40),
// the argument by the 2^-25 of its rounding to fp32.  An fp32 product t * f_p
// would be off by t f_p 2^-24 radians, 2^-7 at position 131072.
//
// Bound by HBM: x read once, y written once.  A warp takes a row (token), or
// with few rows a part of its heads: it finds the token's place, forms the
// pairs' (cos, sin) once for all heads in its part of shared memory, and moves
// 16-byte words, four loads in flight per lane.  No block-wide barrier: the
// other 31 warps of the SM (registers held to 64) hide each one's start.  Twice
// the loads in flight at half the warps ran slower: 16,384 rows of 32 heads of
// 128, half of each rotated, 45.2 us (5.9 TB/s) against 52.8; smaller batches
// at more warps too (51.7).
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
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 256;   // rot_dim <= 512

// One tensor of the call.  Rows of `heads` heads; dst is contiguous (place 0)
// or the key (1) or value (2) pages.
struct Seg {
  const uint16_t* src;
  uint16_t* dst;
  long long src_token, src_head;
  int heads, place, rotate;
  int per;             // items per head
  unsigned int magic;  // ceil(2^32 / per): x / per = umulhi(x, magic) for the small x it is used on
};

struct RopeParams {
  Seg seg[3];
  int n_seg;
  int rows, parts;              // warps per row
  int d, rot, in_place;
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
__device__ __forceinline__ void locate(const RopeParams& p, long long row, long long& pos, long long& at) {
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
  pos = static_cast<long long>(i) + (p.offsets ? __ldg(p.offsets + b) : 0);   // (past 2^31, if so)
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

// Items of a head.  VEC: 8 pairs in two 16-byte words (GPT-NeoX: features 8e ..
// and half + 8e ..), 4 pairs in one (GPT-J), or 8 copied features; else one
// pair or one feature.
template <bool BF16, bool GPTJ, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(const __grid_constant__ RopeParams p) {
  // (A cos, A sin) of the row's pairs, per warp.  VEC: word i of item e (two
  // pairs) at [i][e], so that neighbouring items are neighbouring words
  extern __shared__ float4 tables[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = p.rot >> 1;
  constexpr int PI = !VEC ? 1 : GPTJ ? 4 : 8;   // pairs per item
  constexpr int W = VEC ? 8 : 1;                // features per word
  constexpr bool kTwo = !GPTJ || !VEC;          // the pair's members are apart
  constexpr int U = !VEC ? 2 : GPTJ ? 4 : 2;    // items in flight
  const int groups = half / PI;
  float2* cs = reinterpret_cast<float2*>(tables) + warp * half;
  const float4* cs4 = reinterpret_cast<const float4*>(cs);
  if (p.append && blockIdx.x == 0) {
    // offsets that no row lookup meets
    int first;
    for (int b = threadIdx.x; b < p.B; b += kThreads) chunk_len(p.cu, b, p.total, first, p.err);
  }
  const long long tasks = static_cast<long long>(p.rows) * p.parts;
  for (long long task = static_cast<long long>(blockIdx.x) * kWarps + warp; task < tasks;
       task += static_cast<long long>(gridDim.x) * kWarps) {
    const int row = static_cast<int>(task / p.parts), part = static_cast<int>(task - static_cast<long long>(row) * p.parts);
    long long pos, at;
    locate(p, row, pos, at);
    if (at < 0) continue;
    __syncwarp();   // the table's readers of the row before
    for (int i = lane; i < half; i += 32) {
      const unsigned long long turn = p.turns[i] * static_cast<unsigned long long>(pos);
      float sn, c;
      sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f, &sn, &c);   // 2^-31
      const int to = VEC ? (((i % PI) >> 1) * groups + i / PI) * 2 + (i & 1) : i;
      cs[to] = make_float2(c * p.amplitude, sn * p.amplitude * p.sin_sign);
    }
    __syncwarp();
    for (int k = 0; k < p.n_seg; ++k) {
      const Seg& s = p.seg[k];
      const uint16_t* src = s.src + row * s.src_token;
      uint16_t* dst = s.place == 0 ? s.dst + static_cast<long long>(row) * s.heads * p.d : s.dst + at;
      const long long dst_head = s.place == 0 ? p.d : p.cache.s_head;
      const int turned = s.rotate ? groups : 0;   // items below this are rotated
      const int first = s.rotate ? p.rot : 0;     // first copied feature
      const int stride = 32 * p.parts, start = lane + 32 * part;
      const int dh = s.per == 1 ? stride : __umulhi(stride, s.magic), de = stride - dh * s.per;
      int h = s.per == 1 ? start : __umulhi(start, s.magic), e = start - h * s.per;
      while (h < s.heads) {
        uint4 va[U], vb[U];
        float sa[U], sb[U];
        int hh[U], ee[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          hh[u] = h;
          ee[u] = e;
          if (h < s.heads) {
            const bool t = e < turned;
            const uint16_t* x = src + h * s.src_head + (t ? (GPTJ ? 2 * PI * e : PI * e) : first + W * (e - turned));
            if constexpr (VEC) {
              va[u] = *reinterpret_cast<const uint4*>(x);
              if (kTwo && t) vb[u] = *reinterpret_cast<const uint4*>(x + half);
            } else {
              sa[u] = ld1<BF16>(x);
              if (t) sb[u] = ld1<BF16>(x + (GPTJ ? 1 : half));
            }
          }
          h += dh;
          e += de;
          if (e >= s.per) {
            e -= s.per;
            ++h;
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (hh[u] >= s.heads) continue;
          const int g = ee[u];
          const bool t = g < turned;
          uint16_t* y = dst + hh[u] * dst_head + (t ? (GPTJ ? 2 * PI * g : PI * g) : first + W * (g - turned));
          if constexpr (VEC) {
            uint32_t a[4] = {va[u].x, va[u].y, va[u].z, va[u].w};
            if (t) {
              if constexpr (GPTJ) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const float4 c = cs4[i * groups + g];
                  const float2 x = unpack<BF16>(a[2 * i]), z = unpack<BF16>(a[2 * i + 1]);
                  a[2 * i] = pack<BF16>(x.x * c.x - x.y * c.y, x.x * c.y + x.y * c.x);
                  a[2 * i + 1] = pack<BF16>(z.x * c.z - z.y * c.w, z.x * c.w + z.y * c.z);
                }
              } else {
                uint32_t b[4] = {vb[u].x, vb[u].y, vb[u].z, vb[u].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float4 c = cs4[i * groups + g];
                  const float2 x = unpack<BF16>(a[i]), z = unpack<BF16>(b[i]);
                  a[i] = pack<BF16>(x.x * c.x - z.x * c.y, x.y * c.z - z.y * c.w);
                  b[i] = pack<BF16>(x.x * c.y + z.x * c.x, x.y * c.w + z.y * c.z);
                }
                *reinterpret_cast<uint4*>(y + half) = make_uint4(b[0], b[1], b[2], b[3]);
              }
            }
            *reinterpret_cast<uint4*>(y) = make_uint4(a[0], a[1], a[2], a[3]);
          } else if (t) {
            const float2 c = cs[g];
            st1<BF16>(y, sa[u] * c.x - sb[u] * c.y);
            st1<BF16>(y + (GPTJ ? 1 : half), sa[u] * c.y + sb[u] * c.x);
          } else {
            st1<BF16>(y, sa[u]);
          }
        }
      }
    }
  }
}

// The fraction of x in 64-bit fixed point, modulo 1 (both steps are exact but for
// what lies below 2^-64).
unsigned long long fixed_fraction(double x) {
  const double h = x - std::nearbyint(x);   // [-0.5, 0.5]
  const auto v = static_cast<unsigned long long>(std::fabs(h) * 18446744073709551616.0);
  return h < 0.0 ? 0 - v : v;
}

// f / 2 pi modulo 1: 1 / 2 pi in two doubles, the product's high part and, by the
// fused multiplication and addition, what it leaves.  (The high part comes from
// std::fma too, so that no compiler fuses it into the subtraction that takes its
// fraction.)
unsigned long long turn_of(double f) {
  constexpr double kHigh = 0.15915494309189533577, kLow = -9.839338337591243e-18;   // 1 / (2 pi)
  const double high = std::fma(f, kHigh, 0.0);
  const double low = std::fma(f, kLow, std::fma(f, kHigh, -high));
  return fixed_fraction(high) + fixed_fraction(low);
}

// Checks the rotation's arguments and fills the turn table.
int fill_turns(RopeParams& p, int rot_dim, int d, const double* freqs, float amplitude, int interleaved) {
  if (rot_dim <= 0 || rot_dim > d || (rot_dim & 1) || rot_dim > 2 * kMaxPairs || !freqs) return ATTN_EINVAL;
  if (!std::isfinite(amplitude) || (interleaved != 0 && interleaved != 1)) return ATTN_EINVAL;
  for (int i = 0; i < rot_dim / 2; ++i) {
    if (!std::isfinite(freqs[i])) return ATTN_EINVAL;
    p.turns[i] = turn_of(freqs[i]);
  }
  p.rot = rot_dim;
  p.amplitude = amplitude;
  return ATTN_OK;
}

template <bool BF16, bool GPTJ>
void run(const RopeParams& p, bool vec, int grid, size_t smem, cudaStream_t stream) {
  if (vec) rope_kernel<BF16, GPTJ, true><<<grid, kThreads, smem, stream>>>(p);
  else rope_kernel<BF16, GPTJ, false><<<grid, kThreads, smem, stream>>>(p);
}

int launch(RopeParams& p, bool vec, bool bf16, bool gptj, cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ELAUNCH;
  DeviceInfo info;
  if (int rc = device_info(dev, info)) return rc;
  if (!info.supported) return ATTN_EUNSUPPORTED;
  p.err = info.err_word;
  const int pairs = !vec ? 1 : gptj ? 4 : 8, feats = vec ? 8 : 1;
  int items = 0;
  for (int k = 0; k < p.n_seg; ++k) {
    Seg& s = p.seg[k];
    // in place the features past rot_dim stay where they are
    s.per = s.rotate ? p.rot / 2 / pairs + (p.in_place && s.place == 0 ? 0 : (p.d - p.rot) / feats) : p.d / feats;
    s.magic = static_cast<unsigned int>((0x100000000ull + s.per - 1) / s.per);
    items = std::max(items, s.heads * s.per);
  }
  // a warp per row once the rows fill the GPU's warps; below that a row's
  // items are shared by up to 8 warps, of at least one item a lane
  const long long slots = 4LL * kWarps * info.sm_count;   // resident warps
  p.parts = static_cast<int>(std::max<long long>(1, std::min<long long>({8, slots / std::max(p.rows, 1), (items + 31) / 32})));
  const long long tasks = static_cast<long long>(p.rows) * p.parts;
  const int grid = static_cast<int>(std::min<long long>((tasks + kWarps - 1) / kWarps, 4LL * info.sm_count));
  const size_t smem = static_cast<size_t>(kWarps) * (p.rot / 2) * sizeof(float2);
  if (bf16) gptj ? run<true, true>(p, vec, grid, smem, stream) : run<true, false>(p, vec, grid, smem, stream);
  else gptj ? run<false, true>(p, vec, grid, smem, stream) : run<false, false>(p, vec, grid, smem, stream);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ELAUNCH;
  count_launch();
  return ATTN_OK;
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
  const unsigned long long rows = packed ? static_cast<unsigned long long>(total) : static_cast<unsigned long long>(B) * L;
  if (rows > 0x7fffffffull || rows * H > (1ull << 40) / d) return ATTN_EINVAL;
  if (static_cast<long long>(H) * d > (1 << 26)) return ATTN_EINVAL;   // a row's items are 32-bit
  p.rows = static_cast<int>(rows);
  const bool same = x == y;
  if (same && (x_stride_head != d || x_stride_token != static_cast<long long>(H) * d)) return ATTN_EINVAL;
  if (!same && overlap(x, extent(rows, x_stride_token, H, x_stride_head, d), y, rows * H * d * 2))
    return ATTN_EINVAL;
  if (rows == 0) return ATTN_OK;
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
  return launch(p, vec, fp16 == 0, interleaved != 0, stream);
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
  return launch(p, !freqs_or_null || rot_dim % 16 == 0, cache->fp16 == 0, freqs_or_null && interleaved != 0, stream);
}

}  // extern "C"
