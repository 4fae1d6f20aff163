// What the kernels with a rotation share: 16-bit features in 32-bit words, the
// rotation of an item (16 features, 8 pairs), the fixed-point turns of a
// frequency (see attn_rope_scaled.cu) and the angle that a position makes of them.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ptx.cuh"

namespace attn {

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

// The 16 features of two words as pairs of neighbours, for packed arithmetic.
template <bool BF16>
__device__ __forceinline__ void widen2x(const uint4& a, const uint4& b, float2 (&x)[8]) {
  const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = unpack<BF16>(u[i]);
}
template <bool BF16>
__device__ __forceinline__ void narrow2x(const float2 (&x)[8], uint4& a, uint4& b) {
  a = make_uint4(pack<BF16>(x[0].x, x[0].y), pack<BF16>(x[1].x, x[1].y), pack<BF16>(x[2].x, x[2].y),
                 pack<BF16>(x[3].x, x[3].y));
  b = make_uint4(pack<BF16>(x[4].x, x[4].y), pack<BF16>(x[5].x, x[5].y), pack<BF16>(x[6].x, x[6].y),
                 pack<BF16>(x[7].x, x[7].y));
}

// Turns the item's 8 pairs (BACK: back) by cs, the cosines of pairs 2i and 2i + 1 in
// cs[i], the sines in cs[4 + i].  GPT-NeoX: pairs 2i and 2i + 1 are (x[i], x[4 + i]) by
// components; GPT-J: pair i is the components of x[i].
template <bool GPTJ, bool BACK>
__device__ __forceinline__ void turn2(float2 (&x)[8], const float2 (&cs)[8]) {
  if constexpr (GPTJ) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = i & 1 ? cs[i >> 1].y : cs[i >> 1].x, t = i & 1 ? cs[4 + (i >> 1)].y : cs[4 + (i >> 1)].x;
      const float s = BACK ? -t : t;
      x[i] = ffma2(make_float2(x[i].y, x[i].y), make_float2(-s, c), fmul2(make_float2(x[i].x, x[i].x), make_float2(c, s)));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 c = cs[i], s = BACK ? make_float2(-cs[4 + i].x, -cs[4 + i].y) : cs[4 + i];
      const float2 a = x[i], b = x[4 + i];
      x[i] = ffma2(b, make_float2(-s.x, -s.y), fmul2(a, c));
      x[4 + i] = ffma2(a, s, fmul2(b, c));
    }
  }
}

// (cos, sin) of the fraction of a turn that position pos makes.
__device__ __forceinline__ float2 turned(unsigned long long turns, long long pos) {
  const unsigned long long turn = turns * static_cast<unsigned long long>(pos);
  float sn, c;
  sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f, &sn, &c);   // 2^-31
  return make_float2(c, sn);
}

// The same, an eighth of a turn from a quarter at the most going through fp32: sine and
// cosine are off by 2^-25 from the argument instead of 2^-23, as much as by their own
// rounding (keys that are rounded to 8 bits next keep what the angle gives them).
__device__ __forceinline__ float2 turned_near(unsigned long long turns, long long pos) {
  const unsigned long long turn = turns * static_cast<unsigned long long>(pos);
  const uint32_t h = static_cast<uint32_t>((turn + 0x80000000ull) >> 32), q = (h + 0x20000000u) >> 30;   // nearest quarter
  float sn, c;
  sincospif(static_cast<float>(static_cast<int>(h - (q << 30))) * 4.656612873077393e-10f, &sn, &c);   // 2^-31
  const float a = q & 1 ? -sn : c, b = q & 1 ? c : sn;   // a quarter on: (-sin, cos)
  return q & 2 ? make_float2(-a, -b) : make_float2(a, b);
}

// The fraction of x in 64-bit fixed point, modulo 1 (both steps are exact but for
// what lies below 2^-64).
inline unsigned long long fixed_fraction(double x) {
  const double h = x - std::nearbyint(x);   // [-0.5, 0.5]
  const auto v = static_cast<unsigned long long>(std::fabs(h) * 18446744073709551616.0);
  return h < 0.0 ? 0 - v : v;
}

// f / 2 pi modulo 1: 1 / 2 pi in two doubles, the product's high part and, by the
// fused multiplication and addition, what it leaves.  (The high part comes from
// std::fma too, so that no compiler fuses it into the subtraction that takes its
// fraction.)
inline unsigned long long turn_of(double f) {
  constexpr double kHigh = 0.15915494309189533577, kLow = -9.839338337591243e-18;   // 1 / (2 pi)
  const double high = std::fma(f, kHigh, 0.0);
  const double low = std::fma(f, kLow, std::fma(f, kHigh, -high));
  return fixed_fraction(high) + fixed_fraction(low);
}

// Bytes from the first to past the last element of a strided (rows, heads, d)
// tensor of 16-bit elements.
inline unsigned long long extent(unsigned long long rows, long long st, int heads, long long sh, int d) {
  return rows == 0 ? 0 : 2 * ((rows - 1) * st + (heads - 1) * sh + d);
}

}  // namespace attn
