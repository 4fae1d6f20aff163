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
// itself, or 2^-10 s below 2^-6 s.  The quotient is the rounded one: a product with
// 1 / s is off by an ulp, which moves values that lie on a border between two
// e4m3 values, and rows whose largest is a power of two have many of those.
//
// Bound by HBM: q, k and v read once; q written in 16 bits, k and v in 8 and a
// scale per row (reading back: the other way round).  A lane holds 16 features of a head
// as two 16-byte words that contain its pairs whole, 4 or 8 lanes a head, so the row's
// maximum is 2 or 3 shuffles.  A warp takes a token (with few tokens a part of its
// heads); the next heads' loads, over the token's end, are on their way while one's are
// worked on, the token's place is looked up behind them.
//
// Measured: 8,000 new tokens of eight sequences, 32 + 2 x 8 heads of 128, 37.7 us (4.8
// TB/s; a copy of as many bytes 26.7): neither HBM (47 % of its nominal rate under the
// profiler) nor issue (52 % of the schedulers' cycles) is full, 16 warps per SM with a step
// of loads each on its way; 84,500 keys of 8 heads read back 85 us (6.2 TB/s; 77).
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
  int heads[3];
  int rows, parts, B;     // warps per token
  int d, lg;              // log2 of the lanes per head
  int rot;
  float amplitude;
  const int* cu;
  const int* positions;
  PagedKV8 c;
  int* err;
  unsigned long long turns[kMaxPairs];
};

// x / s, inv the rounded 1 / s: the product, and one correction by its exact remainder
// (P. Markstein, IBM J. Res. Dev. 34, 1990).
__device__ __forceinline__ float2 quotients(float2 x, float s, float inv) {
  const float2 i2 = make_float2(inv, inv), q = fmul2(x, i2);
  return ffma2(ffma2(q, make_float2(-s, -s), x), i2, q);
}

// The last b < B with cu[b] <= row (0 if there is none), by the warp, 32 offsets at a
// time.
__device__ __forceinline__ int find(const int* cu, int B, int row, int lane) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5, at = lo + (lane + 1) * step;
    const int n = __popc(__ballot_sync(0xffffffffu, at < hi && __ldg(cu + at) <= row));
    hi = min(lo + (n + 1) * step, hi);
    lo += n * step;
  }
  return lo;
}

template <bool BF16, bool GPTJ>
__global__ void __launch_bounds__(kThreads, 2) append_kernel(const __grid_constant__ AppendParams p) {
  extern __shared__ float4 tables[];
  constexpr int U = 2;   // heads per lane and step
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lanes = 1 << p.lg, sub = lane >> p.lg, e = lane & (lanes - 1), per = 32 >> p.lg;
  const int groups = p.rot >> 4, half = p.rot >> 1;
  const bool turns_here = e < groups;
  const int lo = !GPTJ && turns_here ? 8 * e : 16 * e;
  const int hi = !GPTJ && turns_here ? half + 8 * e : lo + 8;
  // the token's (A cos, A sin): of pair 8e + i at [i / 4][e] of float4s
  float4* tab = tables + warp * (p.rot >> 2);
  float* tab_f = reinterpret_cast<float*>(tab);
  if (blockIdx.x == 0) {
    // offsets that no row lookup meets
    int first;
    for (int b = threadIdx.x; b < p.B; b += kThreads) chunk_len(p.cu, b, p.rows, first, p.err);
  }
  const long long tasks = static_cast<long long>(p.rows) * p.parts, stride = static_cast<long long>(gridDim.x) * kWarps;
  const int step = U * p.parts * per;
  // steps j of a token: q's heads, k's, v's
  const int steps_q = (p.heads[0] + step - 1) / step, steps_k = (p.heads[1] + step - 1) / step, steps = steps_q + 2 * steps_k;
  struct Batch {
    uint4 a[U], b[U];
  };
  auto part_of = [&](int j, int& h0) {   // which of q, k and v step j is of; its first head (of part 0)
    const int k = j < steps_q ? 0 : j < steps_q + steps_k ? 1 : 2;
    h0 = (k == 0 ? j : j - steps_q - (k == 2 ? steps_k : 0)) * step;
    return k;
  };
  auto load = [&](int row, int part, int j, Batch& t) {
    int h0;
    const int k = part_of(j, h0);
    const uint16_t* src = p.x[k] + row * p.s_token[k];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + (part + u * p.parts) * per + sub;
      t.a[u] = t.b[u] = make_uint4(0, 0, 0, 0);
      if (h < p.heads[k]) {
        t.a[u] = *reinterpret_cast<const uint4*>(src + h * p.d + lo);
        t.b[u] = *reinterpret_cast<const uint4*>(src + h * p.d + hi);
      }
    }
  };
  auto enter = [&](long long task, int& row, int& part) {
    row = static_cast<int>(p.parts == 1 ? task : task / p.parts);
    part = static_cast<int>(task - static_cast<long long>(row) * p.parts);
  };
  float2 cs[8];
  Batch cur, next;
  long long task = static_cast<long long>(blockIdx.x) * kWarps + warp;
  int row = 0, part = 0;
  if (task < tasks) {
    enter(task, row, part);
    load(row, part, 0, cur);
  }
  while (task < tasks) {
    // the token's place
    int page = -1, slot = 0, pos = 0;
    {
      const int b = find(p.cu, p.B, row, lane);
      int m, first, len;
      chunk_and_keys(p.c.t, p.cu, b, p.rows, m, first, len, p.err);
      const int i = row - first;
      if (i >= 0 && i < m) {
        const int key = len - m + i;
        if (key < 0) {
          if (lane == 0) atomicCAS(p.err, 0, ATTN_DEVERR_BAD_SEQLENS);
        } else {
          page = paged_page(p.c.t, b, key >> p.c.t.page_log2, p.err);
          slot = key & ((1 << p.c.t.page_log2) - 1);
          pos = p.positions ? __ldg(p.positions + row) : key;
        }
      }
    }
    const long long task_n = task + stride;
    int row_n = 0, part_n = 0;
    if (task_n < tasks) enter(task_n, row_n, part_n);
    {
      if (p.rot && page >= 0) {
        __syncwarp();   // the table's readers of the token before
#pragma unroll 1
        for (int t = lane; t < half; t += 32) {
          const float2 f = turned_near(p.turns[t], pos);
          const int to = ((((t & 7) >> 2) * groups + (t >> 3)) << 2) + (t & 3);
          tab_f[to] = f.x * p.amplitude;
          tab_f[to + half] = f.y * p.amplitude;
        }
        __syncwarp();
        if (turns_here) {
          const float4 c0 = tab[e], c1 = tab[groups + e], s0 = tab[2 * groups + e], s1 = tab[3 * groups + e];
          cs[0] = make_float2(c0.x, c0.y), cs[1] = make_float2(c0.z, c0.w), cs[2] = make_float2(c1.x, c1.y);
          cs[3] = make_float2(c1.z, c1.w), cs[4] = make_float2(s0.x, s0.y), cs[5] = make_float2(s0.z, s0.w);
          cs[6] = make_float2(s1.x, s1.y), cs[7] = make_float2(s1.z, s1.w);
        }
      }
#pragma unroll 1
      for (int j = 0; j < steps; ++j) {
        if (j + 1 < steps) load(row, part, j + 1, next);
        else if (task_n < tasks) load(row_n, part_n, 0, next);
        int h0;
        const int k = part_of(j, h0);
        if (page >= 0) {
          uint8_t* dst = (k == 1 ? p.c.k : p.c.v) + page * p.c.s_page + slot * p.c.s_token;
          float* scales = (k == 1 ? p.c.ks : p.c.vs) + page * p.c.c_page + slot * p.c.c_token;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int h = h0 + (part + u * p.parts) * per + sub;
            const bool live = h < p.heads[k];
            float2 z[8];
            widen2x<BF16>(cur.a[u], cur.b[u], z);
            if (turns_here && k < 2) turn2<GPTJ, false>(z, cs);
            if (k == 0) {
              if (live) {
                uint4 oa, ob;
                narrow2x<BF16>(z, oa, ob);
                uint16_t* y = p.q_out + (static_cast<long long>(row) * p.heads[0] + h) * p.d;
                *reinterpret_cast<uint4*>(y + lo) = oa;
                *reinterpret_cast<uint4*>(y + hi) = ob;
              }
              continue;
            }
            // the row's largest magnitude, as bits: a NaN counts above infinity
            uint32_t top = 0;
#pragma unroll
            for (int t = 0; t < 8; ++t)
              top = max(top, max(__float_as_uint(z[t].x) & 0x7fffffffu, __float_as_uint(z[t].y) & 0x7fffffffu));
            for (int o = lanes >> 1; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            const bool finite = top < 0x7f800000u;
            const float s = finite ? fmaxf(__uint_as_float(top) / kE4M3Top, kLeastScale) : __uint_as_float(0x7fffffffu);
            const float inv = 1.0f / s;
            uint32_t w[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const uint32_t l = __nv_cvt_float2_to_fp8x2(quotients(z[2 * t], s, inv), __NV_SATFINITE, __NV_E4M3);
              const uint32_t r = __nv_cvt_float2_to_fp8x2(quotients(z[2 * t + 1], s, inv), __NV_SATFINITE, __NV_E4M3);
              w[t] = finite ? l | r << 16 : 0;
            }
            if (live) {
              uint8_t* y = dst + h * p.c.s_head;
              *reinterpret_cast<uint2*>(y + lo) = make_uint2(w[0], w[1]);
              *reinterpret_cast<uint2*>(y + hi) = make_uint2(w[2], w[3]);
              if (e == 0) scales[h * p.c.c_head] = s;
            }
          }
        }
        cur = next;
      }
    }
    task = task_n;
    row = row_n;
    part = part_n;
  }
}

struct ReadParams {
  uint16_t* k;
  uint16_t* v;
  const int* cu;
  const int* starts;   // or null: 0
  int rows, parts, B;
  int d, lg;
  int wide;            // k and v are 32-byte aligned
  PagedKV8 c;
  int* err;
};

// 16 e4m3 values times s, rounded once to 16 bits.
template <bool BF16>
__device__ __forceinline__ void scaled(const uint4& x, float s, uint4& a, uint4& b) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
  const float2 s2 = make_float2(s, s);
  float2 z[8];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u[t] >> (16 * i)), __NV_E4M3);
      z[2 * t + i] = fmul2(__half22float2(__half2(h)), s2);
    }
  }
  narrow2x<BF16>(z, a, b);
}
// Stored as one 32-byte word where it is aligned (half a sector at a time is twice the
// requests).
template <bool BF16>
__device__ __forceinline__ void store16(uint16_t* y, const uint4& x, float s, bool wide) {
  uint4 a, b;
  scaled<BF16>(x, s, a, b);
  if (wide) {
    const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    st_global_v8(y, v);
  } else {
    reinterpret_cast<uint4*>(y)[0] = a;
    reinterpret_cast<uint4*>(y)[1] = b;
  }
}

// Keys and values of one head and 16 features per lane and step, the next step's on
// their way.
template <bool BF16>
__global__ void __launch_bounds__(kThreads, 4) read_kernel(const __grid_constant__ ReadParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lanes = 1 << p.lg, sub = lane >> p.lg, e = lane & (lanes - 1), per = 32 >> p.lg, heads = p.c.t.hkv;
  if (blockIdx.x == 0) {
    int first;
    for (int b = threadIdx.x; b < p.B; b += kThreads) chunk_len(p.cu, b, p.rows, first, p.err);
  }
  const long long tasks = static_cast<long long>(p.rows) * p.parts;
  const int step = p.parts * per;
  for (long long task = static_cast<long long>(blockIdx.x) * kWarps + warp; task < tasks;
       task += static_cast<long long>(gridDim.x) * kWarps) {
    const int row = static_cast<int>(p.parts == 1 ? task : task / p.parts);
    const int part = static_cast<int>(task - static_cast<long long>(row) * p.parts);
    // the row's place
    const int b = find(p.cu, p.B, row, lane);
    int m, first, len;
    chunk_and_keys(p.c.t, p.cu, b, p.rows, m, first, len, p.err);
    const int i = row - first;
    if (i < 0 || i >= m) continue;
    const long long key = static_cast<long long>(i) + (p.starts ? __ldg(p.starts + b) : 0);
    if (key < 0 || key >= len) {
      if (lane == 0) atomicCAS(p.err, 0, ATTN_DEVERR_BAD_SEQLENS);
      continue;
    }
    const int page = paged_page(p.c.t, b, static_cast<int>(key) >> p.c.t.page_log2, p.err);
    if (page < 0) continue;
    const int slot = static_cast<int>(key) & ((1 << p.c.t.page_log2) - 1);
    const long long from = page * p.c.s_page + slot * p.c.s_token + 16 * e;
    const long long scale = page * p.c.c_page + slot * p.c.c_token;
    struct Item {
      uint4 k, v;
      float ks, vs;
    };
    auto load = [&](int h, Item& x) {
      if (h < heads) {
        x.k = *reinterpret_cast<const uint4*>(p.c.k + from + h * p.c.s_head);
        x.v = *reinterpret_cast<const uint4*>(p.c.v + from + h * p.c.s_head);
        x.ks = p.c.ks[scale + h * p.c.c_head];
        x.vs = p.c.vs[scale + h * p.c.c_head];
      }
    };
    Item cur, next;
    int h = part * per + sub;
    load(h, cur);
    for (int h0 = part * per; h0 < heads; h0 += step, h += step) {
      if (h0 + step < heads) load(h + step, next);
      if (h < heads) {
        const long long to = (static_cast<long long>(row) * heads + h) * p.d + 16 * e;
        store16<BF16>(p.k + to, cur.k, cur.ks, p.wide != 0);
        store16<BF16>(p.v + to, cur.v, cur.vs, p.wide != 0);
      }
      cur = next;
    }
  }
}

int device(DeviceInfo& info) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ELAUNCH;
  if (int rc = device_info(dev, info)) return rc;
  return info.supported ? ATTN_OK : ATTN_EUNSUPPORTED;
}

// Warps per row, and blocks: a warp per row once the rows fill the GPU's warps, below
// that a row's heads are shared by up to 8.  (Runs of 8 rows per warp, their places
// looked up at once, were slower: warps side by side then read places far apart.  Reading
// 84,500 rows of 8 heads of 128 back 95 us against the 83 of that time.)
int shape(int rows, int heads, int lg, int per_sm, int sms, int& parts) {
  const long long slots = static_cast<long long>(per_sm) * kWarps * sms;
  const int per = 32 >> lg;
  parts = static_cast<int>(std::max<long long>(1, std::min<long long>({8, slots / std::max(rows, 1), (heads + per - 1) / per})));
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
  for (int i = 0; i < 3; ++i) p.heads[i] = heads[i];
  p.rows = total;
  p.B = B;
  p.d = d;
  p.lg = d == 128 ? 3 : 2;
  p.cu = cu_seqlens;
  p.positions = positions_or_null;
  p.err = info.err_word;
  const int grid = shape(total, std::max(heads[0], hkv), p.lg, 2, info.sm_count, p.parts);
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
  p.wide = ptr_aligned(k, 32) && ptr_aligned(v, 32);
  p.rows = total;
  p.B = B;
  p.d = d;
  p.lg = d == 128 ? 3 : 2;
  p.err = info.err_word;
  const int grid = shape(total, hkv, p.lg, 4, info.sm_count, p.parts);
  if (fp16 == 0) read_kernel<true><<<grid, kThreads, 0, stream>>>(p);
  else read_kernel<false><<<grid, kThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ELAUNCH;
  count_launch();
  return ATTN_OK;
}

}  // extern "C"
