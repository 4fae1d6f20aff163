// Norms of the queries' and keys' heads with their rotary embedding in the same
// pass (attn_qk_norm_rotary), and the gradients (attn_qk_norm_rotary_bwd).
//
// A head x of d features becomes
//   z = x r,  r = 1 / sqrt(mean x^2 + eps),   y = A R(a) (w z),
// R(a) the rotation of pair p by a_p = positions[axis(p)] f_p.  With g = A R(-a) dy,
//   dw = sum over tokens and heads of g z,   dx = r (g w - z mean(g w z)).
// All of it in fp32 from the 16-bit values on, one rounding at the end; the
// angles as in attn_rope_scaled.cu.
//
// Bound by HBM: x read once, y written once (backward: x and dy read, dx
// written).  A lane holds 16 features of a head, two 16-byte words that contain
// its pairs whole, a group of d / 16 lanes (rounded up to a power of two) a head:
// the mean is log2 of that many shuffles, and neither x nor the angles pass
// through shared memory again.  A warp takes a token, forms the pairs' (cos, sin)
// once for all of its heads, and keeps them in registers; the weights lie in shared
// memory as fp32.  The next heads' loads, over the token's end, are on their way while
// one's are worked on, in pairs of fp32 (packed instructions: fewer to issue).  With few
// tokens, and for the last ones when every warp has had as many as the others, a
// token's heads are shared by several warps.
//
// dw: a lane's features are the same in every head, so it sums its own over all heads
// and tokens that its warp meets, one side's in registers, the other's in shared memory;
// the warps' sums are joined in a fixed order, in shared memory and then over the
// blocks by a second launch (sum_weights_kernel).  The same sizes give the same bits.
//
// Measured: 8,192 tokens of 32 + 8 heads of 128 over three axes 34.3 us (4.9 TB/s; a
// copy of as many bytes 24.8), the gradients of 16,384 101 us (5.0 TB/s; 74).  Neither
// HBM (45 and 60 % of its nominal rate under the profiler) nor issue (52 and 55 % of the
// schedulers' cycles) is full: what is left is the latency of the loads, of which the 16
// warps that an SM has at these registers (two blocks) keep one step each on its way.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attn.h"
#include "attn_paged.h"
#include "attn_turns.cuh"
#include "ptx.cuh"

namespace attn {
namespace norm {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 256;   // d <= 512
constexpr int kMaxAxes = 8;

struct Side {            // the queries or the keys
  const uint16_t* x;
  const uint16_t* dy;    // contiguous
  uint16_t* out;         // y, or dx; contiguous
  const void* w;         // weights, or null: ones
  long long s_token, s_head;
  int heads;
};

struct Params {
  Side side[2];
  int rows, parts;       // warps per token
  int d, items, lg;      // items of 16 features per head; log2 of the lanes per head
  int rot;
  int w32;               // weights in fp32
  float eps, inv_d, amplitude;
  const int* positions;  // (axes, rows)
  float* partial;        // dw of each block, (blocks, 2, d)
  unsigned long long turns[kMaxPairs];
  uint8_t axis[kMaxPairs];
};

template <bool BF16>
__device__ __forceinline__ float weight(const void* w, bool fp32, int at) {
  if (fp32) return __ldg(static_cast<const float*>(w) + at);
  const unsigned short v = __ldg(static_cast<const unsigned short*>(w) + at);
  return BF16 ? __bfloat162float(__ushort_as_bfloat16(v)) : __half2float(__ushort_as_half(v));
}
// An item's features times the weights, which lie in shared memory.
__device__ __forceinline__ void scale_by(float2 (&x)[8], const float* w, int lo, int hi) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = *reinterpret_cast<const float4*>(w + (i < 2 ? lo + 4 * i : hi + 4 * i - 8));
    x[2 * i] = fmul2(x[2 * i], make_float2(v.x, v.y));
    x[2 * i + 1] = fmul2(x[2 * i + 1], make_float2(v.z, v.w));
  }
}

__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Where the item's two words lie in its head.
template <bool GPTJ>
__device__ __forceinline__ void place(const Params& p, int e, int& lo, int& hi, bool& turned_item) {
  const int groups = p.rot >> 4;
  turned_item = e < groups;
  if (!GPTJ && turned_item) {
    lo = 8 * e;
    hi = (p.rot >> 1) + 8 * e;
  } else {
    lo = 16 * e;   // (NeoX: rot + 16 (e - groups))
    hi = lo + 8;
  }
}

template <bool BF16, bool GPTJ, bool BWD>
__global__ void __launch_bounds__(kThreads, 2) norm_kernel(const __grid_constant__ Params p) {
  extern __shared__ float4 tables[];
  // heads per lane and step; the next step's are on their way meanwhile
  constexpr int U = BWD ? 1 : 2;
  constexpr int P = 2;   // pairs per lane whose positions are read ahead
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lanes = 1 << p.lg, sub = lane >> p.lg, e = lane & (lanes - 1), per = 32 >> p.lg;   // heads per warp and step
  const bool on = e < p.items;
  const int groups = p.rot >> 4, half = p.rot >> 1;
  // the token's (A cos, A sin), and the weights: of pair 8e + i (feature lo + i, hi + i)
  // at [i / 4][e] of float4s, so that the lanes of a head read neighbouring words
  float4* tab = tables + warp * (p.rot >> 2);   // cos [2][groups], then sin
  float* tab_f = reinterpret_cast<float*>(tab);
  float* weights = reinterpret_cast<float*>(tables) + kWarps * p.rot;   // [2][d]
  float* sums = weights + 2 * p.d;   // dw: of a thread and side, [side][4][thread] of float4s; at the end [warp][2][d]
  int lo, hi;
  bool turns_here;
  place<GPTJ>(p, on ? e : 0, lo, hi, turns_here);
  for (int i = threadIdx.x; i < 2 * p.d; i += kThreads) {
    const Side& s = p.side[i < p.d ? 0 : 1];
    const int f = i < p.d ? i : i - p.d;
    weights[i] = s.w == nullptr ? 1.0f : weight<BF16>(s.w, p.w32 != 0, f);
  }
  __syncthreads();
  // Tokens: whole ones while there are enough for every warp, then parts of the rest.
  const long long warps = static_cast<long long>(gridDim.x) * kWarps;
  const int full = static_cast<int>(p.rows / warps * warps);
  const long long tasks = full + static_cast<long long>(p.rows - full) * p.parts;
  float dw[16];
  float4* mine = reinterpret_cast<float4*>(sums) + threadIdx.x;
  if constexpr (BWD) {
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[i] = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) mine[i * kThreads] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  // the weight sums in registers are of one side, the other's wait in shared memory
  auto put_sums = [&](int k) {
#pragma unroll
    for (int i = 0; i < 4; ++i) mine[(4 * k + i) * kThreads] = make_float4(dw[4 * i], dw[4 * i + 1], dw[4 * i + 2], dw[4 * i + 3]);
  };
  auto get_sums = [&](int k) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = mine[(4 * k + i) * kThreads];
      dw[4 * i] = v.x, dw[4 * i + 1] = v.y, dw[4 * i + 2] = v.z, dw[4 * i + 3] = v.w;
    }
  };
  {
    struct Batch {
      uint4 xa[U], xb[U], ga[BWD ? U : 1], gb[BWD ? U : 1];
    };
    struct Task {
      int row, part, parts;   // part of `parts` of a token's heads
      int steps0, steps;      // steps of the queries' heads, and in all
    };
    auto enter = [&](long long task) {
      Task t;
      t.parts = task < full ? 1 : p.parts;
      t.row = static_cast<int>(task);
      t.part = 0;
      if (t.parts > 1) {
        const int rest = static_cast<int>(task - full);   // (below 8 warps' worth)
        t.row = full + rest / t.parts;
        t.part = rest % t.parts;
      }
      const int step = U * t.parts * per;
      t.steps0 = (p.side[0].heads + step - 1) / step;
      t.steps = t.steps0 + (p.side[1].heads + step - 1) / step;
      return t;
    };
    auto load = [&](const Task& a, int j, Batch& t) {
      const int k = j >= a.steps0, row = a.row;
      const Side& s = p.side[k];
      const uint16_t* x = s.x + row * s.s_token;
      const int h0 = ((j - (k ? a.steps0 : 0)) * U * a.parts + a.part) * per + sub;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * a.parts * per;
        t.xa[u] = t.xb[u] = make_uint4(0, 0, 0, 0);
        if constexpr (BWD) t.ga[u] = t.gb[u] = make_uint4(0, 0, 0, 0);
        if (h < s.heads && on) {
          const uint16_t* src = x + h * s.s_head;
          t.xa[u] = *reinterpret_cast<const uint4*>(src + lo);
          t.xb[u] = *reinterpret_cast<const uint4*>(src + hi);
          if constexpr (BWD) {
            const uint16_t* g = s.dy + (static_cast<long long>(row) * s.heads + h) * p.d;
            t.ga[u] = *reinterpret_cast<const uint4*>(g + lo);
            t.gb[u] = *reinterpret_cast<const uint4*>(g + hi);
          }
        }
      }
    };
    int pos[P];
    auto position = [&](int i, int row) { return __ldg(p.positions + static_cast<long long>(p.axis[i]) * p.rows + row); };
    auto positions = [&](int row) {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (lane + 32 * i < half) pos[i] = position(lane + 32 * i, row);
    };
    float2 cs[8];   // cos, then sin, of pairs 2i and 2i + 1
    Batch cur, next;
    long long task = static_cast<long long>(blockIdx.x) * kWarps + warp;
    Task at = {};
    if (task < tasks) {
      at = enter(task);
      load(at, 0, cur);
      if (p.rot) positions(at.row);
    }
    while (task < tasks) {
      if (p.rot) {
        __syncwarp();   // the table's readers of the token before
        auto turn_pair = [&](int i, int position_i) {
          const float2 t = turned_near(p.turns[i], position_i);
          const int to = ((((i & 7) >> 2) * groups + (i >> 3)) << 2) + (i & 3);
          tab_f[to] = t.x * p.amplitude;
          tab_f[to + half] = t.y * p.amplitude;
        };
#pragma unroll
        for (int i = 0; i < P; ++i)
          if (lane + 32 * i < half) turn_pair(lane + 32 * i, pos[i]);
#pragma unroll 1
        for (int i = lane + 32 * P; i < half; i += 32) turn_pair(i, position(i, at.row));
        __syncwarp();
        if (turns_here) {
          const int eo = on ? e : 0;
          const float4 c0 = tab[eo], c1 = tab[groups + eo], s0 = tab[2 * groups + eo], s1 = tab[3 * groups + eo];
          cs[0] = make_float2(c0.x, c0.y), cs[1] = make_float2(c0.z, c0.w), cs[2] = make_float2(c1.x, c1.y);
          cs[3] = make_float2(c1.z, c1.w), cs[4] = make_float2(s0.x, s0.y), cs[5] = make_float2(s0.z, s0.w);
          cs[6] = make_float2(s1.x, s1.y), cs[7] = make_float2(s1.z, s1.w);
        }
      }
      const long long task_n = task + warps;
      Task then = {};
      if (task_n < tasks) {
        then = enter(task_n);
        if (p.rot) positions(then.row);
      }
#pragma unroll 1
      for (int j = 0; j < at.steps; ++j) {
        if (j + 1 < at.steps) load(at, j + 1, next);
        else if (task_n < tasks) load(then, 0, next);
        const int k = j >= at.steps0;
        if (BWD && (j == 0 || j == at.steps0)) {
          if (j > 0) put_sums(0);
          get_sums(k);
        }
        const Side& s = p.side[k];
        const float* wk = weights + k * p.d;
        const int h0 = ((j - (k ? at.steps0 : 0)) * U * at.parts + at.part) * per + sub;
        uint16_t* out = s.out + static_cast<long long>(at.row) * s.heads * p.d;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = h0 + u * at.parts * per;
          const bool live = h < s.heads && on;
          float2 z[8];
          widen2x<BF16>(cur.xa[u], cur.xb[u], z);
          float2 sq = fmul2(z[0], z[0]);
#pragma unroll
          for (int i = 1; i < 8; ++i) sq = ffma2(z[i], z[i], sq);
          const float r = rsqrtf(fmaf(group_sum(sq.x + sq.y, lanes), p.inv_d, p.eps));
          const float2 r2 = make_float2(r, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = fmul2(z[i], r2);
          uint4 oa, ob;
          if constexpr (!BWD) {
            scale_by(z, wk, lo, hi);
            if (turns_here) turn2<GPTJ, false>(z, cs);
            narrow2x<BF16>(z, oa, ob);
          } else {
            float2 g[8];
            widen2x<BF16>(cur.ga[u], cur.gb[u], g);
            if (turns_here) turn2<GPTJ, true>(g, cs);
            if (live) {   // (no head here: z = 0 / 0 where eps = 0)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 t = ffma2(g[i], z[i], make_float2(dw[2 * i], dw[2 * i + 1]));
                dw[2 * i] = t.x;
                dw[2 * i + 1] = t.y;
              }
            }
            scale_by(g, wk, lo, hi);
            float2 dot = fmul2(g[0], z[0]);
#pragma unroll
            for (int i = 1; i < 8; ++i) dot = ffma2(g[i], z[i], dot);
            const float m = group_sum(live ? dot.x + dot.y : 0.0f, lanes) * -p.inv_d;
            const float2 m2 = make_float2(m, m);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = fmul2(r2, ffma2(z[i], m2, g[i]));
            narrow2x<BF16>(g, oa, ob);
          }
          if (live) {
            uint16_t* y = out + h * p.d;
            *reinterpret_cast<uint4*>(y + lo) = oa;
            *reinterpret_cast<uint4*>(y + hi) = ob;
          }
        }
        cur = next;
      }
      if constexpr (BWD) put_sums(at.steps > at.steps0);
      task = task_n;
      at = then;
    }
  }
  if constexpr (BWD) {
    if (p.partial == nullptr) return;
    // over the lanes that hold the same features, then over the warps
    float v[2][16];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      get_sums(k);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        v[k][i] = dw[i];
        for (int o = lanes; o < 32; o <<= 1) v[k][i] += __shfl_xor_sync(0xffffffffu, v[k][i], o);
      }
    }
    __syncthreads();   // (the threads' sums have been read)
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (sub == 0 && on) sums[(warp * 2 + k) * p.d + (i < 8 ? lo + i : hi + i - 8)] = v[k][i];
    __syncthreads();
    grid_launch_dependents();
    for (int i = threadIdx.x; i < 2 * p.d; i += kThreads) {
      float v = 0.0f;
      if (i < p.d || p.side[1].heads > 0) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += sums[w * 2 * p.d + i];
      }
      p.partial[static_cast<long long>(blockIdx.x) * 2 * p.d + i] = v;
    }
  }
}

// The blocks' sums, 8 features per block: 32 threads of a feature take every
// 32nd block's, then a tree.
template <bool BF16>
__global__ void __launch_bounds__(256) sum_weights_kernel(const float* partial, int blocks, int d, void* dwq, void* dwk,
                                                          int w32) {
  __shared__ float s[32][9];
  const int f = threadIdx.x & 7, t = threadIdx.x >> 3, i = blockIdx.x * 8 + f;
  grid_wait_prerequisites();
  float v = 0.0f;
  for (int b = t; b < blocks; b += 32) v += __ldcg(partial + static_cast<long long>(b) * 2 * d + i);
  s[t][f] = v;
  for (int o = 16; o > 0; o >>= 1) {
    __syncthreads();
    if (t < o) s[t][f] += s[t + o][f];
  }
  if (t != 0) return;
  void* out = i < d ? dwq : dwk;
  const int at = i < d ? i : i - d;
  if (out == nullptr) return;
  if (w32) static_cast<float*>(out)[at] = s[0][f];
  else if constexpr (BF16) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(s[0][f]);
  else static_cast<__half*>(out)[at] = __float2half_rn(s[0][f]);
}

constexpr int kBlocksPerSM = 2;   // of the backward, as its workspace is sized
int bwd_blocks(int sms) { return kBlocksPerSM * sms; }

struct Call {   // the arguments that both directions share
  const void *q, *k, *qw, *kw;
  long long q_token, q_head, k_token, k_head;
  int rows, Hq, Hk, d, w32, rot, axes, interleaved, fp16;
  float eps, amplitude;
  const double* freqs;
  const int* axis;
  const int* positions;
};

int fill(const Call& c, Params& p) {
  if (c.rows < 0 || c.Hq <= 0 || c.Hk < 0 || c.d <= 0 || c.Hq > (1 << 20) || c.Hk > (1 << 20)) return ATTN_EINVAL;
  if ((c.fp16 != 0 && c.fp16 != 1) || (c.w32 != 0 && c.w32 != 1) || (c.interleaved != 0 && c.interleaved != 1)) return ATTN_EINVAL;
  if (!std::isfinite(c.eps) || c.eps < 0.0f || !std::isfinite(c.amplitude)) return ATTN_EINVAL;
  if (c.rot < 0 || c.rot > c.d || (c.rot & 1) || (c.rot > 0 && !c.freqs)) return ATTN_EINVAL;
  if (c.rot > 0 && (c.axes < 1 || c.axes > kMaxAxes || (c.rows > 0 && !c.positions) || !ptr_aligned(c.positions, 4)))
    return ATTN_EINVAL;
  if (c.d % 16 != 0 || c.d > 512 || c.rot % 16 != 0) return ATTN_EUNSUPPORTED;
  if ((c.rows > 0 && (!c.q || (c.Hk > 0 && !c.k)))) return ATTN_EINVAL;
  const void* x[2] = {c.q, c.k};
  const void* w[2] = {c.qw, c.kw};
  const long long st[2] = {c.q_token, c.k_token}, sh[2] = {c.q_head, c.k_head};
  const int heads[2] = {c.Hq, c.Hk};
  for (int i = 0; i < 2; ++i) {
    Side& s = p.side[i];
    s.heads = heads[i];
    if (heads[i] == 0) continue;
    if (!ptr_aligned(x[i], 16) || !ptr_aligned(w[i], 16)) return ATTN_EINVAL;
    if (st[i] < c.d || sh[i] < c.d || st[i] % 8 || sh[i] % 8 || st[i] > (1LL << 40) || sh[i] > (1LL << 40)) return ATTN_EINVAL;
    if (static_cast<long long>(c.rows) * heads[i] > (1LL << 40) / c.d) return ATTN_EINVAL;
    s.x = static_cast<const uint16_t*>(x[i]);
    s.w = w[i];
    s.s_token = st[i];
    s.s_head = sh[i];
  }
  for (int i = 0; i < c.rot / 2; ++i) {
    if (!std::isfinite(c.freqs[i])) return ATTN_EINVAL;
    const int a = c.axis ? c.axis[i] : 0;
    if (a < 0 || a >= c.axes) return ATTN_EINVAL;
    p.turns[i] = turn_of(c.freqs[i]);
    p.axis[i] = static_cast<uint8_t>(a);
  }
  p.rows = c.rows;
  p.d = c.d;
  p.items = c.d / 16;
  p.lg = 0;
  while ((1 << p.lg) < p.items) ++p.lg;
  p.rot = c.rot;
  p.w32 = c.w32;
  p.eps = c.eps;
  p.inv_d = 1.0f / static_cast<float>(c.d);
  p.amplitude = c.amplitude;
  p.positions = c.positions;
  return ATTN_OK;
}

unsigned long long in_bytes(const Params& p, int i) {
  return extent(p.rows, p.side[i].s_token, p.side[i].heads, p.side[i].s_head, p.d);
}
unsigned long long out_bytes(const Params& p, int i) {
  return 2ull * p.rows * p.side[i].heads * p.d;
}

// Checks the two outputs against each other and against the inputs; x itself
// (contiguous) may be its own output.
int check_outputs(const Params& p, void* const (&out)[2], const void* const (&more)[2]) {
  for (int i = 0; i < 2; ++i) {
    if (p.side[i].heads == 0) continue;
    if ((p.rows > 0 && !out[i]) || !ptr_aligned(out[i], 16)) return ATTN_EINVAL;
    for (int j = 0; j < 2; ++j) {
      if (p.side[j].heads == 0) continue;
      if (j != i && overlap(out[i], out_bytes(p, i), out[j], out_bytes(p, j))) return ATTN_EINVAL;
      const bool same = i == j && out[i] == p.side[i].x;
      if (same && (p.side[i].s_head != p.d || p.side[i].s_token != static_cast<long long>(p.side[i].heads) * p.d)) return ATTN_EINVAL;
      if (!same && overlap(out[i], out_bytes(p, i), p.side[j].x, in_bytes(p, j))) return ATTN_EINVAL;
      if (more[j] && !(i == j && out[i] == more[j]) && overlap(out[i], out_bytes(p, i), more[j], out_bytes(p, j))) return ATTN_EINVAL;
    }
  }
  return ATTN_OK;
}

int device(DeviceInfo& info) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ELAUNCH;
  if (int rc = device_info(dev, info)) return rc;
  return info.supported ? ATTN_OK : ATTN_EUNSUPPORTED;
}

// Blocks, and the parts of the tokens that are left when every warp has had as many
// whole ones as the others (all of them, where there are fewer tokens than warps).
int shape(Params& p, int sms, int per_sm) {
  const long long slots = static_cast<long long>(per_sm) * kWarps * sms;
  const int per = 32 >> p.lg, steps = (std::max(p.side[0].heads, p.side[1].heads) + per - 1) / per;
  const long long rest = std::max<long long>(p.rows % slots, 1);
  p.parts = static_cast<int>(std::max<long long>(1, std::min<long long>({8, slots / rest, steps})));
  if (p.rows >= slots) return per_sm * sms;
  return static_cast<int>((static_cast<long long>(p.rows) * p.parts + kWarps - 1) / kWarps);
}

template <bool BWD>
void smem_allowed(bool bf16, bool gptj) {
  const auto f = bf16 ? (gptj ? norm_kernel<true, true, BWD> : norm_kernel<true, false, BWD>)
                      : (gptj ? norm_kernel<false, true, BWD> : norm_kernel<false, false, BWD>);
  cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
}

template <bool BWD>
void run(const Params& p, bool bf16, bool gptj, int grid, cudaStream_t stream) {
  size_t smem = (static_cast<size_t>(kWarps) * p.rot + 2 * p.d) * sizeof(float);
  if (BWD) smem += std::max(static_cast<size_t>(kWarps) * 2 * p.d, static_cast<size_t>(kThreads) * 32) * sizeof(float);
  if (smem > 48 * 1024) smem_allowed<BWD>(bf16, gptj);   // (backward, from 8 rot + 2 d > 4,096 on: d = rot from 416)
  if (bf16) gptj ? norm_kernel<true, true, BWD><<<grid, kThreads, smem, stream>>>(p)
                 : norm_kernel<true, false, BWD><<<grid, kThreads, smem, stream>>>(p);
  else gptj ? norm_kernel<false, true, BWD><<<grid, kThreads, smem, stream>>>(p)
            : norm_kernel<false, false, BWD><<<grid, kThreads, smem, stream>>>(p);
}

}  // namespace norm
}  // namespace attn

extern "C" {

int attn_qk_norm_rotary(const void* q, const void* k, void* q_out, void* k_out, long long q_stride_token,
                        long long q_stride_head, long long k_stride_token, long long k_stride_head, int rows, int Hq,
                        int Hk, int d, const void* q_weight_or_null, const void* k_weight_or_null, int weight_fp32,
                        float eps, int rot_dim, const double* freqs, const int* axis_of_pair_or_null, int axes,
                        float amplitude, int interleaved, const int* positions, int fp16, cudaStream_t stream) {
  using namespace attn;
  using namespace attn::norm;
  static thread_local Params p;
  p = Params{};
  const Call c{q, k, q_weight_or_null, k_weight_or_null, q_stride_token, q_stride_head, k_stride_token, k_stride_head,
               rows, Hq, Hk, d, weight_fp32, rot_dim, axes, interleaved, fp16, eps, amplitude, freqs,
               axis_of_pair_or_null, positions};
  if (int rc = fill(c, p)) return rc;
  void* const out[2] = {q_out, k_out};
  const void* const none[2] = {nullptr, nullptr};
  if (int rc = check_outputs(p, out, none)) return rc;
  if (rows == 0) return ATTN_OK;
  for (int i = 0; i < 2; ++i) p.side[i].out = static_cast<uint16_t*>(out[i]);
  DeviceInfo info;
  if (int rc = device(info)) return rc;
  const int grid = shape(p, info.sm_count, 2);
  run<false>(p, fp16 == 0, interleaved != 0, grid, stream);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ELAUNCH;
  count_launch();
  return ATTN_OK;
}

long long attn_qk_norm_workspace_bytes(int d) {
  using namespace attn;
  if (d <= 0) return ATTN_EINVAL;
  if (d % 16 != 0 || d > 512) return ATTN_EUNSUPPORTED;
  DeviceInfo info;
  if (int rc = norm::device(info)) return rc;
  return static_cast<long long>(norm::bwd_blocks(info.sm_count)) * 2 * d * sizeof(float);
}

int attn_qk_norm_rotary_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k, void* dq, void* dk,
                            void* dq_weight_or_null, void* dk_weight_or_null, long long q_stride_token,
                            long long q_stride_head, long long k_stride_token, long long k_stride_head, int rows, int Hq,
                            int Hk, int d, const void* q_weight_or_null, const void* k_weight_or_null, int weight_fp32,
                            float eps, int rot_dim, const double* freqs, const int* axis_of_pair_or_null, int axes,
                            float amplitude, int interleaved, const int* positions, int fp16, void* workspace,
                            long long workspace_bytes, cudaStream_t stream) {
  using namespace attn;
  using namespace attn::norm;
  static thread_local Params p;
  p = Params{};
  const Call c{q, k, q_weight_or_null, k_weight_or_null, q_stride_token, q_stride_head, k_stride_token, k_stride_head,
               rows, Hq, Hk, d, weight_fp32, rot_dim, axes, interleaved, fp16, eps, amplitude, freqs,
               axis_of_pair_or_null, positions};
  if (int rc = fill(c, p)) return rc;
  void* const out[2] = {dq, dk};
  const void* const dy[2] = {dq_out, Hk > 0 ? dk_out : nullptr};
  if (rows > 0 && (!dq_out || (Hk > 0 && !dk_out))) return ATTN_EINVAL;
  if (!ptr_aligned(dy[0], 16) || !ptr_aligned(dy[1], 16)) return ATTN_EINVAL;
  if (int rc = check_outputs(p, out, dy)) return rc;
  void* const dw[2] = {dq_weight_or_null, Hk > 0 ? dk_weight_or_null : nullptr};
  for (int i = 0; i < 2; ++i)
    if (!ptr_aligned(dw[i], weight_fp32 ? 4 : 2)) return ATTN_EINVAL;
  const bool sums = dw[0] || dw[1];
  if (sums && (!workspace || !ptr_aligned(workspace, 256) || workspace_bytes < 256)) return ATTN_EINVAL;
  DeviceInfo info;
  if (int rc = device(info)) return rc;
  if (sums && workspace_bytes < static_cast<long long>(bwd_blocks(info.sm_count)) * 2 * d * static_cast<long long>(sizeof(float)))
    return ATTN_EINVAL;
  for (int i = 0; i < 2; ++i) {
    p.side[i].out = static_cast<uint16_t*>(out[i]);
    p.side[i].dy = static_cast<const uint16_t*>(dy[i]);
  }
  p.partial = sums ? static_cast<float*>(workspace) : nullptr;
  int grid = 0;
  if (rows > 0) {
    grid = shape(p, info.sm_count, kBlocksPerSM);
    run<true>(p, fp16 == 0, interleaved != 0, grid, stream);
    if (cudaGetLastError() != cudaSuccess) return ATTN_ELAUNCH;
    count_launch();
  }
  if (!sums) return ATTN_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * d / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const float* partial = p.partial;
  const cudaError_t e = fp16 ? cudaLaunchKernelEx(&cfg, sum_weights_kernel<false>, partial, grid, d, dw[0], dw[1], weight_fp32)
                             : cudaLaunchKernelEx(&cfg, sum_weights_kernel<true>, partial, grid, d, dw[0], dw[1], weight_fp32);
  if (e != cudaSuccess) return ATTN_ELAUNCH;
  count_launch();
  return ATTN_OK;
}

}  // extern "C"
