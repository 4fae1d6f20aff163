// What the two kernels of the attention over caches of 8-bit floating point share
// (attn_tree_fp8_kernel.cuh, attn_tree_fp8_rows.cuh): the walk over the work, the
// producers of K, V and their scales, the warps that widen V, the queries'
// e4m3 pieces, and the join of a cut unit's pieces.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_paged_line.cuh"
#include "attn_params.h"
#include "attn_tree_fp8.h"
#include "ptx.cuh"

namespace attn {
namespace tree {

// Warps: the loads of K, the MMAs, the loads of V, and the queries (in the kernel with
// rows the MMAs of S, and those of P V); four of softmax; four that widen V; four more of
// softmax.
constexpr int kWarpK = 0, kWarpMMA = 1, kWarpV = 2, kWarpQ = 3, kWarpSoft1 = 4, kWarpWiden = 8, kWarpSoft2 = 12;
constexpr int kThreads = 512;
// Registers: of the launch's 4 x 128 a thread per warpgroup, the softmax warps take what
// the others do without.
constexpr int kRegsFew = 88, kRegsMany = 168;
static_assert(2 * (kRegsFew + kRegsMany) <= 512, "the launch's registers");
constexpr int kRing = 8;                // stages of scales
// A key that a row (a query's column) sees weighs p = 2^s, s its score in powers of two, and
// its value row's scale is vs.  The row's reference m is the running maximum of s + log2 vs
// over what it sees (it may lag by 8), so that P' = p vs 2^-m is measured by what reaches the
// row's output: neither a key that it does not see nor one without weight counts there,
// however large its value row.  P' is held times 2^kHeldUp in fp16, which has 2^8 to spare
// above (the lag) and keeps P' to 2^-32 below.  Scales count in m as 2^-70 at the least
// (rows of zeros have 2^-126).  l sums p itself in fp32, relative to m: times 2^(kHeldUp +
// kMiddle), and P' takes 2^-kMiddle with the scale, which puts scales from 2^-70 to 2^119
// (the largest there is) around the middle of fp32's range.
constexpr float kHeldUp = 7.0f, kMiddle = 15.0f;
constexpr float kScaleDown = 0x1p-15f, kScaleUp = 0x1p15f;
constexpr float kLeastInRef = 0x1p-70f;
constexpr float kPieceUp = 0x1p4f, kPieceDown = 0x1p-4f;   // of the queries' pieces (convert_queries)
constexpr float kMostScale = 3.402823466e38f;   // (larger: none, or no number)

// The CTA's walk over units: (b, hc) in order, unit at position p of the line
// of steps with T steps and one more for its fixed cost.
struct Walk {
  int b, hc;          // hc: group of p.abreast units; this CTA's is hc * abreast + its place
  long long p, end;   // unit start; end of this CTA's range
  long long begin;
  int n, T;           // keys, steps
  int cols, row0, ctx;   // columns (token, head) of a key/value head; first row of q; keys before the new tokens
  int t0, t1;         // this CTA's steps of the unit
};

// Keys and new tokens of sequence b; one without new tokens takes no time, so it
// has no keys either.
__device__ __forceinline__ void sequence(const Params& p, int b, int& n, int& tokens, int& row0) {
  if (p.cu == nullptr) {
    tokens = 1;
    row0 = b;
    n = paged_len(p.c.t, b, p.err);
    return;
  }
  chunk_and_keys(p.c.t, p.cu, b, p.total, tokens, row0, n, p.err);
  if (tokens > p.max_tokens) {
    atomicCAS(p.err, 0, ATTN_DEVERR_BAD_SEQLENS);
    tokens = 0;
  }
  if (tokens == 0) n = 0;
}

template <int KS>
__device__ __forceinline__ int steps_of(int n) { return (n + KS - 1) / KS; }

template <int KS>
__device__ __forceinline__ void enter(const Params& p, Walk& w) {
  int tokens;
  sequence(p, w.b, w.n, tokens, w.row0);
  w.T = steps_of<KS>(w.n);
  w.cols = tokens * p.group;
  w.ctx = w.n - tokens;
}

// The next unit that has something to do here; false at the range's end.
template <int KS>
__device__ __forceinline__ bool next_unit(const Params& p, Walk& w, bool first) {
  const int nh = p.c.t.hkv * p.parts / p.abreast;
  while (true) {
    if (!first) {
      w.p += w.T + 1;
      if (++w.hc == nh) {
        w.hc = 0;
        if (++w.b < p.B) enter<KS>(p, w);
      }
    }
    first = false;
    if (w.b >= p.B || w.p >= w.end) return false;
    if (part_of<kMinSteps>(w.p, w.T, w.begin, w.end, w.t0, w.t1)) return true;
  }
}

// The table's entry for a key, read a step before it is used so that nothing waits
// for it, and the page that it names.  -1: past the last key; no page: num_pages
// (its rows lie past the pool and read as zeros).
__device__ __forceinline__ int entry_of(const Params& p, const Walk& w, int key) {
  return key < w.n ? __ldg(p.c.t.table + static_cast<long long>(w.b) * p.c.t.table_stride + (key >> p.c.t.page_log2)) : -1;
}
__device__ __forceinline__ int page_of(const Params& p, const Walk& w, int entry, int key) {
  if (key >= w.n) return -1;
  if (entry >= 0 && entry < p.c.t.num_pages) return entry;
  atomicCAS(p.err, 0, ATTN_DEVERR_BAD_PAGE);
  return p.c.t.num_pages;
}

// cc / p.group for cc < 2^20: the rounding of the product (2^-23 of it, twice) stays
// below the half that keeps it off the quotient's borders.
__device__ __forceinline__ int token_of(const Params& p, int cc) {
  return static_cast<int>((static_cast<float>(cc) + 0.5f) * p.inv_group);
}

// A unit's place among the heads: key/value head and first column.
struct Unit {
  int g, col0, cols;   // cols: of this unit, none where the sequence's tree ends before
};
template <int N>
__device__ __forceinline__ Unit unit_of(const Params& p, const Walk& w, int place) {
  const int unit = w.hc * p.abreast + place;
  Unit u;
  u.g = unit / p.parts;
  u.col0 = (unit - u.g * p.parts) * N;
  u.cols = min(N, w.cols - u.col0);
  return u;
}

// Byte offset of byte `at` of row `row` in a K-major tile of rows of ROW bytes (128
// or 64) under the swizzle of that width.
template <int ROW>
__device__ __forceinline__ uint32_t swizzled(int row, int at) {
  const int x = ROW == 128 ? (row & 7) : ((row >> 1) & 3);
  return static_cast<uint32_t>(row * ROW + ((((at >> 4) ^ x) << 4) | (at & 15)));
}

// The halves of a shared-memory matrix descriptor (sdesc_sw128): the lower has the
// address and the leading byte offset, the upper is a constant, the stride byte offset
// and the swizzle mode (2: 128 bytes, 4: 64).
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t lbo_bytes) {
  return (saddr & 0x3FFFFu) >> 4 | lbo_bytes >> 4 << 16;
}
constexpr uint32_t desc_high(uint32_t sbo_bytes, uint32_t mode) { return sbo_bytes >> 4 | 1u << 14 | mode << 29; }
constexpr uint32_t kHigh = desc_high(1024, 2);   // rows of 128 bytes
template <int ROW>
constexpr uint32_t kHighRows = ROW == 128 ? kHigh : desc_high(8 * ROW, 4);   // K-major e4m3 rows of ROW bytes

// The MMAs by the descriptors' lower halves.  D[tmem] (+)= A[smem] * B[smem]^T, 8-bit
// operands; the same, 16-bit; A in tensor memory, 16-bit.  fp32 accumulation.
template <uint32_t H>
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n\t}"
      :: "r"(d_tmem), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(H)
      : "memory");
}
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}"
      :: "r"(d_tmem), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kHigh)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}"
      :: "r"(d_tmem), "r"(a_tmem), "r"(b), "r"(idesc), "r"(accumulate), "n"(kHigh)
      : "memory");
}
// What lane 0 has, uniform over the warp to the compiler too: the MMAs take their operands
// from uniform registers, and moving each of them there from a thread's is what an issuing
// thread spends most of its time on.  The warps that issue MMAs run with all their lanes.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
  return on != 0;
}
// kind::f8f6f4, A of e4m3 or e5m2 and B of e4m3, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_e5m2 = false) {
  return (1u << 4) | ((a_e5m2 ? 1u : 0u) << 7) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// 4-byte asynchronous copy to shared memory, and the arrival of this thread's
// copies so far on a barrier that counts its threads.
__device__ __forceinline__ void copy4(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(bar) : "memory");
}

// The waits of this kernel (ptx.cuh's in fewer instructions: many warps run code of
// their own here, and fetching it counts): every lane polls, the limit is looked at
// with each failed poll.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const WaitCtl& w, int code) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (*w.abort_flag) return false;
    if (global_timer_ns() - t0 > w.timeout_ns) {
      report_error(w, code);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const WaitCtl& w, int code) {
  return __all_sync(0xffffffffu, wait(bar, parity, w, code));
}

// W consecutive 32-bit columns of this thread's TMEM lane (W = 1, 4, 8 or 16); the
// values are there after tld_wait.
template <int W>
__device__ __forceinline__ void tld_start(uint32_t taddr, float (&x)[W]) {
  if constexpr (W == 1) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=f"(x[0]) : "r"(taddr));
  } else if constexpr (W == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(taddr));
  } else if constexpr (W == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                 : "r"(taddr));
  } else {
    static_assert(W == 16, "columns");
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]),
                   "=f"(x[8]), "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15])
                 : "r"(taddr));
  }
}
// Waits for this thread's loads, and ties the values to the wait, so that no use of
// them can be scheduled above it.
template <int W>
__device__ __forceinline__ void tie(float (&x)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) asm volatile("" : "+f"(x[i]));
}
template <int W>
__device__ __forceinline__ void tld_wait(float (&x)[W], float (&y)[W]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  tie<W>(x);
  tie<W>(y);
}
template <int W>
__device__ __forceinline__ void tld(uint32_t taddr, float (&x)[W]) {
  tld_start<W>(taddr, x);
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  tie<W>(x);
}
__device__ __forceinline__ void tst16(uint32_t taddr, const float (&x)[16]) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(x[i]);
  tmem_st_32x32b_x16(taddr, r);
}

__device__ __forceinline__ void store16(uint32_t at, uint32_t x) {
  asm volatile("st.shared.b16 [%0], %1;" :: "r"(at), "h"(static_cast<unsigned short>(x)) : "memory");
}
constexpr uint32_t kNan2 = 0x7fff7fffu;   // two fp16 NaN

// log2 of a value's scale, as the rows' references count it (none, where it is no number).
__device__ __forceinline__ float scale_log2(float vs) {
  return vs <= kMostScale ? __log2f(fmaxf(vs, kLeastInRef)) : -70.0f;
}

// What joins two parts (m, l) of a row: log2 of the sum of its weights (-inf: none), and the
// factors that bring each part's u to O (negative: it saw no key, and its u is nothing).
// By the logarithms of the sums, which do not depend on the parts' references.
struct Joined {
  float sum, f0, f1;
  bool some;
};
__device__ __forceinline__ Joined join(float m0, float l0, float m1, float l1) {
  const bool has0 = l0 != 0.0f, has1 = l1 != 0.0f;   // (a NaN is something, and stays)
  const float a = m0 + __log2f(l0), b = m1 + __log2f(l1);
  const float top = !has1 ? a : has0 ? fmaxf(a, b) : b;
  const float w0 = has0 ? ex2_approx(a - top) : 0.0f, w1 = has1 ? ex2_approx(b - top) : 0.0f, w = w0 + w1;
  Joined r;
  r.some = has0 || has1;
  r.sum = r.some ? top + __log2f(w) - (kHeldUp + kMiddle) : -INFINITY;
  r.f0 = has0 ? w0 / (l0 * w) * kScaleUp : -1.0f;
  r.f1 = has1 ? w1 / (l1 * w) * kScaleUp : -1.0f;
  return r;
}

// Combines n columns (a power of two, at most 8 here) over the warp's lanes: each
// exchange halves the columns that a lane holds, n - 1 shuffles and the rest of five
// instead of 5 n.  Returns the result of column lane >> (5 - log2 n).
template <int n, typename Op>
__device__ __forceinline__ float fold_columns(float (&v)[n], int lane, Op op) {
  int o = 16;
#pragma unroll
  for (int half = n / 2; half > 0; half >>= 1, o >>= 1) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = upper ? v[i + half] : v[i], give = upper ? v[i] : v[i + half];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
#pragma unroll
  for (; o > 0; o >>= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
  return v[0];
}

// Two e4m3 values as the fp16 pair.
__device__ __forceinline__ uint32_t widen2(uint32_t x) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(x)));
  return h;
}
// x as two fp16 pairs: the nearest, and 2^11 times the rest.
__device__ __forceinline__ void split2(float2 x, uint32_t& high, uint32_t& rest) {
  high = pack2<false>(x.x, x.y);
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&high));
  const float2 r = fmul2(fadd2(x, make_float2(-h.x, -h.y)), make_float2(2048.0f, 2048.0f));
  rest = pack2<false>(r.x, r.y);
}
// Two floats as the nearest e4m3 pair, which is taken off them.
__device__ __forceinline__ uint32_t take2(float& a, float& b) {
  const uint32_t v = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t h = widen2(v);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  a -= f.x;
  b -= f.y;
  return v;
}

// Bytes of a step's K (and V) as they are stored, and of its V in fp16, chunks of 64
// features by 128 keys of 128-byte rows.
template <int DA, int TPS>
struct Tiles {
  static constexpr int KS = kKeys * TPS;
  static constexpr int kRaw = KS * DA, kWide = 2 * kRaw, kWideChunk = kKeys * 128;
};

// a / b for a >= 0, b > 0: in 32 bits where that does, which every call of usual size
// does, in a fifth of the instructions.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}
// range_of (attn_paged_line.cuh) with these divisions.
__device__ __forceinline__ long long range_length(long long total, long long units, int ranges) {
  const long long share = quotient(total + ranges - 1, ranges);
  if (share >= kMinSteps) return share;
  return max(share, min(static_cast<long long>(kMinSteps), units > 0 ? quotient(total, units) : 1));
}

// Finds where this CTA's range of the line begins; __syncthreads, then enter_line.
// The line of steps: each thread a strip of sequences, then a prefix sum.
struct Line {
  long long begin, end, range;
  int place, range_id;
};
template <int KS>
__device__ __forceinline__ Line find_line(const Params& p, volatile int* start_b, volatile long long* start_p,
                                          long long* warp_sums) {
  Line r;
  const int nh = p.c.t.hkv * p.parts / p.abreast;
  const int ranges = gridDim.x / p.abreast;
  r.place = blockIdx.x % p.abreast;
  r.range_id = blockIdx.x / p.abreast;
  const int tid = threadIdx.x, strip = (p.B + kThreads - 1) / kThreads;
  const int b_lo = min(tid * strip, p.B), b_hi = min(b_lo + strip, p.B);
  auto cost_of = [&](int b) {
    int n, tokens, row0;
    sequence(p, b, n, tokens, row0);
    return static_cast<long long>(nh) * (steps_of<KS>(n) + 1);
  };
  long long mine = 0, total, units;
#pragma unroll 1
  for (int b = b_lo; b < b_hi; ++b) mine += cost_of(b);
  const long long before = block_prefix<kThreads>(
      mine, static_cast<int>(min(static_cast<long long>(nh) * (b_hi - b_lo), 1LL << 24)), warp_sums, total, units);
  r.range = range_length(total, units, ranges);
  // (SMs past the last whole range idle)
  r.begin = r.range_id < ranges ? r.range_id * r.range : total;
  r.end = min(r.begin + r.range, total);
  if (r.begin >= before && r.begin < before + mine) {
    long long at = before;
#pragma unroll 1
    for (int b = b_lo; b < b_hi; ++b) {
      const long long cost = cost_of(b);
      if (r.begin < at + cost) {
        *start_b = b;
        *start_p = at;
        break;
      }
      at += cost;
    }
  }
  if (tid == 0) p.rec[blockIdx.x] = make_int4(0, 0, 0, 0);
  return r;
}
template <int KS>
__device__ __forceinline__ Walk enter_line(const Params& p, const Line& line, int start_b, long long start_p) {
  Walk w = {};
  w.b = start_b;
  w.begin = line.begin;
  w.end = line.end;
  w.p = start_p;
  if (w.b < p.B) {
    enter<KS>(p, w);
    w.hc = static_cast<int>(quotient(w.begin - w.p, w.T + 1));
    w.p += static_cast<long long>(w.hc) * (w.T + 1);
  }
  return w;
}

// A warp that loads K, or V, of every step: stages of kRaw bytes from `stages` on, a
// box per page and tile; and the keys' or the values' scales, KS floats a step at
// `to_scales` + 2 KS (step % kRing), by 4-byte asynchronous copies.  (The scales' ring
// needs no barrier for its empty stages: a stage of K or V is empty kStages steps later,
// once S, or the widening, of that step is through, which P of the step two before it
// goes ahead of; and kStages + 2 < kRing.)
template <int DA, int TPS, int N, int kStages>
__device__ __forceinline__ void produce(const Params& p, Walk w, int place, const CUtensorMap* map, uint32_t stages,
                                        uint32_t b_full, uint32_t b_empty, const float* scales, uint32_t to_scales,
                                        uint32_t b_c_full, const WaitCtl& wc) {
  using T = Tiles<DA, TPS>;
  constexpr int KS = T::KS, L = KS / 32;   // scales per lane: of keys 32 i + lane
  static_assert(kStages + 2 < kRing, "the scales' ring");
  const int lane = threadIdx.x & 31;
  uint32_t cnt = 0;
  const int box = min(1 << p.c.t.page_log2, kKeys);   // tokens per box
  const int n_pg = kKeys / box;                       // boxes along a tile
  // this lane's box: page `pg` of tile `y` of the step
  const int pg = lane % n_pg, y = lane / n_pg;
  const bool has = lane < TPS * n_pg;
  const int key_off = y * kKeys + pg * box;
  const uint32_t dst0 = stages + key_off * DA;
  auto box_entry = [&](int t) { return has ? entry_of(p, w, t * KS + key_off) : -1; };
  bool ok = true;
  for (bool more = next_unit<KS>(p, w, true); more && ok; more = next_unit<KS>(p, w, false)) {
    const Unit u = unit_of<N>(p, w, place);
    if (w.t1 <= w.t0 || u.cols <= 0) continue;
    const float* head = scales + u.g * p.c.c_head;
    int entry = box_entry(w.t0), of_key[L];
    auto key_entries = [&](int t) {
#pragma unroll
      for (int i = 0; i < L; ++i) of_key[i] = entry_of(p, w, t * KS + 32 * i + lane);
    };
    key_entries(w.t0);
    for (int t = w.t0; t < w.t1; ++t) {
      const int st = cnt % kStages;
      const int next = t + 1 < w.t1 ? box_entry(t + 1) : -1;
      if (!wait_warp(b_empty + 8 * st, ((cnt / kStages) & 1) ^ 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteKEmpty))) {
        ok = false;
        break;
      }
      const int page = has ? page_of(p, w, entry, t * KS + key_off) : -1;
      const uint32_t n_box = __popc(__ballot_sync(0xffffffffu, page >= 0));
      if (lane == 0) mbar_arrive_expect_tx(b_full + 8 * st, n_box * box * DA);
      __syncwarp();
      if (page >= 0)
        tma_load_4d(dst0 + st * T::kRaw, map, b_full + 8 * st, 0, u.g, (t * KS + key_off) & ((1 << p.c.t.page_log2) - 1),
                    page);
      const uint32_t ring = cnt % kRing, dst = to_scales + ring * (2 * KS * 4) + lane * 4;
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const int key = t * KS + 32 * i + lane;
        if (key < w.n && static_cast<unsigned>(of_key[i]) < static_cast<unsigned>(p.c.t.num_pages))   // (a box has reported other pages)
          copy4(dst + 32 * i * 4, head + of_key[i] * p.c.c_page + (key & ((1 << p.c.t.page_log2) - 1)) * p.c.c_token);
      }
      copies_arrive(b_c_full + 8 * ring);
      if (t + 1 < w.t1) key_entries(t + 1);
      entry = next;
      ++cnt;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (lane == 0 && *wc.abort_flag) {
    // let the loads already issued land before the CTA exits
    for (int s = 0; s < kStages; ++s) {
      const uint32_t n = (cnt + kStages - 1 - s) / kStages;
      if (n > 0) mbar_wait(b_full + 8 * s, (n - 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteDrain), false);
    }
  }
}

// Waits until the P.V of this CTA's step i (over all units) has completed: phase i >> 1
// of pv_done(i & 1).  Parity tells that phase from its neighbours alone, so step i - 2's
// has to have been seen to complete (by this warp, or by one that it has waited for), and
// step i + 2's must not until the caller goes on.
__device__ __forceinline__ bool wait_pv(uint32_t b_pv_done, uint32_t i, const WaitCtl& wc) {
  return wait_warp(b_pv_done + 8 * (i & 1), (i >> 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSitePvDone));
}

// Four warps that widen V of every step to fp16 (two buffers at off_wide).
template <int DA, int TPS, int N, int kStages>
__device__ __forceinline__ void widen(const Params& p, Walk w, int place, uint8_t* smem, int off_raw, int off_wide,
                                      uint32_t b_v_full, uint32_t b_v_empty, uint32_t b_w_full, uint32_t b_pv_done,
                                      const WaitCtl& wc) {
  using T = Tiles<DA, TPS>;
  constexpr int KS = T::KS, kItems = KS * DA / 16 / 128;   // of 16 features, per thread
  const int me = threadIdx.x - 32 * kWarpWiden, lane = threadIdx.x & 31;
  // Of head dimension 128 a thread takes 16 features of rows 16 i + row: eight lanes
  // 4 words of two rows that differ in bits 0 and 2, so that they meet eight different
  // words of the banks in the swizzled stage as well as in the fp16 tile.  Of 64, 16
  // features of rows 32 i + row (tile i / 4): eight lanes two rows side by side.
  const int row = DA == 128 ? 8 * (me >> 6) + (((me >> 4) & 3) ^ (((me >> 2) & 1) * 5)) : me >> 2;
  const int c = DA == 128 ? 4 * ((me >> 3) & 1) + (me & 3) : me & 3;
  const uint32_t from = DA == 128 ? swizzled<128>(row, 16 * c) : row * 64 + 16 * c;
  const uint32_t to = (DA == 128 ? (c >> 2) * T::kWideChunk : 0) + row * 128 + ((2 * (c & 3) ^ (row & 7)) << 4);   // (the second word: bit 4 flipped)
  uint32_t step = 0;
  bool ok = true;
  for (bool more = next_unit<KS>(p, w, true); more && ok; more = next_unit<KS>(p, w, false)) {
    const Unit u = unit_of<N>(p, w, place);
    if (w.t1 <= w.t0 || u.cols <= 0) continue;
    for (int t = w.t0; t < w.t1; ++t) {
      const int st = step % kStages;
      if (step >= 2 && !wait_pv(b_pv_done, step - 2, wc)) { ok = false; break; }
      if (!wait_warp(b_v_full + 8 * st, (step / kStages) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteVFull))) {
        ok = false;
        break;
      }
      const uint8_t* src = smem + off_raw + st * T::kRaw + from;
      uint8_t* dst = smem + off_wide + (step & 1) * T::kWide;
      const int left = w.n - t * KS;   // keys from here on
      uint4 x[kItems];
#pragma unroll
      for (int i = 0; i < kItems; ++i) x[i] = *reinterpret_cast<const uint4*>(src + i * 2048);
      if (left < KS) {
        // rows past the last key may hold anything: 0 * NaN would be NaN
#pragma unroll
        for (int i = 0; i < kItems; ++i)
          if ((DA == 128 ? 16 * i : 32 * i) + row >= left) x[i] = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int at = DA == 128 ? i * 2048 : (i >> 2) * T::kWideChunk + (i & 3) * 4096;
        *reinterpret_cast<uint4*>(dst + to + at) =
            make_uint4(widen2(x[i].x), widen2(x[i].x >> 16), widen2(x[i].y), widen2(x[i].y >> 16));
        *reinterpret_cast<uint4*>(dst + (to ^ 16) + at) =
            make_uint4(widen2(x[i].z), widen2(x[i].z >> 16), widen2(x[i].w), widen2(x[i].w >> 16));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(b_v_empty + 8 * st);
        mbar_arrive(b_w_full + 8 * (step & 1));
      }
      ++step;
    }
  }
}

// The rows of q that are columns c0, c0 + dc, ... of the unit, as 8-bit pieces (two or three of
// `piece` bytes, rows of DA bytes, swizzled), their factors (scale, log2 e and the power
// of two, in one) and masks.  A row, its largest value in (224, 448], is the sum of its
// pieces, each the nearest to what the one before leaves, which is half its step.  STEPPED:
// e4m3 pieces, each kPieceUp times the scale of the one before (what is left reaches 2^8 then,
// of 448).  Otherwise their products are summed as they are: e4m3 pieces, the last e5m2,
// whose three bits are what is left of 8 (after one) or 11 (after two) and which reaches
// down to 2^-16.  A feature is off by 2^-14, 2^-21.8 of the row's largest, at the most, and
// by nothing from 2^-6 on.  A warp takes F rows at a time, the next 2 F on their
// way, in a loop: it runs once per unit, so fetching its code counts.  (Rows past u.cols
// hold anything: nothing reads their results.)
template <int DA, int F, bool STEPPED>
__device__ __forceinline__ void convert_queries(const Params& p, const Walk& w, const Unit& u, int c0, int dc, uint8_t* dst,
                                                int piece, float* col, unsigned long long* mask) {
  constexpr int E = DA / 32;      // features per lane
  const int lane = threadIdx.x & 31;
  int head;
  auto place_of = [&](int c) {   // row of q, and head
    const int cc = u.col0 + c, token = token_of(p, cc);
    head = u.g * p.group + cc - token * p.group;
    return w.row0 + token;
  };
  auto load = [&](int c) {
    uint2 v = make_uint2(0, 0);
    if (c < u.cols) {
      const long long row = place_of(c);
      const uint16_t* src = p.q + (row * p.Hq + head) * DA + E * lane;
      if constexpr (E == 4) v = __ldg(reinterpret_cast<const uint2*>(src));
      else v.x = __ldg(reinterpret_cast<const uint32_t*>(src));
    }
    return v;
  };
  // the masks, a lane each, on their way first (a warp has 32 rows at the most)
  const int my = c0 + lane * dc;
  unsigned long long my_mask = 0;
  if (my < u.cols) {
    const int row = place_of(my);
    my_mask = p.mask ? static_cast<unsigned long long>(__ldg(p.mask + row)) : (2ull << (row - w.row0)) - 1;
  }
  uint2 next[F], after[F];
#pragma unroll
  for (int f = 0; f < F; ++f) next[f] = load(c0 + f * dc);
#pragma unroll
  for (int f = 0; f < F; ++f) after[f] = load(c0 + (F + f) * dc);
#pragma unroll 1
  for (int c = c0; c < u.cols; c += F * dc) {
    float x[F][4];
    uint32_t top[F];
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const uint2 now = next[f];
      next[f] = after[f];
      after[f] = load(c + (2 * F + f) * dc);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t v = h == 0 ? now.x : now.y;
        const float2 t = p.fp16 ? __half22float2(*reinterpret_cast<const __half2*>(&v))
                                : make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
        x[f][2 * h] = t.x;
        x[f][2 * h + 1] = t.y;
      }
      top[f] = 0;   // as bits: a NaN counts above infinity
#pragma unroll
      for (int e = 0; e < 4; ++e) top[f] = max(top[f], __float_as_uint(x[f][e]) & 0x7fffffffu);
    }
#pragma unroll
    for (int f = 0; f < F; ++f) top[f] = __reduce_max_sync(0xffffffffu, top[f]);
#pragma unroll
    for (int f = 0; f < F; ++f) {
      // 2^k with max 2^k in (224, 448]: 448 = 1.75 2^8
      int k = 135 - static_cast<int>(top[f] >> 23) - ((top[f] & 0x7fffffu) > 0x600000u ? 1 : 0);
      k = min(k, 120);   // (rows below 2^-112)
      const float up = __uint_as_float(static_cast<uint32_t>(max(127 + k, 1)) << 23);
      const float down = __uint_as_float(static_cast<uint32_t>(min(127 - k, 254)) << 23);
      const int at = c + f * dc;
      if (lane == 0 && at < u.cols) col[at] = fmaxf(p.scale_log2 * down, 0x1p-126f);   // (positive: -inf stays -inf)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[f][e] = top[f] < 0x7f800000u ? x[f][e] * up : __uint_as_float(0x7fffffffu);
    }
    uint8_t* to = dst;
#pragma unroll 1
    for (int s = (p.fp16 ? 3 : 2) - (STEPPED ? 0 : 1); s > 0; --s, to += piece) {
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const int at = c + f * dc;
        uint32_t a = take2(x[f][0], x[f][1]), b = 0;
        if constexpr (E == 4) b = take2(x[f][2], x[f][3]);
        if constexpr (STEPPED) {
#pragma unroll
          for (int e = 0; e < E; ++e) x[f][e] *= kPieceUp;
        }
        uint8_t* y = to + swizzled<DA>(at, E * lane);
        if (F > 1 && at >= u.cols) continue;
        if constexpr (E == 4) *reinterpret_cast<uint32_t*>(y) = a | b << 16;
        else *reinterpret_cast<uint16_t*>(y) = static_cast<uint16_t>(a);
      }
    }
    if constexpr (!STEPPED) {
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const int at = c + f * dc;
        const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(x[f][0], x[f][1]), __NV_SATFINITE, __NV_E5M2);
        const uint32_t b = E == 4 ? __nv_cvt_float2_to_fp8x2(make_float2(x[f][2], x[f][3]), __NV_SATFINITE, __NV_E5M2) : 0;
        uint8_t* y = to + swizzled<DA>(at, E * lane);
        if (F > 1 && at >= u.cols) continue;
        if constexpr (E == 4) *reinterpret_cast<uint32_t*>(y) = a | b << 16;
        else *reinterpret_cast<uint16_t*>(y) = static_cast<uint16_t>(a);
      }
    }
  }
  if (my < u.cols) mask[my] = my_mask;
}

// Joins the pieces of the unit that block x's CTA began, for columns y, y + gridDim.y, ...
// of the unit: M = max m_s, w_s = 2^(m_s - M) l_s, O = sum w_s O_s / sum w_s.  Four
// warps take every fourth piece, a lane DA / 32 features; a programmatic
// dependent of the attention kernel.
template <int N, int DA>
__global__ void __launch_bounds__(128) tree_merge_kernel(const __grid_constant__ Params p) {
  constexpr int E = DA / 32;
  __shared__ float s_m[4], s_l[4];
  __shared__ float s_o[4][DA];
  const int c = blockIdx.x, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_wait_prerequisites();
  const int4 rec = __ldcg(p.rec + c);
  const int pieces = rec.z;
  if (pieces <= 1) return;
  const int g = rec.y / p.parts, col0 = (rec.y - g * p.parts) * N;
  const int row0 = p.cu ? __ldg(p.cu + rec.x) : rec.x;
  for (int h = blockIdx.y; h < rec.w; h += gridDim.y) {
    float M = -INFINITY, L = 0.0f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    auto slot = [&](int s) { return s == 0 ? 2 * c + 1 : 2 * (c + s * p.abreast); };
    for (int s0 = w; s0 < pieces; s0 += 16) {
      float2 ml[4];
      float x[4][E];
#pragma unroll
      for (int u = 0; u < 4; ++u) {   // four pieces in flight
        const int s = s0 + 4 * u;
        const bool in = s < pieces;
        ml[u] = in ? __ldcg(p.part_ml + slot(s) * N + h) : make_float2(-INFINITY, 0.0f);
        const float* src = p.part_o + (static_cast<size_t>(in ? slot(s) : 0) * N + h) * DA + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 v = in ? __ldcg(reinterpret_cast<const float2*>(src + e)) : make_float2(0.0f, 0.0f);
          x[u][e] = v.x;
          x[u][e + 1] = v.y;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (ml[u].y == 0.0f) continue;   // (l of NaN: the sums become NaN, whatever m)
        const float mn = fmaxf(M, ml[u].x);
        const float r = M == -INFINITY ? 0.0f : ex2_approx(M - mn), wt = ex2_approx(ml[u].x - mn) * ml[u].y;
        M = mn;
        L = L * r + wt;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * r + wt * x[u][e];
      }
    }
    if (lane == 0) {
      s_m[w] = M;
      s_l[w] = L;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[w][lane * E + e] = acc[e];
    __syncthreads();
    const int i = threadIdx.x;
    if (i < DA) {
      const float Mx = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
      float Lt = 0.0f, at = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (s_l[k] == 0.0f) continue;
        const float r = ex2_approx(s_m[k] - Mx);
        Lt += s_l[k] * r;
        at += s_o[k][i] * r;
      }
      const int token = token_of(p, col0 + h), head = g * p.group + (col0 + h) - token * p.group;
      const long long row = row0 + token;
      const float v = Lt != 0.0f ? at / Lt : 0.0f;
      p.o[(row * p.Hq + head) * DA + i] =
          p.fp16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
      if (i == 0)
        p.lse[static_cast<long long>(head) * p.total + row] =
            Lt != 0.0f ? Mx * 0.69314718055994531f + __logf(Lt) : -INFINITY;
    }
    __syncthreads();
  }
}

template <int N, int DA>
cudaError_t launch_merge(const Params& p, int cols, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, cols < 16 ? cols : 16);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, tree_merge_kernel<N, DA>, p);
  if (e == cudaSuccess) count_launch();
  return e;
}

// Launches `kernel` with its shared memory allowed (once per device: `done`), and the
// join of cut units.
template <int N, int DA>
cudaError_t launch_with_merge(void (*kernel)(Params), int smem, bool (&done)[64], const Params& p, int cols, int grid,
                              cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev] = true;
  }
  kernel<<<grid, kThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launch();
  return p.cuts ? launch_merge<N, DA>(p, cols, grid, stream) : cudaSuccess;
}

}  // namespace tree
}  // namespace attn
