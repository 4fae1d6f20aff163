// The attention weight that each cached key receives from a chunk of queries
// (attn_key_weights):
//   weights[b, g, j] = decay weights[b, g, j] + sum_h sum_i exp(scale q_ih . k_j - lse_ih)
// The forward's lse makes every weight independent of the others, so no
// softmax statistics are needed, only the scores again.
//
// S^T = K Q^T on tcgen05: the keys on the MMA's M dimension, (token, query
// head) rows on N, so each thread owns one key, sums its columns in registers,
// and the sum needs no exchange.  A CTA's unit is 256 keys of one key/value
// head, two M = 128 tiles whose K stays in shared memory, against the
// sequence's query tiles (all heads of the group), streamed through a ring: a
// query tile serves both key tiles, which halves what the ring draws from L2.
// Each key tile has its warpgroup and two S^T buffers in TMEM.
//
// The lse is a column's, the same for all threads.  Read from shared memory it
// costs as much of the 128 bytes a clock that an SM returns to registers as the
// scores themselves (with TMEM's 64 KB a tile, 2,300 clocks a query tile).  So
// the MMA subtracts it: K gets 16 more features (ALPHA, BETA, 1, 0 ...), and a
// query row -lse / scale in three pieces of the 16-bit type, each the rest that
// the one before leaves (24 bits and more), times those.  One MMA more a tile,
// and the thread's work is a multiplication, an exponential and an addition a
// score.
//
// A query with an infinite lse is left out: a number far below any score takes
// the place of -lse / scale, and its row of Q is zeroed in shared memory, so that
// it adds nothing whatever it holds (a NaN included).
//
// NT, the columns of a query tile: 128 for chunks; 16 when a sequence has few
// rows (one token's heads), where a 128-row box would fetch mostly other
// sequences' queries.  The sums are fp32 in a fixed order.
//
// Work: the units' query tiles form a line cut into equal ranges, one per CTA;
// a unit that reaches over a cut leaves 256 partial sums per piece, which
// weights_merge_kernel adds in order (no atomics: the same bits every time).
//
// Bound: one exponential a pair (32 a clock and SM) and 2 d FLOPs for chunks;
// K read once (HBM) for single tokens.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "attn_paged.h"
#include "attn_paged_launch.h"
#include "attn_paged_line.cuh"
#include "attn_params.h"
#include "ptx.cuh"

namespace attn {
namespace pwts {

// warps 0 and 2 load K and warps 1 and 4 issue the MMAs (a key tile each: with
// one token a sequence, a unit is one tile of 9 small MMAs per key tile, and one
// issuer's waits and walk over units were what it took: 57 -> 48 us), warp 3
// loads Q, and the warps from kWSum sum
constexpr int kWMma = 1, kWMma1 = 4;
constexpr int kWQ = 3;
constexpr int kWSum = 5;
constexpr int kKeys = 256;       // keys per unit
constexpr int kMinTiles = 4;     // pieces of a cut unit are at least about this long
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
  CUtensorMap tm_q;    // (d, Hq, total, 1), box 64 x heads x span x 1
  CUtensorMap tm_k;    // (d, Hkv, page_size, num_pages), box 64 x 1 x min(page_size, 128) x 1
  PagedKV c;
  const float* lse;    // (Hq, total)
  float* weights;      // (B, Hkv, len)
  const int* cu;
  int4* rec;           // per CTA: the unit whose first piece it ran (sequence, head, block, pieces)
  float* part;         // partial sums [2 CTAs][256]
  int* err;
  unsigned long long timeout_ns;
  int B, Hq, total, len, group, heads, parts, span;
  unsigned long long span_inv;   // ceil(2^64 / span), span > 1
  float scale_log2, decay;
  int abreast;       // key/value heads that walk the line side by side (heads_abreast)
  int cuts;          // the chunk can be long enough for a unit to be cut
  float inv_scale;   // 1 / scale; 1 for scale 0 (then the products are left out)
  int products;
};

struct Walk {
  int b, g, kb;              // g: this CTA's head of a group of p.abreast
  int q_len, k_len, row_q, n_kb;
  long long p, begin, end;   // unit start on the line; this CTA's range
  int n, t0, t1;             // query tiles of the unit; this CTA's part
};

// Unit kb of a sequence: keys 256 kb .. and the tokens that see them, the last
// min(q_len, k_len - 256 kb) of the chunk (all, without the causal mask).
template <bool CAUSAL>
struct Line {
  const Params& p;
  __device__ int tokens(const Walk& w, int kb) const {
    return CAUSAL ? min(w.q_len, w.k_len - kb * kKeys) : w.q_len;
  }
  // x / span, exact for every 32-bit x: a multiplication, where the roles walk
  // units a division of some 200 cycles would show
  __device__ int by_span(int x) const { return p.span == 1 ? x : static_cast<int>(__umul64hi(x, p.span_inv)); }
  __device__ int tiles(const Walk& w, int kb) const { return by_span(tokens(w, kb) + p.span - 1) * p.parts; }
  // cost of the units before kb of one head: query tiles, and one for K
  __device__ long long before(const Walk& w, int kb) const {
    if (kb <= 0) return 0;
    const long long all = by_span(w.q_len + p.span - 1);
    long long sum;
    if (kb <= 32) {   // few: one by one, without the closed form's divisions
      sum = kb;
      for (int i = 0; i < kb; ++i) sum += tiles(w, i);
      return sum;
    }
    if (!CAUSAL) {
      sum = all * kb;
    } else {
      const int off = w.k_len - w.q_len;
      const int full = off < 0 ? 0 : min(kb, off / kKeys + 1);   // units that every token sees
      sum = all * full;
      if (kb > full)
        sum += floor_sum(kb - full, p.span, kKeys, static_cast<long long>(w.k_len) - static_cast<long long>(kKeys) * (kb - 1) + p.span - 1);
    }
    return sum * p.parts + kb;
  }
  __device__ void load(Walk& w) const {
    chunk_and_keys(p.c, p.cu, w.b, p.total, w.q_len, w.row_q, w.k_len, p.err);
    if (w.k_len > p.len) {
      atomicCAS(p.err, 0, ATTN_DEVERR_BAD_SEQLENS);
      w.k_len = 0;
    }
    w.n_kb = (w.k_len + kKeys - 1) / kKeys;
  }
  __device__ long long cost(const Walk& w) const { return before(w, w.n_kb) * (p.c.hkv / p.abreast); }
  __device__ int units(const Walk& w) const {
    return static_cast<int>(min(static_cast<long long>(w.n_kb) * (p.c.hkv / p.abreast), 1LL << 24));
  }
  __device__ void advance(Walk& w) const {
    w.p += w.n + 1;
    if (++w.kb == w.n_kb) {
      w.kb = 0;
      if ((w.g += p.abreast) >= p.c.hkv) {
        w.g = blockIdx.x % p.abreast;
        while (++w.b < p.B) {
          load(w);
          if (w.n_kb > 0) break;
        }
      }
    }
    if (w.b < p.B) w.n = tiles(w, w.kb);
  }
  __device__ bool next(Walk& w, bool first) const {
    if (!first) advance(w);
    while (w.b < p.B && w.p < w.end) {
      if (part_of<kMinTiles>(w.p, w.n, w.begin, w.end, w.t0, w.t1)) return true;
      advance(w);
    }
    return false;
  }
};

// The query tiles of a piece, from its first: head part and first token, and
// which key tiles see the tile (kept as running values: the roles are single
// threads or few warps, whose dependent integer divisions would show).
template <bool CAUSAL>
struct Tiles {
  int part, tok, tok0, q_len, span;
  int tok_min[2];   // key tile x is seen by a tile that starts at tok >= tok_min[x]
  __device__ Tiles(const Params& p, const Walk& w, const Line<CAUSAL>& line) {
    const int per = line.by_span(line.tokens(w, w.kb) + p.span - 1);   // tiles of a head part
    span = p.span;
    q_len = w.q_len;
    tok0 = w.q_len - line.tokens(w, w.kb);
    part = p.parts > 1 && per > 0 ? w.t0 / per : 0;
    tok = tok0 + (w.t0 - part * per) * p.span;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int key = w.kb * kKeys + x * 128;
      // the tile's last token, tok + span - 1, sees keys up to it + k_len - q_len
      tok_min[x] = key >= w.k_len ? 0x7fffffff : CAUSAL ? key - (w.k_len - w.q_len) - p.span + 1 : -0x7fffffff;
    }
  }
  __device__ void next() {
    tok += span;
    if (tok >= q_len) {
      tok = tok0;
      ++part;
    }
  }
  __device__ bool active(int x) const { return tok >= (x == 0 ? tok_min[0] : tok_min[1]); }
};

// lse / scale = kAlpha p0 + kBeta p1 + p2, pieces in the 16-bit type.  bf16 has
// the range of fp32.  In fp16 |p0| <= 65504, and half its largest step times
// kAlpha, 2^19, is the most that is left for p1: 2^14 with kBeta, whose half step
// times kBeta, 2^8, is left for p2.
template <bool BF16>
constexpr float kAlpha = BF16 ? 1.0f : 32768.0f;
template <bool BF16>
constexpr float kBeta = BF16 ? 1.0f : 32.0f;
// The largest |lse / scale|, exactly kAlpha times a p0: about 2^31 in fp16.
// exp2(-kFar scale log2 e) is 0 for every scale from 2^-20, so a larger lse gives
// the formula's weights, 0 or infinity, for scores up to kFar / 2.
template <bool BF16>
constexpr float kFar = BF16 ? 0x1p120f : 61024.0f * 32768.0f;

// Byte offset of row r of a tile of 16 features without swizzle: 8 x 16-byte
// core matrices, the two of a row group side by side.
__device__ __forceinline__ int lse_row(int r) { return (r >> 3) * 256 + (r & 7) * 16; }
__device__ __forceinline__ uint64_t lse_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(128 >> 4) << 16 |
         static_cast<uint64_t>(256 >> 4) << 32 | static_cast<uint64_t>(1) << 46;
}

template <int D, int NT>
struct WCfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kKTile = 128 * D * 2;              // one key tile
  static constexpr int kKStage = 2 * kKTile;
  static constexpr int kQStage = NT * D * 2;
  static constexpr int kKS = NT == 128 ? (D == 128 ? 2 : 3) : (D == 128 ? 3 : 6);
  static constexpr int kQS = NT == 128 ? (D == 128 ? 2 : 4) : 4;
  static constexpr int kOffK = 0;
  static constexpr int kOffQ = kOffK + kKS * kKStage;
  static constexpr int kOffA = kOffQ + kQS * kQStage;     // the 16 more features: of the keys ...
  static constexpr int kOffL = kOffA + 128 * 32;          // ... and of each stage's query rows
  static constexpr int kThr = 32 * (kWSum + 8);
  static constexpr int kOffBar = kOffL + kQS * NT * 32;
  static constexpr int kNBars = 3 * kKS + 3 * kQS + 8 + 2;
  static constexpr int kOffMisc = kOffBar + (kNBars + 1) / 2 * 16;
  static constexpr int kSmem = kOffMisc + 384 + 1024;   // (2 sums a warp from kOffMisc + 32)
  static constexpr uint32_t kTmemCols = 4 * NT;           // [key tile][buffer]
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

// Adds exp2(c (s - lse / scale)) of CB columns to sum; MASK drops those outside
// [lo, hi), whatever their score.
template <int CB, bool MASK>
__device__ __forceinline__ void add_columns(const uint32_t (&r)[CB], float2 c2, int lo, int hi, float2 (&sum)[2]) {
#pragma unroll
  for (int k = 0; k < CB; k += 4) {
    const float2 a = fmul2(make_float2(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), c2);
    const float2 b = fmul2(make_float2(__uint_as_float(r[k + 2]), __uint_as_float(r[k + 3])), c2);
    float2 e0 = make_float2(ex2_approx(a.x), ex2_approx(a.y));
    float2 e1 = make_float2(ex2_approx(b.x), ex2_approx(b.y));
    if constexpr (MASK) {
      e0.x = (k >= lo && k < hi) ? e0.x : 0.0f;
      e0.y = (k + 1 >= lo && k + 1 < hi) ? e0.y : 0.0f;
      e1.x = (k + 2 >= lo && k + 2 < hi) ? e1.x : 0.0f;
      e1.y = (k + 3 >= lo && k + 3 < hi) ? e1.y : 0.0f;
    }
    sum[0] = fadd2(sum[0], e0);
    sum[1] = fadd2(sum[1], e1);
  }
}

// The columns of an S^T tile, of this thread's key; the next ones load while
// these are added.
template <int NT, bool MASK, class Release>
__device__ __forceinline__ void add_tile(uint32_t t_s, float2 c2, int lo, int hi, float2 (&sum)[2], Release release) {
  if constexpr (NT == 16) {
    uint32_t r[16];
    tmem_ld_32x32b_x16(t_s, r);
    tmem_wait_ld(r);
    release();
    add_columns<16, MASK>(r, c2, lo, hi, sum);
  } else {
    uint32_t r0[32], r1[32];
    tmem_ld_32x32b_x32(t_s, r0);
    tmem_wait_ld(r0);
#pragma unroll
    for (int c0 = 0; c0 < NT; c0 += 64) {
      tmem_ld_32x32b_x32(t_s + c0 + 32, r1);
      add_columns<32, MASK>(r0, c2, lo - c0, hi - c0, sum);
      tmem_wait_ld(r1);
      if (c0 + 64 < NT) tmem_ld_32x32b_x32(t_s + c0 + 64, r0);
      else release();
      add_columns<32, MASK>(r1, c2, lo - c0 - 32, hi - c0 - 32, sum);
      if (c0 + 64 < NT) tmem_wait_ld(r0);
    }
  }
}

// Zeroes this lane's rows of a query tile whose lse is infinite (bit k of `out`:
// row lane + 32 k), once the tile has landed.  Rare, and out of line: inlined it
// costs every call (a decoding step's weights 49.6 us against 48.7).
__device__ __noinline__ bool zero_rows(uint32_t bar, uint32_t parity, WaitCtl wc, uint8_t* tile, int chunk, int chunks,
                                       uint32_t out) {
  if (!mbar_wait_warp(bar, parity, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteQFull))) return false;
  for (int r = threadIdx.x & 31; out; r += 32, out >>= 1)
    if (out & 1)
      for (int y = 0; y < 8 * chunks; ++y)
        *reinterpret_cast<uint4*>(tile + (y >> 3) * chunk + r * 128 + (y & 7) * 16) = make_uint4(0, 0, 0, 0);
  return true;
}

template <int D, int NT, bool BF16, bool CAUSAL>
__global__ void __launch_bounds__(WCfg<D, NT>::kThr, 1) weights_kernel(const __grid_constant__ Params p) {
  using C = WCfg<D, NT>;
  constexpr int kThr = C::kThr;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sK = sbase + C::kOffK, sQ = sbase + C::kOffQ;
  const uint32_t bar0 = sbase + C::kOffBar;
  auto b_k_full = [&](int x, int s) { return bar0 + 8 * (x * C::kKS + s); };
  auto b_k_empty = [&](int s) { return bar0 + 8 * (2 * C::kKS + s); };
  const uint32_t bar1 = bar0 + 24 * C::kKS;
  auto b_q_full = [&](int s) { return bar1 + 8 * s; };
  auto b_q_empty = [&](int s) { return bar1 + 8 * (C::kQS + s); };
  const uint32_t bar2 = bar1 + 16 * C::kQS;
  auto b_s_full = [&](int x, int s) { return bar2 + 8 * (2 * x + s); };
  auto b_s_free = [&](int x, int s) { return bar2 + 32 + 8 * (2 * x + s); };
  auto b_drain = [&](int x) { return bar2 + 64 + 8 * x; };
  auto b_l_full = [&](int s) { return bar2 + 80 + 8 * s; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  volatile int* start = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);   // b, g, kb
  volatile long long* start_p = reinterpret_cast<volatile long long*>(smem + C::kOffMisc + 24);
  long long* warp_sums = reinterpret_cast<long long*>(smem + C::kOffMisc + 32);
  WaitCtl wc{p.err, abort_flag, p.timeout_ns};

  if (tid == 0) {
    *abort_flag = 0;
    start[0] = p.B;
    for (int s = 0; s < C::kKS; ++s) {
      mbar_init(b_k_full(0, s), 1);
      mbar_init(b_k_full(1, s), 1);
      mbar_init(b_k_empty(s), 2);   // the two issuers
    }
    for (int s = 0; s < C::kQS; ++s) {
      mbar_init(b_q_full(s), 1);
      mbar_init(b_q_empty(s), 2);
      mbar_init(b_l_full(s), 1);   // the lse features (and zeroed rows)
    }
    for (int x = 0; x < 2; ++x)
      for (int s = 0; s < 2; ++s) {
        mbar_init(b_s_full(x, s), 1);
        mbar_init(b_s_free(x, s), 4);   // the warps that read the buffer
      }
    mbar_init(b_drain(0), 1);
    mbar_init(b_drain(1), 1);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_k);
  }
  if (warp == kWMma) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }

  // the features that take the lse: (ALPHA, BETA, 1, 0 ...) for every key; of the
  // query rows only the first three change
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  for (int i = tid; i < 128; i += kThr) {
    const T a(kAlpha<BF16>), b(kBeta<BF16>), one(1.0f), zero(0.0f);
    T f[8] = {a, b, one, zero, zero, zero, zero, zero};
    *reinterpret_cast<uint4*>(smem + C::kOffA + lse_row(i)) = *reinterpret_cast<const uint4*>(f);
    *reinterpret_cast<uint4*>(smem + C::kOffA + lse_row(i) + 128) = make_uint4(0, 0, 0, 0);
  }
  for (int i = tid; i < C::kQS * NT * 2; i += kThr)
    reinterpret_cast<uint4*>(smem + C::kOffL)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();

  const Line<CAUSAL> line{p};
  Walk w0;
  const int strip = (p.B + kThr - 1) / kThr;
  const int b_lo = min(tid * strip, p.B), b_hi = min(b_lo + strip, p.B);
  long long mine = 0, total, units;
  int count = 0;
  for (w0.b = b_lo; w0.b < b_hi; ++w0.b) {
    line.load(w0);
    mine += line.cost(w0);
    count = min(count + line.units(w0), 1 << 24);   // (for a mean: the largest need not be exact)
  }
  const long long before = block_prefix<kThr>(mine, count, warp_sums, total, units);
  const long long range = range_of<kMinTiles>(total, units, gridDim.x / p.abreast);
  const int range_id = blockIdx.x / p.abreast;   // (SMs past the last whole range idle)
  const long long begin = range_id < static_cast<int>(gridDim.x) / p.abreast ? range_id * range : total;
  const long long end = min(begin + range, total);
  if (begin >= before && begin < before + mine) {
    long long at = before;
    for (w0.b = b_lo; w0.b < b_hi; ++w0.b) {
      line.load(w0);
      const long long cost = line.cost(w0);
      if (begin < at + cost) {
        const long long per = line.before(w0, w0.n_kb);
        const int g = static_cast<int>((begin - at) / per);
        at += g * per;
        int lo = 0, hi = w0.n_kb;   // the last unit that starts at or before `begin`
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (at + line.before(w0, mid) <= begin) lo = mid; else hi = mid;
        }
        start[0] = w0.b;
        start[1] = g * p.abreast + blockIdx.x % p.abreast;
        start[2] = lo;
        *start_p = at + line.before(w0, lo);
        break;
      }
      at += cost;
    }
  }
  if (tid == 0) p.rec[blockIdx.x] = make_int4(0, 0, 0, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_launch_dependents();
  w0.b = start[0];
  w0.begin = begin;
  w0.end = end;
  w0.p = 0;
  w0.g = w0.kb = w0.n = w0.n_kb = 0;
  if (w0.b < p.B) {
    w0.g = start[1];
    w0.kb = start[2];
    w0.p = *start_p;
    line.load(w0);
    w0.n = line.tiles(w0, w0.kb);
  }

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------------ TMA producer of key tile x
    const int x = warp >> 1;
    uint32_t k_cnt = 0;
    const int box = min(1 << p.c.page_log2, 128);   // tokens per box
    const int n_pg = 128 / box;                     // boxes along the tile
    const int pg = lane % n_pg, ch = lane / n_pg;   // this lane's box: page, feature chunk
    const bool has = lane < C::kChunks * n_pg;
    const uint32_t dst0 = sK + x * C::kKTile + ch * 16384 + pg * box * 128;
    // the page of this lane's box of a unit, -1: none to load
    auto page_of = [&](const Walk& u) {
      const int key = u.kb * kKeys + x * 128 + pg * box;
      if (!has || key >= u.k_len || u.t1 <= u.t0) return -1;
      const int id = paged_page(p.c, u.b, key >> p.c.page_log2, p.err);
      return id < 0 ? p.c.num_pages : id;   // no page: rows past the pool read as zeros
    };
    Walk w = w0, ahead;   // the next unit, whose page is read while this one is issued
    bool more = line.next(w, true), more_ahead = false;
    int page = more ? page_of(w) : -1, page_ahead = -1;
    for (; more; w = ahead, more = more_ahead, page = page_ahead) {
      ahead = w;
      more_ahead = line.next(ahead, false);
      page_ahead = more_ahead ? page_of(ahead) : -1;
      if (w.t1 <= w.t0) continue;
      const int key = w.kb * kKeys + x * 128 + pg * box;
      const int ks = k_cnt % C::kKS;
      if (!mbar_wait_warp(b_k_empty(ks), ((k_cnt / C::kKS) & 1) ^ 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteKEmpty))) break;
      const uint32_t n_box = __popc(__ballot_sync(0xffffffffu, page >= 0));
      if (lane == 0) mbar_arrive_expect_tx(b_k_full(x, ks), n_box * box * 128);
      __syncwarp();
      if (page >= 0)
        tma_load_4d(dst0 + ks * C::kKStage, &p.tm_k, b_k_full(x, ks), ch * 64, w.g, key & ((1 << p.c.page_log2) - 1), page);
      ++k_cnt;
    }
    if (lane == 0 && *abort_flag) {
      // let the loads already issued land before the CTA exits
      for (int s = 0; s < C::kKS; ++s) {
        const uint32_t n = (k_cnt + C::kKS - 1 - s) / C::kKS;
        if (n > 0) mbar_wait(b_k_full(x, s), (n - 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteDrain), false);
      }
    }
  } else if (warp == kWQ) {
    // ------------------------------------------------------------------ query tiles and their lse features
    constexpr int NC = (NT + 31) / 32;   // lane's rows are lane, lane + 32, ...
    int row_tok[NC], row_head[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      row_tok[k] = (lane + 32 * k) / p.heads;
      row_head[k] = lane + 32 * k - row_tok[k] * p.heads;
    }
    uint32_t q_cnt = 0;
    bool ok = true;
    Walk w = w0;
    for (bool more = line.next(w, true); more && ok; more = line.next(w, false)) {
      Tiles<CAUSAL> it(p, w, line);
      for (int i = w.t0; i < w.t1; ++i, it.next()) {
        const int qs = q_cnt % C::kQS, head0 = w.g * p.group + it.part * p.heads, row0 = w.row_q + it.tok;
        float l[NC];   // on its way while the stage is waited for
#pragma unroll
        for (int k = 0; k < NC; ++k) {
          l[k] = 0.0f;   // rows past the chunk: their columns are dropped by index
          if (lane + 32 * k < NT && row_tok[k] < p.span && it.tok + row_tok[k] < w.q_len)
            l[k] = __ldg(p.lse + static_cast<long long>(head0 + row_head[k]) * p.total + row0 + row_tok[k]);
        }
        if (!mbar_wait_warp(b_q_empty(qs), ((q_cnt / C::kQS) & 1) ^ 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteQEmpty))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(b_q_full(qs), C::kChunks * p.heads * p.span * 128);
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_4d(sQ + qs * C::kQStage + c * NT * 128, &p.tm_q, b_q_full(qs), c * 64, head0, row0, 0);
        }
        ++q_cnt;
        uint32_t out = 0;   // this lane's queries that are left out
#pragma unroll
        for (int k = 0; k < NC; ++k) out |= isinf(l[k]) ? 1u << k : 0u;
        if (__any_sync(0xffffffffu, out != 0) &&
            !zero_rows(b_q_full(qs), ((q_cnt - 1) / C::kQS) & 1, wc, smem + C::kOffQ + qs * C::kQStage, NT * 128,
                       C::kChunks, out)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int k = 0; k < NC; ++k) {
          // -lse / scale, within what the pieces hold; of a query left out far below every score
          constexpr float kF = kFar<BF16>, kA = kAlpha<BF16>, kB = kBeta<BF16>;
          const float v = isinf(l[k]) ? -kF : fminf(fmaxf(-l[k] * p.inv_scale, -kF), kF);
          const T p0 = T(v * (1.0f / kA));
          const float r1 = l[k] != l[k] ? l[k] : v - static_cast<float>(p0) * kA;
          const T p1 = T(r1 * (1.0f / kB));
          const T p2 = T(r1 - static_cast<float>(p1) * kB);
          T f[4] = {p0, p1, p2, T(0.0f)};
          if (lane + 32 * k < NT)
            *reinterpret_cast<uint2*>(smem + C::kOffL + qs * NT * 32 + lse_row(lane + 32 * k)) = *reinterpret_cast<const uint2*>(f);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_l_full(qs));
      }
    }
    if (lane == 0 && *abort_flag) {
      // let the loads already issued land before the CTA exits
      for (int s = 0; s < C::kQS; ++s) {
        const uint32_t n = (q_cnt + C::kQS - 1 - s) / C::kQS;
        if (n > 0) mbar_wait(b_q_full(s), (n - 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteDrain), false);
      }
    }
  } else if (warp == kWMma || warp == kWMma1) {
    // ------------------------------------------------------------------ MMA issuer of key tile x
    const int x = warp == kWMma1 ? 1 : 0;
    if (lane == 0) {
      constexpr uint32_t kIdesc = idesc_f16_f32acc(128, NT, BF16, false);
      const uint64_t dk0 = sdesc_sw128(sK, 16, 1024);
      const uint64_t dq0 = sdesc_sw128(sQ, 16, 1024);
      const uint64_t da0 = lse_desc(sbase + C::kOffA), dl0 = lse_desc(sbase + C::kOffL);
      uint32_t k_cnt = 0, q_cnt = 0, s_cnt = 0;
      bool ok = true;
      // the next unit and its tiles, worked out while the tensor core is busy
      // with this one's first tile
      Walk w = w0, ahead;
      bool more = line.next(w, true), more_ahead = false;
      ahead = w;
      Tiles<CAUSAL> it(p, w, line), it_ahead = it;
      for (; more && ok; w = ahead, it = it_ahead, more = more_ahead) {
        auto look_ahead = [&] {
          ahead = w;
          more_ahead = line.next(ahead, false);
          if (more_ahead) it_ahead = Tiles<CAUSAL>(p, ahead, line);
        };
        if (w.t1 <= w.t0) {
          look_ahead();
          continue;
        }
        const int ks = k_cnt % C::kKS;
        if (!mbar_wait(b_k_full(x, ks), (k_cnt / C::kKS) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteKFull))) break;
        ++k_cnt;
        for (int i = w.t0; i < w.t1 && ok; ++i, it.next()) {
          const int qs = q_cnt % C::kQS;
          if (!mbar_wait(b_l_full(qs), (q_cnt / C::kQS) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteQFull)) ||
              !mbar_wait(b_q_full(qs), (q_cnt / C::kQS) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteQFull))) {
            ok = false;
            break;
          }
          ++q_cnt;
          if (it.active(x)) {
            const int sb = s_cnt & 1;
            if (!mbar_wait(b_s_free(x, sb), ((s_cnt >> 1) & 1) ^ 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteSFree))) {
              ok = false;
              break;
            }
            ++s_cnt;
            tc_fence_after();
            // the products, then -lse / scale: the larger accumulator last, as every
            // addition of the tensor core truncates to fp32
            if (p.products) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t a = dk0 + ((ks * C::kKStage + x * C::kKTile + (kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
                const uint64_t b = dq0 + ((qs * C::kQStage + (kk >> 2) * NT * 128 + (kk & 3) * 32) >> 4);
                umma_ss(tmem + (2 * x + sb) * NT, a, b, kIdesc, kk > 0 ? 1u : 0u);
              }
            }
            umma_ss(tmem + (2 * x + sb) * NT, da0, dl0 + ((qs * NT * 32) >> 4), kIdesc, p.products ? 1u : 0u);
            umma_commit(b_s_full(x, sb));
          }
          umma_commit(b_q_empty(qs));
          if (i == w.t1 - 1) umma_commit(b_k_empty(ks));
          if (i == w.t0) look_ahead();
        }
      }
      umma_commit(b_drain(x));
      mbar_wait(b_drain(x), 0, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteDrain), false);
    }
  } else {
    // ------------------------------------------------------------------ sums: one warpgroup per key tile
    const int x = (warp - kWSum) >> 2;
    const int quarter = warp & 3;
    const int lrow = quarter * 32 + lane;   // TMEM lane: key of the tile
    const uint32_t t_s = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + 2 * x * NT;
    const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
    uint32_t s_cnt = 0;
    bool ok = true;
    auto out_of = [&](const Walk& u) {
      return p.weights + (static_cast<long long>(u.b) * p.c.hkv + u.g) * p.len + u.kb * kKeys + x * 128 + lrow;
    };
    auto old_of = [&](const Walk& u) {
      return p.decay != 0.0f && u.t1 - u.t0 == u.n && u.kb * kKeys + x * 128 + lrow < u.k_len ? *out_of(u) : 0.0f;
    };
    Walk w = w0, ahead;   // the next unit, whose old weights are read while this one is summed
    bool more = line.next(w, true), more_ahead = false;
    float old = more ? old_of(w) : 0.0f, old_ahead = 0.0f;
    for (; more && ok; w = ahead, more = more_ahead, old = old_ahead) {
      ahead = w;
      more_ahead = line.next(ahead, false);
      if (more_ahead) old_ahead = old_of(ahead);
      const int key = w.kb * kKeys + x * 128 + lrow, off = w.k_len - w.q_len;
      float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
      Tiles<CAUSAL> it(p, w, line);
      for (int i = w.t0; i < w.t1; ++i, it.next()) {
        if (!it.active(x)) continue;
        const int sb = s_cnt & 1;
        if (!mbar_wait_warp(b_s_full(x, sb), (s_cnt >> 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteSFull))) {
          ok = false;
          break;
        }
        ++s_cnt;
        tc_fence_after();
        // columns this key sees: from c_lo (causal) to the chunk's end
        const int c_lo = CAUSAL ? max(0, key - off - it.tok) * p.heads : 0;
        const int c_hi = min(p.span, w.q_len - it.tok) * p.heads;
        const bool full = (!CAUSAL || w.kb * kKeys + x * 128 + 127 - off <= it.tok) && c_hi == NT;
        auto release = [&] {   // the scores are in registers: the buffer may be overwritten
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_s_free(x, sb));
        };
        if (full) add_tile<NT, false>(t_s + sb * NT, c2, 0, NT, sum, release);
        else add_tile<NT, true>(t_s + sb * NT, c2, c_lo, c_hi, sum, release);
      }
      if (!ok) break;
      const float s = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      if (w.t1 - w.t0 == w.n) {
        if (key < w.k_len) *out_of(w) = p.decay * old + s;
      } else {
        p.part[(2 * blockIdx.x + (w.t0 == 0 ? 1 : 0)) * kKeys + x * 128 + lrow] = s;
        if (w.t0 == 0 && warp == kWSum && lane == 0)
          p.rec[blockIdx.x] = make_int4(w.b, w.g, w.kb,
                                        static_cast<int>((w.p + w.n - 1) / range) - range_id + 1);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Adds the pieces of the unit that block x's CTA began, in order.
__global__ void __launch_bounds__(kKeys) weights_merge_kernel(const __grid_constant__ Params p) {
  grid_wait_prerequisites();
  const int c = blockIdx.x;
  const int4 rec = __ldcg(p.rec + c);
  if (rec.w <= 1) return;
  const int key = rec.z * kKeys + threadIdx.x;
  float s = __ldcg(p.part + (2 * c + 1) * kKeys + threadIdx.x);
  for (int i = 1; i < rec.w; ++i) s += __ldcg(p.part + 2 * (c + i * p.abreast) * kKeys + threadIdx.x);
  if (key >= __ldg(p.c.seqlens + rec.x)) return;
  float* out = p.weights + (static_cast<long long>(rec.x) * p.c.hkv + rec.y) * p.len + key;
  *out = (p.decay != 0.0f ? p.decay * *out : 0.0f) + s;
}

template <int D, int NT, bool BF16, bool CAUSAL>
cudaError_t launch(const Params& p, int grid, cudaStream_t stream) {
  constexpr int smem = WCfg<D, NT>::kSmem;
  static bool attr_done[64] = {};   // per instantiation
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_done[dev]) {
    e = cudaFuncSetAttribute(weights_kernel<D, NT, BF16, CAUSAL>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_done[dev] = true;
  }
  weights_kernel<D, NT, BF16, CAUSAL><<<grid, WCfg<D, NT>::kThr, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launch();
  if (!p.cuts) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kKeys);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, weights_merge_kernel, p);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <int D, int NT>
cudaError_t pick(const Params& p, bool bf16, bool causal, int grid, cudaStream_t stream) {
  if (bf16) return causal ? launch<D, NT, true, true>(p, grid, stream) : launch<D, NT, true, false>(p, grid, stream);
  return causal ? launch<D, NT, false, true>(p, grid, stream) : launch<D, NT, false, false>(p, grid, stream);
}

size_t rec_bytes(int sms) { return (static_cast<size_t>(sms) * sizeof(int4) + 255) / 256 * 256; }

}  // namespace pwts

long long paged_weights_workspace(int sms) {
  return static_cast<long long>(pwts::rec_bytes(sms) + static_cast<size_t>(2 * sms) * pwts::kKeys * sizeof(float));
}

int paged_weights(const void* q, const float* lse, float* weights, int weights_len, int B, int Hq, int total,
                  const PagedKV& c, int d, bool bf16, int page_size, const int* cu, bool causal, float scale,
                  float decay, void* ws, int sms, int* err, cudaStream_t stream) {
  pwts::Params p;
  p.c = c;
  p.group = Hq / c.hkv;
  // few rows per sequence: tiles of 16 columns
  const bool few = static_cast<long long>(total) * p.group <= 16LL * B;
  const int nt = few ? 16 : 128;
  // equal parts of a group, so that every row of a tile is a query head of it
  for (p.heads = p.group < nt ? p.group : nt; p.group % p.heads != 0;) --p.heads;
  p.parts = p.group / p.heads;
  p.span = nt / p.heads;
  p.span_inv = ~0ull / p.span + 1;   // (span = 1: not used)
  // with no rows at all nothing is loaded through the map
  const int rows = total > 0 ? total : 1;
  if (int rc = tile_map(q, bf16, d, Hq, rows, 1, d, static_cast<long long>(Hq) * d,
                        static_cast<long long>(rows) * Hq * d, p.heads, p.span, p.tm_q))
    return rc;
  const int box = page_size < 128 ? page_size : 128;
  if (int rc = tile_map(c.k, bf16, d, c.hkv, page_size, c.num_pages, c.s_head, c.s_token, c.s_page, 1, box, p.tm_k)) return rc;
  char* w = static_cast<char*>(ws);
  p.rec = reinterpret_cast<int4*>(w);
  p.part = reinterpret_cast<float*>(w + pwts::rec_bytes(sms));
  p.lse = lse;
  p.weights = weights;
  p.cu = cu;
  p.err = err;
  p.timeout_ns = wait_timeout_ns();
  p.B = B;
  p.Hq = Hq;
  p.total = total;
  p.len = weights_len;
  p.abreast = heads_abreast(c.hkv, sms);
  p.cuts = static_cast<long long>((total + p.span - 1) / p.span) * p.parts > pwts::kMinTiles;
  p.products = scale > 0.0f;
  p.inv_scale = scale > 0.0f ? 1.0f / scale : 1.0f;
  p.scale_log2 = (scale > 0.0f ? scale : 1.0f) * pwts::kLog2e;
  p.decay = decay;
  cudaError_t e;
  if (d == 64) e = few ? pwts::pick<64, 16>(p, bf16, causal, sms, stream) : pwts::pick<64, 128>(p, bf16, causal, sms, stream);
  else e = few ? pwts::pick<128, 16>(p, bf16, causal, sms, stream) : pwts::pick<128, 128>(p, bf16, causal, sms, stream);
  return e == cudaSuccess ? ATTN_OK : ATTN_ELAUNCH;
}

}  // namespace attn
