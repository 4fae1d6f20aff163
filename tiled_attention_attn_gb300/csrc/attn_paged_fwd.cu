// Attention of a chunk of new tokens over a paged cache (attn_fwd_paged).
//
// The tile work is the packed forward's: two query sub-tiles of 128 rows per
// CTA, S = Q K^T and u += P V on tcgen05 with S, P and u in TMEM, one softmax
// thread per row with the running maximum m and sum l (softmax_tile), K and V
// through one ring of TMA stages.  A row is a (token, query head) pair: the
// heads of a key/value head share a tile, so that a key tile is read once for
// all of them: 128 / heads tokens x heads rows (any group; rows left over are
// zero queries).  P is rounded to the 16-bit type for the second product,
// whose operands tcgen05.mma takes in one type (half a step of each weight; the
// rest of the rounding as a third product would cost half as many MMAs again;
// kLift); everything else is fp32.
//
// Pages: a 128-key tile is 128 / min(page_size, 128) boxes of 64 features for
// K and as many for V; each lane of the producer warp loads one box at the page
// that it read from the table a tile ahead.  Slots past the last key may hold
// anything: their scores are dropped by index and their V rows zeroed in shared
// memory by the softmax threads (0 * NaN would be NaN).
//
// Work: the units (sequence, head group, block of 256 rows) with their key
// tiles (up to the causal limit) form a line of tiles, cut into equal ranges,
// one per CTA, wherever the cuts fall.  The lengths are on the device, so the
// cuts are computed there, from a closed form of the tiles before a block.  A
// unit that reaches over a cut leaves fp32 partials, at most two per CTA,
// which fwd_merge_kernel joins.  Few rows over a long cache are thus spread
// over every SM, and ragged batches end together.
//
// Bound by the tensor cores (4 d FLOPs a pair) for chunks of hundreds of
// tokens, by HBM for a few tokens.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_kernel.cuh"
#include "attn_paged.h"
#include "attn_paged_line.cuh"
#include "attn_paged_launch.h"

namespace attn {
namespace pfwd {

constexpr int kUnitCost = 2;   // a unit's fixed cost (Q, first S, epilogue) in tiles
constexpr int kMinTiles = 6;   // pieces of a cut unit are at least about this long

struct Params {
  CUtensorMap tm_q;    // q (total, Hq, d) as (d, Hq, total, 1), box 64 x heads x span x 1
  CUtensorMap tm_k;    // (d, Hkv, page_size, num_pages), box 64 x 1 x min(page_size, 128) x 1
  CUtensorMap tm_v;
  PagedKV c;
  void* o;
  float* lse;          // (Hq, total)
  const int* cu;
  int4* rec;           // per CTA: the unit whose first piece it ran (sequence, group, block, pieces)
  float* part_ml;      // (m, l) [2 CTAs][2][128] float2
  float4* part_o;      // u / l  [2 CTAs][2][d / 4][128]
  int* err;
  unsigned long long timeout_ns;
  int B, Hq, total, group;
  int heads, parts;    // query heads per unit, units per key/value head
  int span;            // tokens per sub-tile
  int cuts;            // the table can hold a unit long enough to be cut
  float scale_log2;
};

// The CTA's walk over units.
struct Walk {
  int b, hc, mb;
  int q_len, k_len, row_q, n_mb;   // sequence
  long long p, begin, end;         // unit start on the line; this CTA's range
  int n, t0, t1;                   // key tiles of the unit; this CTA's part
};

template <bool CAUSAL>
struct Line {
  const Params& p;
  __device__ int tok() const { return 2 * p.span; }
  __device__ int units_per_block() const { return p.c.hkv * p.parts; }
  // key tiles of block mb
  __device__ int tiles(const Walk& w, int mb) const {
    const long long e = CAUSAL ? static_cast<long long>(w.k_len) - w.q_len + min((mb + 1) * tok(), w.q_len) : w.k_len;
    return e <= 0 ? 0 : static_cast<int>((e + kBN - 1) / kBN);
  }
  // cost of the blocks before mb (of one head group)
  __device__ long long before(const Walk& w, int mb) const {
    long long sum = static_cast<long long>(kUnitCost) * mb;
    if (mb <= 0) return 0;
    const long long last = (w.k_len + kBN - 1) / kBN;
    if (!CAUSAL) return sum + last * mb;
    if (mb <= 32) {   // short chunks: one by one, without the closed form's divisions
      for (int i = 0; i < mb; ++i) sum += tiles(w, i);
      return sum;
    }
    // whole blocks: ceil((off + (i + 1) tok) / kBN), from the first that sees a key
    const int whole = min(mb, w.n_mb - 1);
    const int off = w.k_len - w.q_len, step = tok();
    const int i0 = off + step > 0 ? 0 : (-off) / step;   // off + (i0 + 1) step > 0
    if (whole > i0) sum += floor_sum(whole - i0, kBN, step, off + (i0 + 1) * step + kBN - 1);
    if (mb == w.n_mb) sum += last;
    return sum;
  }
  __device__ void load(Walk& w) const {
    chunk_and_keys(p.c, p.cu, w.b, p.total, w.q_len, w.row_q, w.k_len, p.err);
    w.n_mb = (w.q_len + tok() - 1) / tok();
  }
  __device__ long long cost(const Walk& w) const { return before(w, w.n_mb) * units_per_block(); }
  __device__ int units(const Walk& w) const {
    return static_cast<int>(min(static_cast<long long>(w.n_mb) * units_per_block(), 1LL << 24));
  }
  __device__ void advance(Walk& w) const {
    w.p += w.n + kUnitCost;
    if (++w.mb == w.n_mb) {
      w.mb = 0;
      if (++w.hc == units_per_block()) {
        w.hc = 0;
        while (++w.b < p.B) {
          load(w);
          if (w.n_mb > 0) break;
        }
      }
    }
    if (w.b < p.B) w.n = tiles(w, w.mb);
  }
  // the next unit that has something to do here; false at the range's end
  __device__ bool next(Walk& w, bool first) const {
    if (!first) advance(w);
    while (w.b < p.B && w.p < w.end) {
      if (part_of<kMinTiles>(w.p, w.n, w.begin, w.end, w.t0, w.t1)) return true;
      advance(w);
    }
    return false;
  }
};

template <int D>
struct PCfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kTile = kBM * D * 2;
  // ring of key/value stages: stage use i of a piece holds K tile t0 + i and V
  // tile t0 + i - 1 (the first K only, the last V only)
  static constexpr int kNS = (D == 128) ? 2 : 4;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kNSub * kTile;
  static constexpr int kOffV = kOffK + kNS * kTile;
  static constexpr int kOffBar = kOffV + kNS * kTile;
  static constexpr int kNBars = 2 + 2 * kNS + 7;
  static constexpr int kOffMisc = kOffBar + (kNBars + 1) / 2 * 16;
  static constexpr int kSmem = kOffMisc + 256 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

// softmax_tile of a tile some of whose keys are hidden (diagonal and ragged
// tiles): keys past `lim` are dropped by index.  The scores are read from TMEM
// twice, 32 columns at a time in rolled loops, instead of held in 128
// registers: an eighth of the code, which a short call fetches cold, for one more
// read of the tile (8 chunks of 512 tokens over their own keys, four query heads a
// key/value head: 37.2 us against 41.1 with the 128-register form).
template <bool BF16, int D>
__device__ __forceinline__ void softmax_masked(uint32_t t_s, uint32_t t_o, int lim, float c_log2, RowState& st, bool first) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int c0 = 0; c0 < kBN; c0 += 32) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(t_s + c0, r);
    tmem_wait_ld(r);
#pragma unroll
    for (int i = 0; i < 32; ++i) mx = fmaxf(mx, c0 + i <= lim ? __uint_as_float(r[i]) : -INFINITY);
  }
  const float m_tile = (mx == -INFINITY) ? -INFINITY : mx * c_log2, m_old = st.m;
  const bool resc = m_tile > m_old && (first || m_old == -INFINITY || m_tile - m_old > 8.0f);
  if (resc) st.m = m_tile;
  const float moff = (st.m == -INFINITY) ? 0.0f : st.m - kLift<BF16>;
  float sum = 0.0f;
  // P of columns c0 .. c0 + 31 goes to words c0 / 2 .., below the scores still to be read
#pragma unroll 1
  for (int c0 = 0; c0 < kBN; c0 += 32) {
    uint32_t r[32], pk[16];
    tmem_ld_32x32b_x32(t_s + c0, r);
    tmem_wait_ld(r);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float a = c0 + 2 * i <= lim ? ex2_approx(__uint_as_float(r[2 * i]) * c_log2 - moff) : 0.0f;
      const float b = c0 + 2 * i + 1 <= lim ? ex2_approx(__uint_as_float(r[2 * i + 1]) * c_log2 - moff) : 0.0f;
      sum += a + b;
      pk[i] = pack2<BF16>(a, b);
    }
    tmem_st_32x32b_x16(t_s + c0 / 2, pk);
  }
  const float r = resc ? ((m_old == -INFINITY) ? 0.0f : ex2_approx(m_old - st.m)) : 1.0f;
  st.l = st.l * r + sum;
  if (!first && __any_sync(0xffffffffu, resc)) {
#pragma unroll 1
    for (int c = 0; c < D / 16; ++c) {
      uint32_t o[16];
      tmem_ld_32x32b_x16(t_o + c * 16, o);
      tmem_wait_ld(o);
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * r);
      tmem_st_32x32b_x16(t_o + c * 16, o);
    }
  }
  tmem_wait_st();
}

template <int D, bool BF16, bool CAUSAL>
__global__ void __launch_bounds__(kThreads, 1) fwd_kernel(const __grid_constant__ Params p) {
  using C = PCfg<D>;
  using T = typename IO<BF16>::T;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + C::kOffQ, sK = sbase + C::kOffK, sV = sbase + C::kOffV;
  const uint32_t bar0 = sbase + C::kOffBar;
  const uint32_t b_q_full = bar0, b_q_empty = bar0 + 8;
  auto b_kv_full = [&](int s) { return bar0 + 16 + 8 * s; };
  auto b_kv_empty = [&](int s) { return bar0 + 16 + 8 * (C::kNS + s); };
  const uint32_t bar_sp = bar0 + 16 + 16 * C::kNS;
  auto b_s_full = [&](int t) { return bar_sp + 8 * t; };
  auto b_p_full = [&](int t) { return bar_sp + 16 + 8 * t; };
  auto b_o_done = [&](int t) { return bar_sp + 32 + 8 * t; };
  const uint32_t b_drain = bar_sp + 48;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  volatile int* start = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);   // b, hc, mb
  volatile long long* start_p = reinterpret_cast<volatile long long*>(smem + C::kOffMisc + 24);
  long long* warp_sums = reinterpret_cast<long long*>(smem + C::kOffMisc + 32);
  WaitCtl wc{p.err, abort_flag, p.timeout_ns};

  if (tid == 0) {
    *abort_flag = 0;
    start[0] = p.B;
    mbar_init(b_q_full, 1);
    mbar_init(b_q_empty, 1);
    for (int s = 0; s < C::kNS; ++s) {
      mbar_init(b_kv_full(s), 1);
      mbar_init(b_kv_empty(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(b_s_full(t), 1);
      mbar_init(b_p_full(t), kBM / 32);   // one arrival per softmax warp
      mbar_init(b_o_done(t), 1);
    }
    mbar_init(b_drain, 1);
    fence_mbar_init();
  }
  if (warp == kWarpTMA && lane == 0) {
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  if (warp == kWarpMMA) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (p.heads * p.span < kBM) {
    // rows past the box: zero queries
    for (int i = tid; i < kNSub * C::kTile / 16; i += kThreads)
      reinterpret_cast<uint4*>(smem + C::kOffQ)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }

  // the line: each thread a strip of sequences, then a prefix sum
  const Line<CAUSAL> line{p};
  Walk w0;
  const int strip = (p.B + kThreads - 1) / kThreads;
  const int b_lo = min(tid * strip, p.B), b_hi = min(b_lo + strip, p.B);
  long long mine = 0, total, units;
  int count = 0;
  for (w0.b = b_lo; w0.b < b_hi; ++w0.b) {
    line.load(w0);
    mine += line.cost(w0);
    count = min(count + line.units(w0), 1 << 24);   // (for a mean: the largest need not be exact)
  }
  const long long before = block_prefix<kThreads>(mine, count, warp_sums, total, units);
  const long long range = range_of<kMinTiles>(total, units, gridDim.x);
  const long long begin = blockIdx.x * range, end = min(begin + range, total);
  if (begin >= before && begin < before + mine) {
    long long at = before;
    for (w0.b = b_lo; w0.b < b_hi; ++w0.b) {
      if (strip > 1) line.load(w0);   // else still there
      const long long cost = strip > 1 ? line.cost(w0) : mine;
      if (begin < at + cost) {
        const long long per = line.before(w0, w0.n_mb);
        const int hc = static_cast<int>((begin - at) / per);
        at += hc * per;
        int lo = 0, hi = w0.n_mb;   // the last block that starts at or before `begin`
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (at + line.before(w0, mid) <= begin) lo = mid; else hi = mid;
        }
        start[0] = w0.b;
        start[1] = hc;
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
  w0.hc = w0.mb = w0.n = w0.n_mb = 0;
  if (w0.b < p.B) {
    w0.hc = start[1];
    w0.mb = start[2];
    w0.p = *start_p;
    line.load(w0);
    w0.n = line.tiles(w0, w0.mb);
  }
  auto last_tile = [&](const Walk& w, int t) {
    return kv_last_tile(w.mb * line.tok(), t, w.q_len, w.k_len, CAUSAL, p.span);
  };

  if (warp == kWarpTMA) {
    // ------------------------------------------------------------------ TMA producer
    uint32_t q_cnt = 0, kv_cnt = 0;
    const int box = min(1 << p.c.page_log2, kBN);   // tokens per box
    const int n_pg = kBN / box;
    // this lane's box: page `pg` of a tile, feature chunk `ch`, of K or V
    const int pg = lane % n_pg, ch = (lane / n_pg) % C::kChunks;
    const bool of_v = lane >= C::kChunks * n_pg, has = lane < 2 * C::kChunks * n_pg;
    const CUtensorMap* map = of_v ? &p.tm_v : &p.tm_k;
    const uint32_t dst0 = (of_v ? sV : sK) + ch * 16384 + pg * box * 128;
    const int lag = of_v ? 1 : 0;   // V runs one stage use behind K
    Walk w = w0;
    bool ok = true;
    for (bool more = line.next(w, true); more && ok; more = line.next(w, false)) {
      if (w.t1 <= w.t0) continue;
      const int n = w.t1 - w.t0;
      // the page of this lane's box in stage use i, -1: none to load
      auto page_at = [&](int i) {
        const int t = i - lag, key = (w.t0 + t) * kBN + pg * box;
        if (!has || t < 0 || t >= n || key >= w.k_len) return -1;
        const int id = paged_page(p.c, w.b, key >> p.c.page_log2, p.err);
        return id < 0 ? p.c.num_pages : id;   // no page: rows past the pool read as zeros
      };
      if (!mbar_wait_warp(b_q_empty, (q_cnt & 1) ^ 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteQEmpty))) break;
      const int g = w.hc / p.parts, head0 = g * p.group + (w.hc - g * p.parts) * p.heads;
      if (lane == 0) {
        mbar_arrive_expect_tx(b_q_full, kNSub * C::kChunks * p.heads * p.span * 128);
        for (int t = 0; t < kNSub; ++t)
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_4d(sQ + t * C::kTile + c * 16384, &p.tm_q, b_q_full, c * 64, head0,
                        w.row_q + w.mb * line.tok() + t * p.span, 0);
      }
      ++q_cnt;
      int page = page_at(0);
      for (int i = 0; i <= n; ++i) {
        const int st = kv_cnt % C::kNS;
        const int next = page_at(i + 1);
        if (!mbar_wait_warp(b_kv_empty(st), ((kv_cnt / C::kNS) & 1) ^ 1, wc,
                            ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteKEmpty))) { ok = false; break; }
        const uint32_t n_box = __popc(__ballot_sync(0xffffffffu, page >= 0));
        if (lane == 0) mbar_arrive_expect_tx(b_kv_full(st), n_box * box * 128);
        __syncwarp();
        if (page >= 0)
          tma_load_4d(dst0 + st * C::kTile, map, b_kv_full(st), ch * 64, g,
                      ((w.t0 + i - lag) * kBN + pg * box) & ((1 << p.c.page_log2) - 1), page);
        page = next;
        ++kv_cnt;
      }
    }
    if (lane == 0 && *abort_flag) {
      // let the loads already issued land before the CTA exits
      for (int s = 0; s < C::kNS; ++s) {
        const uint32_t n = (kv_cnt + C::kNS - 1 - s) / C::kNS;
        if (n > 0) mbar_wait(b_kv_full(s), (n - 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteDrain), false);
      }
      if (q_cnt > 0) mbar_wait(b_q_full, (q_cnt - 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteDrain), false);
    }
  } else if (warp == kWarpMMA) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t kIdescO = idesc_f16_f32acc(kBM, D, BF16, true);
      constexpr uint32_t kIdescS = idesc_f16_f32acc(kBM, kBN, BF16, false);
      const uint64_t dq0 = sdesc_sw128(sQ, 16, 1024);
      const uint64_t dk0 = sdesc_sw128(sK, 16, 1024);
      const uint64_t dv0 = sdesc_sw128(sV, 16384, 1024);
      uint32_t q_cnt = 0, kv_cnt = 0;
      uint32_t p_cnt0 = 0, p_cnt1 = 0;
      auto issue_s = [&](int t, int st) {
        const uint64_t a0 = dq0 + ((t * C::kTile) >> 4);
        const uint64_t b0 = dk0 + ((st * C::kTile) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
          umma_ss(tmem + t * 128, a0 + off, b0 + off, kIdescS, kk > 0 ? 1u : 0u);
        }
        umma_commit(b_s_full(t));
      };
      bool ok = true;
      Walk w = w0;
      for (bool more = line.next(w, true); more && ok; more = line.next(w, false)) {
        if (w.t1 <= w.t0) continue;
        const int last[2] = {last_tile(w, 0), last_tile(w, 1)};
        if (!mbar_wait(b_q_full, q_cnt & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteQFull))) break;
        bool first_pv0 = true, first_pv1 = true;
        {
          // first stage use: K of the first tile, S for it
          const int st = kv_cnt % C::kNS;
          if (!mbar_wait(b_kv_full(st), (kv_cnt / C::kNS) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteKFull))) break;
#pragma unroll
          for (int t = 0; t < kNSub; ++t)
            if (w.t0 <= last[t]) issue_s(t, st);
          umma_commit(b_kv_empty(st));
          ++kv_cnt;
        }
        // Per tile j: u_t += P_t(j) V(j), then S_t(j + 1), for t = 0, 1: the
        // commit that signals S_t(j + 1) also covers P_t(j) V(j)
        for (int j = w.t0; j < w.t1; ++j) {
          const int st = kv_cnt % C::kNS;
          if (!mbar_wait(b_kv_full(st), (kv_cnt / C::kNS) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteVFull))) {
            ok = false;
            break;
          }
          const bool have_next = j + 1 < w.t1;
#pragma unroll
          for (int t = 0; t < kNSub; ++t) {
            uint32_t& p_cnt = (t == 0) ? p_cnt0 : p_cnt1;
            bool& first_pv = (t == 0) ? first_pv0 : first_pv1;
            const bool next_s = have_next && j + 1 <= last[t];
            if (j <= last[t]) {
              if (!mbar_wait(b_p_full(t), p_cnt & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSitePFull))) {
                ok = false;
                break;
              }
              ++p_cnt;
              tc_fence_after();   // the softmax threads' P (tcgen05.st) before the MMA that reads it
              const uint64_t bv = dv0 + ((st * C::kTile) >> 4);
#pragma unroll
              for (int kk = 0; kk < kBN / 16; ++kk)
                umma_ts(tmem + 256 + t * 128, tmem + t * 128 + kk * 8, bv + ((kk * 2048) >> 4), kIdescO,
                        (first_pv && kk == 0) ? 0u : 1u);
              if (!next_s) umma_commit(b_o_done(t));
              first_pv = false;
            }
            if (next_s) issue_s(t, st);
          }
          if (!ok) break;
          umma_commit(b_kv_empty(st));
          ++kv_cnt;
        }
        if (!ok) break;
        umma_commit(b_q_empty);
        ++q_cnt;
      }
      umma_commit(b_drain);
      mbar_wait(b_drain, 0, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteDrain), false);
    }
  } else {
    // ------------------------------------------------------------------ softmax warpgroups
    const int t = warp >> 2;                 // query sub-tile
    const int quarter = warp & 3;            // TMEM lane quarter of this warp
    const int row = quarter * 32 + lane;     // row within the sub-tile
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lane_off + t * 128;
    const uint32_t t_o = tmem + lane_off + 256 + t * 128;
    const float c_log2 = p.scale_log2;
    uint32_t s_cnt = 0, o_cnt = 0, kv_cnt = 0;
    T* out = reinterpret_cast<T*>(p.o);
    const int r_tok = row / p.heads, r_head = row - r_tok * p.heads;   // this row's token and head in the tile
    Walk w = w0;
    for (bool more = line.next(w, true); more; more = line.next(w, false)) {
      const int q_first = w.mb * line.tok() + t * p.span;   // first token of the sub-tile
      const int qrow = q_first + r_tok;
      const int g = w.hc / p.parts, part = w.hc - g * p.parts;
      const int head0 = g * p.group + part * p.heads;
      const int n_heads = min(p.heads, p.group - part * p.heads);
      const bool row_valid = r_tok < p.span && r_head < n_heads && qrow < w.q_len;
      int lim_key = w.k_len - 1;   // allowed keys of this row: key <= lim_key
      if (CAUSAL) lim_key = min(lim_key, qrow + (w.k_len - w.q_len));
      const int last = last_tile(w, t);
      RowState st{-INFINITY, 0.0f};
      int n_act = 0;
      bool ok = true;
      for (int j = w.t0; j < w.t1; ++j) {
        if (j > last) break;
        if (!mbar_wait_warp(b_s_full(t), s_cnt & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteSFull))) { ok = false; break; }
        ++s_cnt;
        tc_fence_after();
        const int lim = lim_key - j * kBN;
        const bool ragged = j * kBN + kBN > w.k_len;
        if (ragged || (CAUSAL && j * kBN + kBN - 1 > q_first + (w.k_len - w.q_len))) {
          if (ragged) {
            // rows of V past the last key become zero, once the tile has landed
            const uint32_t use = kv_cnt + (j - w.t0) + 1;
            const int vs = use % C::kNS;
            if (!mbar_wait_warp(b_kv_full(vs), (use / C::kNS) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteVFull))) {
              ok = false;
              break;
            }
            if (j * kBN + row >= w.k_len) {
#pragma unroll
              for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  reinterpret_cast<uint4*>(smem + C::kOffV + vs * C::kTile + c * 16384 + row * 128)[i] =
                      make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
          softmax_masked<BF16, D>(t_s, t_o, lim, c_log2, st, n_act == 0);
        } else {
          softmax_tile<false, BF16, D, kLift<BF16>>(t_s, t_o, lim, c_log2, st, n_act == 0);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_p_full(t));
        ++n_act;
      }
      if (!ok) break;
      if (w.t1 > w.t0) kv_cnt += w.t1 - w.t0 + 1;
      if (n_act > 0) {
        if (!mbar_wait_warp(b_o_done(t), o_cnt & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteODone))) break;
        ++o_cnt;
        tc_fence_after();
      }
      const bool whole = w.t1 - w.t0 == w.n;
      const float inv_l = (st.l != 0.0f) ? 1.0f / st.l : 0.0f;   // 0: saw no key; a NaN stays one
      if (whole) {
        // O = u / l, lse = m / log2(e) + ln l
        T* dst = out + (static_cast<size_t>(w.row_q + qrow) * p.Hq + head0 + r_head) * D;
        const bool v8 = (reinterpret_cast<uintptr_t>(p.o) & 31) == 0;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (n_act > 0) {
            tmem_ld_32x32b_x32(t_o + c * 32, o);
            tmem_wait_ld(o);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            pk[i] = pack2<BF16>(__uint_as_float(o[2 * i]) * inv_l, __uint_as_float(o[2 * i + 1]) * inv_l);
          if (row_valid && v8) {
            st_global_v8(dst + c * 32, pk);
            st_global_v8(dst + c * 32 + 16, pk + 8);
          } else if (row_valid) {
            uint4* d4 = reinterpret_cast<uint4*>(dst + c * 32);
#pragma unroll
            for (int i = 0; i < 4; ++i) d4[i] = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
          }
        }
        if (row_valid)
          p.lse[static_cast<size_t>(head0 + r_head) * p.total + w.row_q + qrow] =
              (st.l != 0.0f) ? st.m * 0.69314718055994531f + __logf(st.l * kDrop<BF16>) : -INFINITY;
      } else {
        // a piece: O_s = u_s / l_s and (m, l) in fp32; a warp's 32 rows of one
        // 4-column group are 512 contiguous bytes
        const size_t slot = static_cast<size_t>(2 * blockIdx.x + (w.t0 == 0 ? 1 : 0)) * kNSub + t;
        if (n_act > 0) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(t_o + c * 32, o);
            tmem_wait_ld(o);
            if (row_valid) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                p.part_o[(slot * (D / 4) + c * 8 + i) * kBM + row] =
                    make_float4(__uint_as_float(o[4 * i]) * inv_l, __uint_as_float(o[4 * i + 1]) * inv_l,
                                __uint_as_float(o[4 * i + 2]) * inv_l, __uint_as_float(o[4 * i + 3]) * inv_l);
            }
          }
        }
        if (row_valid)
          reinterpret_cast<float2*>(p.part_ml)[slot * kBM + row] = make_float2(st.m, st.l * kDrop<BF16>);
        // the unit's pieces lie on CTAs p / range ... (p + n - 1) / range
        if (w.t0 == 0 && warp == 0 && lane == 0)
          p.rec[blockIdx.x] = make_int4(w.b, w.hc, w.mb,
                                        static_cast<int>((w.p + w.n - 1) / range) - static_cast<int>(blockIdx.x) + 1);
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMMA) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of the unit that block x's CTA began: M = max m_s, w_s =
// 2^(m_s - M) l_s, O = sum w_s O_s / sum w_s.  Block (CTA, sub-tile, 32
// columns), one thread per row and 16 columns, two pieces (the usual count) in
// flight; a programmatic dependent of the forward.
template <int D, bool BF16>
__global__ void __launch_bounds__(2 * kBM, 4) fwd_merge_kernel(const __grid_constant__ Params p) {
  using T = typename IO<BF16>::T;
  const int c0 = blockIdx.x, t = blockIdx.y, cb = blockIdx.z * 2 + threadIdx.x / kBM, row = threadIdx.x % kBM;
  grid_wait_prerequisites();
  const int4 rec = __ldcg(p.rec + c0);
  const int pieces = rec.w;
  if (pieces <= 1) return;
  int row_q;
  const int q_len = chunk_len(p.cu, rec.x, p.total, row_q, p.err);
  const int r_tok = row / p.heads, r_head = row - r_tok * p.heads;
  const int qrow = (2 * rec.z + t) * p.span + r_tok;
  const int g = rec.y / p.parts, part = rec.y - g * p.parts;
  if (r_tok >= p.span || qrow >= q_len || r_head >= p.group - part * p.heads) return;
  // piece s of this row: the first on the CTA's slot for a unit that goes on,
  // the others on the next CTAs' slots for one that came
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + row;
  auto slot = [&](int s) { return static_cast<size_t>(s == 0 ? 2 * c0 + 1 : 2 * (c0 + s)) * kNSub + t; };
  float M = -INFINITY;
#pragma unroll 4
  for (int s = 0; s < pieces; ++s) M = fmaxf(M, __ldcg(ml + slot(s) * kBM).x);
  float L = 0.0f, acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
  for (int s0 = 0; s0 < pieces; s0 += 2) {
    float2 mlv[2];
    float4 x[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool in = s0 + i < pieces;
      const size_t sl = slot(in ? s0 + i : 0);
      mlv[i] = in ? __ldcg(ml + sl * kBM) : make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        x[i][c] = in ? __ldcg(p.part_o + (sl * (D / 4) + cb * 4 + c) * kBM + row) : make_float4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (mlv[i].y == 0.0f) continue;   // a piece that saw no key (its O_s was never written)
      const float wt = ex2_approx(mlv[i].x - M) * mlv[i].y;   // (l of NaN: NaN, whatever m)
      L += wt;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[4 * c] += wt * x[i][c].x;
        acc[4 * c + 1] += wt * x[i][c].y;
        acc[4 * c + 2] += wt * x[i][c].z;
        acc[4 * c + 3] += wt * x[i][c].w;
      }
    }
  }
  const float inv = (L != 0.0f) ? 1.0f / L : 0.0f;
  const int head = g * p.group + part * p.heads + r_head;
  uint4* d4 = reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.o) +
                                       (static_cast<size_t>(row_q + qrow) * p.Hq + head) * D + cb * 16);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    d4[i] = make_uint4(pack2<BF16>(acc[8 * i] * inv, acc[8 * i + 1] * inv),
                       pack2<BF16>(acc[8 * i + 2] * inv, acc[8 * i + 3] * inv),
                       pack2<BF16>(acc[8 * i + 4] * inv, acc[8 * i + 5] * inv),
                       pack2<BF16>(acc[8 * i + 6] * inv, acc[8 * i + 7] * inv));
  if (cb == 0)
    p.lse[static_cast<size_t>(head) * p.total + row_q + qrow] =
        (L != 0.0f) ? M * 0.69314718055994531f + __logf(L) : -INFINITY;
}

template <int D, bool BF16, bool CAUSAL>
cudaError_t launch(const Params& p, int grid, cudaStream_t stream) {
  constexpr int smem = PCfg<D>::kSmem;
  static bool attr_done[64] = {};   // per instantiation
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_done[dev]) {
    e = cudaFuncSetAttribute(fwd_kernel<D, BF16, CAUSAL>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_done[dev] = true;
  }
  fwd_kernel<D, BF16, CAUSAL><<<grid, kThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launch();
  if (!p.cuts) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, kNSub, D / 32);
  cfg.blockDim = dim3(2 * kBM);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, fwd_merge_kernel<D, BF16>, p);
  if (e == cudaSuccess) count_launch();
  return e;
}

size_t rec_bytes(int sms) { return (static_cast<size_t>(sms) * sizeof(int4) + 255) / 256 * 256; }
size_t ml_bytes(int sms) { return static_cast<size_t>(2 * sms) * kNSub * kBM * sizeof(float2); }

}  // namespace pfwd

long long paged_fwd_workspace(int sms, int d) {
  return static_cast<long long>(pfwd::rec_bytes(sms) + pfwd::ml_bytes(sms) +
                                static_cast<size_t>(2 * sms) * kNSub * kBM * d * sizeof(float));
}

int paged_fwd(const void* q, void* o, float* lse, int B, int Hq, int total, const PagedKV& c, int d, bool bf16,
              int page_size, const int* cu, bool causal, float scale, void* ws, int sms, int* err, cudaStream_t stream) {
  pfwd::Params p;
  p.c = c;
  p.group = Hq / c.hkv;
  // a tile holds up to 128 query heads of a key/value head
  p.parts = (p.group + kBM - 1) / kBM;
  p.heads = (p.group + p.parts - 1) / p.parts;
  p.parts = (p.group + p.heads - 1) / p.heads;
  p.span = kBM / p.heads;
  if (int rc = tile_map(q, bf16, d, Hq, total, 1, d, static_cast<long long>(Hq) * d,
                        static_cast<long long>(total) * Hq * d, p.heads, p.span, p.tm_q))
    return rc;
  const int box = page_size < kBN ? page_size : kBN;
  if (int rc = tile_map(c.k, bf16, d, c.hkv, page_size, c.num_pages, c.s_head, c.s_token, c.s_page, 1, box, p.tm_k)) return rc;
  if (int rc = tile_map(c.v, bf16, d, c.hkv, page_size, c.num_pages, c.s_head, c.s_token, c.s_page, 1, box, p.tm_v)) return rc;
  char* w = static_cast<char*>(ws);
  p.rec = reinterpret_cast<int4*>(w);
  p.part_ml = reinterpret_cast<float*>(w + pfwd::rec_bytes(sms));
  p.part_o = reinterpret_cast<float4*>(w + pfwd::rec_bytes(sms) + pfwd::ml_bytes(sms));
  p.o = o;
  p.lse = lse;
  p.cu = cu;
  p.err = err;
  p.timeout_ns = wait_timeout_ns();
  p.B = B;
  p.Hq = Hq;
  p.total = total;
  p.cuts = (c.max_pages << c.page_log2) > pfwd::kMinTiles * kBN;
  p.scale_log2 = scale * 1.4426950408889634f;
  cudaError_t e;
  if (d == 64) {
    if (causal) e = bf16 ? pfwd::launch<64, true, true>(p, sms, stream) : pfwd::launch<64, false, true>(p, sms, stream);
    else e = bf16 ? pfwd::launch<64, true, false>(p, sms, stream) : pfwd::launch<64, false, false>(p, sms, stream);
  } else {
    if (causal) e = bf16 ? pfwd::launch<128, true, true>(p, sms, stream) : pfwd::launch<128, false, true>(p, sms, stream);
    else e = bf16 ? pfwd::launch<128, true, false>(p, sms, stream) : pfwd::launch<128, false, false>(p, sms, stream);
  }
  return e == cudaSuccess ? ATTN_OK : ATTN_ELAUNCH;
}

}  // namespace attn
