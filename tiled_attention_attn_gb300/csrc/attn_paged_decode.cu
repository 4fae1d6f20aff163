// One decoding step over a paged cache on tensor cores (attn_decode_paged).
//
// The products are transposed, as in the packed decode kernel: the tile's 128
// keys on the MMA's M dimension, the query heads of a key/value head on N,
//   S^T = K Q^T    (M = 128 keys, N = 16 head columns, K = d)
//   u^T += V^T P^T (M = d, N = 16, K = 128 keys)
// so that each softmax thread owns one key.  The statistics are those of the
// online softmax: running maximum m, sum l and accumulator u, rescaled by
// 2^(m_old - m_new); m may lag by up to 2^8, which cancels in u / l.  P is
// rounded to the cache's 16-bit type for the second product, whose operands
// tcgen05.mma takes in one type (half a step of each weight, as much again as the
// rounding of O; kLift); S, m, l, u and the pieces' partial results are fp32.
//
// Bound by HBM: K and V of every sequence once.  A ring of three stages of 64
// KB (K and V of a step) keeps up to 192 KB per SM in flight.  A page holds at
// least 16 tokens, so a 128-key tile is up to 8 pages; the producer's lanes
// each load one box (64 features x the tokens of a page) of K or V at the page
// that the lane has read from the table, one step ahead.
//
// Work: the steps of all (sequence, head group) units, one after the other (the
// key/value heads side by side, heads_abreast), cut into equal ranges, one per
// CTA, wherever the cut falls (the host does not know the lengths, and ragged
// caches need no other balancing).  A unit that reaches over a cut leaves fp32
// partials, at most two per CTA, which a second launch (decode_merge_kernel)
// joins.
//
// Slots past a sequence's last key may hold anything: their scores are dropped
// by index, and their rows of V are zeroed in shared memory before the product
// (0 * NaN would be NaN).
//
// Head dimension 64: a step covers two tiles, one P.V serves both: V read
// MN-major with M = 128 spans the stage's two chunks (rows 0-63 = d of tile a,
// 64-127 = d of tile b), P^T has 2 x 16 rows, and the product's diagonal
// blocks are u_a and u_b, summed at the unit's end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "attn_paged.h"
#include "attn_paged_line.cuh"
#include "attn_paged_launch.h"
#include "attn_params.h"
#include "ptx.cuh"

namespace attn {
namespace pdec {

constexpr int kThreads = 224;
constexpr int kWarpTMA = 0;    // loads Q and K
constexpr int kWarpMMA = 1;
constexpr int kWarpTMAV = 6;   // loads V
constexpr int kKeys = 128;   // keys per tile
constexpr int kNQ = 16;      // head columns
constexpr int kStages = 3;
constexpr int kMinSteps = 4;   // pieces of a cut unit are at least about this long
constexpr int kTile = kKeys * 128 * 2;   // one stage of K or of V: two 64-column chunks
constexpr int kChunk = kTile / 2;

template <int DA>
struct Cfg {
  static constexpr int kTPS = 128 / DA;           // tiles per step
  static constexpr int kQChunk = kNQ * 128;
  static constexpr int kQ = (DA / 64) * kQChunk;
  static constexpr int kRows = kTPS * kNQ;        // P^T rows of a step (the P.V's N)
  static constexpr int kPChunk = kRows * 128;
  static constexpr int kP = 2 * kPChunk;
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kOffK + kStages * kTile;
  static constexpr int kOffQ = kOffV + kStages * kTile;   // two Q slots
  static constexpr int kOffP = kOffQ + 2 * kQ;            // two P^T buffers
  static constexpr int kOffRed = kOffP + 2 * kP;          // [parity][warp][kNQ] floats
  static constexpr int kOffBar = kOffRed + 2 * 4 * kNQ * 4;
  static constexpr int kNBars = 4 * kStages + 14;
  static constexpr int kOffMisc = kOffBar + kNBars * 8;
  static constexpr int kSmem = kOffMisc + 256 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // S^T: two buffers of kTPS tiles, then u^T (kRows columns)
  static constexpr int kUsedCols = 3 * kTPS * kNQ;
  static constexpr uint32_t kTmemCols = kUsedCols <= 64 ? 64 : 128;
};

struct Params {
  CUtensorMap tm_q;    // q (B, Hq, d) as (d, Hq, B, 1), box 64 x heads x 1 x 1
  CUtensorMap tm_k;    // (d, Hkv, page_size, num_pages), box 64 x 1 x min(page_size, 128) x 1
  CUtensorMap tm_v;
  PagedKV c;
  void* o;             // (B, Hq, d)
  float* lse;          // (Hq, B)
  int4* rec;           // per CTA: the unit whose first piece it ran (sequence, group, pieces, 0)
  float2* part_ml;     // (m, l) [2 CTAs][kNQ]
  float* part_o;       // u / l  [2 CTAs][kNQ][DA]
  int* err;
  unsigned long long timeout_ns;
  int B, Hq, group, heads, parts;   // heads per unit; units per key/value head
  int abreast;         // unit groups that walk the line side by side (heads_abreast)
  int cuts;            // the table can hold a unit long enough to be cut
  float scale_log2;
};

// The CTA's walk over units: (b, hc) in order, unit at position p of the line
// of steps with T steps and one more for its fixed cost.
struct Walk {
  int b, hc;          // hc: group of p.abreast units; this CTA's is hc * abreast + its place
  long long p, end;   // unit start; end of this CTA's range
  long long begin;
  int n, T;           // keys, steps
  int t0, t1;         // this CTA's steps of the unit
};

template <int KS>
__device__ __forceinline__ int steps_of(int n) { return (n + KS - 1) / KS; }

// The next unit that has something to do here; false at the range's end.
template <int KS>
__device__ __forceinline__ bool next_unit(const Params& p, Walk& w, bool first) {
  const int nh = p.c.hkv * p.parts / p.abreast;
  if (!first) {
    w.p += w.T + 1;
    if (++w.hc == nh) {
      w.hc = 0;
      if (++w.b < p.B) {
        w.n = paged_len(p.c, w.b, p.err);
        w.T = steps_of<KS>(w.n);
      }
    }
  }
  while (w.b < p.B && w.p < w.end) {
    if (part_of<kMinSteps>(w.p, w.T, w.begin, w.end, w.t0, w.t1)) return true;
    w.p += w.T + 1;
    if (++w.hc == nh) {
      w.hc = 0;
      if (++w.b < p.B) {
        w.n = paged_len(p.c, w.b, p.err);
        w.T = steps_of<KS>(w.n);
      }
    }
  }
  return false;
}

// Shared-memory byte offset of element (row, col) in a K-major tile of
// 128-byte rows under the 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128(int row, int col) {
  return static_cast<uint32_t>(row * 128 + ((((col >> 3) ^ (row & 7)) << 4) | ((col & 7) << 1)));
}

__device__ __forceinline__ void tld(uint32_t taddr, float (&x)[kNQ]) {
  uint32_t r[16];
  tmem_ld_32x32b_x16(taddr, r);
  tmem_wait_ld(r);
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tst(uint32_t taddr, const float (&x)[kNQ]) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(x[i]);
  tmem_st_32x32b_x16(taddr, r);
}

__host__ __device__ constexpr uint32_t idesc_a_mn(int M, int N, bool bf16) {
  return idesc_f16_f32acc(M, N, bf16, false) | (1u << 15);
}

// GT: head columns whose softmax is computed (p.heads of them are stored).
template <int GT, bool BF16, int DA>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const __grid_constant__ Params p) {
  using C = Cfg<DA>;
  constexpr int kTPS = C::kTPS;
  constexpr int KS = kKeys * kTPS;   // keys per step
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sK = sbase + C::kOffK, sV = sbase + C::kOffV, sQ = sbase + C::kOffQ, sP = sbase + C::kOffP;
  float* red = reinterpret_cast<float*>(smem + C::kOffRed);
  const uint32_t bar0 = sbase + C::kOffBar;
  auto b_k_full = [&](int s) { return bar0 + 8 * s; };
  auto b_v_full = [&](int s) { return bar0 + 8 * (kStages + s); };
  // head dimension 64 frees K's stage as soon as S^T is computed (131,072 keys
  // 50.1 -> 48.3 us); at 128 both are freed together, K running ahead of V
  // costs there (85.3 -> 88.6 us)
  auto b_v_empty = [&](int s) { return bar0 + 8 * (2 * kStages + s); };
  auto b_k_empty = [&](int s) { return DA == 64 ? bar0 + 8 * (3 * kStages + s) : b_v_empty(s); };
  const uint32_t bar1 = bar0 + 8 * 4 * kStages;
  auto b_q_full = [&](int s) { return bar1 + 8 * s; };
  auto b_q_empty = [&](int s) { return bar1 + 8 * (2 + s); };
  auto b_s_full = [&](int s) { return bar1 + 8 * (4 + s); };
  auto b_p_full = [&](int s) { return bar1 + 8 * (6 + s); };
  // p_free(b): the P.V that read P^T buffer b has completed (one phase per use)
  auto b_p_free = [&](int s) { return bar1 + 8 * (8 + s); };
  const uint32_t b_o_free = bar1 + 8 * 10;
  const uint32_t b_red = bar1 + 8 * 11;
  const uint32_t b_drain = bar1 + 8 * 12;
  const uint32_t b_xch = bar1 + 8 * 13;   // u_b handed over (head_dim 64)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  volatile int* start_b = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
  volatile long long* start_p = reinterpret_cast<volatile long long*>(smem + C::kOffMisc + 16);
  long long* warp_sums = reinterpret_cast<long long*>(smem + C::kOffMisc + 32);
  WaitCtl wc{p.err, abort_flag, p.timeout_ns};

  if (tid == 0) {
    *abort_flag = 0;
    *start_b = p.B;
    *start_p = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(b_k_full(s), 1);
      mbar_init(b_v_full(s), 1);
      mbar_init(b_v_empty(s), 1);
      if constexpr (DA == 64) mbar_init(b_k_empty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(b_q_full(s), 1);
      mbar_init(b_q_empty(s), 1);
      mbar_init(b_s_full(s), 1);
      mbar_init(b_p_full(s), 4);   // the four softmax warps
      mbar_init(b_p_free(s), 1);
    }
    mbar_init(b_o_free, 4);
    mbar_init(b_red, 4);
    mbar_init(b_drain, 1);
    mbar_init(b_xch, 2);
    fence_mbar_init();
  }
  if (warp == kWarpMMA) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == kWarpTMA && lane == 0) {
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  // head columns past p.heads: zero queries (their results are not stored)
  for (int i = tid; i < 2 * C::kQ / 16; i += kThreads)
    reinterpret_cast<uint4*>(smem + C::kOffQ)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();

  // the line of steps: each thread a strip of sequences, then a prefix sum
  const int nh = p.c.hkv * p.parts / p.abreast;
  const int place = blockIdx.x % p.abreast, ranges = gridDim.x / p.abreast, range_id = blockIdx.x / p.abreast;
  const int strip = (p.B + kThreads - 1) / kThreads;
  const int b_lo = min(tid * strip, p.B), b_hi = min(b_lo + strip, p.B);
  long long mine = 0, total, units;
  for (int b = b_lo; b < b_hi; ++b) mine += static_cast<long long>(nh) * (steps_of<KS>(paged_len(p.c, b, p.err)) + 1);
  const long long before = block_prefix<kThreads>(
      mine, static_cast<int>(min(static_cast<long long>(nh) * (b_hi - b_lo), 1LL << 24)), warp_sums, total, units);
  const long long range = range_of<kMinSteps>(total, units, ranges);
  // (SMs past the last whole range idle)
  const long long begin = range_id < ranges ? range_id * range : total, end = min(begin + range, total);
  if (begin >= before && begin < before + mine) {
    long long at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      const long long cost = static_cast<long long>(nh) * (steps_of<KS>(paged_len(p.c, b, p.err)) + 1);
      if (begin < at + cost) {
        *start_b = b;
        *start_p = at;
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
  Walk w0;
  w0.b = *start_b;
  w0.begin = begin;
  w0.end = end;
  w0.n = 0;
  w0.T = 0;
  w0.hc = 0;
  w0.p = *start_p;
  if (w0.b < p.B) {
    w0.n = paged_len(p.c, w0.b, p.err);
    w0.T = steps_of<KS>(w0.n);
    w0.hc = static_cast<int>((begin - w0.p) / (w0.T + 1));
    w0.p += static_cast<long long>(w0.hc) * (w0.T + 1);
  }

  if (warp == kWarpTMA || warp == kWarpTMAV) {
    // ------------------------------------------------------------------ TMA producer
    uint32_t q_cnt = 0, kv_cnt = 0;
    const int box = min(1 << p.c.page_log2, kKeys);   // tokens per box
    const int n_pg = kKeys / box;                     // boxes along a tile
    // this lane's box: page `pg` of a tile, chunk `ch`
    const int pg = lane % n_pg, ch = (lane / n_pg) & 1;
    const bool of_v = warp == kWarpTMAV, has = lane < 2 * n_pg;
    const CUtensorMap* map = of_v ? &p.tm_v : &p.tm_k;
    const uint32_t dst0 = (of_v ? sV : sK) + ch * kChunk + pg * box * 128;
    auto b_full = [&](int s) { return of_v ? b_v_full(s) : b_k_full(s); };
    auto b_empty = [&](int s) { return of_v ? b_v_empty(s) : b_k_empty(s); };
    const int key_off = (kTPS == 1 ? 0 : ch * kKeys) + pg * box;
    const int col = kTPS == 1 ? ch * 64 : 0;
    auto page_at = [&](const Walk& w, int t) {   // the page of this lane's box in step t, -1: past the last key
      const int key = t * KS + key_off;
      if (!has || key >= w.n) return -1;
      const int id = paged_page(p.c, w.b, key >> p.c.page_log2, p.err);
      return id < 0 ? p.c.num_pages : id;   // no page: rows past the pool read as zeros
    };
    Walk w = w0;
    bool ok = true;
    for (bool more = next_unit<KS>(p, w, true); more && ok; more = next_unit<KS>(p, w, false)) {
      if (w.t1 <= w.t0) continue;
      const int unit = w.hc * p.abreast + place, g = unit / p.parts, part = unit - g * p.parts;
      if (!of_v) {
        const int qs = q_cnt & 1;
        if (!mbar_wait_warp(b_q_empty(qs), ((q_cnt >> 1) & 1) ^ 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteQEmpty))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(b_q_full(qs), (DA / 64) * p.heads * 128);
          for (int c = 0; c < DA / 64; ++c)
            tma_load_4d(sQ + qs * C::kQ + c * C::kQChunk, &p.tm_q, b_q_full(qs), c * 64, g * p.group + part * p.heads,
                        w.b, 0);
        }
        ++q_cnt;
      }
      int page = page_at(w, w.t0);
      for (int t = w.t0; t < w.t1; ++t) {
        const int st = kv_cnt % kStages;
        const int next = t + 1 < w.t1 ? page_at(w, t + 1) : -1;
        if (!mbar_wait_warp(b_empty(st), ((kv_cnt / kStages) & 1) ^ 1, wc,
                            ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteKEmpty))) { ok = false; break; }
        const uint32_t n_box = __popc(__ballot_sync(0xffffffffu, page >= 0));
        if (lane == 0) mbar_arrive_expect_tx(b_full(st), n_box * box * 128);
        __syncwarp();
        if (page >= 0)
          tma_load_4d(dst0 + st * kTile, map, b_full(st), col, g,
                      (t * KS + key_off) & ((1 << p.c.page_log2) - 1), page);
        page = next;
        ++kv_cnt;
      }
    }
    if (lane == 0 && *abort_flag) {
      // let the loads already issued land before the CTA exits
      for (int s = 0; s < kStages; ++s) {
        const uint32_t n = (kv_cnt + kStages - 1 - s) / kStages;
        if (n > 0) mbar_wait(b_full(s), (n - 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteDrain), false);
      }
      for (int s = 0; s < 2; ++s) {
        const uint32_t n = (q_cnt + 1 - s) / 2;
        if (n > 0) mbar_wait(b_q_full(s), (n - 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteDrain), false);
      }
    }
  } else if (warp == kWarpMMA) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t kIdescS = idesc_f16_f32acc(kKeys, kNQ, BF16, false);   // A = K, B = Q: both K-major
      constexpr uint32_t kIdescO = idesc_a_mn(128, C::kRows, BF16);            // A = V read MN-major, B = P^T
      const uint64_t dq0 = sdesc_sw128(sQ, 16, 1024);
      const uint64_t dk0 = sdesc_sw128(sK, 16, 1024);
      const uint64_t dv0 = sdesc_sw128(sV, kChunk, 1024);
      const uint64_t dp0 = sdesc_sw128(sP, 16, 1024);
      const uint32_t t_u = tmem + 2 * kTPS * kNQ;   // u^T columns
      uint32_t q_cnt = 0, kv_cnt = 0, v_cnt = 0, s_cnt = 0, p_cnt = 0, units_done = 0;
      bool ok = true;
      Walk w = w0;
      for (bool more = next_unit<KS>(p, w, true); more && ok; more = next_unit<KS>(p, w, false)) {
        if (w.t1 <= w.t0) continue;
        const int qs = q_cnt & 1;
        if (!mbar_wait(b_q_full(qs), (q_cnt >> 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteQFull))) break;
        ++q_cnt;
        tc_fence_after();
        // u^T += V^T P^T of the step in stage vst, P^T buffer pb; V (and K: see
        // b_k_empty) is released after it.  Before a unit's first product, which
        // overwrites u^T, the previous unit's epilogue must have read it
        auto do_pv = [&](int vst, int pb, bool first) -> bool {
          if (!mbar_wait(b_v_full(vst), (v_cnt / kStages) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteVFull))) return false;
          ++v_cnt;
          if (!mbar_wait(b_p_full(pb), (p_cnt >> 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSitePFull))) return false;
          ++p_cnt;
          if (first && units_done > 0 &&
              !mbar_wait(b_o_free, (units_done - 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteODone)))
            return false;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk) {
            const uint64_t a = dv0 + ((vst * kTile + kk * 2048) >> 4);
            const uint64_t b = dp0 + ((pb * C::kP + (kk >> 2) * C::kPChunk + (kk & 3) * 32) >> 4);
            umma_ss(t_u, a, b, kIdescO, (first && kk == 0) ? 0u : 1u);
          }
          umma_commit(b_v_empty(vst));
          umma_commit(b_p_free(pb));
          return true;
        };
        int prev_st = -1, prev_pb = -1;
        bool first_pv = true;
        for (int t = w.t0; t < w.t1; ++t) {
          const int st = kv_cnt % kStages;
          const int nt = kTPS == 1 ? 1 : (w.n - t * KS > kKeys ? 2 : 1);
          if (!mbar_wait(b_k_full(st), (kv_cnt / kStages) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteKFull))) {
            ok = false;
            break;
          }
          ++kv_cnt;
          tc_fence_after();
          // S^T of the step's tiles into buffer s_cnt & 1: its previous
          // contents (two steps back) were consumed, since this thread has
          // waited for that step's P
          const int sb = s_cnt & 1;
          for (int x = 0; x < nt; ++x) {
#pragma unroll
            for (int kk = 0; kk < DA / 16; ++kk) {
              const uint32_t off = ((x + (kk >> 2)) * kChunk + (kk & 3) * 32) >> 4;
              const uint32_t offq = ((qs * C::kQ + (kk >> 2) * C::kQChunk + (kk & 3) * 32) >> 4);
              umma_ss(tmem + (sb * kTPS + x) * kNQ, dk0 + ((st * kTile) >> 4) + off, dq0 + offq, kIdescS,
                      kk > 0 ? 1u : 0u);
            }
          }
          umma_commit(b_s_full(sb));
          if constexpr (DA == 64) umma_commit(b_k_empty(st));
          ++s_cnt;
          if (prev_pb >= 0) {
            if (!do_pv(prev_st, prev_pb, first_pv)) {
              ok = false;
              break;
            }
            first_pv = false;
          }
          prev_st = st;
          prev_pb = sb;
        }
        if (!ok) break;
        // the unit's last step
        if (!do_pv(prev_st, prev_pb, first_pv)) break;
        umma_commit(b_q_empty(qs));
        ++units_done;
      }
      umma_commit(b_drain);
      mbar_wait(b_drain, 0, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteDrain), false);
    }
  } else {
    // ------------------------------------------------------------------ softmax warps
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    const int sw = warp - 2;                       // softmax warp 0..3
    const int quarter = warp & 3;                  // TMEM lane quarter this warp may address
    const int lrow = quarter * 32 + lane;          // TMEM lane: key of the tile (S^T), d (u^T)
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    // u^T columns this thread's lane holds: at DA = 64 lanes 64-127 keep u_b
    const uint32_t t_u = tmem + lane_off + 2 * kTPS * kNQ + ((kTPS == 2 && lrow >= 64) ? kNQ : 0);
    const float c = p.scale_log2;
    uint32_t s_cnt = 0, red_cnt = 0, xch_cnt = 0;
    uint32_t free_seen[2] = {0, 0};   // phases of p_free(b) observed
    uint32_t steps_total = 0;         // steps (stage and P^T buffer uses) so far, all units
    bool ok = true;
    // reduces v over the 128 softmax threads (max or sum), all get the result
    auto reduce = [&](float (&v)[GT], bool is_max) -> bool {
#pragma unroll
      for (int h = 0; h < GT; ++h) {
        float x = v[h];
        if (is_max) {
          asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(x) : "f"(v[h]));
        } else {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        }
        v[h] = x;
      }
      const int par = red_cnt & 1;
      if (lane == 0) {
#pragma unroll
        for (int h = 0; h < GT; ++h) red[(par * 4 + sw) * kNQ + h] = v[h];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(b_red);
      if (!mbar_wait_warp(b_red, red_cnt & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteXchg))) return false;
      ++red_cnt;
#pragma unroll
      for (int h = 0; h < GT; ++h) {
        const float a = red[(par * 4 + 0) * kNQ + h], b = red[(par * 4 + 1) * kNQ + h];
        const float e = red[(par * 4 + 2) * kNQ + h], f = red[(par * 4 + 3) * kNQ + h];
        v[h] = is_max ? fmaxf(fmaxf(a, b), fmaxf(e, f)) : (a + b) + (e + f);
      }
      return true;
    };
    // waits until the P.V of this CTA's step i (over all units) has completed:
    // phase i >> 1 of p_free(i & 1); phases of one buffer are observed in order
    // and never fall two behind (step i + 2 writes the buffer only after this)
    auto pv_wait = [&](uint32_t i) -> bool {
      const int b = i & 1;
      while (free_seen[b] <= (i >> 1)) {
        if (!mbar_wait_warp(b_p_free(b), free_seen[b] & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSitePvDone)))
          return false;
        ++free_seen[b];
      }
      tc_fence_after();
      return true;
    };
    Walk w = w0;
    for (bool more = next_unit<KS>(p, w, true); more && ok; more = next_unit<KS>(p, w, false)) {
      const int unit = w.hc * p.abreast + place, g = unit / p.parts, part = unit - g * p.parts;
      const int head0 = g * p.group + part * p.heads;
      const int G = min(p.heads, p.group - part * p.heads);   // heads of this unit
      const size_t orow0 = static_cast<size_t>(w.b) * p.Hq + head0;   // first output row (b, head)
      if (w.T == 0) {
        // a sequence without keys: O = 0, lse = -inf
        T* dst = reinterpret_cast<T*>(p.o);
        if (lrow < DA)
          for (int h = 0; h < G; ++h) dst[(orow0 + h) * DA + lrow] = T(0.0f);
        if (sw == 0 && lane < G) p.lse[static_cast<size_t>(head0 + lane) * p.B + w.b] = -INFINITY;
        continue;
      }
      float m[GT], l[GT];
#pragma unroll
      for (int h = 0; h < GT; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.0f;
      }
      for (int t = w.t0; t < w.t1; ++t) {
        const int sb = s_cnt & 1;
        if (!mbar_wait_warp(b_s_full(sb), (s_cnt >> 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteSFull))) {
          ok = false;
          break;
        }
        ++s_cnt;
        tc_fence_after();
        // this thread's key in each tile of the step
        float s[kTPS][kNQ];
        bool valid[kTPS];
#pragma unroll
        for (int y = 0; y < kTPS; ++y) {
          tld(tmem + lane_off + (sb * kTPS + y) * kNQ, s[y]);
          valid[y] = t * KS + y * kKeys + lrow < w.n;
        }
        float x[GT];
#pragma unroll
        for (int h = 0; h < GT; ++h) {
          x[h] = valid[0] ? s[0][h] : -INFINITY;
#pragma unroll
          for (int y = 1; y < kTPS; ++y) x[h] = fmaxf(x[h], valid[y] ? s[y][h] : -INFINITY);
        }
        if (!reduce(x, true)) { ok = false; break; }
        // running max (scaled units): rescale only when it grows by more than 2^8
        float r[GT];
        bool any_resc = false;
#pragma unroll
        for (int h = 0; h < GT; ++h) {
          r[h] = 1.0f;
          const float mt = (x[h] == -INFINITY) ? -INFINITY : x[h] * c;
          if (mt > m[h] && (m[h] == -INFINITY || mt - m[h] > 8.0f)) {
            r[h] = (m[h] == -INFINITY) ? 0.0f : ex2_approx(m[h] - mt);
            m[h] = mt;
            any_resc = true;
          }
        }
        // P^T of these keys into buffer sb, once the P.V that read it two
        // steps back has completed
        if (steps_total >= 2 && !pv_wait(steps_total - 2)) { ok = false; break; }
#pragma unroll
        for (int h = 0; h < GT; ++h) {
          const float mh = (m[h] == -INFINITY) ? 0.0f : m[h] - kLift<BF16>;
          float e_sum = 0.0f;
#pragma unroll
          for (int y = 0; y < kTPS; ++y) {
            const float e = valid[y] ? ex2_approx(s[y][h] * c - mh) : 0.0f;
            e_sum += e;
            uint8_t* pbuf = smem + C::kOffP + sb * C::kP + (lrow >> 6) * C::kPChunk;
            *reinterpret_cast<T*>(pbuf + sw128(y * kNQ + h, lrow & 63)) = T(e);
          }
          l[h] = l[h] * r[h] + e_sum;
        }
        if (t * KS + KS > w.n) {
          // the sequence's last step: rows of V past its last key become zero,
          // once the stage's V has landed
          const int st = steps_total % kStages;
          if (!mbar_wait_warp(b_v_full(st), (steps_total / kStages) & 1, wc,
                              ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteVFull))) { ok = false; break; }
#pragma unroll
          for (int y = 0; y < 2; ++y)
            if (!valid[kTPS == 1 ? 0 : y]) {
              uint4* row = reinterpret_cast<uint4*>(smem + C::kOffV + st * kTile + y * kChunk + lrow * 128);
#pragma unroll
              for (int i = 0; i < 8; ++i) row[i] = make_uint4(0, 0, 0, 0);
            }
        }
        // u^T rescale (rare): needs the previous step's P.V complete.  m is
        // the same in every thread, so the decision is too; the vote keeps the
        // warp-collective TMEM accesses below uniform regardless.
        any_resc = __any_sync(0xffffffffu, any_resc);
        if (t > w.t0 && any_resc) {
          if (!pv_wait(steps_total - 1)) { ok = false; break; }
          float o[kNQ];
          tld(t_u, o);
#pragma unroll
          for (int h = 0; h < GT; ++h) o[h] *= r[h];
          tst(t_u, o);
          tmem_wait_st();
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_p_full(sb));
        ++steps_total;
      }
      if (!ok) break;
      // the piece's exp-sums over all its keys, then u^T / l
      if (!reduce(l, false)) break;
      if (!pv_wait(steps_total - 1)) break;
      float o[kNQ];
      tld(t_u, o);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_o_free);   // u^T may be overwritten by the next unit
      if constexpr (kTPS == 2) {
        // u = u_a + u_b: lanes 64-127 hand u_b over through the first P^T
        // buffer, idle now that every P.V so far has completed; the next
        // P^T write follows the next max exchange, which all four warps
        // reach only after this
        float* xch = reinterpret_cast<float*>(smem + C::kOffP);
        if (lrow >= 64) {
#pragma unroll
          for (int h = 0; h < GT; ++h) xch[h * 64 + (lrow - 64)] = o[h];
          __syncwarp();
          if (lane == 0) mbar_arrive(b_xch);
        } else {
          if (!mbar_wait_warp(b_xch, xch_cnt & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteXchg))) break;
#pragma unroll
          for (int h = 0; h < GT; ++h) o[h] += xch[h * 64 + lrow];
        }
        ++xch_cnt;
      }
      const bool whole = w.t0 == 0 && w.t1 == w.T;
      const int slot = 2 * blockIdx.x + (w.t0 == 0 ? 1 : 0);
      if (lrow < DA) {
#pragma unroll
        for (int h = 0; h < GT; ++h) {
          if (h >= G) break;
          const float v = (l[h] != 0.0f) ? o[h] / l[h] : 0.0f;   // 0: saw no key; a NaN stays one
          if (whole) reinterpret_cast<T*>(p.o)[(orow0 + h) * DA + lrow] = T(v);
          else p.part_o[(static_cast<size_t>(slot) * kNQ + h) * DA + lrow] = v;
        }
      }
      if (sw == 0 && lane < G) {
        float lv = 0.0f, mv = -INFINITY;
#pragma unroll
        for (int h = 0; h < GT; ++h)
          if (h == lane) {
            lv = l[h] * kDrop<BF16>;
            mv = m[h];
          }
        if (whole)
          p.lse[static_cast<size_t>(head0 + lane) * p.B + w.b] =
              (lv != 0.0f) ? mv * 0.69314718055994531f + __logf(lv) : -INFINITY;
        else
          p.part_ml[slot * kNQ + lane] = make_float2(mv, lv);
        // the unit's pieces lie on the ranges p / range ... (p + T - 1) / range
        if (!whole && w.t0 == 0 && lane == 0)
          p.rec[blockIdx.x] = make_int4(w.b, unit, static_cast<int>((w.p + w.T - 1) / range) - range_id + 1, 0);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMMA) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins the pieces of the unit that block x's CTA began, for head y of the
// unit: M = max m_s, w_s = 2^(m_s - M) l_s, O = sum w_s O_s / sum w_s.  Four
// warps take every fourth piece, a lane DA / 32 features; a programmatic
// dependent of the decode kernel.
template <bool BF16, int DA>
__global__ void __launch_bounds__(128) decode_merge_kernel(const __grid_constant__ Params p) {
  constexpr int E = DA / 32;
  __shared__ float s_m[4], s_l[4];
  __shared__ float s_o[4][DA];
  const int c = blockIdx.x, h = blockIdx.y, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_wait_prerequisites();
  const int4 rec = __ldcg(p.rec + c);
  const int pieces = rec.z;
  if (pieces <= 1) return;
  const int g = rec.y / p.parts, part = rec.y - g * p.parts;
  if (h >= p.group - part * p.heads) return;
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
      ml[u] = in ? __ldcg(p.part_ml + slot(s) * kNQ + h) : make_float2(-INFINITY, 0.0f);
      const float* src = p.part_o + (static_cast<size_t>(in ? slot(s) : 0) * kNQ + h) * DA + lane * E;
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
    using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
    const int head = g * p.group + part * p.heads + h;
    reinterpret_cast<T*>(p.o)[(static_cast<size_t>(rec.x) * p.Hq + head) * DA + i] = T(Lt != 0.0f ? at / Lt : 0.0f);
    if (i == 0)
      p.lse[static_cast<size_t>(head) * p.B + rec.x] = Lt != 0.0f ? Mx * 0.69314718055994531f + __logf(Lt) : -INFINITY;
  }
}

template <int GT, bool BF16, int DA>
cudaError_t launch(const Params& p, int grid, cudaStream_t stream) {
  constexpr int smem = Cfg<DA>::kSmem;
  static bool attr_done[64] = {};   // per instantiation
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_done[dev]) {
    e = cudaFuncSetAttribute(decode_kernel<GT, BF16, DA>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_done[dev] = true;
  }
  decode_kernel<GT, BF16, DA><<<grid, kThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launch();
  if (!p.cuts) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, p.heads);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, decode_merge_kernel<BF16, DA>, p);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <bool BF16, int DA>
cudaError_t pick(const Params& p, int grid, cudaStream_t stream) {
  if (p.heads <= 1) return launch<1, BF16, DA>(p, grid, stream);
  if (p.heads <= 2) return launch<2, BF16, DA>(p, grid, stream);
  if (p.heads <= 4) return launch<4, BF16, DA>(p, grid, stream);
  if (p.heads <= 8) return launch<8, BF16, DA>(p, grid, stream);
  return launch<16, BF16, DA>(p, grid, stream);
}

constexpr size_t kRecBytes(int sms) { return (static_cast<size_t>(sms) * sizeof(int4) + 255) / 256 * 256; }
constexpr size_t kMlBytes(int sms) { return static_cast<size_t>(2 * sms) * kNQ * sizeof(float2); }

}  // namespace pdec

long long paged_decode_workspace(int sms, int d) {
  return static_cast<long long>(pdec::kRecBytes(sms) + pdec::kMlBytes(sms) +
                                static_cast<size_t>(2 * sms) * pdec::kNQ * d * sizeof(float));
}

int paged_decode(const void* q, void* o, float* lse, int B, int Hq, const PagedKV& c, int d, bool bf16, int page_size,
                 float scale, void* ws, int sms, int* err, cudaStream_t stream) {
  pdec::Params p;
  p.c = c;
  p.group = Hq / c.hkv;
  // a unit holds up to 16 query heads of a key/value head; a wider group is cut
  // into equal parts, each of which reads the keys
  p.parts = (p.group + pdec::kNQ - 1) / pdec::kNQ;
  p.heads = (p.group + p.parts - 1) / p.parts;
  p.parts = (p.group + p.heads - 1) / p.heads;
  if (int rc = tile_map(q, bf16, d, Hq, B, 1, static_cast<long long>(d), static_cast<long long>(Hq) * d,
                        static_cast<long long>(B) * Hq * d, p.heads, 1, p.tm_q))
    return rc;
  const int box = page_size < 128 ? page_size : 128;
  if (int rc = tile_map(c.k, bf16, d, c.hkv, page_size, c.num_pages, c.s_head, c.s_token, c.s_page, 1, box, p.tm_k)) return rc;
  if (int rc = tile_map(c.v, bf16, d, c.hkv, page_size, c.num_pages, c.s_head, c.s_token, c.s_page, 1, box, p.tm_v)) return rc;
  char* w = static_cast<char*>(ws);
  p.rec = reinterpret_cast<int4*>(w);
  p.part_ml = reinterpret_cast<float2*>(w + pdec::kRecBytes(sms));
  p.part_o = reinterpret_cast<float*>(w + pdec::kRecBytes(sms) + pdec::kMlBytes(sms));
  p.o = o;
  p.lse = lse;
  p.err = err;
  p.timeout_ns = wait_timeout_ns();
  p.B = B;
  p.Hq = Hq;
  p.abreast = heads_abreast(c.hkv * p.parts, sms);
  p.cuts = (c.max_pages << c.page_log2) > pdec::kMinSteps * (d == 64 ? 256 : 128);
  p.scale_log2 = scale * 1.4426950408889634f;
  cudaError_t e;
  if (d == 64) e = bf16 ? pdec::pick<true, 64>(p, sms, stream) : pdec::pick<false, 64>(p, sms, stream);
  else e = bf16 ? pdec::pick<true, 128>(p, sms, stream) : pdec::pick<false, 128>(p, sms, stream);
  return e == cudaSuccess ? ATTN_OK : ATTN_ELAUNCH;
}

}  // namespace attn
