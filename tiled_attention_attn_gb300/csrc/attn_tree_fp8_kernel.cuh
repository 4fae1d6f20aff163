// Attention of single tokens and of trees of drafted tokens over a paged cache of
// 8-bit floating point, on tensor cores (attn_tree_fp8).
//
// The new tokens' query heads that share a key/value head, T tokens x G heads, are
// the columns of transposed products, as in the 16-bit decode kernel:
//   S^T = K Q^T    (M = 128 keys, N columns, K = d)
//   u^T += V^T P^T (M = d, N columns, K = 128 keys)
// with the online softmax's running reference m, sum l and accumulator u per column;
// m may lag by up to 2^8, which cancels in u / l.
//
// K stays in e4m3 from HBM to the tensor core (kind::f8f6f4): what has 16 bits is
// the query, and it is small.  A query row, times the power of two that brings its
// largest value into (224, 448], is held as a sum of e4m3 values, two for bf16 and
// three for fp16 (4 significant bits each, so 8 and 11 exactly; see convert_queries for
// the small features), and S^T sums the products in fp32.  The key's
// scale and the row's power of two are applied to S.
//
// V is widened to fp16, which holds e4m3 exactly, by four warps between the TMA's
// stage and the second product: P in e4m3 would lose the light keys of a long
// cache.  A value's scale goes into its weight, P' = p vs 2^-m, and m follows the
// largest p vs of what the column sees (see kHeldUp): a reference for the scales of all
// keys would let a large value row that a column does not see, or sees without weight,
// take the bits of its other weights.  P' is a sum of two fp16 values, the second 2^11
// times what the first leaves, in columns of P^T that the product has anyway: off by
// 2^-22 of itself.
//
// Bound by HBM: per key and head d bytes of K and of V, and 8 of scales.  TMA
// stages of 16 KB of K and 16 of V (three or four), per page one box per tile; the
// warps that load them bring the scales too, with 4-byte asynchronous copies.  The
// queries' pieces are further columns of S^T, whose parts the softmax adds: at these
// widths the number of products counts, not their columns (a product per piece, and all
// softmax warps on one step: 120 us for 32 caches of ~3,550 keys, 32 heads on 8 of
// 128).  So does what it takes to issue one: with the operands in one thread's registers
// about 85 cycles each, whatever their size, and 61 us for those caches; uniform over the
// warp (see uniform()) 55.  Measured (device time, merge included): those caches 56.1 us,
// of which the 236 MB take 35 at the copy rate; one of 131,072 keys 55.3 of 41, its line
// of steps at 6.6 TB/s.  What is left is the start (4 us to the first S: prologue, the
// walk, the queries' conversion), the epilogue and 3 to 4 of the merge.
//
// Work is cut as in the 16-bit decode kernel: the steps of all (sequence, unit) on
// one line, equal ranges per CTA, pieces of a cut unit joined by tree_merge_kernel.
// A unit has up to 8 columns; more are the rows of attn_tree_fp8_rows.cuh.
//
// Slots past a sequence's last key may hold anything: their scores are dropped by
// index, their V is zeroed as it is widened.
//
// Head dimension 64: a step covers two tiles, one P.V serves both (M = 128 spans
// the two tiles' d; the product's diagonal blocks are u_a and u_b).
#pragma once
#include "attn_tree_fp8_parts.cuh"

namespace attn {
namespace tree {

constexpr int kRaw = kKeys * 128;       // a stage of K, or of V, in bytes
constexpr int kWide = 2 * kRaw;         // a step's V in fp16: two chunks of 128-byte rows
constexpr int kWideChunk = kRaw;

// GT columns.  Two groups of four softmax warps take turns, step by step, with references,
// sums and accumulators of their own that are joined at the unit's end (one group's
// chain of waits is longer than a step takes to arrive).  Two buffers of S^T, so that a
// group meets every phase of its buffer's barriers: with three it would see every
// second, which parity cannot tell from the one before.
template <int GT_, int DA>
struct Cfg {
  static constexpr int GT = GT_, N = 16;
  static_assert(GT <= kMostCols, "columns");
  static constexpr int kTPS = 128 / DA;            // tiles per step
  static constexpr int KS = kKeys * kTPS;          // keys per step
  static constexpr int kRows = kTPS * N;           // rows of P^T (the P.V's N)
  static constexpr int kStages = DA == 128 ? 4 : 3;
  static constexpr int kQSlots = 2;
  static constexpr int kSCols = 3 * N;   // columns of S^T per tile: the queries' pieces as further columns
  static constexpr int kQPiece = N * DA;
  static constexpr int kQ = 3 * kQPiece;
  static constexpr int kPChunk = kRows * 128;
  static constexpr int kP = 2 * kPChunk;
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kOffK + kStages * kRaw;
  static constexpr int kOffW = kOffV + kStages * kRaw;     // V in fp16, two buffers
  static constexpr int kOffP = kOffW + 2 * kWide;          // P^T, two buffers
  static constexpr int kOffQ = kOffP + 2 * kP;
  static constexpr int kOffScale = kOffQ + kQSlots * kQ;   // [kRing][k, v][KS] floats
  static constexpr int kOffMask = kOffScale + kRing * 2 * KS * 4;   // [slot][N] 64-bit words
  static constexpr int kOffCol = kOffMask + kQSlots * N * 8;        // [slot][N] floats
  static constexpr int kOffRed = kOffCol + kQSlots * N * 4;         // [group][parity][GT][4] floats
  static constexpr int kOffMax = kOffRed + 2 * 2 * GT * 16;  // references, [softmax warp][GT] floats
  static constexpr int kOffFin = kOffMax + 8 * GT * 4;   // the second group's (m, l)
  static constexpr int kOffFactor = (kOffFin + 2 * GT * 4 + 15) / 16 * 16;   // [softmax warp][GT][4] floats
  static constexpr int kOffBar = kOffFactor + 8 * GT * 16;
  static constexpr int kNBars = 4 * kStages + 12 + kRing + 6;
  static constexpr int kOffMisc = kOffBar + (kNBars * 8 + 15) / 16 * 16;
  static constexpr int kSmem = kOffMisc + 512 + 1024;
  // S^T: two buffers of kTPS tiles, then u^T (kRows columns) of each group with its own
  static constexpr int kColU = 2 * kTPS * kSCols;
  static constexpr int kUsedCols = kColU + 2 * kRows;
  static constexpr uint32_t kTmemCols = kUsedCols <= 128 ? 128 : kUsedCols <= 256 ? 256 : 512;
  static_assert(kSmem <= 227 * 1024 && kUsedCols <= 512, "shared and tensor memory");
};

template <int GT, int DA>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const __grid_constant__ Params p) {
  using C = Cfg<GT, DA>;
  constexpr int N = C::N, kTPS = C::kTPS, KS = C::KS, kStages = C::kStages, kSlots = C::kQSlots;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // (by an offset, not through an integer: the accesses stay ones of shared memory)
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);
  uint32_t bar_at = sbase + C::kOffBar;
  auto take = [&](int n) { const uint32_t a = bar_at; bar_at += 8 * n; return a; };
  const uint32_t b_k_full = take(kStages), b_k_empty = take(kStages), b_v_full = take(kStages), b_v_empty = take(kStages);
  const uint32_t b_q_full = take(2), b_q_empty = take(2), b_s_full = take(2), b_p_full = take(2), b_w_full = take(2);
  const uint32_t b_pv_done = take(2);   // the P.V that read P^T and V buffer i has completed (one phase per use)
  const uint32_t b_c_full = take(kRing);
  const uint32_t b_o_free = take(1), b_drain = take(1), b_red = take(2), b_xch = take(1), b_fin = take(1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  volatile int* start_b = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
  volatile long long* start_p = reinterpret_cast<volatile long long*>(smem + C::kOffMisc + 16);
  long long* warp_sums = reinterpret_cast<long long*>(smem + C::kOffMisc + 32);   // 2 kThreads / 32
  WaitCtl wc{p.err, abort_flag, p.timeout_ns};

  if (tid == 0) {
    *abort_flag = 0;
    *start_b = p.B;
    *start_p = 0;
  }
  // barriers, a thread each
  if (tid < C::kNBars) {
    const uint32_t bar = sbase + C::kOffBar + 8 * tid;
    auto in = [&](uint32_t first, int n) { return bar >= first && bar < first + 8 * n; };
    const int arrivals = in(b_v_empty, kStages) || in(b_w_full, 2) || in(b_red, 2) ? 4   // the warps that widen; a group
                         : in(b_q_empty, 2)                          ? 1 + 8     // the MMA, the softmax warps
                         : in(b_p_full, 2) || in(b_o_free, 1)        ? 4         // the softmax warps of a step; those that read u^T
                         : in(b_c_full, kRing)                       ? 64        // the copying threads
                         : in(b_xch, 1)                              ? 2
                                                                     : 1;
    mbar_init(bar, arrivals);
    fence_mbar_init();
  }
  if (warp == kWarpMMA) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == kWarpK && lane == 0) {
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }

  const Line line = find_line<KS>(p, start_b, start_p, warp_sums);
  const int place = line.place;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_launch_dependents();
  const bool softmax = warp >= kWarpSoft2 || (warp >= kWarpSoft1 && warp < kWarpWiden);   // (by warpgroup)
  Walk w = enter_line<KS>(p, line, *start_b, *start_p);

  if (!softmax) {
    regs_dec<kRegsFew>();
    auto any = [](bool x) { return __any_sync(0xffffffffu, x) != 0; };   // (uniform to the compiler too)
    if (warp == kWarpK) {
      produce<DA, kTPS, N, kStages>(p, w, place, &p.tm_k, sbase + C::kOffK, b_k_full, b_k_empty, p.c.ks,
                                   sbase + C::kOffScale, b_c_full, wc);
    } else if (warp == kWarpV) {
      produce<DA, kTPS, N, kStages>(p, w, place, &p.tm_v, sbase + C::kOffV, b_v_full, b_v_empty, p.c.vs,
                                   sbase + C::kOffScale + KS * 4, b_c_full, wc);
    } else if (warp >= kWarpWiden && warp < kWarpWiden + 4) {
      widen<DA, kTPS, N, kStages>(p, w, place, smem, C::kOffV, C::kOffW, b_v_full, b_v_empty, b_w_full, b_pv_done, wc);
    } else if (warp == kWarpQ) {
      // ------------------------------------------------------------------ queries
      uint32_t cnt = 0;
      bool ok = true;
      for (bool more = next_unit<KS>(p, w, true); more && ok; more = next_unit<KS>(p, w, false)) {
        const Unit u = unit_of<N>(p, w, place);
        if (w.t1 <= w.t0 || u.cols <= 0) continue;
        const int slot = cnt % kSlots;
        uint8_t* dst = smem + C::kOffQ + slot * C::kQ;
        float* col = reinterpret_cast<float*>(smem + C::kOffCol) + slot * N;
        unsigned long long* mask = reinterpret_cast<unsigned long long*>(smem + C::kOffMask) + slot * N;
        if (!wait_warp(b_q_empty + 8 * slot, ((cnt / kSlots) & 1) ^ 1, wc,
                            ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteQEmpty))) break;
        convert_queries<DA, 1, true>(p, w, u, 0, 1, dst, C::kQPiece, col, mask);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_q_full + 8 * slot);
        ++cnt;
      }
    } else if (warp == kWarpMMA) {
      // ------------------------------------------------------------------ MMA issuer
      const uint32_t idesc_s = idesc_e4m3(kKeys, N * (p.fp16 ? 3 : 2));
      constexpr uint32_t kIdescO = idesc_f16_f32acc(128, C::kRows, false, false) | (1u << 15);   // A = V read MN-major
      const uint32_t dq0 = desc_low(sbase + C::kOffQ, 16);
      const uint32_t dk0 = desc_low(sbase + C::kOffK, 16);
      const uint32_t dv0 = desc_low(sbase + C::kOffW, kWideChunk);
      const uint32_t dp0 = desc_low(sbase + C::kOffP, 16);
      const uint32_t t_u = tmem + C::kColU;   // u^T columns
      uint32_t q_cnt = 0, k_cnt = 0, pv_cnt = 0, units_done = 0;
      bool ok = true;
      for (bool more = any(next_unit<KS>(p, w, true)); more && ok; more = any(next_unit<KS>(p, w, false))) {
        const Unit u = unit_of<N>(p, w, place);
        if (w.t1 <= w.t0 || u.cols <= 0) continue;
        const int qs = q_cnt % kSlots;
        if (!wait_warp(b_q_full + 8 * qs, (q_cnt / kSlots) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteQFull))) break;
        ++q_cnt;
        tc_fence_after();
        // u^T += V^T P^T of the next step in line.  Before a unit's first products,
        // which overwrite u^T, the previous unit's epilogue must have read it
        int pv_unit = 0;
        auto do_pv = [&]() -> bool {
          const bool first = pv_unit++ < 2;
          const int b = pv_cnt & 1;
          if (!wait_warp(b_w_full + 8 * b, (pv_cnt >> 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteVFull))) return false;
          if (!wait_warp(b_p_full + 8 * b, (pv_cnt >> 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSitePFull))) return false;
          ++pv_cnt;
          if (pv_unit == 1 && units_done > 0 &&
              !wait_warp(b_o_free, (units_done - 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteODone)))
            return false;
          tc_fence_after();
          const uint32_t tu = uniform(t_u + b * C::kRows), a0 = uniform(dv0 + (b * kWide >> 4));
          const uint32_t b0 = uniform(dp0 + (b * C::kP >> 4)), done = uniform(b_pv_done + 8 * b);
          const uint32_t more_of_it = uniform(first ? 0u : 1u);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              mma_f16(tu, a0 + (kk * 2048 >> 4), b0 + (((kk >> 2) * C::kPChunk + (kk & 3) * 32) >> 4), kIdescO,
                      kk == 0 ? more_of_it : 1u);
            umma_commit(done);
          }
          __syncwarp();
          return true;
        };
        // S^T of a step's tiles into its buffer, whose last contents were consumed:
        // this warp has waited for that step's P
        auto issue_s = [&](int t) -> bool {
          const int st = k_cnt % kStages, sb = k_cnt & 1;
          const int nt = kTPS == 1 ? 1 : (w.n - t * KS > kKeys ? 2 : 1);
          if (!wait_warp(b_k_full + 8 * st, (k_cnt / kStages) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteKFull))) return false;
          ++k_cnt;
          tc_fence_after();
          const uint32_t ts = uniform(tmem + sb * kTPS * C::kSCols), a0 = uniform(dk0 + (st * kRaw >> 4));
          const uint32_t b0 = uniform(dq0 + (qs * C::kQ >> 4));
          const uint32_t full = uniform(b_s_full + 8 * sb), empty = uniform(b_k_empty + 8 * st);
          if (elect_one()) {
#pragma unroll
            for (int x = 0; x < kTPS; ++x) {
              if (x >= nt) break;
#pragma unroll
              for (int kk = 0; kk < DA / 32; ++kk)
                mma_f8<kHighRows<DA>>(ts + x * C::kSCols, a0 + ((x * (kKeys * DA) + kk * 32) >> 4), b0 + 2 * kk, idesc_s,
                                      kk > 0 ? 1u : 0u);
            }
            umma_commit(full);
            umma_commit(empty);
          }
          __syncwarp();
          return true;
        };
        // S^T of a step goes before P.V of the one before it
        for (int t = w.t0; t <= w.t1 && ok; ++t) {
          if (t < w.t1) ok = issue_s(t);
          if (ok && t > w.t0) ok = do_pv();
        }
        if (!ok) break;
        if (elect_one()) umma_commit(b_q_empty + 8 * qs);
        __syncwarp();
        ++units_done;
      }
      if (elect_one()) {
        umma_commit(b_drain);
        mbar_wait(b_drain, 0, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteDrain), false);
      }
      __syncwarp();
    }
  } else {
    regs_inc<kRegsMany>();
    auto pv_wait = [&](uint32_t i) { return wait_pv(b_pv_done, i, wc); };
    uint32_t step = 0;   // steps so far, all units
    bool ok = true;
    // ---------------------------------------------------------------- softmax warps
    const int grp = warp >= kWarpSoft2 ? 1 : 0;
    const int sw = warp - (grp ? kWarpSoft2 : kWarpSoft1);  // softmax warp 0..3 of its group
    const int quarter = warp & 3;                  // TMEM lane quarter this warp may address
    const int lrow = quarter * 32 + lane;          // TMEM lane: key of the tile (S^T), d (u^T)
    constexpr int LD = GT < 4 ? 4 : GT;            // columns as they are read
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    // u^T columns this thread's lane holds: at DA = 64 lanes 64-127 keep u_b
    const uint32_t t_u = t_lane + C::kColU + ((kTPS == 2 && lrow >= 64) ? N : 0) + grp * C::kRows;
    float4* red = reinterpret_cast<float4*>(smem + C::kOffRed) + grp * 2 * GT;   // [parity][GT], a float per warp
    const uint32_t bar_red = b_red + 8 * grp;
    uint32_t q_cnt = 0, red_cnt = 0, xch_cnt = 0, units_done = 0;
    float* m = reinterpret_cast<float*>(smem + C::kOffMax) + (4 * grp + sw) * GT;   // this warp's copy of the references
    // A warp hands GT values over to the group: column h by put(h, v) of one
    // lane, then meet(); then red[par * GT + h] has the four warps'
    auto put = [&](int h, float v) { reinterpret_cast<float*>(red + (red_cnt & 1) * GT)[4 * h + sw] = v; };
    constexpr int kOwn = GT == 8 ? 2 : GT == 4 ? 3 : GT == 2 ? 4 : 5;   // log2 of the lanes per column of fold_columns
    auto put_folded = [&](float v) {
      if ((lane & ((1 << kOwn) - 1)) == 0) put(lane >> kOwn, v);
    };
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_red);
      if (!wait_warp(bar_red, red_cnt & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteXchg))) return false;
      ++red_cnt;
      return true;
    };
    // S^T of LD columns, the pieces' products summed, times the key's scale; -inf
    // where the bits say that a column does not see the key
    auto scores = [&](uint32_t at, float scale, bool all, uint32_t bits, float (&x)[LD]) {
      {
        float y[LD];
        tld_start<LD>(at, x);
        tld_start<LD>(at + N, y);
        tld_wait<LD>(x, y);
#pragma unroll
        for (int i = 0; i < LD; ++i) x[i] = fmaf(y[i], kPieceDown, x[i]);
        if (p.fp16) {
          tld<LD>(at + 2 * N, y);
#pragma unroll
          for (int i = 0; i < LD; ++i) x[i] = fmaf(y[i], kPieceDown * kPieceDown, x[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < LD; ++i) x[i] *= scale;
      if (!all) {
#pragma unroll
        for (int i = 0; i < GT; ++i)
          if (!((bits >> i) & 1)) x[i] = -INFINITY;
      }
    };
    for (bool more = next_unit<KS>(p, w, true); more && ok; more = next_unit<KS>(p, w, false)) {
      const Unit u = unit_of<N>(p, w, place);
      if (u.cols <= 0) continue;
      const int G = min(GT, u.cols);   // columns
      // row of q and head of column h
      auto out_row = [&](int h, int& head) {
        const int cc = u.col0 + h, token = token_of(p, cc);
        head = u.g * p.group + cc - token * p.group;
        return w.row0 + token;
      };
      if (w.T == 0) {
        // a sequence without keys: O = 0, lse = -inf
        for (int h = 0; h < G && grp == 0; ++h) {
          int head;
          const long long row = out_row(h, head);
          if (lrow < DA) p.o[(row * p.Hq + head) * DA + lrow] = 0;
          if (lrow == 0) p.lse[static_cast<long long>(head) * p.total + row] = -INFINITY;
        }
        continue;
      }
      if (w.t1 <= w.t0) continue;
      const int qs = q_cnt % kSlots;
      if (!wait_warp(b_q_full + 8 * qs, (q_cnt / kSlots) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteQFull))) break;
      ++q_cnt;
      const float* col = reinterpret_cast<const float*>(smem + C::kOffCol) + qs * N;
      const unsigned long long* mask = reinterpret_cast<const unsigned long long*>(smem + C::kOffMask) + qs * N;
      float l[GT];
#pragma unroll
      for (int h = 0; h < GT; ++h) l[h] = 0.0f;
      if (lane < GT) m[lane] = -INFINITY;
      __syncwarp();
      const uint32_t step0 = step;   // of the unit
      int first_t = -1;              // this group's first step
      for (int t = w.t0; t < w.t1; ++t) {
        if (static_cast<int>(step & 1) != grp) {   // the other group's
          ++step;
          continue;
        }
        if (first_t < 0) first_t = t;
        const int sb = step & 1, ring = step % kRing;   // buffer of S^T and of P^T; stage of the scales
        if (!wait_warp(b_c_full + 8 * ring, (step / kRing) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteSFree))) {
          ok = false;
          break;
        }
        // this thread's key in each tile of the step: its scales, and the columns that see it
        const float* scales = reinterpret_cast<const float*>(smem + C::kOffScale) + ring * 2 * KS;
        float ks[kTPS], vs[kTPS];
        float cs[GT], lv[kTPS];   // the columns' factors; log2 of the values' scales
        uint32_t vis[kTPS];
#pragma unroll
        for (int y = 0; y < kTPS; ++y) {
          const int key = t * KS + y * kKeys + lrow, at = key - w.ctx;   // at: place among the new tokens
          ks[y] = scales[y * kKeys + lrow];
          vs[y] = scales[KS + y * kKeys + lrow];
          lv[y] = scale_log2(vs[y]);
          vis[y] = key < w.n ? 0xffffffffu : 0u;
          if (key < w.n) {
            if (at >= 0) {
              uint32_t bits = 0;
#pragma unroll 1
              for (int h = 0; h < GT; ++h) bits |= static_cast<uint32_t>((mask[h] >> at) & 1) << h;
              vis[y] = bits;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < GT; ++i) cs[i] = col[i];
        if (!wait_warp(b_s_full + 8 * sb, (step >> 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteSFull))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t t_s = t_lane + sb * kTPS * C::kSCols;
        float s[kTPS][LD];
        bool all = vis[0] == 0xffffffffu;   // every column sees every key of this warp
        if constexpr (kTPS == 2) all = all && vis[1] == 0xffffffffu;
        all = __all_sync(0xffffffffu, all);
        {
          float x[GT];
#pragma unroll
          for (int y = 0; y < kTPS; ++y) {
            scores(t_s + y * C::kSCols, ks[y], all, vis[y], s[y]);
#pragma unroll
            for (int i = 0; i < GT; ++i) {
              const float z = fmaf(s[y][i], cs[i], lv[y]);
              x[i] = y == 0 ? z : fmaxf(x[i], z);
            }
          }
          put_folded(fold_columns<GT>(x, lane, [](float a, float b) { return fmaxf(a, b); }));
        }
        if (!meet()) { ok = false; break; }
        const float4* got = red + ((red_cnt - 1) & 1) * GT;
        auto top4 = [](const float4& v) { return fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)); };
        // P^T of these keys into buffer sb, once the P.V that read it two
        // steps back has completed
        if (step >= 2 && !pv_wait(step - 2)) { ok = false; break; }
        // (no weight of a slot past the last key; a scale that is no number is dealt with below)
        float f[kTPS];
        bool strange = false;
#pragma unroll
        for (int y = 0; y < kTPS; ++y) {
          f[y] = vis[y] == 0 ? 0.0f : vs[y] * kScaleDown;
          if (!(f[y] <= kMostScale)) {
            strange = true;
            f[y] = 0.0f;
          }
        }
        // where P^T of this thread's key lies: row r at (pbuf ^ (r & 7) << 4) + 128 r
        const uint32_t pbuf = sbase + C::kOffP + sb * C::kP + (lrow >> 6) * C::kPChunk +
                              ((lrow & 63) >> 3 << 4) + 2 * (lrow & 7);
        // the references: rescale only when one grows by more than 2^8
        // (loads first, and no branches among them: a load behind a condition would
        // wait for the one before)
        float mt[GT], old[GT];
#pragma unroll
        for (int i = 0; i < GT; ++i) {
          mt[i] = top4(got[i]);   // (-inf where no column sees a key)
          old[i] = m[i];
        }
        bool any = false;
#pragma unroll
        for (int i = 0; i < GT; ++i) {
          // grows past old + 8, or past -inf at all
          const bool grows = mt[i] > fmaxf(old[i] + 8.0f, -3.0e38f);
          mt[i] = grows ? mt[i] : old[i];
          any |= grows;
        }
        // m is the same in every thread, so the decision is too; the vote
        // keeps the warp-collective TMEM accesses below uniform regardless.
        any = __any_sync(0xffffffffu, any);
        if (any) {
          float r[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) r[i] = 1.0f;
#pragma unroll
          for (int i = 0; i < GT; ++i) {
            // (from -inf: 0; by halves, since l has the range for 2^-189, from rows of zeros to the largest scale)
            const float h = old[i] == mt[i] ? 1.0f : ex2_approx(0.5f * (old[i] - mt[i]));
            l[i] = l[i] * h * h;
            r[i] = r[8 + i] = h * h;
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < GT; ++i)
            if (lane == i) m[i] = mt[i];
          __syncwarp();
          // u^T rescale (rare): this group's last P.V has completed
          if (t > first_t) {
            tc_fence_after();
            float o[16];
            tld<16>(t_u, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= r[i];
            tst16(t_u, o);
            tmem_wait_st();
          }
        }
        // P^T, and 2^11 times its rest as columns 8 on, whose products cost nothing more
        auto weight = [&](int i, int y) {
          const float e = ex2_approx(fmaf(s[y][i], cs[i], (kHeldUp + kMiddle) - fmaxf(mt[i], -3.0e38f)));
          l[i] += e;
          return e * f[y];
        };
        auto store = [&](int i, int y, uint32_t high, uint32_t rest) {
          const uint32_t at = (pbuf ^ ((i & 7) << 4)) + (y * N + i) * 128;
          store16(at, high);
          store16(at + 8 * 128, rest);
        };
        if constexpr (kTPS == 2 || GT == 1) {
#pragma unroll
          for (int i = 0; i < GT; ++i) {
            uint32_t high, rest;
            const float a = weight(i, 0);
            split2(make_float2(a, kTPS == 2 ? weight(i, kTPS - 1) : 0.0f), high, rest);
            store(i, 0, high, rest);
            if constexpr (kTPS == 2) store(i, 1, high >> 16, rest >> 16);
          }
        } else {
#pragma unroll
          for (int i = 0; i < GT; i += 2) {
            uint32_t high, rest;
            const float a = weight(i, 0);
            split2(make_float2(a, weight(i + 1, 0)), high, rest);
            store(i, 0, high, rest);
            store(i + 1, 0, high >> 16, rest >> 16);
          }
        }
        if (strange) {
          // a value's scale that is no number reaches the columns that see its key
#pragma unroll 1
          for (int i = 0; i < kTPS * GT; ++i) {
            const int y = i / GT, h = i - y * GT;
            const float v = y == 0 ? vs[0] : vs[kTPS - 1];
            const uint32_t seen = y == 0 ? vis[0] : vis[kTPS - 1];
            if (!(v <= kMostScale) && ((seen >> h) & 1)) store16((pbuf ^ ((h & 7) << 4)) + (y * N + h) * 128, kNan2);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_p_full + 8 * sb);
        ++step;
      }
      if (!ok) break;
      if (lane == 0) mbar_arrive(b_q_empty + 8 * qs);   // (what it read of the slot: the columns' factors and masks)
      // the piece's exp-sums over all its keys, then u^T / l (rolled over the
      // columns: this code runs once per unit)
      put_folded(fold_columns<GT>(l, lane, [](float a, float b) { return a + b; }));
      if (!meet()) break;
      const float4* got = red + ((red_cnt - 1) & 1) * GT;
      auto sum_of = [&](int h) {
        const float4 v = got[h];
        return (v.x + v.y) + (v.z + v.w);
      };
      float* fin_m = reinterpret_cast<float*>(smem + C::kOffFin);
      float* fin_l = fin_m + GT;
      if (grp == 1) {
        // hands its references and sums over (of no step: -inf and 0), once the first group
        // has read those of the unit before
        if (units_done > 0 &&
            !wait_warp(b_o_free, (units_done - 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteODone)))
          break;
        if (sw == 0) {
          if (lane < GT) {
            fin_m[lane] = m[lane];
            fin_l[lane] = sum_of(lane);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(b_fin);
        }
        ++units_done;
        continue;
      }
      // The second group's sums first: it has handed over all of its steps then, and seen
      // the phase of its barrier before each, so that the waits for both groups' last
      // products below cannot take an earlier phase for theirs
      if (!wait_warp(b_fin, units_done & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteMerge))) break;
      if (!pv_wait(step - 1)) break;
      if (step - step0 >= 2 && !pv_wait(step - 2)) break;
      tc_fence_after();
      const bool whole = w.t0 == 0 && w.t1 == w.T;
      const int slot = 2 * blockIdx.x + (w.t0 == 0 ? 1 : 0);
      // log2 of a column's sum, and the factors of the groups' u^T (join); a lane per
      // column, left in shared memory for the warp
      float4* factors = reinterpret_cast<float4*>(smem + C::kOffFactor) + (4 * grp + sw) * GT;
      if (lane < GT) {
        const Joined r = join(m[lane], sum_of(lane), fin_m[lane], fin_l[lane]);
        factors[lane] = make_float4(r.sum, r.some ? 1.0f : 0.0f, r.f0, r.f1);
      }
      __syncwarp();
      auto joined = [&](int h) {
        const float4 f = factors[h];
        float a[1], b[1], ar[1], br[1];   // of P^T, and of its rest
        tld_start<1>(t_u + h, a);
        tld_start<1>(t_u + h + 8, ar);
        tld_start<1>(t_u + C::kRows + h, b);
        tld_start<1>(t_u + C::kRows + h + 8, br);
        tld_wait<1>(a, b);
        tie<1>(ar);
        tie<1>(br);
        return (f.z < 0.0f ? 0.0f : fmaf(ar[0], 0x1p-11f, a[0]) * f.z) + (f.w < 0.0f ? 0.0f : fmaf(br[0], 0x1p-11f, b[0]) * f.w);
      };
      // u = u_a + u_b at head dimension 64: lanes 64-127 hand u_b over in the
      // first P^T buffer, idle now that every P.V that read
      // it has completed; this group writes them next after its next meeting
      auto handed = [&](int h, int i) {
        return reinterpret_cast<float*>(smem + C::kOffP + (i >> 5) * C::kPChunk + h * 128 + (i & 31) * 4);
      };
      if constexpr (kTPS == 2) {
        if (lrow >= 64) {
#pragma unroll 1
          for (int h = 0; h < G; ++h) {
            *handed(h, lrow - 64) = joined(h);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(b_xch);
        } else {
          if (!wait_warp(b_xch, xch_cnt & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteXchg))) break;
        }
        ++xch_cnt;
      }
      if (kTPS == 1 || lrow < 64) {
#pragma unroll 1
        for (int h = 0; h < G; ++h) {
          float v = joined(h);
          if constexpr (kTPS == 2) v += *handed(h, lrow);
          if (whole) {
            int head;
            const long long at = (static_cast<long long>(out_row(h, head)) * p.Hq + head) * DA + lrow;
            p.o[at] = p.fp16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
          } else {
            p.part_o[(static_cast<size_t>(slot) * N + h) * DA + lrow] = v;
          }
        }
      }
      if (sw == 0 && lane < G) {
        const float4 r = factors[lane];
        if (whole) {
          int head;
          const long long row = out_row(lane, head);
          p.lse[static_cast<long long>(head) * p.total + row] = r.x * 0.69314718055994531f;
        } else {
          p.part_ml[slot * N + lane] = make_float2(r.x, r.y);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_o_free);   // u^T may be overwritten by the next unit
      ++units_done;
      // the unit's pieces lie on the ranges p / range ... (p + T - 1) / range
      if (!whole && w.t0 == 0 && tid == 32 * kWarpSoft1)
        p.rec[blockIdx.x] = make_int4(w.b, w.hc * p.abreast + place,
                                      static_cast<int>((w.p + w.T - 1) / line.range) - line.range_id + 1, u.cols);
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

template <int GT, int DA>
cudaError_t launch(const Params& p, int cols, int grid, cudaStream_t stream) {
  using C = Cfg<GT, DA>;
  static bool done[64] = {};   // per instantiation
  return launch_with_merge<C::N, DA>(tree_kernel<GT, DA>, C::kSmem, done, p, cols, grid, stream);
}

template <int DA>
cudaError_t pick(const Params& p, int cols, int grid, cudaStream_t stream) {
  if (cols <= 1) return launch<1, DA>(p, cols, grid, stream);
  if (cols <= 2) return launch<2, DA>(p, cols, grid, stream);
  if (cols <= 4) return launch<4, DA>(p, cols, grid, stream);
  return launch<8, DA>(p, cols, grid, stream);
}

}  // namespace tree
}  // namespace attn
