// The attention over caches of 8-bit floating point for trees with many columns
// (token, head) per key/value head: they are the rows of the products,
//   S = Q K^T   (M = 128 rows, N = 128 keys, K = d; 8 bits, Q's pieces one after another)
//   u += P V    (M = 128 rows, N = d, K = 128 keys; P in tensor memory)
// so that a softmax thread owns a row and needs no other thread for its maximum and
// sum.  (With the columns on N, as in attn_tree_fp8_kernel.cuh, their maxima over the
// keys are exchanges between threads: eight trees of 64 tokens, 32 heads on 8 of 128,
// over 16,384 keys took 579 us; 141 us here.)
//
// Two groups of four softmax warps take 64 of a step's 128 keys each, with references, sums
// and an accumulator of their own, joined at the unit's end, while S of the next step and
// P V of the last run.  P overwrites the S that it comes from.  (Taking whole steps in
// turns, a group waited for the P V and the S that have to follow its P: 220 us against
// 199 then; with more registers for the softmax warps, so that they hold their 64 values
// of S, 173; with the scales further ahead 162, the masks read ahead 158.)  S and P V are
// issued by a warp each, so that neither waits in the other's queue (155), from uniform
// operands (143); with the scales copied by the loading warps 138.  Bound by the
// chains of the softmax warps (at work for 1,500 to 2,100 of a step's 2,200 cycles when that
// took 138 us); the tensor pipe is 35 % busy (its floor for the 64 tokens is 51 us).
// The rest is as in attn_tree_fp8_kernel.cuh, but that P' is one fp16 value, off by 2^-11 of
// itself: a second one would double the products of P V, and V and P as bf16 values, which
// need no reference, took 180 us (its widening 14, the two values 9).  The references
// by p vs instead of p and a common one of the scales cost 5 of 143 us.  (A step looks
// for the largest p vs with an addition per key.  A cheaper bound that is exact where the
// scales are much the same, with a branch for where they are not, took 153 us, the branch
// taken or not.)
#pragma once
#include "attn_tree_fp8_parts.cuh"

namespace attn {
namespace tree {

template <int DA>
struct RowsCfg {
  using T = Tiles<DA, 1>;
  static constexpr int kStages = DA == 128 ? 3 : 4;
  static constexpr int kQPiece = 128 * DA;
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kOffK + kStages * T::kRaw;
  static constexpr int kOffW = kOffV + kStages * T::kRaw;
  static constexpr int kOffQ = kOffW + 2 * T::kWide;
  static constexpr int kOffScale = kOffQ + 3 * kQPiece;          // [kRing][k, v][128] floats
  static constexpr int kOffF = kOffScale + kRing * 2 * 128 * 4;  // [softmax warp][2][64] floats: vs 2^-kMiddle, log2 vs
  static constexpr int kOffMask = kOffF + 8 * 2 * 64 * 4;           // [128] 64-bit words
  static constexpr int kOffCol = kOffMask + 128 * 8;             // [128] floats
  static constexpr int kOffFin = kOffCol + 128 * 4;              // the second group's (m, l) per row
  static constexpr int kOffBar = kOffFin + 128 * 8;
  static constexpr int kNBars = 4 * kStages + 10 + kRing + 3;
  static constexpr int kOffMisc = kOffBar + (kNBars * 8 + 15) / 16 * 16;
  static constexpr int kSmem = kOffMisc + 512 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static constexpr uint32_t kTmemCols = 512;   // S: two buffers of 128 columns; u: two of d
  static constexpr int kColU = 256;
};

__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1; }

template <int DA>
__global__ void __launch_bounds__(kThreads, 1) tree_rows_kernel(const __grid_constant__ Params p) {
  using C = RowsCfg<DA>;
  using T = Tiles<DA, 1>;
  constexpr int N = kRowsPerUnit, KS = 128, kStages = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // (by an offset, not through an integer: the accesses stay ones of shared memory)
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);
  uint32_t bar_at = sbase + C::kOffBar;
  auto take = [&](int n) { const uint32_t a = bar_at; bar_at += 8 * n; return a; };
  const uint32_t b_k_full = take(kStages), b_k_empty = take(kStages), b_v_full = take(kStages), b_v_empty = take(kStages);
  const uint32_t b_s_full = take(2), b_p_full = take(2), b_w_full = take(2), b_pv_done = take(2), b_q_full = take(1),
                 b_q_empty = take(1), b_c_full = take(kRing), b_o_free = take(1), b_drain = take(1), b_fin = take(1);
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
    const int arrivals = in(b_v_empty, kStages) || in(b_w_full, 2) || in(b_o_free, 1) || in(b_fin, 1) ? 4   // the warps that widen; a group
                         : in(b_p_full, 2) || in(b_q_full, 1) ? 8       // the softmax warps, which convert the queries too
                         : in(b_q_empty, 1)                   ? 1 + 8   // the MMA, the softmax warps
                         : in(b_c_full, kRing)                ? 64      // the copying threads
                         : in(b_drain, 1)                     ? 2       // the two that issue MMAs
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
      produce<DA, 1, N, kStages>(p, w, place, &p.tm_k, sbase + C::kOffK, b_k_full, b_k_empty, p.c.ks,
                                sbase + C::kOffScale, b_c_full, wc);
    } else if (warp == kWarpV) {
      produce<DA, 1, N, kStages>(p, w, place, &p.tm_v, sbase + C::kOffV, b_v_full, b_v_empty, p.c.vs,
                                sbase + C::kOffScale + KS * 4, b_c_full, wc);
    } else if (warp >= kWarpWiden && warp < kWarpWiden + 4) {
      widen<DA, 1, N, kStages>(p, w, place, smem, C::kOffV, C::kOffW, b_v_full, b_v_empty, b_w_full, b_pv_done, wc);
    } else if (warp == kWarpMMA) {
      // ------------------------------------------------------------------ S's issuer
      constexpr uint32_t kIdescS = idesc_e4m3(128, 128), kIdescLast = idesc_e4m3(128, 128, true);
      const uint32_t idesc_1 = uniform(p.fp16 ? kIdescS : kIdescLast);   // (the last piece is e5m2)
      const uint32_t dq0 = desc_low(sbase + C::kOffQ, 16);
      const uint32_t dk0 = desc_low(sbase + C::kOffK, 16);
      uint32_t k_cnt = 0, units_done = 0;
      bool ok = true;
      for (bool more = any(next_unit<KS>(p, w, true)); more && ok; more = any(next_unit<KS>(p, w, false))) {
        const Unit u = unit_of<N>(p, w, place);
        if (w.t1 <= w.t0 || u.cols <= 0) continue;
        if (!wait_warp(b_q_full, units_done & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteQFull))) break;
        tc_fence_after();
        for (int t = w.t0; t < w.t1; ++t) {
          const int st = k_cnt % kStages, sb = k_cnt & 1;
          // into buffer sb, once the P.V that reads the P there has completed
          if ((k_cnt >= 2 && !wait_warp(b_pv_done + 8 * sb, ((k_cnt >> 1) - 1) & 1, wc,
                                   ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSitePvDone))) ||
              !wait_warp(b_k_full + 8 * st, (k_cnt / kStages) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteKFull))) {
            ok = false;
            break;
          }
          ++k_cnt;
          tc_fence_after();
          const uint32_t tm = uniform(tmem + sb * 128), a0 = uniform(dq0), b0 = uniform(dk0 + (st * T::kRaw >> 4));
          const uint32_t full = uniform(b_s_full + 8 * sb), empty = uniform(b_k_empty + 8 * st);
          if (elect_one()) {
#pragma unroll
            for (int s = 0; s < 3; ++s) {
              if (s == 2 && !p.fp16) break;
#pragma unroll
              for (int kk = 0; kk < DA / 32; ++kk)
                mma_f8<kHighRows<DA>>(tm, a0 + ((s * C::kQPiece + kk * 32) >> 4), b0 + 2 * kk, s == 0 ? kIdescS : s == 1 ? idesc_1 : kIdescLast,
                                      (s > 0 || kk > 0) ? 1u : 0u);
            }
            umma_commit(full);
            umma_commit(empty);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) umma_commit(b_q_empty);
        __syncwarp();
        ++units_done;
      }
      if (elect_one()) {
        umma_commit(b_drain);
        mbar_wait(b_drain, 0, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteDrain), false);
      }
      __syncwarp();
    } else if (warp == kWarpQ) {
      // ------------------------------------------------------------------ P V's issuer
      constexpr uint32_t kIdescO = idesc_f16_f32acc(128, DA, false, true);   // B = V read MN-major
      const uint32_t dv0 = desc_low(sbase + C::kOffW, T::kWideChunk);
      uint32_t pv_cnt = 0, units_done = 0;
      bool ok = true;
      for (bool more = any(next_unit<KS>(p, w, true)); more && ok; more = any(next_unit<KS>(p, w, false))) {
        const Unit u = unit_of<N>(p, w, place);
        if (w.t1 <= w.t0 || u.cols <= 0) continue;
        // u += P V, each group's keys into its accumulator.  Before a unit's first
        // products, which overwrite them, the previous unit's epilogue must have read both
        for (int t = w.t0; t < w.t1; ++t, ++pv_cnt) {
          const int b = pv_cnt & 1;
          const bool first = t == w.t0;
          if (!wait_warp(b_w_full + 8 * b, (pv_cnt >> 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteVFull)) ||
              !wait_warp(b_p_full + 8 * b, (pv_cnt >> 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSitePFull)) ||
              (first && units_done > 0 &&
               !wait_warp(b_o_free, (units_done - 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteODone)))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t tm = uniform(tmem), ta = uniform(tmem + b * 128), b0 = uniform(dv0 + (b * T::kWide >> 4));
          const uint32_t done = uniform(b_pv_done + 8 * b);
          const uint32_t more_of_it = uniform(first ? 0u : 1u);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              mma_f16_ts(tm + C::kColU + (kk >> 2) * DA, ta + (kk >> 2) * 64 + (kk & 3) * 8, b0 + (kk * 2048 >> 4), kIdescO,
                         (kk & 3) == 0 ? more_of_it : 1u);
            umma_commit(done);
          }
          __syncwarp();
        }
        if (!ok) break;
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
    // ------------------------------------------------------------------ softmax warps
    const int grp = warp >= kWarpSoft2 ? 1 : 0;
    const int sw = grp ? 4 + warp - kWarpSoft2 : warp - kWarpSoft1;   // softmax warp 0..7
    const int quarter = warp & 3;                  // TMEM lane quarter this warp may address
    const int row = quarter * 32 + lane;           // of the unit
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t t_u = t_lane + C::kColU;
    float* factor = reinterpret_cast<float*>(smem + C::kOffF) + sw * 128;   // this warp's, of the values' scales
    float2* fin = reinterpret_cast<float2*>(smem + C::kOffFin);
    uint32_t step = 0, units_done = 0;
    bool ok = true;
    for (bool more = next_unit<KS>(p, w, true); more && ok; more = next_unit<KS>(p, w, false)) {
      const Unit u = unit_of<N>(p, w, place);
      if (u.cols <= 0) continue;
      const int cc = u.col0 + row, token = token_of(p, cc), head = u.g * p.group + cc - token * p.group;
      const long long q_row = w.row0 + token;
      const bool mine = row < u.cols;
      uint16_t* out = p.o + (q_row * p.Hq + head) * DA;
      if (w.T == 0) {
        // a sequence without keys: O = 0, lse = -inf
        if (grp == 0 && mine) {
          for (int i = 0; i < DA; i += 8) *reinterpret_cast<uint4*>(out + i) = make_uint4(0, 0, 0, 0);
          p.lse[static_cast<long long>(head) * p.total + q_row] = -INFINITY;
        }
        continue;
      }
      if (w.t1 <= w.t0) continue;
      // the queries, by all eight warps, once the unit before is done with the last
      if (!wait_warp(b_q_empty, (units_done & 1) ^ 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteQEmpty))) break;
      convert_queries<DA, 4, false>(p, w, u, sw, 8, smem + C::kOffQ, C::kQPiece, reinterpret_cast<float*>(smem + C::kOffCol),
                          reinterpret_cast<unsigned long long*>(smem + C::kOffMask));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_q_full);
      if (!wait_warp(b_q_full, units_done & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteQFull))) break;
      const float cs = mine ? reinterpret_cast<const float*>(smem + C::kOffCol)[row] : 1.0f;
      const unsigned long long mask = mine ? reinterpret_cast<const unsigned long long*>(smem + C::kOffMask)[row] : 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(b_q_empty);
      // warps without a row leave their part of P as it is: rows of their own alone
      const bool idle = quarter * 32 >= u.cols;
      float m = -INFINITY, l = 0.0f;
      // which of the 32 keys from `key` on this row sees
      auto seen = [&](int key) {
        const int at = key - w.ctx;   // the first among the new tokens
        const uint32_t tree = at >= 64 ? 0u : at >= 0 ? static_cast<uint32_t>(mask >> at)
                              : at > -32 ? static_cast<uint32_t>(mask) << -at : 0u;
        return (low_bits(-at) | tree) & low_bits(w.n - key);
      };
      for (int t = w.t0; t < w.t1; ++t) {
        const int sb = step & 1, ring = step % kRing;
        if (!wait_warp(b_c_full + 8 * ring, (step / kRing) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteSFree))) {
          ok = false;
          break;
        }
        const uint32_t t_s = t_lane + sb * 128 + grp * 64;   // this group's keys
        const float* ks = reinterpret_cast<const float*>(smem + C::kOffScale) + ring * 2 * 128 + grp * 64;
        const int k0 = t * KS + grp * 64;
        // the values' scales: two keys per lane, for the warp
        uint32_t strange = 0;   // bit i: the lane's key i has no number for a scale
        {
          const float2 v2 = reinterpret_cast<const float2*>(ks + 128)[lane];
          float v[2] = {v2.x, v2.y};
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            v[i] = k0 + 2 * lane + i < w.n ? v[i] : 0.0f;
            if (!(v[i] <= kMostScale)) {
              strange |= 1u << i;
              v[i] = 0.0f;
            }
          }
          reinterpret_cast<float2*>(factor)[lane] = make_float2(v[0] * kScaleDown, v[1] * kScaleDown);
          reinterpret_cast<float2*>(factor)[32 + lane] = make_float2(scale_log2(v[0]), scale_log2(v[1]));
          __syncwarp();
        }
        if (!wait_warp(b_s_full + 8 * sb, (step >> 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteSFull))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (idle) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_p_full + 8 * sb);
          ++step;
          continue;
        }
        // which keys this row sees: all, but in the tiles that hold new tokens or the end
        const bool all = k0 + 64 <= min(w.ctx, w.n);
        uint32_t vis[2] = {0xffffffffu, 0xffffffffu};
        if (!all) {
#pragma unroll
          for (int i = 0; i < 2; ++i) vis[i] = seen(k0 + 32 * i);
        }
        // S of the 64 keys, times the keys' scales, -inf where this row does not see the key
        float s[64];
        {
          uint32_t r[64];
          tmem_ld_32x32b_x64(t_s, r);
          tmem_wait_ld(r);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float4 k4 = reinterpret_cast<const float4*>(ks)[i];
            const float2 x = fmul2(make_float2(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1])), make_float2(k4.x, k4.y));
            const float2 y = fmul2(make_float2(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])), make_float2(k4.z, k4.w));
            s[4 * i] = x.x, s[4 * i + 1] = x.y, s[4 * i + 2] = y.x, s[4 * i + 3] = y.y;
          }
        }
        if (!all) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (!((vis[i >> 5] >> (i & 31)) & 1)) s[i] = -INFINITY;
        }
        // the largest s + log2 vs
        float mt = -INFINITY;
        {
          float a = mt, b = mt, c = mt;
#pragma unroll
          for (int i = 0; i < 64; i += 8) {
            const float4 u4 = reinterpret_cast<const float4*>(factor)[16 + i / 4], v4 = reinterpret_cast<const float4*>(factor)[17 + i / 4];
            const float2 cs2 = make_float2(cs, cs);
            const float2 x0 = ffma2(make_float2(s[i], s[i + 1]), cs2, make_float2(u4.x, u4.y));
            const float2 x1 = ffma2(make_float2(s[i + 2], s[i + 3]), cs2, make_float2(u4.z, u4.w));
            const float2 x2 = ffma2(make_float2(s[i + 4], s[i + 5]), cs2, make_float2(v4.x, v4.y));
            const float2 x3 = ffma2(make_float2(s[i + 6], s[i + 7]), cs2, make_float2(v4.z, v4.w));
            mt = fmax3(mt, x0.x, x0.y);
            a = fmax3(a, x1.x, x1.y);
            b = fmax3(b, x2.x, x2.y);
            c = fmax3(c, x3.x, x3.y);
          }
          mt = fmaxf(fmax3(mt, a, b), c);
        }
        // the reference: rescale only when it grows by more than 2^8, or past -inf at all
        const bool grows = mt > fmaxf(m + 8.0f, -3.0e38f);
        if (__any_sync(0xffffffffu, grows)) {
          // (from -inf: 0; by halves, since l has the range for 2^-189, from rows of zeros to the largest scale)
          const float h = grows ? ex2_approx(0.5f * (m - mt)) : 1.0f, q = h * h;
          l = l * h * h;
          m = grows ? mt : m;
          if (t > w.t0) {
            if (!wait_pv(b_pv_done, step - 1, wc)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < DA; c += 16) {   // (by 32: 146 us against 141)
              float o[16];
              tld<16>(t_u + grp * DA + c, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= q;
              tst16(t_u + grp * DA + c, o);
            }
          }
        }
        const float mh = fmaxf(m, -3.0e38f) - (kHeldUp + kMiddle);   // (finite)
        const float2 cs2 = make_float2(cs, cs), mh2 = make_float2(-mh, -mh);
        float2 la = make_float2(0.0f, 0.0f), lb = la;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 f4 = reinterpret_cast<const float4*>(factor)[4 * c + i];
            float2 x = ffma2(make_float2(s[16 * c + 4 * i], s[16 * c + 4 * i + 1]), cs2, mh2);
            float2 y = ffma2(make_float2(s[16 * c + 4 * i + 2], s[16 * c + 4 * i + 3]), cs2, mh2);
            x = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            y = make_float2(ex2_approx(y.x), ex2_approx(y.y));
            la = fadd2(la, x);
            lb = fadd2(lb, y);
            x = fmul2(x, make_float2(f4.x, f4.y));
            y = fmul2(y, make_float2(f4.z, f4.w));
            pk[2 * i] = pack2<false>(x.x, x.y);
            pk[2 * i + 1] = pack2<false>(y.x, y.y);
          }
          // P over S, which is in registers
          asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t_s + 8 * c),
                       "r"(pk[0]), "r"(pk[1]), "r"(pk[2]), "r"(pk[3]), "r"(pk[4]), "r"(pk[5]), "r"(pk[6]), "r"(pk[7]));
        }
        l += (la.x + la.y) + (lb.x + lb.y);
        if (__any_sync(0xffffffffu, strange != 0)) {
          // a value's scale that is no number reaches the rows that see its key
          uint32_t hit = 0;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll 1
            for (int j = 0; j < 32; ++j)
              hit |= __shfl_sync(0xffffffffu, strange, 16 * i + (j >> 1)) >> (j & 1) & vis[i] >> j & 1u;
          }
          uint32_t one[1];
          tmem_wait_st();
          asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
                       : "=r"(one[0]) : "r"(t_s) : "memory");
          if (hit) one[0] = kNan2;
          asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" :: "r"(t_s), "r"(one[0]) : "memory");
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_p_full + 8 * sb);
        ++step;
      }
      if (!ok) break;
      if (grp == 1) {
        // hands its maxima and sums over, once the first group has read those of the unit
        // before
        if (units_done > 0 &&
            !wait_warp(b_o_free, (units_done - 1) & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteODone)))
          break;
        fin[row] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(b_fin);
        ++units_done;
        continue;
      }
      if (!wait_pv(b_pv_done, step - 1, wc)) break;
      if (!wait_warp(b_fin, units_done & 1, wc, ATTN_DEVERR_WAIT_TIMEOUT_SITE(kSiteMerge))) break;
      tc_fence_after();
      if (!idle) {
        const float2 other = fin[row];
        const Joined f = join(m, l, other.x, other.y);
        const bool whole = w.t0 == 0 && w.t1 == w.T;
        const int slot = 2 * blockIdx.x + (w.t0 == 0 ? 1 : 0);
        float* part = p.part_o + (static_cast<size_t>(slot) * N + row) * DA;
#pragma unroll 1
        for (int c = 0; c < DA; c += 16) {
          float a[16], b[16];
          tld_start<16>(t_u + c, a);
          tld_start<16>(t_u + DA + c, b);
          tld_wait<16>(a, b);
#pragma unroll
          for (int i = 0; i < 16; ++i) a[i] = (f.f0 < 0.0f ? 0.0f : a[i] * f.f0) + (f.f1 < 0.0f ? 0.0f : b[i] * f.f1);
          if (mine && whole) {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              v[i] = p.fp16 ? pack2<false>(a[2 * i], a[2 * i + 1]) : pack2<true>(a[2 * i], a[2 * i + 1]);
            reinterpret_cast<uint4*>(out + c)[0] = make_uint4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<uint4*>(out + c)[1] = make_uint4(v[4], v[5], v[6], v[7]);
          } else if (mine) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              reinterpret_cast<float4*>(part + c)[i] = make_float4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
          }
        }
        if (mine) {
          if (whole) p.lse[static_cast<long long>(head) * p.total + q_row] = f.sum * 0.69314718055994531f;
          else p.part_ml[slot * N + row] = make_float2(f.sum, f.some ? 1.0f : 0.0f);
        }
        // the unit's pieces lie on the ranges p / range ... (p + T - 1) / range
        if (!whole && w.t0 == 0 && row == 0)
          p.rec[blockIdx.x] = make_int4(w.b, w.hc * p.abreast + place,
                                        static_cast<int>((w.p + w.T - 1) / line.range) - line.range_id + 1, u.cols);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_o_free);   // u may be overwritten by the next unit
      ++units_done;
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

template <int DA>
cudaError_t launch_rows(const Params& p, int cols, int grid, cudaStream_t stream) {
  static bool done[64] = {};   // per instantiation
  return launch_with_merge<kRowsPerUnit, DA>(tree_rows_kernel<DA>, RowsCfg<DA>::kSmem, done, p, cols, grid, stream);
}

}  // namespace tree
}  // namespace attn
