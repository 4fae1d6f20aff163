// Cutting a batch's work into equal ranges on the device: the units of all
// sequences form a line, each as long as its cost, and range r of them is what
// lies in [r range, (r + 1) range).
#pragma once
#include <cuda_runtime.h>

namespace attn {

// How many key/value heads (units of a sequence, equally long) walk the line
// side by side, each on a CTA of its own: the heads of a token lie next to one
// another in memory, and CTAs that read them at the same time keep to open DRAM
// rows.  The largest divisor of `heads` that leaves at most 5 % of the SMs idle.
// (One token over 32 caches of ~3,550 keys, 8 heads of 64: 47.1 us
// against 58.4 one head after the other.)
inline int heads_abreast(int heads, int sms) {
  for (int m = heads; m > 1; --m)
    if (heads % m == 0 && m <= sms && 20 * (sms / m) * m >= 19 * sms) return m;
  return 1;
}

// The sum of `mine` over the threads before this one, and the sums of `mine`
// and of `units` over all of them.  Has one __syncthreads; warp_sums holds
// 2 kThreads / 32 entries.
template <int kThreads>
__device__ __forceinline__ long long block_prefix(long long mine, int units, long long* warp_sums, long long& total,
                                                  long long& total_units) {
  constexpr int kW = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  units = __reduce_add_sync(0xffffffffu, units);
  if (lane == 31) {
    warp_sums[warp] = incl;
    warp_sums[kW + warp] = units;
  }
  __syncthreads();
  long long before = incl - mine;
  total = total_units = 0;
#pragma unroll
  for (int w = 0; w < kW; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
    total_units += warp_sums[kW + w];
  }
  return before;
}

// The length of a range: equal shares, but not below the mean unit, nor,
// when units are longer than that, below kLeast: shorter pieces cost more than
// they save (their merge, and a start each).  Units of up to kLeast are not
// cut: they belong to the range that they start in.
template <int kLeast>
__device__ __forceinline__ long long range_of(long long total, long long units, int ranges) {
  const long long share = (total + ranges - 1) / ranges;
  if (share >= kLeast) return share;
  return max(share, min(static_cast<long long>(kLeast), units > 0 ? total / units : 1));
}

// A unit of n steps that starts at p on the line: the steps [t0, t1) that fall
// to the range [begin, end); false where none does.  A unit of none falls to
// the range that it starts in.
template <int kLeast>
__device__ __forceinline__ bool part_of(long long p, int n, long long begin, long long end, int& t0, int& t1) {
  const long long lo = begin - p, hi = end - p;
  if (n <= kLeast) {
    t0 = 0;
    t1 = n;
    return lo <= 0 && hi > 0;
  }
  t0 = lo > 0 ? static_cast<int>(min(lo, static_cast<long long>(n))) : 0;
  t1 = hi > 0 ? static_cast<int>(min(hi, static_cast<long long>(n))) : 0;
  return t0 < t1;
}

// sum over i < n of floor((a i + b) / m), for a, b >= 0: the whole multiples of
// m in a and b are summed directly; of what is left, points under a line of
// slope a / m < 1 are counted by columns of the transposed line, as in
// Euclid's algorithm.  a n + b fits in 32 bits.
__device__ inline long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  long long sum = 0;
  while (n > 0) {
    const unsigned qa = a / m, qb = b / m;
    sum += static_cast<long long>(n) * (n - 1) / 2 * qa + static_cast<long long>(n) * qb;
    a -= qa * m;
    b -= qb * m;
    const unsigned top = a * n + b;   // the line's end, in m-ths
    if (top < m) break;
    // rows 1 .. top / m, each crossed at the column where the line reaches it
    n = top / m;
    b = top - n * m;
    const unsigned t = m;
    m = a;
    a = t;
  }
  return sum;
}

}  // namespace attn
