// Cutting a batch's work into equal ranges on the device: the units of all
// sequences form a line, each as long as its cost, and CTA c takes what lies
// in [c range, (c + 1) range).
#pragma once
#include <cuda_runtime.h>

namespace attn {

// The sum of `mine` over the threads before this one, and over all of them.
// Has one __syncthreads; warp_sums holds kThreads / 32 entries.
template <int kThreads>
__device__ __forceinline__ long long block_prefix(long long mine, long long* warp_sums, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  long long before = incl - mine;
  total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  return before;
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
