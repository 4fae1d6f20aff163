// Eviction from a paged cache by accumulated attention weight
// (attn_cache_evict): per sequence and key/value head, the `recent` last keys
// and the heaviest of the others are kept, in order, and their rows moved to
// the front.
//
// Selection (evict_select_kernel, one cluster per sequence and head): the
// weights' bit patterns are mapped to unsigned integers of the same order, and
// the k-th largest is found digit by digit (11, 11 and 10 bits, most
// significant first): a histogram of the digit over the keys that match the
// digits so far, then the digit whose count from above passes k.  Keys above
// it are kept, and the first of those equal to it, so that exactly k are;
// counts of the warps before (and of the CTAs before, over distributed shared
// memory) give each kept key its place in order.  The weights are read from
// HBM once and stay in shared memory.
//
// Moving (evict_move_kernel): row s of the kept keys goes from key kept[s] to
// key s.  Into other pages, blocks take rows in any order.  In place (some page
// is written where it lies) a block owns a 32-byte column of the rows of one
// (sequence, head, K or V) and walks the rows in order, a batch at a time,
// every load of a batch before its stores: kept[s] >= s, so a store to key s
// can only meet loads of keys kept[s'] = s with s' <= s, which came in the same
// batch or an earlier one.  Bound by HBM: each kept row read and written once.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attn_paged.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;            // 11-bit digits
constexpr int kMaxKeys = 48 * 1024;    // weights that a CTA keeps in shared memory; more are read again
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 4;           // rows in flight per thread, in any order
constexpr int kWalkRows = 8;           // and in place

struct EvictParams {
  const float* weights;
  float* weights_out;
  int* kept;
  int* seqlens_out;
  PagedKV c;            // source
  const int* dst_table;
  int dst_stride, dst_max_pages;
  int weights_len, weights_out_len, budget, recent, d;
  int key_slots;        // weights per CTA that shared memory holds
  int* err;
};

// Unsigned key of the same order as the float: NaNs largest.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  if (u == 0x80000000u) return 0x80000000u;   // -0 is 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Keys of sequence b, bounded by the weights' row too.
__device__ __forceinline__ int evict_len(const EvictParams& p, int b) {
  const int n = paged_len(p.c, b, p.err);
  if (n <= p.weights_len) return n;
  atomicCAS(p.err, 0, ATTN_DEVERR_BAD_SEQLENS);
  return 0;
}

__device__ __forceinline__ int ld_dsmem_s32(uint32_t a) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Grid (CTAs of a cluster, heads, sequences).  Every CTA of a cluster takes the
// same path, so all reach each cluster barrier.  32 registers, so that two CTAs
// share an SM (256 heads in one wave: 32 x 4096 keys 104 -> 99.5 us).  Each digit
// costs one cluster barrier and two rounds of reads from the peers, about 4,500
// clocks of the 36,000 that 131,072 keys on 8 CTAs take (35.2 us with their
// moving; with two barriers a digit and one key a lane 37.4).
__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  // counts of each digit apart, so that a peer may still read one digit's while
  // the next digit is counted
  __shared__ __align__(8) int hists[3][kBins];
  __shared__ int coarses[3][32], from_peer[kMaxCluster][64];
  __shared__ int n_gt[kSelWarps + 1], n_eq[kSelWarps + 1];   // per warp; last: the CTA's
  __shared__ uint32_t s_prefix;
  __shared__ int s_need, s_group;
  const int CS = gridDim.x, rank = blockIdx.x;
  const int g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_launch_dependents();
  const int n = evict_len(p, b), m = min(n, p.budget);
  const long long row = static_cast<long long>(b) * p.c.hkv + g;
  const float* w = p.weights + row * p.weights_len;
  int* kept = p.kept + row * p.budget;
  if (g == 0 && rank == 0 && tid == 0) p.seqlens_out[b] = m;
  const int t0 = rank * kSelThreads + tid, step = CS * kSelThreads;
  for (int s = m + t0; s < p.budget; s += step) kept[s] = -1;
  if (n <= p.budget) {
    for (int s = t0; s < n; s += step) kept[s] = s;
    return;
  }
  const int cand = n - p.recent;       // keys that compete
  const int k = p.budget - p.recent;   // of which this many stay
  for (int s = t0; s < p.recent; s += step) kept[k + s] = cand + s;
  if (k == 0) return;
  // this CTA's keys [lo, hi)
  const int per = ((cand + CS - 1) / CS + 31) & ~31;
  const int lo = min(rank * per, cand), hi = min(lo + per, cand);
  const bool held = per <= p.key_slots;
  for (int i = tid; i < 3 * kBins; i += kSelThreads) hists[0][i] = 0;
  const int quads = lo + ((hi - lo + 3) & ~3);   // the keys by fours
  if (held && hi + tid < quads) keys[hi + tid - lo] = 0;   // below every key
  __syncthreads();
  // the weights, eight loads in flight, and the first digit's histogram
  for (int j0 = lo + tid; j0 < hi; j0 += 8 * kSelThreads) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = j0 + i * kSelThreads < hi ? __ldg(w + j0 + i * kSelThreads) : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int j = j0 + i * kSelThreads;
      if (j >= hi) break;
      const uint32_t u = order_key(x[i]);
      if (held) keys[j - lo] = u;
      atomicAdd(&hists[0][u >> 21], 1);
    }
  }
  // keys j .. j + 3; 0, which is below every key, past the last
  auto four_at = [&](int j) {
    if (held) return *reinterpret_cast<const uint4*>(keys + (j - lo));
    auto one = [&](int i) { return i < hi ? order_key(__ldg(w + i)) : 0u; };
    return make_uint4(one(j), one(j + 1), one(j + 2), one(j + 3));
  };
  uint32_t prefix = 0, mask = 0;
  int need = k;   // still to take among the keys that match the prefix
#pragma unroll 1
  for (int shift = 21, digits = 0;; shift = shift == 21 ? 10 : 0, ++digits) {
    const uint32_t digit = shift == 0 ? 0x3ffu : 0x7ffu;
    int *hist = hists[digits], *coarse = coarses[digits];
    if (shift != 21) {
      // no key's first digit is 0, so the zeros past the last match no prefix
      auto count = [&](uint32_t u) {
        if ((u & mask) == prefix) atomicAdd(&hist[(u >> shift) & digit], 1);
      };
      for (int j = lo + 4 * tid; j < quads; j += 4 * kSelThreads) {
        const uint4 u = four_at(j);
        count(u.x);
        count(u.y);
        count(u.z);
        count(u.w);
      }
    }
    __syncthreads();
    // The digit, in two steps: which group of 64 bins, then which bin; each
    // step adds one count per CTA and bin over the cluster (all 2,048 bins of
    // every CTA would be 64 KB to read per CTA and digit).
    {
      const int2 two = reinterpret_cast<const int2*>(hist)[warp * 32 + lane];
      const int c = __reduce_add_sync(0xffffffffu, two.x + two.y);
      if (lane == 0) coarse[warp] = c;
    }
    if (CS > 1) cluster_sync();
    else __syncthreads();
    if (warp < CS) from_peer[warp][lane] = ld_dsmem_s32(mapa_shared(smem_u32(&coarse[lane]), warp));
    __syncthreads();
    if (warp == 0) {
      int c = 0;
      for (int r = 0; r < CS; ++r) c += from_peer[r][lane];
      int above = c;   // keys of this group and the larger ones
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_down_sync(0xffffffffu, above, o);
        if (lane + o < 32) above += y;
      }
      if (above >= need && above - c < need) {
        s_group = lane;
        s_need = need - (above - c);
      }
    }
    __syncthreads();
    if (tid < 64 * CS) {
      const int i = tid & 63;
      from_peer[tid >> 6][i] = ld_dsmem_s32(mapa_shared(smem_u32(&hist[s_group * 64 + i]), tid >> 6));
    }
    __syncthreads();
    if (warp == 0) {
      const int need2 = s_need;
      int c0 = 0, c1 = 0;   // bins 2 lane and 2 lane + 1 of the group
      for (int r = 0; r < CS; ++r) {
        c0 += from_peer[r][2 * lane];
        c1 += from_peer[r][2 * lane + 1];
      }
      int above = c0 + c1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_down_sync(0xffffffffu, above, o);
        if (lane + o < 32) above += y;
      }
      const int before = above - (c0 + c1);
      __syncwarp();
      if (above >= need2 && before < need2) {
        const bool upper = before + c1 >= need2;
        s_prefix = prefix | static_cast<uint32_t>(s_group * 64 + 2 * lane + (upper ? 1 : 0)) << shift;
        s_need = need2 - (upper ? before : before + c1);
      }
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    mask |= digit << shift;
    __syncthreads();
    if (shift == 0) break;
  }
  // keys above the threshold, and the first `need` of those equal to it: counts
  // of each warp's run of keys, then their places
  const int run = ((per + kSelWarps - 1) / kSelWarps + 127) & ~127;
  const int r0 = min(lo + warp * run, quads), r1 = min(r0 + run, quads);
  int gt = 0, eq = 0;
  for (int j = r0 + 4 * lane; j < r1; j += 128) {
    const uint4 u = four_at(j);
    gt += (u.x > prefix) + (u.y > prefix) + (u.z > prefix) + (u.w > prefix);
    eq += (u.x == prefix) + (u.y == prefix) + (u.z == prefix) + (u.w == prefix);
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    n_gt[warp] = gt;
    n_eq[warp] = eq;
  }
  __syncthreads();
  if (warp == 0) {   // exclusive sums over the warps
    int a = n_gt[lane], e = n_eq[lane];
    const int a0 = a, e0 = e;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, e, o);
      if (lane >= o) {
        a += x;
        e += y;
      }
    }
    n_gt[lane] = a - a0;
    n_eq[lane] = e - e0;
    if (lane == 31) {
      n_gt[kSelWarps] = a;
      n_eq[kSelWarps] = e;
    }
  }
  __syncthreads();
  gt = n_gt[warp];
  eq = n_eq[warp];
  if (CS > 1) {
    cluster_sync();
    // lane r: the counts of CTA r, of which those before this one are added
    const int x = lane < CS ? ld_dsmem_s32(mapa_shared(smem_u32(&n_gt[kSelWarps]), lane)) : 0;
    const int y = lane < CS ? ld_dsmem_s32(mapa_shared(smem_u32(&n_eq[kSelWarps]), lane)) : 0;
    gt += __reduce_add_sync(0xffffffffu, lane < rank ? x : 0);
    eq += __reduce_add_sync(0xffffffffu, lane < rank ? y : 0);
    cluster_arrive();
  }
  for (int j0 = r0; j0 < r1; j0 += 128) {
    const int j = j0 + 4 * lane;
    const uint4 u = j < r1 ? four_at(j) : make_uint4(0, 0, 0, 0);
    const uint32_t x[4] = {u.x, u.y, u.z, u.w};
    int c = 0;   // above in the low half, equal in the high half
#pragma unroll
    for (int i = 0; i < 4; ++i) c += (x[i] > prefix) + ((x[i] == prefix) << 16);
    int to = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, to, o);
      if (lane >= o) to += y;
    }
    const int all = __shfl_sync(0xffffffffu, to, 31);
    to -= c;
    int above = gt + (to & 0xffff), e = eq + (to >> 16);   // before this lane's keys
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool is_gt = x[i] > prefix, is_eq = x[i] == prefix;
      if (is_gt || (is_eq && e < need)) kept[above + min(e, need)] = j + i;
      above += is_gt;
      e += is_eq;
    }
    gt += all & 0xffff;
    eq += all >> 16;
  }
  if (CS > 1) cluster_wait();   // no CTA leaves before its counts have been read
}

// Grid (blocks, heads, sequences); the last block of x moves the weights.  Four
// blocks per SM (64 registers): 32 x 4096 keys in place 103 us against 124 with
// three.
__global__ void __launch_bounds__(kMoveThreads, 4) evict_move_kernel(const __grid_constant__ EvictParams p) {
  const int blocks = gridDim.x - 1;
  const int g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int n = evict_len(p, b), m = min(n, p.budget);
  const long long row = static_cast<long long>(b) * p.c.hkv + g;
  const int* kept = p.kept + row * p.budget;
  const int lg = p.c.page_log2, pm = (1 << lg) - 1;
  const int* src_row = p.c.table + static_cast<long long>(b) * p.c.table_stride;
  const int* dst_row = p.dst_table + static_cast<long long>(b) * p.dst_stride;
  // whether any page is written where it lies
  bool lies = src_row == dst_row;
  if (!lies) {
    bool same = false;
    for (int i = tid; i < min((m + pm) >> lg, p.dst_max_pages); i += kMoveThreads) same |= src_row[i] == dst_row[i];
    lies = __syncthreads_or(same);
  }
  grid_wait_prerequisites();   // `kept` is written
  if (static_cast<int>(blockIdx.x) == blocks) {
    // the weights themselves, in the same order
    const float* w = p.weights + row * p.weights_len;
    float* out = p.weights_out + row * p.weights_out_len;
    for (int s0 = 0; s0 < m; s0 += kMoveThreads * kWalkRows) {
      float x[kWalkRows];
#pragma unroll
      for (int u = 0; u < kWalkRows; ++u) {
        const int s = s0 + u * kMoveThreads + tid;
        x[u] = s < m ? w[kept[s]] : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kWalkRows; ++u)
        if (s0 + u * kMoveThreads + tid < m) out[s0 + u * kMoveThreads + tid] = x[u];
    }
    __syncthreads();
    for (int s = m + tid; s < p.weights_out_len; s += kMoveThreads) out[s] = 0.0f;
    return;
  }
  if (lies && n <= p.budget && src_row == dst_row) return;   // nothing moves
  // offsets of row s's source and place; false where it stays or has no page
  auto places = [&](int s, long long& from, long long& to) {
    const int j = kept[s];
    const int f = paged_page(p.c, b, j >> lg, p.err);
    const int t = (s >> lg) < p.dst_max_pages ? __ldg(dst_row + (s >> lg)) : -1;
    if (t < 0 || t >= p.c.num_pages) {
      atomicCAS(p.err, 0, ATTN_DEVERR_BAD_PAGE);
      return false;
    }
    from = f * p.c.s_page + (j & pm) * p.c.s_token;
    to = t * p.c.s_page + (s & pm) * p.c.s_token;
    return f >= 0 && from != to;
  };
  if (!lies) {
    // whole rows of K and V, 16 bytes a thread
    const int lanes = p.d / 8, rows = kMoveThreads / lanes;
    const long long at = g * p.c.s_head + tid % lanes * 8;
    const int step = blocks * rows * kMoveRows;
    long long from[kMoveRows], to[kMoveRows];
    auto find = [&](int s0) {
#pragma unroll
      for (int u = 0; u < kMoveRows; ++u) {
        const int s = s0 + u * rows + tid / lanes;
        if (s >= m || !places(s, from[u], to[u])) to[u] = -1;
      }
    };
    int s0 = blockIdx.x * rows * kMoveRows;
    if (s0 < m) find(s0);
    for (; s0 < m; s0 += step) {
      uint4 x[kMoveRows], y[kMoveRows];
      long long put[kMoveRows];
#pragma unroll
      for (int u = 0; u < kMoveRows; ++u) {
        put[u] = to[u];
        if (to[u] >= 0) {
          x[u] = *reinterpret_cast<const uint4*>(p.c.k + from[u] + at);
          y[u] = *reinterpret_cast<const uint4*>(p.c.v + from[u] + at);
        }
      }
      if (s0 + step < m) find(s0 + step);   // while the rows are on their way
#pragma unroll
      for (int u = 0; u < kMoveRows; ++u)
        if (put[u] >= 0) {
          *reinterpret_cast<uint4*>(p.c.k + put[u] + at) = x[u];
          *reinterpret_cast<uint4*>(p.c.v + put[u] + at) = y[u];
        }
    }
    return;
  }
  const int n_col = p.d / 16;   // 32-byte columns
  if (static_cast<int>(blockIdx.x) >= 2 * n_col) return;
  const int which = blockIdx.x / n_col, col = blockIdx.x - which * n_col;
  uint16_t* base = (which == 0 ? p.c.k : p.c.v) + g * p.c.s_head + col * 16 + (tid & 1) * 8;
  constexpr int kRows = kMoveThreads / 2;
  for (int s0 = 0; s0 < m; s0 += kRows * kWalkRows) {
    uint4 x[kWalkRows];
    long long to[kWalkRows];
#pragma unroll
    for (int u = 0; u < kWalkRows; ++u) {
      const int s = s0 + u * kRows + (tid >> 1);
      long long from;
      if (s < m && places(s, from, to[u])) x[u] = *reinterpret_cast<const uint4*>(base + from);
      else to[u] = -1;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kWalkRows; ++u)
      if (to[u] >= 0) *reinterpret_cast<uint4*>(base + to[u]) = x[u];
    __syncthreads();
  }
}

}  // namespace
}  // namespace attn

extern "C" int attn_cache_evict(const float* weights, int weights_len, int* kept, int* seqlens_out, float* weights_out,
                                int weights_out_len, int B, const attn_paged_kv* cache, const int* dst_page_table,
                                int dst_stride, int dst_max_pages, int budget, int recent, cudaStream_t stream) {
  using namespace attn;
  EvictParams p = {};
  if (int rc = paged_check(cache, B, true, p.c)) return rc;
  if (!weights || !kept || !seqlens_out || !weights_out || weights_len <= 0) return ATTN_EINVAL;
  for (const void* x : {static_cast<const void*>(weights), static_cast<const void*>(kept),
                        static_cast<const void*>(seqlens_out), static_cast<const void*>(weights_out)})
    if (!ptr_aligned(x, 4)) return ATTN_EINVAL;
  if (budget < 1 || recent < 0 || recent > budget || weights_out_len < budget || budget > (1 << 30)) return ATTN_EINVAL;
  if (seqlens_out == cache->seqlens_k || (weights_out == weights && weights_out_len != weights_len)) return ATTN_EINVAL;
  const unsigned long long rows = 4ull * B * p.c.hkv;   // bytes of an entry of every row
  if (weights_out != weights && overlap(weights, rows * weights_len, weights_out, rows * weights_out_len)) return ATTN_EINVAL;
  if (dst_page_table) {
    if (dst_max_pages <= 0 || dst_stride < dst_max_pages ||
        static_cast<long long>(dst_max_pages) * cache->page_size < std::min<long long>(
            budget, static_cast<long long>(cache->max_pages) * cache->page_size))
      return ATTN_EINVAL;
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ELAUNCH;
  DeviceInfo info;
  if (int rc = device_info(dev, info)) return rc;
  if (!info.supported) return ATTN_EUNSUPPORTED;
  p.weights = weights;
  p.weights_out = weights_out;
  p.kept = kept;
  p.seqlens_out = seqlens_out;
  p.dst_table = dst_page_table ? dst_page_table : cache->page_table;
  p.dst_stride = dst_page_table ? dst_stride : cache->table_stride;
  p.dst_max_pages = dst_page_table ? dst_max_pages : cache->max_pages;
  p.weights_len = weights_len;
  p.weights_out_len = weights_out_len;
  p.budget = budget;
  p.recent = recent;
  p.d = cache->head_dim;
  p.err = info.err_word;
  // CTAs of a cluster per (sequence, head): as many as fill the SMs, up to 8,
  // of at least 2,048 keys each
  const long long longest = std::min<long long>(weights_len, static_cast<long long>(cache->max_pages) * cache->page_size);
  int cs = kMaxCluster;
  while (cs > 1 && (static_cast<long long>(B) * p.c.hkv * cs > info.sm_count || longest < 2048LL * cs)) cs /= 2;
  p.key_slots = static_cast<int>(std::min<long long>(kMaxKeys, (longest + cs - 1) / cs + 32));
  const int smem = p.key_slots * 4;
  static bool attr_done[64] = {};
  if (dev >= 64 || !attr_done[dev]) {
    if (cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (kMaxKeys + 32) * 4) !=
        cudaSuccess)
      return ATTN_ELAUNCH;
    if (dev < 64) attr_done[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cs, p.c.hkv, B);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, evict_select_kernel, p) != cudaSuccess) return ATTN_ELAUNCH;
  count_launch();
  // blocks per (sequence, head): the columns of K and V in place; in any order
  // up to eight blocks per SM in all, of at least one batch of rows
  const int batch = kMoveThreads / (p.d / 8) * kMoveRows;
  const long long heads = static_cast<long long>(B) * p.c.hkv;
  const int blocks = static_cast<int>(std::max<long long>(
      2 * p.d / 16, std::min<long long>((budget + batch - 1) / batch, 8LL * info.sm_count / heads)));
  cfg.gridDim = dim3(blocks + 1, p.c.hkv, B);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = 0;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  if (cudaLaunchKernelEx(&cfg, evict_move_kernel, p) != cudaSuccess) return ATTN_ELAUNCH;
  count_launch();
  return ATTN_OK;
}
