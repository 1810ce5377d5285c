// The paged key-value cache: geometry and checks shared by its kernels,
// appending tokens, and eviction by accumulated attention weight. (Attention
// over the cache is in sta_decode.cuh.) Both calls here only move data, so HBM
// bounds them: a key or value row (128 or 256 B) is read once and written once
// with 16-byte accesses.
#pragma once
#include "sta_cache_index.h"
#include "sta_common.cuh"

namespace sta {
namespace cache {

// sta_kv_cache as the kernels take it.
struct Args {
  uint4 *k, *v;  // pages, in 16-byte chunks
  const int *table;
  int *lens, *seen, *pos;
  float *weight;
  int B, H, num_pages, max_pages;
  // length of row r = b*H + h, or -1 (recorded) if the page table cannot hold it
  __device__ __forceinline__ int length(int r) const {
    const int n = lens[r];
    if (length_ok(n, max_pages)) return n;
    record_error(DEV_ERR_BAD_CACHE);
    return -1;
  }
  // page of slot j of sequence b, or -1 (recorded) if it is not in the pool;
  // 0 <= j < PAGE * max_pages
  __device__ __forceinline__ int page(int b, int j) const {
    const int p = table[(long long)b * max_pages + j / PAGE];
    if (page_ok(p, num_pages)) return p;
    record_error(DEV_ERR_BAD_CACHE);
    return -1;
  }
  // row (key or value of one token and head) of the pools
  __device__ __forceinline__ long long row(int page, int h, int j) const {
    return ((long long)page * H + h) * PAGE + j % PAGE;
  }
  // index of slot j of row r in slot_pos and weight
  __device__ __forceinline__ long long slot(int r, int j) const { return (long long)r * PAGE * max_pages + j; }
};

// ------------------------------------------------------------------- append
constexpr int APPEND_THREADS = 256;
constexpr int APPEND_UNROLL = 4;

// grid.y = sequence; each thread moves APPEND_UNROLL 16-byte chunks of the
// sequence's new K and of its new V: reads run through the raster rows in
// order, writes are the 2*D-byte rows of the heads' pages.
template <int D>
__global__ void __launch_bounds__(APPEND_THREADS)
append_kernel(Args a, const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new, int n_new,
              const int *__restrict__ counts) {
  constexpr unsigned CPR = D / 8;  // 16-byte chunks per row
  const int b = blockIdx.y;
  const int c = counts != nullptr ? counts[b] : n_new;
  if (c < 0 || c > n_new) {
    if (threadIdx.x == 0) record_error(DEV_ERR_BAD_CACHE);
    return;
  }
  const unsigned total = (unsigned)c * a.H * CPR;
  const unsigned base = blockIdx.x * (APPEND_THREADS * APPEND_UNROLL) + threadIdx.x;
  const long long src0 = (long long)b * n_new * a.H * CPR;
  uint4 k[APPEND_UNROLL], v[APPEND_UNROLL];
  long long dst[APPEND_UNROLL];
#pragma unroll
  for (int u = 0; u < APPEND_UNROLL; ++u) {
    const unsigned idx = base + u * APPEND_THREADS;
    dst[u] = -1;
    if (idx < total) {
      k[u] = __ldcs(k_new + src0 + idx);
      v[u] = __ldcs(v_new + src0 + idx);
      const unsigned chunk = idx % CPR, th = idx / CPR;
      const unsigned i = th / (unsigned)a.H, h = th - i * a.H;
      const int r = b * a.H + (int)h;
      const int len = a.length(r);
      if (len >= 0 && len < c) record_error(DEV_ERR_BAD_CACHE);
      if (len >= c) {
        const int j = len - c + (int)i;
        const int p = a.page(b, j);
        if (p >= 0) dst[u] = a.row(p, (int)h, j) * CPR + chunk;
        if (chunk == 0) {
          if (a.pos != nullptr) a.pos[a.slot(r, j)] = a.seen[r] - c + (int)i;
          if (a.weight != nullptr) a.weight[a.slot(r, j)] = 0.0f;
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < APPEND_UNROLL; ++u)
    if (dst[u] >= 0) {
      a.k[dst[u]] = k[u];
      a.v[dst[u]] = v[u];
    }
}

// -------------------------------------------------------------------- evict
constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_WARPS = PLAN_THREADS / 32;
constexpr int PLAN_BINS = 2048;

// Order of a slot as an unsigned key: the protected ones above every weight,
// NaN below every weight, -0 as +0, else the weight's own order.
__device__ __forceinline__ unsigned evict_key(float w, int pos, int sinks, int recent_from) {
  if (pos < sinks || pos >= recent_from) return 0xFFFFFFFFu;
  if (w != w) return 0u;
  const unsigned u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Inclusive sum over the lanes of a warp.
__device__ __forceinline__ int warp_scan(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// One CTA per (sequence, head): the budget-th largest key by radix selection
// (11 + 11 + 10 bits), then, over one contiguous range of slots per warp, the
// ranks of the ties, of the slots given up below the budget ("holes") and of
// those kept above it ("fills"). holes and fills [rows, cap], count [rows].
// Position, weight and length are updated here; the keys and values by
// move_kernel.
__global__ void __launch_bounds__(PLAN_THREADS)
evict_plan_kernel(Args a, int budget, int recent, int sinks, int cap, int *__restrict__ holes,
                  int *__restrict__ fills, int *__restrict__ count) {
  __shared__ unsigned hist[PLAN_BINS];
  __shared__ int part[3][PLAN_WARPS];
  __shared__ unsigned s_prefix;
  __shared__ int s_left;
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = a.length(r);
  if (len <= budget) {
    if (tid == 0) count[r] = 0;
    return;
  }
  const int from = a.seen[r] - recent;
  int *pos = a.pos + a.slot(r, 0);
  float *weight = a.weight + a.slot(r, 0);
  auto key_of = [&](int j) { return evict_key(weight[j], pos[j], sinks, from); };

  unsigned prefix = 0;  // the bits of the threshold found so far
  int left = budget;    // how many are still to be taken below the bins passed
  int shift = 32;
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10;
    const int next = shift - bits;
    for (int i = tid; i < PLAN_BINS; i += PLAN_THREADS) hist[i] = 0;
    __syncthreads();
    for (int j0 = 0; j0 < len; j0 += PLAN_THREADS) {
      const int j = j0 + tid;
      if (j < len) {
        const unsigned k = key_of(j);
        if (pass == 0 || (k >> shift) == prefix) atomicAdd(&hist[(k >> next) & ((1u << bits) - 1u)], 1u);
      }
    }
    __syncthreads();
    // the bin, counted from the top, in which the left-th key lies: thread t
    // holds bins 2047 - 2t and 2046 - 2t
    const int hi = (int)hist[PLAN_BINS - 1 - 2 * tid], lo = (int)hist[PLAN_BINS - 2 - 2 * tid];
    const int sum = warp_scan(hi + lo);
    if (lane == 31) part[0][warp] = sum;
    __syncthreads();
    if (warp == 0) part[0][lane] = warp_scan(part[0][lane]);
    __syncthreads();
    const int before = (warp > 0 ? part[0][warp - 1] : 0) + sum - hi - lo;
    if (before < left && left <= before + hi + lo) {
      const bool top = left <= before + hi;
      s_prefix = (prefix << bits) | (unsigned)(PLAN_BINS - 1 - 2 * tid - (top ? 0 : 1));
      s_left = left - before - (top ? 0 : hi);
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
    shift = next;
    __syncthreads();
  }
  // keep: above the threshold, and the first `left` of its equals
  const unsigned threshold = prefix;
  const int seg = (len + PLAN_THREADS - 1) / PLAN_THREADS * 32;
  const int lo = min(len, warp * seg), hi = min(len, lo + seg);
  const unsigned below_lane = (1u << lane) - 1u;
  int ties = 0;
  for (int j0 = lo; j0 < hi; j0 += 32)
    ties += __popc(__ballot_sync(0xFFFFFFFFu, j0 + lane < hi && key_of(j0 + lane) == threshold));
  if (lane == 0) part[0][warp] = ties;
  __syncthreads();
  if (warp == 0) {
    const int v = part[0][lane];
    part[0][lane] = warp_scan(v) - v;
  }
  __syncthreads();
  // twice over the range: count the holes and fills of the range, then list them
  int n_holes = 0, n_fills = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int tie = part[0][warp];
    int hole = pass ? part[1][warp] : 0, fill = pass ? part[2][warp] : 0;
    for (int j0 = lo; j0 < hi; j0 += 32) {
      const int j = j0 + lane;
      const bool in = j < hi;
      const unsigned k = in ? key_of(j) : 0u;
      const bool equal = in && k == threshold;
      const unsigned eq = __ballot_sync(0xFFFFFFFFu, equal);
      const bool keep = in && (k > threshold || (equal && tie + __popc(eq & below_lane) < left));
      const unsigned hm = __ballot_sync(0xFFFFFFFFu, in && !keep && j < budget);
      const unsigned fm = __ballot_sync(0xFFFFFFFFu, keep && j >= budget);
      if (pass) {
        const int at_hole = hole + __popc(hm & below_lane), at_fill = fill + __popc(fm & below_lane);
        if ((hm >> lane & 1u) && at_hole < cap) holes[(long long)r * cap + at_hole] = j;
        if ((fm >> lane & 1u) && at_fill < cap) fills[(long long)r * cap + at_fill] = j;
      }
      tie += __popc(eq);
      hole += __popc(hm);
      fill += __popc(fm);
    }
    if (!pass) {
      if (lane == 0) {
        part[1][warp] = hole;
        part[2][warp] = fill;
      }
      __syncthreads();
      if (warp < 2) {
        const int v = part[1 + warp][lane];
        const int s = warp_scan(v);
        part[1 + warp][lane] = s - v;
        if (lane == 31) hist[warp] = (unsigned)s;
      }
      __syncthreads();
      n_holes = (int)hist[0];
      n_fills = (int)hist[1];
    }
  }
  __syncthreads();
  // as many holes as fills: `budget` slots stay in all (and never more than
  // the lists hold)
  const int n = min(min(n_holes, n_fills), cap);
  for (int i = tid; i < n; i += PLAN_THREADS) {
    const int to = holes[(long long)r * cap + i], of = fills[(long long)r * cap + i];
    pos[to] = pos[of];
    weight[to] = weight[of];
  }
  if (tid == 0) {
    count[r] = n;
    a.lens[r] = budget;
  }
}

constexpr int MOVE_THREADS = 256;
constexpr int MOVE_UNROLL = 4;
// Pairs (fill, hole) one CTA of move_kernel<D> takes per pass.
template <int D>
__host__ __device__ constexpr int move_pairs() {
  return MOVE_THREADS / (D / 8) * MOVE_UNROLL;
}

// grid.x = row, grid.y strides over its pairs; D/8 threads move one pair's key
// and value, MOVE_UNROLL pairs in flight each.
template <int D>
__global__ void __launch_bounds__(MOVE_THREADS)
move_kernel(Args a, int cap, const int *__restrict__ holes, const int *__restrict__ fills,
            const int *__restrict__ count) {
  constexpr int CPR = D / 8;
  constexpr int GROUPS = MOVE_THREADS / CPR;
  const int r = blockIdx.x, b = r / a.H, h = r - b * a.H;
  const int n = count[r];
  const int chunk = threadIdx.x % CPR, group = threadIdx.x / CPR;
  for (int i0 = (int)blockIdx.y * move_pairs<D>(); i0 < n; i0 += (int)gridDim.y * move_pairs<D>()) {
    uint4 k[MOVE_UNROLL], v[MOVE_UNROLL];
    long long dst[MOVE_UNROLL];
#pragma unroll
    for (int u = 0; u < MOVE_UNROLL; ++u) {
      const int i = i0 + u * GROUPS + group;
      dst[u] = -1;
      if (i < n) {
        const int to = holes[(long long)r * cap + i], of = fills[(long long)r * cap + i];
        const int pt = a.page(b, to), pf = a.page(b, of);
        if (pt >= 0 && pf >= 0) {
          const long long src = a.row(pf, h, of) * CPR + chunk;
          dst[u] = a.row(pt, h, to) * CPR + chunk;
          k[u] = a.k[src];
          v[u] = a.v[src];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < MOVE_UNROLL; ++u)
      if (dst[u] >= 0) {
        a.k[dst[u]] = k[u];
        a.v[dst[u]] = v[u];
      }
  }
}

}  // namespace cache
}  // namespace sta
