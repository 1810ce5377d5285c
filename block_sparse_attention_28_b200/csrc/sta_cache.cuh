// The paged key-value cache: geometry and checks shared by its kernels,
// appending tokens, and eviction by accumulated attention weight. (Attention
// over the cache is in sta_decode.cuh.) Both calls here only move data, so HBM
// bounds them: a key or value row (128 or 256 B) is read once and written once
// with 16-byte accesses.
#pragma once
#include <cooperative_groups.h>

#include <type_traits>

#include "sta_cache_index.h"
#include "sta_common.cuh"

namespace sta {
namespace cache {

// Start of every kernel of the cache calls: the next kernel of the stream may
// start up beside this one, and this one goes on when the one before has ended
// and its writes can be seen.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// sta_kv_cache as the kernels take it.
struct Args {
  uint4 *k, *v;  // pages, in 16-byte chunks
  const int *table;
  int *lens, *seen, *pos;
  float *weight;
  int B, H, num_pages, max_pages;
  // length of row r = b*H + h, or -1 (recorded) if the page table cannot hold it
  __device__ __forceinline__ int length(int r) const { return checked_length(lens[r]); }
  __device__ __forceinline__ int checked_length(int n) const {
    if (length_ok(n, max_pages)) return n;
    record_error(DEV_ERR_BAD_CACHE);
    return -1;
  }
  // page of slot j of sequence b, or -1 (recorded) if it is not in the pool;
  // 0 <= j < PAGE * max_pages
  __device__ __forceinline__ int page(int b, int j) const {
    return checked_page(table[(long long)b * max_pages + j / PAGE]);
  }
  __device__ __forceinline__ int checked_page(int p) const {
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
  // (checked build) whether there is such a row, such a slot: what uses one asks
  // first and leaves the access out if not
  __device__ __forceinline__ bool has_row(int page, int h, int j) const {
    return dbg_ok(page >= 0 && page < num_pages && h >= 0 && h < H && j >= 0);
  }
  __device__ __forceinline__ bool has_slot(int r, int j) const {
    return dbg_ok(r >= 0 && r < B * H && j >= 0 && j < PAGE * max_pages);
  }
};

// ------------------------------------------------------------------- append
constexpr int APPEND_THREADS = 256;

// grid.y = sequence; each thread moves a 16-byte chunk of the new K and one of
// the new V (STRIDE: and goes on by the grid's width): reads run through the
// raster rows in order, writes are the 2*D-byte rows of the heads' pages. (Two
// or four chunks at once: 219 and 222 us where one takes 216, 1.35 GB.)
template <int D, bool STRIDE>
__global__ void __launch_bounds__(APPEND_THREADS)
append_kernel(Args a, const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new, int n_new,
              const int *__restrict__ counts) {
  constexpr unsigned CPR = D / 8;  // 16-byte chunks per row
  let_next_start();
  wait_for_previous();
  const int b = blockIdx.y;
  const int c = counts != nullptr ? counts[b] : n_new;
  if (c < 0 || c > n_new) {
    if (threadIdx.x == 0) record_error(DEV_ERR_BAD_CACHE);
    return;
  }
  const unsigned total = (unsigned)c * a.H * CPR;
  for (unsigned idx = blockIdx.x * APPEND_THREADS + threadIdx.x; idx < total; idx += gridDim.x * APPEND_THREADS) {
    const long long src = (long long)b * n_new * a.H * CPR + idx;
    const uint4 k = __ldcs(k_new + src), v = __ldcs(v_new + src);
    const unsigned chunk = idx % CPR, th = idx / CPR;
    const int i = (int)(th / (unsigned)a.H), h = (int)th - i * a.H;
    const int r = b * a.H + h;
    const int len = a.length(r);
    if (len < c) {  // (-1: recorded)
      if (len >= 0) record_error(DEV_ERR_BAD_CACHE);
      if (!STRIDE) break;
      continue;
    }
    const int j = len - c + i;
    const int p = a.page(b, j);
    if (p >= 0 && a.has_row(p, h, j)) {
      const long long dst = a.row(p, h, j) * CPR + chunk;
      a.k[dst] = k;
      a.v[dst] = v;
    }
    if (chunk == 0 && a.has_slot(r, j)) {
      if (a.pos != nullptr) a.pos[a.slot(r, j)] = a.seen[r] - c + i;
      if (a.weight != nullptr) a.weight[a.slot(r, j)] = 0.0f;
    }
    if (!STRIDE) break;
  }
}

// -------------------------------------------------------------------- evict
constexpr int PLAN_BINS = 2048;
constexpr int PLAN_PASSES = 3;              // 11 + 11 + 10 bits of the key
constexpr int PLAN_MAX_KEYS = 44 * 1024;    // keys a CTA holds in shared memory
constexpr int PLAN_UNROLL = 8;
constexpr int PLAN_RANKS = 8;  // CTAs of a cluster, at most

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

// Slots of a range by what becomes of them: equal to the threshold and below /
// from the budget on; given up below it; kept from it on.
struct alignas(16) Tally {
  int tie_below, tie_above, hole, fill;
  // Of the range's ties the first `take` stay (slot order: those below the
  // budget come first): its holes and fills.
  __device__ __forceinline__ int holes(int take) const { return hole + tie_below - min(take, tie_below); }
  __device__ __forceinline__ int fills(int take) const { return fill + take - min(take, tie_below); }
  __device__ __forceinline__ int ties() const { return tie_below + tie_above; }
};

// Moves the n pairs (fill, hole) of row r that one CTA of THREADS threads takes
// at a time, from pair i0 on and then every `step`: a thread each moves position
// and weight, D/8 threads key and value, UNROLL pairs in flight. Sources and
// destinations are disjoint.
template <int D, int THREADS, int UNROLL>
__device__ __forceinline__ void move_pairs(const Args &a, int r, const int *holes, const int *fills, int n, int i0,
                                           int step, int tid) {
  constexpr int CPR = D / 8;
  constexpr int GROUPS = THREADS / CPR, PAIRS = GROUPS * UNROLL;
  static_assert(PAIRS <= THREADS, "a thread for every pair");
  const int b = r / a.H, h = r - b * a.H;
  const int chunk = tid % CPR, group = tid / CPR;
  for (; i0 < n; i0 += step) {
    uint4 k[UNROLL], v[UNROLL];
    long long dst[UNROLL];
    int to = -1, p = 0;
    float w = 0.0f;
    if (tid < PAIRS && i0 + tid < n) {
      to = holes[i0 + tid];
      const int from = fills[i0 + tid];
      if (a.has_slot(r, to) && a.has_slot(r, from)) {
        p = a.pos[a.slot(r, from)];
        w = a.weight[a.slot(r, from)];
      } else {
        to = -1;
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int i = i0 + u * GROUPS + group;
      dst[u] = -1;
      if (i < n) {
        const int into = holes[i], from = fills[i];
        if (!a.has_slot(r, into) || !a.has_slot(r, from)) continue;
        const int pt = a.page(b, into), pf = a.page(b, from);
        if (pt >= 0 && pf >= 0 && a.has_row(pt, h, into) && a.has_row(pf, h, from)) {
          const long long src = a.row(pf, h, from) * CPR + chunk;
          dst[u] = a.row(pt, h, into) * CPR + chunk;
          k[u] = a.k[src];
          v[u] = a.v[src];
        }
      }
    }
    if (to >= 0) {
      a.pos[a.slot(r, to)] = p;
      a.weight[a.slot(r, to)] = w;
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (dst[u] >= 0) {
        a.k[dst[u]] = k[u];
        a.v[dst[u]] = v[u];
      }
  }
}

// What an eviction is asked for, and where its lists go.
struct Evict {
  int budget, recent, sinks;
  int cap;              // pairs a row can have
  int *holes, *fills;   // [rows][cap]
  int *count;           // [rows] pairs that are left to move_kernel
};

// What plans a row: half a CTA of 1024 threads, a CTA, the CTAs of a cluster.
enum : int { BY_HALF, BY_CTA, BY_CLUSTER };
template <int BY>
__device__ __forceinline__ void sync_threads() {  // of a half, or of the CTA
  if (BY == BY_HALF)
    asm volatile("barrier.sync %0, 512;" ::"r"(1 + (int)(threadIdx.x >> 9)) : "memory");
  else
    __syncthreads();
}

// Plans row r, which has len > budget slots: THREADS threads of a CTA, or those
// of a cluster's CTAs, each with an equal range of the slots and their keys in shared
// memory (read once; past key_room they are read again). The budget-th largest
// key is found by radix selection on histograms that every CTA sums up over the
// cluster; one more pass over the keys counts ties, holes (slots given up below
// the budget) and fills (slots kept above it) per warp, and a last one lists
// holes and fills, both in slot order. The length is updated here; how many
// pairs the row has is returned to the first thread of the last CTA's last warp
// (0 to the others). The key reads (8 bytes per slot) are the floor; what bounds
// it is latency: some ten steps that each wait for the one before (and, at
// 25,000 keys to a CTA, the instructions of the five passes over them).
template <int THREADS, int BY>
__device__ __forceinline__ int plan_row(const Args &a, const Evict &ev, int r, int len, unsigned *plan_smem,
                                        int key_room) {
  constexpr int W = THREADS / 32;
  constexpr int PER = PLAN_BINS / THREADS;  // bins of a thread
  constexpr bool CLUSTER = BY == BY_CLUSTER;
  constexpr int MOST = CLUSTER ? PLAN_RANKS : 1;
  constexpr bool ROOM = THREADS == 512;  // for all keys
  constexpr int KEYS = THREADS == 1024 ? 4 : 2;  // keys of a thread read from shared memory at once: what registers hold
  unsigned *hist = plan_smem;                            // [PLAN_PASSES][PLAN_BINS]
  unsigned *keys = plan_smem + PLAN_PASSES * PLAN_BINS;  // [key_room]
  constexpr int HALVES = BY == BY_HALF ? 2 : 1;
  __shared__ int parts[HALVES][W];
  __shared__ Tally tallies[HALVES][W], whole;
  __shared__ unsigned bins[HALVES];
  __shared__ int lefts[HALVES];
  const int half = BY == BY_HALF ? threadIdx.x >> 9 : 0;
  int *part = parts[half];
  Tally *tally = tallies[half];
  unsigned &s_bin = bins[half];
  int &s_left = lefts[half];
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = CLUSTER ? (int)cluster.num_blocks() : 1, rank = CLUSTER ? (int)cluster.block_rank() : 0;
  const int tid = threadIdx.x & (THREADS - 1), lane = tid & 31, warp = tid >> 5;
  if (!a.has_slot(r, 0) || !a.has_slot(r, len - 1)) return 0;  // for all CTAs of the row alike
  const int budget = ev.budget, sinks = ev.sinks, cap = ev.cap, from = a.seen[r] - ev.recent;
  const int seg = ((len + ranks - 1) / ranks + 31) / 32 * 32;
  const int begin = min(len, rank * seg), n = min(len, begin + seg) - begin;
  const int *pos = a.pos + a.slot(r, begin);
  const float *weight = a.weight + a.slot(r, begin);
  auto read_key = [&](int j) { return evict_key(weight[j], pos[j], sinks, from); };
  // KEYS keys of this thread, `step` apart, from first + own on; those past
  // n are read as anything. (512 threads have room for all keys.)
  auto read_keys = [&](unsigned (&k)[KEYS], int first, int own, int step) {
    const bool held = first + KEYS * step <= key_room;
#pragma unroll
    for (int x = 0; x < KEYS; ++x) {
      const int j = first + own + x * step;
      if (ROOM)
        k[x] = j < n ? keys[j] : 0u;
      else if (held)
        k[x] = keys[j];
      else
        k[x] = j >= n ? 0u : (j < key_room ? keys[j] : read_key(j));
    }
  };

  for (int i = tid; i < PLAN_PASSES * PLAN_BINS; i += THREADS) hist[i] = 0;
  sync_threads<BY>();
  for (int j0 = tid; j0 < n; j0 += THREADS * PLAN_UNROLL) {
    float w[PLAN_UNROLL];
    int p[PLAN_UNROLL];
#pragma unroll
    for (int x = 0; x < PLAN_UNROLL; ++x) {
      const int j = j0 + x * THREADS;
      w[x] = j < n ? weight[j] : 0.0f;
      p[x] = j < n ? pos[j] : 0;
    }
#pragma unroll
    for (int x = 0; x < PLAN_UNROLL; ++x) {
      const int j = j0 + x * THREADS;
      if (j < n) {
        const unsigned k = evict_key(w[x], p[x], sinks, from);
        if (ROOM || j < key_room) keys[j] = k;
        atomicAdd(&hist[k >> 21], 1u);
      }
    }
  }
  unsigned threshold = 0;  // its bits found so far
  int left = budget;       // keys still to be taken below the bins passed
  int shift = 21;
  for (int pass = 0; pass < PLAN_PASSES; ++pass) {
    const int bits = pass < 2 ? 11 : 10;
    unsigned *mine = hist + pass * PLAN_BINS;
    if (pass > 0) {
      const int next = shift - bits;
      for (int j0 = 0; j0 < n; j0 += THREADS * KEYS) {
        unsigned k[KEYS];
        read_keys(k, j0, tid, THREADS);
#pragma unroll
        for (int x = 0; x < KEYS; ++x)
          if (j0 + tid + x * THREADS < n && (k[x] >> shift) == threshold)
            atomicAdd(&mine[(k[x] >> next) & ((1u << bits) - 1u)], 1u);
      }
      shift = next;
    }
    if (CLUSTER)
      cluster.sync();
    else
      sync_threads<BY>();
    // the bin, counted from the top, in which the left-th key lies; this
    // thread's bins are PLAN_BINS - 1 - PER tid and the PER - 1 below
    int sum[PER], all = 0;
#pragma unroll
    for (int x = 0; x < PER; ++x) sum[x] = 0;
#pragma unroll
    for (int c = 0; c < MOST; ++c)  // all CTAs' reads on their way at once
      if (c < ranks) {
        const unsigned *theirs = CLUSTER ? cluster.map_shared_rank(mine, c) : mine;
#pragma unroll
        for (int x = 0; x < PER; ++x) sum[x] += (int)theirs[PLAN_BINS - 1 - PER * tid - x];
      }
#pragma unroll
    for (int x = 0; x < PER; ++x) all += sum[x];
    const int upto = warp_scan(all);
    if (lane == 31) part[warp] = upto;
    sync_threads<BY>();
    int before = upto - all + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? part[lane] : 0);
    if (before < left && left <= before + all) {
      int x = 0;
#pragma unroll
      for (int y = 0; y + 1 < PER; ++y)
        if (x == y && left > before + sum[y]) {
          before += sum[y];
          ++x;
        }
      s_bin = (unsigned)(PLAN_BINS - 1 - PER * tid - x);
      s_left = left - before;
    }
    sync_threads<BY>();
    threshold = (threshold << bits) | s_bin;
    left = s_left;
  }
  // keep: above the threshold, and the first `left` of its equals
  const int each = ((n + W - 1) / W + 31) / 32 * 32;  // a warp's slots
  const int lo = min(n, warp * each), hi = min(n, lo + each);
  const int edge = budget - begin;  // first local slot past the budget
  const int mid = max(lo, min(edge, hi));
  auto count_keys = [&](int first, int end, int &equal, int &less) {
    for (int j0 = first; j0 < end; j0 += 32 * KEYS) {
      unsigned k[KEYS];
      read_keys(k, j0, lane, 32);
#pragma unroll
      for (int x = 0; x < KEYS; ++x) {
        const bool in = j0 + lane + 32 * x < end;
        equal += in && k[x] == threshold;
        less += in && k[x] < threshold;
      }
    }
  };
  Tally mine = {0, 0, 0, 0};
  int given_up = 0;  // at and past the budget
  count_keys(lo, mid, mine.tie_below, mine.hole);
  count_keys(mid, hi, mine.tie_above, given_up);
  mine.tie_below = __reduce_add_sync(0xFFFFFFFFu, mine.tie_below);
  mine.tie_above = __reduce_add_sync(0xFFFFFFFFu, mine.tie_above);
  mine.hole = __reduce_add_sync(0xFFFFFFFFu, mine.hole);
  mine.fill = hi - mid - mine.tie_above - __reduce_add_sync(0xFFFFFFFFu, given_up);
  if (lane == 0) tally[warp] = mine;
  sync_threads<BY>();
  if (warp == 0) {
    Tally v = {0, 0, 0, 0};
    if (lane < W) v = tally[lane];
    v.tie_below = __reduce_add_sync(0xFFFFFFFFu, v.tie_below);
    v.tie_above = __reduce_add_sync(0xFFFFFFFFu, v.tie_above);
    v.hole = __reduce_add_sync(0xFFFFFFFFu, v.hole);
    v.fill = __reduce_add_sync(0xFFFFFFFFu, v.fill);
    if (lane == 0) whole = v;
  }
  if (CLUSTER)
    cluster.sync();
  else
    sync_threads<BY>();
  // ties, holes and fills before this warp's range
  int tie = 0, hole = 0, fill = 0;
  auto pass_over = [&](const Tally &v) {  // a lane's each, in the order of the lanes
    const int upto = warp_scan(v.ties());
    const int take = max(0, min(left - tie - (upto - v.ties()), v.ties()));
    hole += __reduce_add_sync(0xFFFFFFFFu, v.holes(take));
    fill += __reduce_add_sync(0xFFFFFFFFu, v.fills(take));
    tie += __shfl_sync(0xFFFFFFFFu, upto, 31);
  };
  if (CLUSTER) {
    Tally v = {0, 0, 0, 0};  // of CTA `lane`
    if (lane < rank) v = *cluster.map_shared_rank(&whole, lane);
    pass_over(v);
  }
  {
    Tally v = {0, 0, 0, 0};  // of warp `lane`
    if (lane < warp) v = tally[lane];
    pass_over(v);
  }
  const unsigned below_lane = (1u << lane) - 1u;
  const bool no_ties = tally[warp].ties() == 0;
  int *hole_list = ev.holes + (long long)r * cap, *fill_list = ev.fills + (long long)r * cap;
  // lists the slots of a range that are kept or given up; how many are listed then
  auto list = [&](int first, int end, bool kept, int *to, int listed) {
    for (int j0 = first; j0 < end; j0 += 32 * KEYS) {
      unsigned k[KEYS];
      bool keep[KEYS];
      read_keys(k, j0, lane, 32);
#pragma unroll
      for (int x = 0; x < KEYS; ++x) keep[x] = k[x] > threshold;
      if (!no_ties)
#pragma unroll
        for (int x = 0; x < KEYS; ++x) {
          const bool equal = j0 + lane + 32 * x < end && k[x] == threshold;
          const unsigned eq = __ballot_sync(0xFFFFFFFFu, equal);
          keep[x] |= equal && tie + __popc(eq & below_lane) < left;
          tie += __popc(eq);
        }
#pragma unroll
      for (int x = 0; x < KEYS; ++x) {
        const int j = j0 + lane + 32 * x;
        const bool is = j < end && keep[x] == kept;
        const unsigned mask = __ballot_sync(0xFFFFFFFFu, is);
        const int at = listed + __popc(mask & below_lane);
        if (is && at < cap) to[at] = begin + j;
        listed += __popc(mask);
      }
    }
    return listed;
  };
  hole = list(lo, mid, false, hole_list, hole);
  fill = list(mid, hi, true, fill_list, fill);
  int pairs = 0;
  if (rank == ranks - 1 && warp == W - 1 && lane == 0) {
    // as many holes as fills: `budget` slots stay in all (and never more than
    // the lists hold)
    pairs = min(min(hole, fill), cap);
    a.lens[r] = budget;
  }
  // the others have read this CTA's memory, and its lists are written
  if (CLUSTER)
    cluster.sync();
  else
    sync_threads<BY>();
  return pairs;
}

// How a row is planned goes by the slots it holds, not by the width of the page
// table, which a caller makes for the longest context it admits: up to
// PLAN_SHORT slots 512 threads (where there are rows enough for that), more than
// those a CTA of 1024, or a cluster.
constexpr int PLAN_SHORT = 4096;

// 512 threads that plan a row also move its pairs where there are PLAN_MOVES at
// most, as in a cache that is cut at every step.
constexpr int PLAN_MOVES = PAGE;
template <int D, int BY>
__device__ __forceinline__ void plan_short_row(const Args &a, const Evict &ev, int r, int len, unsigned *plan_smem,
                                               int key_room) {
  constexpr int HALVES = BY == BY_HALF ? 2 : 1;
  __shared__ int pairs[HALVES];
  const int half = BY == BY_HALF ? threadIdx.x >> 9 : 0, tid = threadIdx.x & 511;
  const int got = plan_row<512, BY>(a, ev, r, len, plan_smem, key_room);
  if (tid == 512 - 32) {
    pairs[half] = got;
    ev.count[r] = got <= PLAN_MOVES ? 0 : got;
  }
  sync_threads<BY>();
  if (pairs[half] <= PLAN_MOVES)
    move_pairs<D, 512, 2>(a, r, ev.holes + (long long)r * ev.cap, ev.fills + (long long)r * ev.cap, pairs[half], 0,
                          512 / (D / 8) * 2, tid);
}

// Under a table of up to PLAN_SHORT slots: a CTA per row.
template <int D>
__global__ void __launch_bounds__(512, 3)
evict_short_kernel(const Args a, const Evict ev, int key_room) {
  extern __shared__ unsigned plan_smem[];
  const int r = blockIdx.x;
  let_next_start();
  wait_for_previous();
  const int len = a.length(r);
  if (len <= ev.budget) {
    if (threadIdx.x == 0) ev.count[r] = 0;
    return;
  }
  plan_short_row<D, BY_CTA>(a, ev, r, len, plan_smem, key_room);
}

// Under a wider one, as many CTAs as run at once. A row is one cluster's, which
// looks its rows up 32 at a time and plans those of more than `alone` slots with
// all of its CTAs, then those of more than `halved` a CTA each, then the others
// half a CTA each. What a warp finds is left in shared memory (held in registers
// it made the plan spill: 134 us at 40 rows of 75,600 slots became 144).
template <int D>
__global__ void __launch_bounds__(1024, 1)
evict_long_kernel(const Args a, const Evict ev, int halved, int alone, int key_room) {
  extern __shared__ unsigned plan_smem[];
  __shared__ int s_row[3][32], s_len[3][32], s_found[3];
  __shared__ long long s_first;
  namespace cg = cooperative_groups;
  let_next_start();
  wait_for_previous();
  if (threadIdx.x == 0) s_first = blockIdx.x / cg::this_cluster().num_blocks();
  while (true) {
    __syncthreads();
    const long long first = s_first;
    if (first >= a.B * a.H) break;
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x, ranks = (int)cg::this_cluster().num_blocks(), clusters = (int)gridDim.x / ranks;
      const long long mine = first + (long long)lane * clusters;
      const int len = mine < a.B * a.H ? a.length((int)mine) : -1;
      const bool cut = len > ev.budget;
      if (mine < a.B * a.H && !cut && cg::this_cluster().block_rank() == 0) ev.count[mine] = 0;
      const int kind = len <= halved ? BY_HALF : (len <= alone ? BY_CTA : BY_CLUSTER);
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const unsigned some = __ballot_sync(0xFFFFFFFFu, cut && kind == k);
        const int at = __popc(some & ((1u << lane) - 1u));
        if (cut && kind == k) {
          s_row[k][at] = (int)mine;
          s_len[k][at] = len;
        }
        if (lane == 0) s_found[k] = __popc(some);
      }
    }
    // all CTAs have read the lengths before any plan changes one
    if (cg::this_cluster().num_blocks() > 1)
      cg::this_cluster().sync();
    else
      __syncthreads();
    // (everyone has read it, and reads it again behind the next barrier)
    if (threadIdx.x == 0) s_first = first + 32LL * (gridDim.x / cg::this_cluster().num_blocks());
    if (cg::this_cluster().num_blocks() > 1)
      for (int i = 0; i < s_found[BY_CLUSTER]; ++i) {
        const int got =
            plan_row<1024, BY_CLUSTER>(a, ev, s_row[BY_CLUSTER][i], s_len[BY_CLUSTER][i], plan_smem, key_room);
        if (threadIdx.x == 1024 - 32 && cg::this_cluster().block_rank() + 1 == cg::this_cluster().num_blocks())
          ev.count[s_row[BY_CLUSTER][i]] = got;
      }
    for (int i = (int)cg::this_cluster().block_rank(); i < s_found[BY_CTA];
         i += (int)cg::this_cluster().num_blocks()) {
      const int got = plan_row<1024, BY_CTA>(a, ev, s_row[BY_CTA][i], s_len[BY_CTA][i], plan_smem, key_room);
      if (threadIdx.x == 1024 - 32) ev.count[s_row[BY_CTA][i]] = got;
    }
    for (int i = 2 * (int)cg::this_cluster().block_rank() + (int)(threadIdx.x >> 9); i < s_found[BY_HALF];
         i += 2 * (int)cg::this_cluster().num_blocks())
      plan_short_row<D, BY_HALF>(a, ev, s_row[BY_HALF][i], s_len[BY_HALF][i],
                                 plan_smem + (threadIdx.x >> 9) * (PLAN_PASSES * PLAN_BINS + PLAN_SHORT), PLAN_SHORT);
  }
}

constexpr int MOVE_THREADS = 128;
constexpr int MOVE_UNROLL = 3;
// Pairs one CTA of move_kernel<D> takes at a time.
template <int D>
__host__ __device__ constexpr int move_share() {
  return MOVE_THREADS / (D / 8) * MOVE_UNROLL;
}

// grid.x = row, grid.y strides over its pairs.
template <int D>
__global__ void __launch_bounds__(MOVE_THREADS)
move_kernel(const Args a, int cap, const int *holes, const int *fills, const int *count) {
  let_next_start();
  wait_for_previous();
  const int r = blockIdx.x;
  move_pairs<D, MOVE_THREADS, MOVE_UNROLL>(a, r, holes + (long long)r * cap, fills + (long long)r * cap, count[r],
                                           (int)blockIdx.y * move_share<D>(), (int)gridDim.y * move_share<D>(),
                                           (int)threadIdx.x);
}

}  // namespace cache
}  // namespace sta
