// Attention of a sequence's newest tokens over its paged key-value cache.
//
//   row r = (b, h): one key head; its M = n_q * group query rows, row
//   m = i * group + g being token i of query head h * group + g
//   s_j = scale q_m . k_j,  o_m = sum_j e^(s_j - lse_m) v_j
// over the slots j that token i sees: all but those of the n_q - 1 - i newest
// tokens, which go by their positions where the cache keeps them. A producer
// then reads the positions (4 bytes a slot) of the pages it looks up, a lane a
// page's, and marks the few pieces that hold a token newer than the oldest
// query; only in those (and where a row ends) the warps mask scores.
//
// Every key and value is read once and used by the M <= 64 query rows of its
// head: at most 64 flop per byte, so HBM is the floor. The matrix products are
// mma.sync tiles with the keys (or the values' columns) along the 16 rows and 8
// query rows across: S^T = K Q^T, O^T = V^T P^T. Up to 16 query rows that keeps
// up with HBM (tensor pipe 15% busy). With 17 to 64 the warps wait for their own
// products instead (a quarter to a third of HBM's rate); tcgen05 tiles, 128
// keys by the query rows, would fit there and have not been built.
//
// attend_kernel: one CTA per SM, 7 or 8 warps. A worker is a warp (for many
// query rows two or four, see rows_per_warp) with a ring of its own in shared
// memory, into which its first warp sends half pages (TMA, 128-byte swizzle)
// ahead of their use. The pages to be read, rows one after another, are cut
// into one equal chunk per worker whatever the lengths are: no worker waits for
// a long sequence, or for another where a row ends. Each warp keeps the running
// maximum and sum and the outputs of its query rows in registers; rows cut by a
// chunk border leave their parts (the sum relative to a maximum) in the
// workspace.
// join_kernel: joins those parts.
// Short rows (attend_kernel with CLUSTER): a cluster of CTAs per row, whose
// workers share its pages and are joined through distributed shared memory; no
// other kernel, and no part leaves the SMs.
// weigh_kernel: adds every slot's attention to its weight now that the rows'
// log-sum-exps are known, from the scores that attend_kernel left (4 bytes per
// slot and query row against 4 d for its key and value).
#pragma once
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "sta_cache.cuh"
#include "sta_tc.cuh"

namespace sta {
namespace decode {

using cache::Args;
using cache::PAGE;

constexpr int MAX_CTAS = 148;  // one per SM of a B200
constexpr int MAX_WARPS = 8;
constexpr int MAX_ROWS = 64;  // query rows per key head
constexpr int KEYS = 32;      // slots of a stage of the ring
constexpr int KT = KEYS / 16;
constexpr int HALF_BYTES = KEYS * 128;  // 64 values of every slot
constexpr int MAX_STAGES = 28;          // of all workers
constexpr int JOIN_BATCH = 4;
constexpr long long DRAIN_LIMIT = 200000000LL;

// Query rows that a warp has: 16, and 32 at d = 64, where their outputs fit in
// its registers. The keys and values are then read from shared memory by half
// as many warps (8 sequences of 8,192 tokens, 8 key heads: with 20 query rows
// 50 us, with 48 76 us; with 16 rows a warp 56 and 99).
__host__ __device__ constexpr int rows_per_warp(int d, int M) { return d == 64 && M > 16 ? 32 : 16; }
// Warps of a worker, workers of a CTA, stages of a worker's ring (16 KB at d =
// 128, 8 at d = 64). Seven workers of one warp have 32 KB each: what shared
// memory holds.
__host__ __device__ inline int tiles_of(int d, int M) {
  const int warps = (M + rows_per_warp(d, M) - 1) / rows_per_warp(d, M);
  return warps <= 2 ? warps : 4;
}
__host__ __device__ inline int workers_of(int d, int M) {
  const int tiles = tiles_of(d, M);
  return tiles == 1 ? 7 : 8 / tiles;
}
__host__ __device__ inline int stages_of(int d, int M) {
  const int tiles = tiles_of(d, M);
  return (tiles == 1 ? 2 : 3 * tiles / 2) * (128 / d);
}
inline int warps_of(int d, int M) { return tiles_of(d, M) * workers_of(d, M); }

template <int D>
struct Cfg {
  static constexpr int TILE_BYTES = HALF_BYTES * (D / 64);  // keys or values of a stage
  static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
  static int smem(int M) { return 1024 + workers_of(D, M) * stages_of(D, M) * STAGE_BYTES; }
  static int most_smem() { return smem(1); }  // seven workers of one warp
};

struct Shape {
  int group, n_q;                  // query heads per key head, newest tokens
  const int *page_ptr, *page_idx;  // page lists (CSR), or NULL
  long long idx_capacity;
  float scale_log2;  // scale * log2 e
  // Which of the n_q newest tokens a slot holds: with more than one of them, by
  // its position where positions are kept (an eviction moves the newest tokens
  // into slots of any number), else by its slot.
  bool by_position;
};
// How much newer than the oldest query a token is, given its position (or slot)
// and the end of these (tokens seen, or slots filled): query i sees the tokens
// up to i. The newest query sees every filled slot.
__device__ __forceinline__ int newness(int n_q, int at, int end) {
  return min((int)((unsigned)at - (unsigned)end) + n_q, n_q - 1);
}

struct Work {
  float *part_o;      // [2 * chunks][M][D]
  float2 *part_ml;    // [2 * chunks][M] maximum (log2) and sum
  int2 *row_units;    // [rows] unit of the first page and pages of a row in parts; pages 0: not in parts
  cache::Chunks *chunks;
  // for weigh_kernel (else NULL)
  int2 *units;        // [units] row, and packed column and filled slots, of a page; else -1
  float *scores;      // [units][M][PAGE] s_j log2 e, -inf out of view
  float *lse2;        // [rows][M] log-sum-exp (log2)
  // (checked build) parts there is room for, units (0 without weights), rows
  int part_room, unit_room, row_room;
  __device__ __forceinline__ bool has_part(int part) const { return dbg_ok(part >= 0 && part < part_room); }
  __device__ __forceinline__ bool has_unit(int unit) const { return dbg_ok(unit >= 0 && unit < unit_room); }
  __device__ __forceinline__ bool has_row(int r) const { return dbg_ok(r >= 0 && r < row_room); }
};

// A page's column (below 2^24) and its filled slots (1 to PAGE).
__device__ __forceinline__ int pack_page(int col, int held) { return col | (min(held, PAGE) - 1) << 24; }

// What a worker's warps are told of a stage.
enum : int { FIRST = 1, LAST = 2, WHOLE = 4, BEGINS = 8, SKIP = 16, END = 32, UPPER = 64, NEWER = 128 };
constexpr int COLUMN = 8;  // flags' bits from here on: the page's column (below 2^24)
struct __align__(16) Piece {
  int row, unit;
  int held;   // filled slots from the piece's first on (may be above KEYS)
  int flags;  // UPPER: the page's second half; NEWER: a slot is newer, by position, than the oldest query
  // the piece's first slot
  __device__ __forceinline__ int slot() const {
    return (int)((unsigned)flags >> COLUMN) * PAGE + (flags & UPPER ? KEYS : 0);
  }
};

// ------------------------------------------------------------ element types
template <typename T>
struct Num;
template <>
struct Num<__nv_bfloat16> {
  // p is at most 1
  static constexpr float SHIFT = 0.0f;
  static constexpr uint32_t NONFINITE = 0x7F80u;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return tc::pack_bf16(lo, hi); }
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  }
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Num<__half> {
  // p is scaled to at most 2^14 (the sum with it): fp16's smallest step is
  // 2^-24, so the second of a weight's two terms is off by up to 2^-25, which
  // is 2^-39 of the largest weight (more than 2^-22 of those below 2^-17 of it)
  static constexpr float SHIFT = 14.0f;
  static constexpr uint32_t NONFINITE = 0x7C00u;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
  }
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

__device__ __forceinline__ void ldmatrix(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Transposes an 8 x 8 matrix of 2-byte elements held two to a register.
__device__ __forceinline__ uint32_t transpose(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(v));
  return r;
}

// Bounded wait, as tc::mbar_wait. A thread that try_wait has suspended is not
// woken by a short limit (on a B200 not within the 5 us of the longest wait
// here, whatever the hint), so under a limit of less than some milliseconds the
// barrier is polled.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile uint32_t *abort, long long limit) {
  const bool sleep = limit >= 4LL * STA_WAIT_SLEEP_NS;
  auto done = [&]() {
    if (sleep) return tc::mbar_try_wait_sleep(bar, parity, STA_WAIT_SLEEP_NS);
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0u;
  };
  if (done()) return true;
  const long long t0 = clock64();
  while (true) {
    if (done()) return true;
    if (*abort) return false;
    if (clock64() - t0 > limit) {
      *abort = 1u;
      record_error(DEV_ERR_TIMEOUT);
      return false;
    }
  }
}

// ------------------------------------------------------------------- rows
struct RowPages {
  int len, n, first;  // length, pages attended to, first entry of its list
};
// (first, next: the row's offsets, where there are lists)
__device__ __forceinline__ RowPages row_pages(const Args &a, const Shape &s, int len, int first, int next) {
  RowPages p;
  p.len = a.checked_length(len);
  p.n = cache::filled_pages(p.len);
  p.first = 0;
  if (s.page_ptr != nullptr) {
    if (!cache::list_ok(first, next, s.idx_capacity, a.max_pages)) {
      record_error(DEV_ERR_BAD_MASK);
      p.n = 0;
    } else {
      p.first = first;
      p.n = p.len >= 0 ? next - first : 0;
    }
  }
  return p;
}
__device__ __forceinline__ RowPages row_pages(const Args &a, const Shape &s, int r) {
  const bool lists = s.page_ptr != nullptr;
  return row_pages(a, s, a.lens[r], lists ? s.page_ptr[r] : 0, lists ? s.page_ptr[r + 1] : 0);
}

// --------------------------------------------------------------- producer
// The next two are calls: few of the kernel's calls need them, and their code
// in line makes it start later behind other kernels (5 us in a step of 384 rows
// of 1,300 slots).

// Which halves of a page with `held` slots hold a token newer than the oldest
// query: NEWER the lower, UPPER the upper.
__device__ __noinline__ int newer_halves(const int *pos, int end, int n_q, int held) {
  int halves = 0;
  auto look = [&](int j, int at) {
    if (j < held && newness(n_q, at, end) > 0) halves |= j < KEYS ? NEWER : UPPER;
  };
  if ((reinterpret_cast<uintptr_t>(pos) & 15u) == 0) {
#pragma unroll 8
    for (int j = 0; j < PAGE; j += 4) {
      const int4 at = *reinterpret_cast<const int4 *>(pos + j);
      look(j, at.x);
      look(j + 1, at.y);
      look(j + 2, at.z);
      look(j + 3, at.w);
    }
  } else {
#pragma unroll 4
    for (int j = 0; j < PAGE; ++j) look(j, pos[j]);
  }
  return halves;
}

// The largest of a list's first n entries, for the whole warp; -1: none.
__device__ __noinline__ int largest_entry(const int *list, int n) {
  constexpr int UNROLL = 8;
  int v = -1;
  for (int j = threadIdx.x & 31; j < n; j += 32 * UNROLL) {
    int e[UNROLL];
#pragma unroll
    for (int x = 0; x < UNROLL; ++x) e[x] = j + 32 * x < n ? list[j + 32 * x] : -1;
#pragma unroll
    for (int x = 0; x < UNROLL; ++x) v = max(v, e[x]);
  }
  return __reduce_max_sync(0xFFFFFFFFu, v);
}

// The first warp of a worker sends its pieces: 32 units at a time a lane each
// finds its unit's row, column and page; the lanes then send them in order.
template <int D>
struct Producer {
  using C = Cfg<D>;
  uint8_t *ring;
  uint64_t *full, *empty;
  Piece *piece;
  int stages;
  int row, off;   // a row and the next unit to be looked up, counted from the row's first
  int u, u0, u1;  // that unit, the chunk's range
  int issued;     // stages sent
  bool ended, ok;
  // this lane's unit of the batch at hand
  int w_row, w_unit, w_held, w_flags, w_y;
  unsigned left;  // lanes of the batch still to be sent
  int upper;      // 1: the first of them has its lower half sent
  int top;        // the largest entry before the next unit's in its row's list

  // Looks up the next units of the chunk, 32 at most.
  __device__ __forceinline__ void batch(const Args &a, const Shape &s, int rows, const Work &work) {
    static_assert(cache::ROW_COST == 1, "what is the chunk's last page");
    const int lane = threadIdx.x & 31;
    const int r0 = row + lane;
    RowPages mine = {0, 0, 0};
    if (r0 < rows) mine = row_pages(a, s, r0);
    const int upto = cache::warp_scan(cache::row_units(mine.n));
    const int total = __shfl_sync(0xFFFFFFFFu, upto, 31);
    left = 0;
    upper = 0;
    if (off >= total) {  // not in these 32 rows
      row += 32;
      off -= total;
      return;
    }
    const int take = min(min(total - off, u1 - u), 32), at = off + lane;
    int k = 0;  // the row of this lane's unit: the first with upto > at
#pragma unroll
    for (int step = 16; step > 0; step >>= 1)
      if (__shfl_sync(0xFFFFFFFFu, upto, k + step - 1) <= at) k += step;
    const int n = __shfl_sync(0xFFFFFFFFu, mine.n, k), first = __shfl_sync(0xFFFFFFFFu, mine.first, k);
    const int len = __shfl_sync(0xFFFFFFFFu, mine.len, k), end = __shfl_sync(0xFFFFFFFFu, upto, k);
    const int i = n - (end - at);  // the row's i-th page; negative: the row's own unit
    const bool page_unit = lane < take && i >= 0;
    int entry = i, before = -1;  // of the row's list, the largest before it
    if (s.page_ptr != nullptr) {
      if (page_unit) entry = s.page_idx[first + i];
      if (u == u0) top = largest_entry(s.page_idx + __shfl_sync(0xFFFFFFFFu, first, 0), __shfl_sync(0xFFFFFFFFu, i, 0));
      // the lanes before this one hold the entries before its own, up to the
      // row's first or (i > lane) the batch's
      int upto = page_unit ? entry : -1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o && i >= o) upto = max(upto, x);
      }
      if (i > lane) upto = max(upto, top);
      const int x = __shfl_up_sync(0xFFFFFFFFu, upto, 1);
      if (i > 0) before = lane > 0 ? x : top;
      top = __shfl_sync(0xFFFFFFFFu, upto, take - 1);
    }
    w_row = row + k;
    w_unit = u + lane;
    w_y = w_held = w_flags = 0;
    int col = -1;
    if (page_unit) {
      const int b = w_row / a.H, h = w_row - b * a.H, start = w_unit - i;
      col = entry;
      if (s.page_ptr != nullptr && !cache::column_ok(entry, before, cache::filled_pages(len))) {
        record_error(DEV_ERR_BAD_MASK);
        col = -1;
      }
      int page = -1, newer = 0;
      if (col >= 0) {
        // (both on their way at once)
        const int given = a.table[(long long)b * a.max_pages + col];
        if (s.by_position && a.has_slot(w_row, col * PAGE))
          newer = newer_halves(a.pos + a.slot(w_row, col * PAGE), a.seen[w_row], s.n_q, len - col * PAGE);
        page = a.checked_page(given);
      }
      if (page >= 0) {
        w_y = (page * a.H + h) * PAGE;
        w_held = len - col * PAGE;
        w_flags = (int)((unsigned)col << COLUMN) | newer;
      } else {
        col = -1;
        w_flags = SKIP;
      }
      const bool begins = start >= u0;
      if (i == 0 || w_unit == u0) w_flags |= FIRST;
      if (i == n - 1 || w_unit == u1 - 1) w_flags |= LAST;
      // a row's own unit follows its last page, if anything does
      if (w_unit == u1 - 1 || (i == n - 1 && w_unit == u1 - 2)) w_flags |= END;
      if (begins) w_flags |= BEGINS;
      if (begins && start + n <= u1) w_flags |= WHOLE;
      if (i == 0 && work.row_units != nullptr && work.has_row(w_row))
        work.row_units[w_row] = make_int2(start, w_flags & WHOLE ? 0 : n);
    }
    if (work.units != nullptr && lane < take && work.has_unit(w_unit))
      work.units[w_unit] = col >= 0 ? make_int2(w_row, pack_page(col, w_held)) : make_int2(-1, -1);
    left = __ballot_sync(0xFFFFFFFFu, page_unit);
    // the unit after these, counted from the last one's row
    const int lk = __shfl_sync(0xFFFFFFFFu, k, take - 1), le = __shfl_sync(0xFFFFFFFFu, end, take - 1);
    const int ln = __shfl_sync(0xFFFFFFFFu, n, take - 1);
    u += take;
    off += take - (le - cache::row_units(ln));
    row += lk;
  }

  // Looks up units until there is a page among them.
  __device__ __forceinline__ void find(const Args &a, const Shape &s, int rows, const Work &work) {
    while (left == 0 && u < u1 && row < rows) batch(a, s, rows, work);
  }

  // Sends the next piece; where a chunk has no page, just the end.
  __device__ __forceinline__ void send(const CUtensorMap &tk, const CUtensorMap &tv, const Args &a, const Shape &s,
                                       int rows, const Work &work, volatile uint32_t *abort, long long limit) {
    const int lane = threadIdx.x & 31, stage = issued % stages;
    const bool none = left == 0;
    const int x = none ? 0 : __ffs(left) - 1;
    int state = 0;
    if (lane == x) {
      const bool last = none || (w_flags & SKIP) || upper || w_held <= KEYS;
      int flags = none ? (SKIP | END) : w_flags;
      if (upper)  // (w_flags has UPPER where the upper half holds a newer token)
        flags = (flags & ~(FIRST | NEWER)) | UPPER | (flags & UPPER ? NEWER : 0);
      else
        flags &= ~UPPER;
      if (!last) flags &= ~(LAST | END);
      const int y = w_y + upper * KEYS;
      if (!(flags & SKIP) && !dbg_ok(y >= 0 && y <= (a.num_pages * a.H - 1) * PAGE + KEYS && (y & (KEYS - 1)) == 0))
        flags |= SKIP;
      if (issued < stages || wait(&empty[stage], ((issued / stages) & 1) ^ 1, abort, limit)) {
        piece[stage] = Piece{w_row, w_unit, w_held - upper * KEYS, flags};
        if (flags & SKIP) {
          tc::mbar_arrive(&full[stage]);
        } else {
          const uint32_t dst = tc::smem_u32(ring + stage * C::STAGE_BYTES);
          tc::mbar_expect_tx(&full[stage], C::STAGE_BYTES);
#pragma unroll
          for (int e = 0; e < D / 64; ++e) tc::tma_load_2d(dst + e * HALF_BYTES, &tk, &full[stage], 64 * e, y);
#pragma unroll
          for (int e = 0; e < D / 64; ++e)
            tc::tma_load_2d(dst + C::TILE_BYTES + e * HALF_BYTES, &tv, &full[stage], 64 * e, y);
        }
        state = 1 | (last ? 2 : 0) | (flags & END);
      }
    }
    state = __shfl_sync(0xFFFFFFFFu, state, x);
    ok = state != 0;
    ended = state & END;
    if (ok) ++issued;
    if (state & 2) {
      upper = 0;
      left &= left - 1;
      find(a, s, rows, work);  // while what was sent is on its way
    } else {
      upper = 1;
    }
  }
};

// --------------------------------------------------------------- consumers
// 8 NT query rows of one warp (NT: 1, 2 or 4). Thread (g, t) = (lane / 4,
// lane % 4) holds, of query rows 8 n + 2 t + y (y = 0, 1): o[c][n][y + 2 x], their outputs
// 16 c + g + 8 x; the running maximum (log2); its share of the sum.
template <int D, int NT>
struct Tile {
  float o[D / 16][NT][4];
  float top[NT][2], sum[NT][2];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[c][n][0] = o[c][n][1] = o[c][n][2] = o[c][n][3] = 0.0f;
      top[n][0] = top[n][1] = -INFINITY;
      sum[n][0] = sum[n][1] = 0.0f;
    }
  }
};

// Query rows m0 .. m0 + 8 NT - 1 as the B operand of D / 16 steps (rows past M:
// zero).
template <int D, int NT, typename T>
__device__ __forceinline__ void load_queries(const T *q, const Args &a, const Shape &s, int r, int m0,
                                             uint32_t (&qb)[NT][D / 16][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int b = r / a.H, h = r - b * a.H;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int m = m0 + 8 * n + g;
    const bool in = m < s.group * s.n_q;
    const int i = in ? m / s.group : 0, hg = in ? m - i * s.group : 0;
    const uint32_t *row = reinterpret_cast<const uint32_t *>(
        q + (((long long)b * s.n_q + i) * (a.H * s.group) + h * s.group + hg) * D);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      qb[n][ks][0] = in ? row[ks * 8 + t] : 0u;
      qb[n][ks][1] = in ? row[ks * 8 + 4 + t] : 0u;
    }
  }
}

// Where a lane's ldmatrix rows lie in a stage (128-byte swizzle: 16-byte piece c
// of slot j is at piece c ^ (j % 8) of its 128 bytes), for pieces 2 j, 2 j + 1.
struct Lanes {
  uint32_t k[4], v[4];
  template <int D>
  __device__ __forceinline__ void init() {
    const int lane = threadIdx.x & 31, l7 = lane & 7, m8 = lane >> 3;  // row l7 of matrix m8
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // A = K: matrices (slots 0..7, 8..15) x (pieces 2 j, 2 j + 1)
      k[j] = (l7 + (m8 & 1) * 8) * 128 + (((m8 >> 1) ^ l7 ^ (2 * j)) << 4);
      // A = V^T: matrices (pieces 2 j, 2 j + 1) x (slots 0..7, 8..15)
      v[j] = Cfg<D>::TILE_BYTES + (l7 + (m8 >> 1) * 8) * 128 + (((m8 & 1) ^ l7 ^ (2 * j)) << 4);
    }
  }
};

// One stage: scores, softmax step, weighted values. token[n][y]: the token (of
// the n_q newest) that query row 8 n + 2 t + y is; held: how many of its slots
// are filled (may be above KEYS). EDGE: some slot is not filled, or newer than
// the oldest query; newer: of slot `lane` how much newer (newness; n_q: not
// filled). scores: where query row 0's scores go (MASS), of which the warp has
// `rows` rows.
template <int D, int NT, typename T, bool MASS, bool EDGE>
__device__ __forceinline__ void attend_slots(uint32_t stage, const Lanes &lanes, const uint32_t (&qb)[NT][D / 16][2],
                                             const Shape &s, const int (&token)[NT][2], int held, int newer,
                                             Tile<D, NT> &acc, float *scores, int rows) {
  using N = Num<T>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  int slot_newer[KT][2];  // of slots 16 x + g + 8 y
  if (EDGE)
#pragma unroll
    for (int x = 0; x < KT; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) slot_newer[x][y] = __shfl_sync(0xFFFFFFFFu, newer, 16 * x + g + 8 * y);
  float p[KT][NT][4];
#pragma unroll
  for (int x = 0; x < KT; ++x)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) p[x][n][e] = 0.0f;
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
    for (int x = 0; x < KT; ++x) {
      uint32_t ka[4];
      ldmatrix(stage + lanes.k[ks & 3] + x * 2048 + (ks >> 2) * HALF_BYTES, ka);
#pragma unroll
      for (int n = 0; n < NT; ++n) N::mma(p[x][n], ka, qb[n][ks][0], qb[n][ks][1]);
    }
#pragma unroll
  for (int x = 0; x < KT; ++x)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p[x][n][e] = __fmul_rn(p[x][n][e], s.scale_log2);  // the score that is kept, with or without MASS
        if (EDGE && slot_newer[x][e >> 1] > token[n][e & 1]) p[x][n][e] = -INFINITY;
      }
  if (MASS) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (const int m = 8 * n + 2 * t + (e & 1); m < rows)
#pragma unroll
          for (int x = 0; x < KT; ++x) scores[m * PAGE + 16 * x + g + 8 * (e >> 1)] = p[x][n][e];
  }
  float keep[NT][2];
  bool grown = false;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float up = acc.top[n][y];
#pragma unroll
      for (int x = 0; x < KT; ++x) up = tc::fmax3(up, p[x][n][y], p[x][n][y + 2]);
      up = fmaxf(up, __shfl_xor_sync(0xFFFFFFFFu, up, 4));
      up = fmaxf(up, __shfl_xor_sync(0xFFFFFFFFu, up, 8));
      up = fmaxf(up, __shfl_xor_sync(0xFFFFFFFFu, up, 16));
      const float from = up == -INFINITY ? 0.0f : up;  // a row that has seen nothing yet
      keep[n][y] = tc::ex2(acc.top[n][y] - from);
      grown |= keep[n][y] != 1.0f;
      acc.top[n][y] = up;
      const float base = from - N::SHIFT;
      float z = 0.0f;
#pragma unroll
      for (int x = 0; x < KT; ++x) {
        p[x][n][y] = tc::ex2(p[x][n][y] - base);
        p[x][n][y + 2] = tc::ex2(p[x][n][y + 2] - base);
        z += p[x][n][y] + p[x][n][y + 2];
      }
      acc.sum[n][y] = acc.sum[n][y] * keep[n][y] + z;
    }
  if (__any_sync(0xFFFFFFFFu, grown)) {
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc.o[c][n][e] *= keep[n][e & 1];
  }
  // Values of slots that are not seen must not reach the products even with a
  // weight of 0 (0 * inf): those of slots >= held are cleared. A slot that only
  // the newer of the n_q tokens see is cleared where it is not finite, and what
  // is not finite added by hand for those who see it.
  auto finite = [](uint32_t v) {
    return ((v & N::NONFINITE) == N::NONFINITE ? 0u : v & 0xFFFFu) |
           ((v >> 16 & N::NONFINITE) == N::NONFINITE ? 0u : v & 0xFFFF0000u);
  };
  auto value = [&](int key, int d) {  // of slot `key`, in the low half
    uint32_t v;
    asm volatile("ld.shared.u16 %0, [%1];"
                 : "=r"(v)
                 : "r"(stage + Cfg<D>::TILE_BYTES + (d >> 6) * HALF_BYTES + key * 128 +
                       ((((d & 63) >> 3) ^ (key & 7)) << 4) + (d & 7) * 2));
    return v;
  };
  bool odd = false;
  if (EDGE && s.n_q > 1) {
    for (unsigned some = __ballot_sync(0xFFFFFFFFu, newer > 0 && newer < s.n_q); some != 0; some &= some - 1)
      for (int d = lane; d < D; d += 32) odd |= (value(__ffs(some) - 1, d) & N::NONFINITE) == N::NONFINITE;
    odd = __any_sync(0xFFFFFFFFu, odd);
  }
#pragma unroll
  for (int x = 0; x < KT; ++x) {
    // the weights of 16 slots as the B operand, split in two terms: one alone
    // would be off by as much as the output's own rounding
    uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float p0 = p[x][n][2 * e], p1 = p[x][n][2 * e + 1];
        const uint32_t v = N::pack(p0, p1);
        const float2 r = N::unpack(v);
        hi[n][e] = transpose(v);
        lo[n][e] = transpose(N::pack(p0 - r.x, p1 - r.y));
      }
    auto below = [&](int key) { return key + 1 < held ? 0xFFFFFFFFu : (key < held ? 0xFFFFu : 0u); };
    uint32_t m0 = 0, m1 = 0;
    if (EDGE) {
      m0 = below(16 * x + 2 * t);
      m1 = below(16 * x + 8 + 2 * t);
    }
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      uint32_t va[4];
      ldmatrix_trans(stage + lanes.v[c & 3] + x * 2048 + (c >> 2) * HALF_BYTES, va);
      if (EDGE) {
        va[0] &= m0;
        va[1] &= m0;
        va[2] &= m1;
        va[3] &= m1;
        if (odd) {
#pragma unroll
          for (int e = 0; e < 4; ++e) va[e] = finite(va[e]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) N::mma(acc.o[c][n], va, hi[n][0], hi[n][1]);
#pragma unroll
      for (int n = 0; n < NT; ++n) N::mma(acc.o[c][n], va, lo[n][0], lo[n][1]);
    }
  }
  if (EDGE && odd)
    for (int key = 0; key < min(KEYS, held); ++key) {
      const int key_newer = __shfl_sync(0xFFFFFFFFu, newer, key);
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t v = value(key, 16 * c + g + 8 * x);
          if ((v & N::NONFINITE) == N::NONFINITE)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int y = 0; y < 2; ++y)
                if (key_newer <= token[n][y]) acc.o[c][n][y + 2 * x] += N::unpack(v).x;
        }
    }
}

// Where row m of row r's result goes.
template <int D, typename T>
struct Sink {
  T *o;
  float *lse;
  __device__ __forceinline__ long long row(const Args &a, const Shape &s, int r, int m) const {
    const int b = r / a.H, h = r - b * a.H, i = m / s.group, g = m - i * s.group;
    return ((long long)b * s.n_q + i) * (a.H * s.group) + h * s.group + g;
  }
  // a row that sees nothing: o = 0, lse = -inf (one thread)
  __device__ __forceinline__ void put_nothing(const Args &a, const Shape &s, int r) const {
    for (int m = 0; m < s.group * s.n_q; ++m) {
      for (int c = 0; c < D / 8; ++c)
        reinterpret_cast<uint4 *>(o + row(a, s, r, m) * D)[c] = make_uint4(0u, 0u, 0u, 0u);
      put_lse(a, s, r, m, -INFINITY);
    }
  }
  // y: log-sum-exp (log2)
  __device__ __forceinline__ void put_lse(const Args &a, const Shape &s, int r, int m, float y) const {
    const int b = r / a.H, h = r - b * a.H, i = m / s.group, g = m - i * s.group;
    if (lse != nullptr)
      lse[((long long)b * (a.H * s.group) + h * s.group + g) * s.n_q + i] = y * 0.69314718055994530942f;
  }
};

// A part of a row's sum: the weights' maximum (log2) and sum, four outputs. A
// sum of 0 is nothing.
struct Part {
  float top, sum;
  float4 o;
  __device__ __forceinline__ void add(const Part &p) {
    if (p.sum == 0.0f) return;
    const float up = sum == 0.0f ? p.top : fmaxf(top, p.top);
    const float x = sum == 0.0f ? 0.0f : tc::ex2(top - up), y = tc::ex2(p.top - up);
    top = up;
    sum = sum * x + p.sum * y;
    o.x = o.x * x + p.o.x * y;
    o.y = o.y * x + p.o.y * y;
    o.z = o.z * x + p.o.z * y;
    o.w = o.w * x + p.o.w * y;
  }
};

__device__ __forceinline__ Part shuffled(const Part &v, int d) {
  Part p;
  p.top = __shfl_xor_sync(0xFFFFFFFFu, v.top, d);
  p.sum = __shfl_xor_sync(0xFFFFFFFFu, v.sum, d);
  p.o.x = __shfl_xor_sync(0xFFFFFFFFu, v.o.x, d);
  p.o.y = __shfl_xor_sync(0xFFFFFFFFu, v.o.y, d);
  p.o.z = __shfl_xor_sync(0xFFFFFFFFu, v.o.z, d);
  p.o.w = __shfl_xor_sync(0xFFFFFFFFu, v.o.w, d);
  return p;
}

// CLUSTER: grid.x = rows x CTAs of a cluster.
template <int D, int NT, typename T, bool MASS, bool CLUSTER>
__global__ void __launch_bounds__(32 * MAX_WARPS, 1)
attend_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const Args a,
              const Shape s, const T *__restrict__ q, const Sink<D, T> sink, const Work work, long long limit) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[MAX_STAGES], empty[MAX_STAGES];  // worker after worker
  __shared__ Piece pieces[MAX_STAGES];
  __shared__ int warp_units[MAX_WARPS];
  __shared__ int row_before[32 * MAX_WARPS];  // units before the rows of each thread
  __shared__ uint32_t abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rows = a.B * a.H, M = s.group * s.n_q;
  const int tiles = tiles_of(D, M), workers = workers_of(D, M), stages = stages_of(D, M);
  const int threads = blockDim.x;
  const int wk = warp / tiles, mt = warp % tiles, g = lane >> 2, t = lane & 3;
  cache::let_next_start();
  if (tid < workers * stages) {
    tc::mbar_init(&full[tid], 1);
    tc::mbar_init(&empty[tid], tiles);
    tc::fence_barrier_init();
  }
  if (tid == 0) {
    abort = 0u;
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tk) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tv) : "memory");
  }
  cache::wait_for_previous();
  namespace cg = cooperative_groups;
  const int ranks = CLUSTER ? (int)cg::this_cluster().num_blocks() : 1;
  const int rank = CLUSTER ? (int)cg::this_cluster().block_rank() : 0;
  const int row = (int)blockIdx.x / ranks;  // CLUSTER: this CTA's
  Producer<D> p;
  int worker, units = 0;
  if constexpr (CLUSTER) {
    // units are the row's own; its pages, shared out evenly
    worker = wk * ranks + rank;
    const int n = row_pages(a, s, row).n, all = workers * ranks;
    p.u = p.u0 = cache::ROW_COST + (int)((long long)n * worker / all);
    p.u1 = cache::ROW_COST + (int)((long long)n * (worker + 1) / all);
    p.row = row;
    p.off = p.u0;
    units = p.u1;
    __syncthreads();  // the barriers are there
  } else {
    // units before each thread's rows; rows without pages get their zeros here
    const int per = (rows + threads - 1) / threads;
    const int lo = (int)min((long long)rows, (long long)tid * per), hi = min(rows, lo + per);
    int mine = 0;
    bool none = false;
    for (int r0 = lo; r0 < hi; r0 += 8) {
      // eight rows' lengths and lists on their way at once
      int len[8], ptr[9];
#pragma unroll
      for (int x = 0; x < 8; ++x) len[x] = r0 + x < hi ? a.lens[r0 + x] : 0;
      if (s.page_ptr != nullptr)
#pragma unroll
        for (int x = 0; x < 9; ++x) ptr[x] = r0 + x <= hi ? s.page_ptr[r0 + x] : 0;
#pragma unroll
      for (int x = 0; x < 8; ++x)
        if (r0 + x < hi) {
          const int n = row_pages(a, s, len[x], ptr[x], ptr[x + 1]).n;
          mine += cache::row_units(n);
          none |= n == 0;
        }
    }
    if (none)
      for (int r = lo; r < hi; ++r)
        if (r % gridDim.x == blockIdx.x && row_pages(a, s, r).n == 0) {
          sink.put_nothing(a, s, r);
          if (work.has_row(r)) work.row_units[r] = make_int2(0, 0);
        }
    const int upto = cache::warp_scan(mine);
    if (lane == 31) warp_units[warp] = upto;
    __syncthreads();
    int before = upto - mine;
#pragma unroll
    for (int w = 0; w < MAX_WARPS; ++w) {
      if (32 * w >= threads) break;
      if (w < warp) before += warp_units[w];
      units += warp_units[w];
    }
    row_before[tid] = before;
    __syncthreads();
    const cache::Chunks chunks = cache::make_chunks(units, workers * gridDim.x);
    if (tid == 0 && blockIdx.x == 0) *work.chunks = chunks;
    worker = wk * gridDim.x + blockIdx.x;  // few units: a worker of every SM before a second one of any
    p.u = p.u0 = chunks.begin(worker);
    p.u1 = chunks.begin(worker + 1);
    if (p.u0 >= p.u1) return;
    if (mt == 0) {
      int n = 0;  // threads whose rows begin at or before the chunk
      for (int i = 0; i < threads; i += 32) n += __popc(__ballot_sync(0xFFFFFFFFu, row_before[i + lane] <= p.u0));
      p.row = (n - 1) * per;
      p.off = p.u0 - row_before[n - 1];
    }
  }
  p.ring = smem_raw + (1024 - (tc::smem_u32(smem_raw) & 1023u)) + wk * stages * C::STAGE_BYTES;
  p.full = full + wk * stages;
  p.empty = empty + wk * stages;
  p.piece = pieces + wk * stages;
  p.stages = stages;
  p.issued = p.upper = 0;
  p.left = 0;
  p.ended = false;
  p.ok = true;
  p.top = -1;
  if (mt == 0) p.find(a, s, rows, work);
  const int m0 = (NT == 4 ? 32 : 16) * mt, tile_rows = min(8 * NT, M - m0);  // may be <= 0
  int token[NT][2];  // of the n_q newest, a query row's
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int m = m0 + 8 * n + 2 * t + y;
      token[n][y] = m < M ? m / s.group : s.n_q - 1;
    }
  bool ok = true;
  Tile<D, NT> acc;
  uint32_t qb[NT][D / 16][2];
  Lanes lanes;
  lanes.init<D>();
  const uint32_t ring = tc::smem_u32(p.ring);
  int stage = 0, parity = 0;
  if (CLUSTER) acc.clear();
  for (int it = 0; !CLUSTER || p.u0 < p.u1; ++it) {
    if (mt == 0)
      while (p.ok && !p.ended && p.issued < it + stages) p.send(tk, tv, a, s, rows, work, &abort, limit);
    if (!p.ok) {
      ok = false;
      break;
    }
    // The warp that sent the piece knows it already, and has the queries of a
    // new row on their way while it waits for the keys.
    __syncwarp();
    Piece d = {};
    if (mt == 0) d = p.piece[stage];
    if (d.flags & FIRST) load_queries<D, NT, T>(q, a, s, d.row, m0, qb);
    ok = __all_sync(0xFFFFFFFFu, wait(&p.full[stage], parity, &abort, limit));
    if (!ok) break;
    if (mt != 0) {
      d = p.piece[stage];
      if (d.flags & FIRST) load_queries<D, NT, T>(q, a, s, d.row, m0, qb);
    }
    if (d.flags & FIRST) acc.clear();
    if (!(d.flags & SKIP) && tile_rows > 0) {
      const uint32_t at = ring + stage * C::STAGE_BYTES;
      float *sc = nullptr;
      int score_rows = tile_rows;
      if (MASS) {
        sc = work.scores + ((long long)d.unit * M + m0) * PAGE + (d.flags & UPPER ? KEYS : 0);
        if (!work.has_unit(d.unit)) score_rows = 0;
      }
      if (s.by_position ? d.held < KEYS || (d.flags & NEWER) : d.held - (s.n_q - 1) < KEYS) {
        int newer = s.n_q;  // of slot `lane`
        if (lane < d.held) {
          if (!s.by_position)
            newer = newness(s.n_q, lane, d.held);
          else
            newer = d.flags & NEWER && a.has_slot(d.row, d.slot() + lane)
                        ? newness(s.n_q, a.pos[a.slot(d.row, d.slot() + lane)], a.seen[d.row])
                        : 0;
        }
        attend_slots<D, NT, T, MASS, true>(at, lanes, qb, s, token, d.held, newer, acc, sc, score_rows);
      } else {
        attend_slots<D, NT, T, MASS, false>(at, lanes, qb, s, token, d.held, 0, acc, sc, score_rows);
      }
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&p.empty[stage]);
    if (++stage == stages) {
      stage = 0;
      parity ^= 1;
    }
    if (!CLUSTER && (d.flags & LAST) &&
        (d.flags & WHOLE ? work.has_row(d.row) : work.has_part(cache::part_of(worker, d.flags & BEGINS)))) {
      const long long part = (long long)cache::part_of(worker, d.flags & BEGINS) * M + m0;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float scale[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float sum = acc.sum[n][y];
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 4);
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
          const float top = (acc.top[n][y] == -INFINITY ? 0.0f : acc.top[n][y]) - Num<T>::SHIFT;
          scale[y] = sum == 0.0f ? 0.0f : 1.0f / sum;
          const int m = 8 * n + 2 * t + y;
          if (g == 0 && m < tile_rows) {
            if (d.flags & WHOLE) {
              const float lse2 = sum == 0.0f ? -INFINITY : top + log2f(sum);
              sink.put_lse(a, s, d.row, m0 + m, lse2);
              if (MASS) work.lse2[(long long)d.row * M + m0 + m] = lse2;
            } else {
              work.part_ml[part + m] = make_float2(top, sum);
            }
          }
        }
        if (d.flags & WHOLE) {
          const int m = 8 * n + g;
          T *to = sink.o + (m < tile_rows ? sink.row(a, s, d.row, m0 + m) : 0) * D + 2 * t;
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t v =
                  transpose(Num<T>::pack(acc.o[c][n][2 * x] * scale[0], acc.o[c][n][2 * x + 1] * scale[1]));
              if (m < tile_rows) *reinterpret_cast<uint32_t *>(to + 16 * c + 8 * x) = v;
            }
        } else {
#pragma unroll
          for (int y = 0; y < 2; ++y)
            if (const int m = 8 * n + 2 * t + y; m < tile_rows)
#pragma unroll
              for (int c = 0; c < D / 16; ++c)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                  work.part_o[(part + m) * D + 16 * c + g + 8 * x] = acc.o[c][n][y + 2 * x];
        }
      }
    }
    if (d.flags & END) break;
  }
  // given up: the loads in flight still write to this CTA's shared memory
  if (mt == 0 && lane == 0 && !(ok && p.ok))
    for (int x = max(0, p.issued - stages); x < p.issued; ++x)
      tc::mbar_wait(&p.full[x % stages], (x / stages) & 1, nullptr, DRAIN_LIMIT);
  if constexpr (CLUSTER) {
    // every worker's part into its own ring, which nobody reads from any more:
    // outputs [M][D], then maximum and sum [M]
    __syncthreads();
    float *part_o = reinterpret_cast<float *>(p.ring);
    float2 *part_ml = reinterpret_cast<float2 *>(part_o + M * D);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float sum = acc.sum[n][y];
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 4);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
        if (const int m = 8 * n + 2 * t + y; m < tile_rows) {
          if (g == 0)
            part_ml[m0 + m] = make_float2((acc.top[n][y] == -INFINITY ? 0.0f : acc.top[n][y]) - Num<T>::SHIFT, sum);
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
#pragma unroll
            for (int x = 0; x < 2; ++x) part_o[(m0 + m) * D + 16 * c + g + 8 * x] = acc.o[c][n][y + 2 * x];
        }
      }
    cg::this_cluster().sync();
    // The outputs, four to an element, are shared out among the CTAs; a warp
    // has four elements at a time, and eight lanes for each that go through the
    // CTAs' parts (ranks: 1, 2, 4 or 8).
    const int elements = M * (D / 4), each = (elements + ranks - 1) / ranks;
    const int e0 = rank * each, e1 = min(elements, e0 + each);
    const int ring_floats = stages * C::STAGE_BYTES / 4, lane_parts = 8 / ranks;
    const float *theirs = cg::this_cluster().map_shared_rank(
        reinterpret_cast<float *>(p.ring - wk * stages * C::STAGE_BYTES), (lane / 4) & (ranks - 1));
    const int first = (lane / 4) / ranks;  // of the workers of that CTA
    for (int eb = e0 + 4 * warp; eb < e1; eb += 4 * (threads / 32)) {
      const int e = min(eb + lane % 4, e1 - 1), m = e / (D / 4);
      Part sum = {0.0f, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
      for (int k = first; k < workers; k += lane_parts * JOIN_BATCH) {
        Part q[JOIN_BATCH];  // on their way at once
#pragma unroll
        for (int x = 0; x < JOIN_BATCH; ++x) {
          const int w = k + lane_parts * x;
          q[x].sum = 0.0f;
          if (w < workers) {
            const float *of = theirs + w * ring_floats;
            const float2 ml = reinterpret_cast<const float2 *>(of + M * D)[m];
            q[x] = Part{ml.x, ml.y, *reinterpret_cast<const float4 *>(of + e * 4)};
          }
        }
#pragma unroll
        for (int x = 0; x < JOIN_BATCH; ++x) sum.add(q[x]);
      }
#pragma unroll
      for (int d = 4; d < 32; d *= 2) sum.add(shuffled(sum, d));
      if (lane < 4 && eb + lane < e1) {
        const float z = sum.sum == 0.0f ? 0.0f : 1.0f / sum.sum;
        *reinterpret_cast<uint2 *>(sink.o + sink.row(a, s, row, m) * D + e % (D / 4) * 4) =
            make_uint2(Num<T>::pack(sum.o.x * z, sum.o.y * z), Num<T>::pack(sum.o.z * z, sum.o.w * z));
        if (e % (D / 4) == 0) sink.put_lse(a, s, row, m, sum.sum == 0.0f ? -INFINITY : sum.top + log2f(sum.sum));
      }
    }
    cg::this_cluster().sync();  // the others have read this CTA's memory
  }
}

constexpr int JOIN_THREADS = 128;
constexpr int JOIN_SPREAD = 200 * 1024;

// grid.x = rows; grid.y shares out a row's outputs, four to an element. Lanes
// run along `wide` elements (a power of two), the rest of the CTA along the
// parts; those sums are added up by shuffles and through shared memory.
template <int D, typename T>
__global__ void __launch_bounds__(JOIN_THREADS)
join_kernel(const Args a, const Shape s, const Sink<D, T> sink, const Work work, int wide) {
  __shared__ Part parts[JOIN_THREADS];
  cache::let_next_start();
  cache::wait_for_previous();
  const int tid = threadIdx.x, M = s.group * s.n_q;
  const cache::Chunks chunks = *work.chunks;
  const int r = blockIdx.x, first = work.row_units[r].x, n = work.row_units[r].y;
  // (the bounds hold for whatever a call that was given up has left here)
  if (first < 0 || n < 1 || n > a.max_pages || first > chunks.units - n) return;
  const int c0 = chunks.of(first), c1 = chunks.of(first + n - 1);
  const int e = (int)blockIdx.y * wide + tid % wide, m = e / (D / 4);
  Part sum = {0.0f, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
  if (m < M)
    for (int c = c0 + tid / wide; c <= c1; c += JOIN_BATCH * (JOIN_THREADS / wide)) {
      Part p[JOIN_BATCH];  // on their way at once
#pragma unroll
      for (int x = 0; x < JOIN_BATCH; ++x) {
        const int cx = c + x * (JOIN_THREADS / wide);
        p[x].sum = 0.0f;
        if (cx <= c1 && work.has_part(cache::part_of(cx, cx == c0))) {
          const long long at = (long long)cache::part_of(cx, cx == c0) * M + m;
          const float2 ml = work.part_ml[at];
          p[x] = Part{ml.x, ml.y, *reinterpret_cast<const float4 *>(work.part_o + at * D + e % (D / 4) * 4)};
        }
      }
#pragma unroll
      for (int x = 0; x < JOIN_BATCH; ++x) sum.add(p[x]);
    }
  for (int d = wide; d < 32; d *= 2) sum.add(shuffled(sum, d));
  parts[tid] = sum;
  __syncthreads();
  if (tid >= wide || m >= M) return;
  const int step = max(wide, 32);
  for (int k = tid + step; k < JOIN_THREADS; k += step) sum.add(parts[k]);
  const float z = sum.sum == 0.0f ? 0.0f : 1.0f / sum.sum;
  *reinterpret_cast<uint2 *>(sink.o + sink.row(a, s, r, m) * D + e % (D / 4) * 4) =
      make_uint2(Num<T>::pack(sum.o.x * z, sum.o.y * z), Num<T>::pack(sum.o.z * z, sum.o.w * z));
  if (e % (D / 4) == 0) {
    const float y = sum.sum == 0.0f ? -INFINITY : sum.top + log2f(sum.sum);
    sink.put_lse(a, s, r, m, y);
    if (work.lse2 != nullptr) work.lse2[(long long)r * M + m] = y;
  }
}

constexpr int WEIGH_THREADS = 256;
constexpr int WEIGH_PAGES = WEIGH_THREADS / PAGE;  // of a CTA at a time

// A thread per slot; the grid strides over the pages.
__global__ void __launch_bounds__(WEIGH_THREADS)
weigh_kernel(const Args a, const int M, const Work work) {
  cache::let_next_start();
  cache::wait_for_previous();
  const int rows = a.B * a.H, units = work.chunks->units;
  const int j = threadIdx.x % PAGE, step = (int)gridDim.x * WEIGH_PAGES;
  int u = (int)blockIdx.x * WEIGH_PAGES + (int)threadIdx.x / PAGE;
  int2 at = u < units ? work.units[u] : make_int2(-1, -1);
  for (; u < units; u += step) {
    const int2 next = u < units - step ? work.units[u + step] : make_int2(-1, -1);
    const int col = at.y & 0xFFFFFF;
    // (the bounds hold for whatever a call that was given up has left here)
    if (at.x >= 0 && at.x < rows && at.y >= 0 && col < a.max_pages && j <= at.y >> 24 && work.has_unit(u) &&
        a.has_slot(at.x, col * PAGE + j)) {
      const float *x = work.scores + (long long)u * M * PAGE + j, *y = work.lse2 + (long long)at.x * M;
      float *w = a.weight + a.slot(at.x, col * PAGE + j);
      const float old = *w;
      float got = 0.0f;
      for (int m0 = 0; m0 < M; m0 += 8) {
        float xs[8], ys[8];
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          xs[m] = m0 + m < M ? x[(m0 + m) * PAGE] : -INFINITY;
          ys[m] = m0 + m < M ? y[m0 + m] : 0.0f;
        }
#pragma unroll
        for (int m = 0; m < 8; ++m)
          if (ys[m] != -INFINITY) got += tc::ex2(xs[m] - ys[m]);  // else the query sees nothing
      }
      if (got != 0.0f) *w = old + got;
    }
    at = next;
  }
}

}  // namespace decode
}  // namespace sta
