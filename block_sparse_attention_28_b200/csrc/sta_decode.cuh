// Attention of a sequence's newest tokens over its paged key-value cache.
//
//   row r = (b, h): one key head; its M = n_q * group query rows, row
//   m = i * group + g being token i of query head h * group + g
//   s_j = scale q_m . k_j,  o_m = sum_j e^(s_j - lse_m) v_j
//
// Every key and value is read once and used by the M <= 64 query rows of its
// head: at most 64 flop per byte, so HBM bounds the call. The matrix products
// are 16-row mma.sync tiles (a tcgen05 tile has at least 64 rows, of which a
// token of a group of 1 to 8 heads would fill a few).
//
// attend_kernel: one CTA per SM. The pages to be read are the units of work,
// rows one after another, cut into one equal chunk per CTA whatever the
// lengths are: no CTA waits for a long sequence. A producer warp streams pages
// through a ring of shared memory (TMA, 128-byte swizzle). Eight warps take
// them: two to a page (32 of its slots each), once for every 16 query rows, and
// with fewer than 64 query rows two or four pages at a time. Each has a running
// maximum and sum and its own output tile; they are merged where a row ends. Rows cut by a chunk border leave their parts (sum
// relative to a maximum) in the workspace.
// join_kernel: joins those parts, and adds every slot's attention to its
// weight once the row's log-sum-exp is known, from the scores that
// attend_kernel left (4 bytes per slot and query row against 4 d for its key
// and value).
#pragma once
#include <cuda_fp16.h>

#include "sta_cache.cuh"
#include "sta_tc.cuh"

namespace sta {
namespace decode {

using cache::Args;
using cache::PAGE;

constexpr int CONSUMERS = 8;  // warps
constexpr int THREADS = 32 * (CONSUMERS + 1);
constexpr int KEYS = PAGE / 2;  // slots of a page one warp takes
constexpr int MAX_ROWS = 64;   // query rows per key head
constexpr int MAX_CTAS = 148;  // one per SM of a B200
constexpr int LEAST_UNITS = 1;
constexpr int JOIN_THREADS = 256;
constexpr int JOIN_SHARES = 8;  // CTAs of join_kernel for one of attend_kernel, when weights are added
constexpr long long DRAIN_LIMIT = 200000000LL;

template <int D>
struct Cfg {
  static constexpr int HALF_BYTES = PAGE * 128;           // 64 values of every token
  static constexpr int TILE_BYTES = HALF_BYTES * (D / 64);  // keys or values of a page
  static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
  static constexpr int STAGES = 131072 / STAGE_BYTES;
  // A warp waits for a stage's next load only after it has had the load before
  // it, because page groups (4, 2 or 1) divide the stages: a barrier's phase
  // parity is read one phase ahead at most.
  static_assert(STAGES % 4 == 0, "page groups divide the stages");
  static constexpr int MERGE_STRIDE = D + 8;  // floats; 8 more spread the rows over the banks
  static constexpr int MERGE_BYTES = CONSUMERS * 16 * MERGE_STRIDE * 4;
  static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + MERGE_BYTES;
};

struct Shape {
  int group, n_q;                  // query heads per key head, newest tokens
  const int *page_ptr, *page_idx;  // page lists (CSR), or NULL
  long long idx_capacity;
  float scale_log2;  // scale * log2 e
};

// A CTA's rows that it does not hold whole (row -1: none): [0] the one it
// goes on with, [1] the one it begins.
struct Split {
  int row[2], start[2], n[2];
  int chunk, units;
};

struct Work {
  float *part_o;      // [2 * MAX_CTAS][M][D]
  float2 *part_ml;    // [2 * MAX_CTAS][M] maximum (log2) and sum
  Split *split;       // [MAX_CTAS]
  int2 *units;        // [units] (row, column of the page table or -1)
  float *scores;      // [units][M][PAGE] s_j log2 e, -inf out of view
  float *lse2;        // [rows][M] log-sum-exp (log2) of the rows held whole
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
  static __device__ __forceinline__ __nv_bfloat16 round(float x) { return __float2bfloat16_rn(x); }
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Num<__half> {
  // p is scaled to at most 2^14 (the sum with it), so that fp16, whose
  // smallest step is 2^-24, keeps weights down to 2^-38 of the largest
  static constexpr float SHIFT = 14.0f;
  static constexpr uint32_t NONFINITE = 0x7C00u;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
  }
  static __device__ __forceinline__ __half round(float x) { return __float2half_rn(x); }
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
// ------------------------------------------------------------------- rows
struct RowPages {
  int len, n, first;  // length, pages attended to, first entry of its list
};
__device__ __forceinline__ RowPages row_pages(const Args &a, const Shape &s, int r) {
  RowPages p;
  p.len = a.length(r);
  p.n = cache::filled_pages(p.len);
  p.first = 0;
  if (s.page_ptr != nullptr) {
    const int first = s.page_ptr[r], next = s.page_ptr[r + 1];
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

// A warp's view of 32 rows, one per lane, from row `base` on.
struct Window {
  int base;
  RowPages mine;
  __device__ __forceinline__ void load(const Args &a, const Shape &s, int from, int rows) {
    base = from;
    const int r = from + (int)(threadIdx.x & 31);
    mine.len = mine.n = mine.first = 0;
    if (r < rows) mine = row_pages(a, s, r);
  }
};

// --------------------------------------------------------------- producer
// One warp: 32 units at a time, a lane each finds its unit's row, column and
// page, then lane 0 issues the loads in order.
template <int D>
__device__ void produce(const CUtensorMap &tk, const CUtensorMap &tv, const Args &a, const Shape &s, int rows,
                        int row, int off, int u, int u1, uint8_t *ring, uint64_t *full, uint64_t *empty,
                        int *stage_col, volatile uint32_t *abort, long long limit) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  int issued = 0;
  bool ok = true;
  while (u < u1 && row < rows && ok) {
    Window w;
    w.load(a, s, row, rows);
    const int skip = lane == 0 ? off : 0;
    const int upto = cache::warp_scan(w.mine.n - skip);  // units of the window up to this lane's row
    const int total = __shfl_sync(0xFFFFFFFFu, upto, 31);
    const int take = min(total, u1 - u);
    for (int t0 = 0; t0 < take && ok; t0 += 32) {
      const int t = t0 + lane;
      int k = 0;  // first row of the window with upto > t
#pragma unroll
      for (int step = 16; step > 0; step >>= 1)
        if (__shfl_sync(0xFFFFFFFFu, upto, k + step - 1) <= t) k += step;
      k = min(k, 31);
      const int n = __shfl_sync(0xFFFFFFFFu, w.mine.n, k), first = __shfl_sync(0xFFFFFFFFu, w.mine.first, k);
      const int len = __shfl_sync(0xFFFFFFFFu, w.mine.len, k), end = __shfl_sync(0xFFFFFFFFu, upto, k);
      const int r = row + k, b = r / a.H, h = r - b * a.H;
      int col = -1, y = 0;
      if (t < take) {
        const int i = n - (end - t);  // the row's i-th page
        col = i;
        if (s.page_ptr != nullptr) {
          col = s.page_idx[first + i];
          if (!cache::column_ok(col, i > 0 ? s.page_idx[first + i - 1] : -1, cache::filled_pages(len))) {
            record_error(DEV_ERR_BAD_MASK);
            col = -1;
          }
        }
        const int page = col >= 0 ? a.page(b, col * PAGE) : -1;
        if (page < 0) col = -1;
        y = page >= 0 ? (page * a.H + h) * PAGE : 0;
      }
      const int count = min(32, take - t0);
      for (int x = 0; x < count && ok; ++x) {
        const int xc = __shfl_sync(0xFFFFFFFFu, col, x), xy = __shfl_sync(0xFFFFFFFFu, y, x);
        const int stage = issued % C::STAGES;
        if (lane == 0) {
          if (issued >= C::STAGES) ok = tc::mbar_wait(&empty[stage], ((issued / C::STAGES) & 1) ^ 1, abort, limit);
          if (ok) {
            stage_col[stage] = xc;
            if (xc < 0) {
              tc::mbar_arrive(&full[stage]);
            } else {
              const uint32_t dst = tc::smem_u32(ring + stage * C::STAGE_BYTES);
              tc::mbar_expect_tx(&full[stage], C::STAGE_BYTES);
#pragma unroll
              for (int e = 0; e < D / 64; ++e) tc::tma_load_2d(dst + e * C::HALF_BYTES, &tk, &full[stage], 64 * e, xy);
#pragma unroll
              for (int e = 0; e < D / 64; ++e)
                tc::tma_load_2d(dst + C::TILE_BYTES + e * C::HALF_BYTES, &tv, &full[stage], 64 * e, xy);
            }
          }
        }
        ok = __shfl_sync(0xFFFFFFFFu, (int)ok, 0) != 0;
        if (ok) ++issued;
      }
    }
    u += take;
    row += 32;
    off = 0;
  }
  // given up: the loads in flight still write to this CTA's shared memory
  if (!ok && lane == 0)
    for (int x = max(0, issued - C::STAGES); x < issued; ++x)
      tc::mbar_wait(&full[x % C::STAGES], (x / C::STAGES) & 1, nullptr, DRAIN_LIMIT);
}

// Rows without any page: o = 0, lse = -inf. Row r is CTA r % CTAs'.
template <int D, typename T>
__device__ void fill_empty_rows(const Args &a, const Shape &s, int rows, T *o, float *lse) {
  const int lane = threadIdx.x & 31;
  const int M = s.group * s.n_q, heads = a.H * s.group;
  for (long long r0 = blockIdx.x; r0 < rows; r0 += 32LL * gridDim.x) {
    const long long mine = r0 + (long long)lane * gridDim.x;
    const bool none = mine < rows && row_pages(a, s, (int)mine).n == 0;
    for (unsigned left = __ballot_sync(0xFFFFFFFFu, none); left != 0; left &= left - 1) {
      const int r = (int)(r0 + (long long)(__ffs(left) - 1) * gridDim.x);
      const int b = r / a.H, h = r - b * a.H;
      for (int e = lane; e < M * (D / 8); e += 32) {
        const int m = e / (D / 8), i = m / s.group, g = m - i * s.group;
        const long long row = ((long long)b * s.n_q + i) * heads + h * s.group + g;
        reinterpret_cast<uint4 *>(o + row * D)[e % (D / 8)] = make_uint4(0u, 0u, 0u, 0u);
      }
      if (lse != nullptr)
        for (int m = lane; m < M; m += 32) {
          const int i = m / s.group, g = m - i * s.group;
          lse[((long long)b * heads + h * s.group + g) * s.n_q + i] = -INFINITY;
        }
    }
  }
}

// --------------------------------------------------------------- consumers
// 16 query rows of one warp: thread (g, t) = (lane / 4, lane % 4) holds rows g
// and g + 8 of the tile, columns 8 n + 2 t and + 1 of each 8-column piece n.
template <int D>
struct Tile {
  float o[D / 8][4];
  float top[2], sum[2];  // running maximum (log2); this thread's share of the sum
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
    top[0] = top[1] = -INFINITY;
    sum[0] = sum[1] = 0.0f;
  }
};

// Query rows of tile mt as the A operand of D / 16 steps (rows past M: zero).
template <int D, typename T>
__device__ __forceinline__ void load_queries(const T *q, const Args &a, const Shape &s, int b, int h, int mt,
                                             uint32_t (&qa)[D / 16][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int m = mt * 16 + g + 8 * half;
    const bool in = m < s.group * s.n_q;
    const int i = in ? m / s.group : 0, hg = in ? m - i * s.group : 0;
    const uint32_t *row = reinterpret_cast<const uint32_t *>(
        q + (((long long)b * s.n_q + i) * (a.H * s.group) + h * s.group + hg) * D);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      qa[ks][half] = in ? row[ks * 8 + t] : 0u;
      qa[ks][2 + half] = in ? row[ks * 8 + 4 + t] : 0u;
    }
  }
}

// KEYS slots of a page (kt, vt: where their keys and values begin): scores, softmax step, weighted
// values. lim[x]: how many of them row g + 8 x sees; held: how many are filled
// (either may be negative or above KEYS). edge: any of these is below KEYS.
// scores: where this tile's scores go (MASS), of which it has `rows` rows.
template <int D, typename T, bool MASS>
__device__ __forceinline__ void attend_slots(uint32_t kt, uint32_t vt, const uint32_t (&qa)[D / 16][4],
                                             const Shape &s, const int (&lim)[2], int held, bool edge, Tile<D> &acc,
                                             float *scores, int rows) {
  using N = Num<T>;
  constexpr int HALF_BYTES = Cfg<D>::HALF_BYTES;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float p[KEYS / 8][4];
  {
    const uint32_t row = kt + (lane & 7) * 128, x = lane & 7, m = lane >> 3;
#pragma unroll
    for (int n = 0; n < KEYS / 8; ++n) {
      p[n][0] = p[n][1] = p[n][2] = p[n][3] = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        uint32_t kb[4];
        // 16-byte pieces 4 j .. 4 j + 3 of keys 8 n .. 8 n + 7
        ldmatrix(row + n * 1024 + (j >> 1) * HALF_BYTES + ((((j & 1) * 4 + m) ^ x) << 4), kb);
        N::mma(p[n], qa[2 * j], kb[0], kb[1]);
        N::mma(p[n], qa[2 * j + 1], kb[2], kb[3]);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < KEYS / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[n][e] *= s.scale_log2;
      if (edge && 8 * n + 2 * t + (e & 1) >= lim[e >> 1]) p[n][e] = -INFINITY;
    }
  if (MASS) {
#pragma unroll
    for (int n = 0; n < KEYS / 8; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (g + 8 * x < rows)
          *reinterpret_cast<float2 *>(scores + (g + 8 * x) * PAGE + 8 * n + 2 * t) =
              make_float2(p[n][2 * x], p[n][2 * x + 1]);
  }
  float base[2], keep[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    float up = -INFINITY;
#pragma unroll
    for (int n = 0; n < KEYS / 8; ++n) up = tc::fmax3(up, p[n][2 * x], p[n][2 * x + 1]);
    up = fmaxf(up, __shfl_xor_sync(0xFFFFFFFFu, up, 1));
    up = fmaxf(up, __shfl_xor_sync(0xFFFFFFFFu, up, 2));
    up = fmaxf(up, acc.top[x]);
    const float from = up == -INFINITY ? 0.0f : up;  // a row that has seen nothing yet
    keep[x] = tc::ex2(acc.top[x] - from);
    acc.top[x] = up;
    base[x] = from - N::SHIFT;
  }
  if (__any_sync(0xFFFFFFFFu, keep[0] != 1.0f || keep[1] != 1.0f)) {
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      acc.o[n][0] *= keep[0];
      acc.o[n][1] *= keep[0];
      acc.o[n][2] *= keep[1];
      acc.o[n][3] *= keep[1];
    }
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    float z = 0.0f;
#pragma unroll
    for (int n = 0; n < KEYS / 8; ++n)
#pragma unroll
      for (int e = 2 * x; e < 2 * x + 2; ++e) {
        p[n][e] = tc::ex2(p[n][e] - base[x]);
        z += p[n][e];
      }
    acc.sum[x] = acc.sum[x] * keep[x] + z;
  }
  // The weights of slots 16 ks .. 16 ks + 15 as the A operand, split in two
  // terms: one alone would be off by as much as the output's own rounding.
  auto weights = [&](int ks, uint32_t(&hi)[4], uint32_t(&lo)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float p0 = p[2 * ks + (e >> 1)][(e & 1) * 2], p1 = p[2 * ks + (e >> 1)][(e & 1) * 2 + 1];
      hi[e] = N::pack(p0, p1);
      const float2 r = N::unpack(hi[e]);
      lo[e] = N::pack(p0 - r.x, p1 - r.y);
    }
  };
  const uint32_t vrow = vt + ((lane & 7) + ((lane >> 3) & 1) * 8) * 128, vx = lane & 7, vc = lane >> 4;
  // Values of slots that are not seen must not reach the products even with a
  // weight of 0 (0 * inf): registers of slots >= held are cleared. A slot that
  // only the newer of the n_q tokens see is cleared where it is not finite,
  // and what is not finite added by hand for those who see it.
  auto slots_below = [&](int key, int upto) { return key + 1 < upto ? 0xFFFFFFFFu : (key < upto ? 0xFFFFu : 0u); };
  auto finite = [](uint32_t v) {
    return ((v & N::NONFINITE) == N::NONFINITE ? 0u : v & 0xFFFFu) |
           ((v >> 16 & N::NONFINITE) == N::NONFINITE ? 0u : v & 0xFFFF0000u);
  };
  auto value_pair = [&](int key, int c) {  // values 8 c + 2 t and + 1
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];"
                 : "=r"(v)
                 : "r"(vt + (c >> 3) * HALF_BYTES + key * 128 + (((c & 7) ^ (key & 7)) << 4) + 4 * t));
    return v;
  };
  bool odd = false;
  if (edge && s.n_q > 1) {
    for (int key = max(0, held - (s.n_q - 1)) + g; key < min(KEYS, held); key += 8)
      for (int c = 0; c < D / 8; ++c) {
        const uint32_t v = value_pair(key, c);
        odd |= finite(v) != v;
      }
    odd = __any_sync(0xFFFFFFFFu, odd);
  }
#pragma unroll
  for (int ks = 0; ks < KEYS / 16; ++ks) {
    // the weights of slots 16 ks .. 16 ks + 15 as the A operand, split in two
    // terms: one alone would be off by as much as the output's own rounding
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float p0 = p[2 * ks + (e >> 1)][(e & 1) * 2], p1 = p[2 * ks + (e >> 1)][(e & 1) * 2 + 1];
      hi[e] = N::pack(p0, p1);
      const float2 r = N::unpack(hi[e]);
      lo[e] = N::pack(p0 - r.x, p1 - r.y);
    }
    const uint32_t m0 = slots_below(16 * ks + 2 * t, held), m1 = slots_below(16 * ks + 8 + 2 * t, held);
#pragma unroll
    for (int c = 0; c < D / 8; c += 2) {
      uint32_t vb[4];
      // keys 16 ks .. 16 ks + 15, 16-byte pieces c and c + 1
      ldmatrix_trans(vrow + ks * 2048 + (c >> 3) * HALF_BYTES + ((((c & 7) + vc) ^ vx) << 4), vb);
      if (edge) {
        vb[0] &= m0;
        vb[1] &= m1;
        vb[2] &= m0;
        vb[3] &= m1;
        if (odd) {
#pragma unroll
          for (int e = 0; e < 4; ++e) vb[e] = finite(vb[e]);
        }
      }
      N::mma(acc.o[c], hi, vb[0], vb[1]);
      N::mma(acc.o[c + 1], hi, vb[2], vb[3]);
      N::mma(acc.o[c], lo, vb[0], vb[1]);
      N::mma(acc.o[c + 1], lo, vb[2], vb[3]);
    }
  }
  if (odd)
    for (int key = 0; key < min(KEYS, held); ++key)
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint32_t v = value_pair(key, c);
        const uint32_t bad = v ^ finite(v);  // the halves that are not finite, as they are
        const float2 x = N::unpack(bad);
        if (bad != 0)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key < lim[e >> 1]) acc.o[c][e] += e & 1 ? x.y : x.x;
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
  // y: log-sum-exp (log2)
  __device__ __forceinline__ void put_lse(const Args &a, const Shape &s, int r, int m, float y) const {
    const int b = r / a.H, h = r - b * a.H, i = m / s.group, g = m - i * s.group;
    if (lse != nullptr)
      lse[((long long)b * (a.H * s.group) + h * s.group + g) * s.n_q + i] = y * 0.69314718055994530942f;
  }
};

template <int D, typename T, bool MASS>
__global__ void __launch_bounds__(THREADS, 1)
attend_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const Args a,
              const Shape s, const T *__restrict__ q, const Sink<D, T> sink, const Work work, long long limit) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[C::STAGES], empty[C::STAGES];
  __shared__ int stage_col[C::STAGES];
  __shared__ float2 merge_ml[CONSUMERS][16];
  __shared__ int warp_units[CONSUMERS + 1];
  __shared__ int begin[2];  // row and page of it that this CTA begins with
  __shared__ uint32_t abort;
  uint8_t *ring = smem_raw + (1024 - (tc::smem_u32(smem_raw) & 1023u));
  float *merge = reinterpret_cast<float *>(ring + C::STAGES * C::STAGE_BYTES);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rows = a.B * a.H, M = s.group * s.n_q;
  // two warps per page and 16 query rows; the rest side by side over the pages
  const int tiles = M <= 16 ? 1 : (M <= 32 ? 2 : 4), groups = CONSUMERS / (2 * tiles);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], 2 * tiles);
    }
    abort = 0u;
    tc::fence_barrier_init();
  }
  // units before each thread's rows
  const int per = (rows + THREADS - 1) / THREADS;
  const int lo = (int)min((long long)rows, (long long)tid * per), hi = min(rows, lo + per);
  int mine = 0;
  for (int r = lo; r < hi; ++r) mine += row_pages(a, s, r).n;
  const int upto = cache::warp_scan(mine);
  if (lane == 31) warp_units[warp] = upto;
  __syncthreads();
  int units = 0, before = upto - mine;
#pragma unroll
  for (int w = 0; w < CONSUMERS + 1; ++w) {
    if (w < warp) before += warp_units[w];
    units += warp_units[w];
  }
  const int chunk = cache::chunk_units(units, gridDim.x, LEAST_UNITS);
  const int u0 = cache::chunk_begin(blockIdx.x, chunk, units), u1 = cache::chunk_begin(blockIdx.x + 1, chunk, units);
  if (u0 < u1 && before <= u0 && u0 < before + mine) {
    int at = before, r = lo;
    for (; r < hi; ++r) {
      const int n = row_pages(a, s, r).n;
      if (u0 < at + n) break;
      at += n;
    }
    begin[0] = r;
    begin[1] = u0 - at;
  }
  __syncthreads();
  if (warp == CONSUMERS) {
    if (u0 < u1)
      produce<D>(tk, tv, a, s, rows, begin[0], begin[1], u0, u1, ring, full, empty, stage_col, &abort, limit);
    fill_empty_rows<D, T>(a, s, rows, sink.o, sink.lse);
    return;
  }

  Split split;
  split.row[0] = split.row[1] = -1;
  split.start[0] = split.start[1] = split.n[0] = split.n[1] = 0;
  split.chunk = chunk;
  split.units = units;
  const int mt = warp % tiles, pg = warp / tiles / 2, g = lane >> 2, t = lane & 3;
  const int key0 = warp / tiles % 2 * KEYS;
  const int tile_rows = min(16, M - 16 * mt);  // may be <= 0
  int u = u0, row = u0 < u1 ? begin[0] : 0, off = u0 < u1 ? begin[1] : 0;
  int done = 0;  // units of this CTA before the row's
  bool ok = true;
  bool pending = false;  // a merge that all warps read may still be being read
  Window win;
  if (u0 < u1) win.load(a, s, row, rows);
  Tile<D> acc;
  while (u < u1 && row < rows) {
    // next row with pages left
    const unsigned has = __ballot_sync(0xFFFFFFFFu, win.mine.n > (win.base + lane == row ? off : 0) &&
                                                        win.base + lane >= row);
    if (has == 0) {
      row = win.base + 32;
      off = 0;
      win.load(a, s, row, rows);
      continue;
    }
    const int k = __ffs(has) - 1;
    if (win.base + k != row) off = 0;
    row = win.base + k;
    const int n = __shfl_sync(0xFFFFFFFFu, win.mine.n, k), len = __shfl_sync(0xFFFFFFFFu, win.mine.len, k);
    const int seg = min(n - off, u1 - u);
    const int b = row / a.H, h = row - b * a.H;
    const bool whole = off == 0 && seg == n;
    if (!whole) {
      const int x = off > 0 ? 0 : 1;
      split.row[x] = row;
      split.start[x] = u - off;
      split.n[x] = n;
    }
    acc.clear();
    const int lead = (pg - done % groups + groups) % groups;  // this warp's first page of the row
    const bool active = lead < seg && tile_rows > 0;
    if (lead < seg) {
      uint32_t qa[D / 16][4];
      load_queries<D, T>(q, a, s, b, h, mt, qa);
      const int m0 = 16 * mt + g, m1 = m0 + 8;
      const int back0 = m0 < M ? s.n_q - 1 - m0 / s.group : 0, back1 = m1 < M ? s.n_q - 1 - m1 / s.group : 0;
      for (int x = lead; x < seg; x += groups) {
        const int it = done + x, stage = it % C::STAGES;
        if (ok) ok = tc::mbar_wait(&full[stage], (it / C::STAGES) & 1, &abort, limit);
        ok = __all_sync(0xFFFFFFFFu, ok);
        const int col = ok ? stage_col[stage] : -1;
        if (MASS && lane == 0 && mt == 0 && key0 == 0) work.units[u + x] = make_int2(row, col);
        if (col >= 0 && tile_rows > 0) {
          const int held = len - col * PAGE - key0;
          const int lim[2] = {held - back0, held - back1};
          const uint32_t kt = tc::smem_u32(ring + stage * C::STAGE_BYTES) + key0 * 128;
          float *sc = MASS ? work.scores + ((long long)(u + x) * M + 16 * mt) * PAGE + key0 : nullptr;
          attend_slots<D, T, MASS>(kt, kt + C::TILE_BYTES, qa, s, lim, held, held - (s.n_q - 1) < KEYS, acc, sc,
                                   tile_rows);
        }
        __syncwarp();
        if (lane == 0 && ok) tc::mbar_arrive(&empty[stage]);
      }
    }
    // the row's sum in this thread's rows
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      acc.sum[x] += __shfl_xor_sync(0xFFFFFFFFu, acc.sum[x], 1);
      acc.sum[x] += __shfl_xor_sync(0xFFFFFFFFu, acc.sum[x], 2);
    }
    const int part = cache::part_of(blockIdx.x, off);
    auto put = [&](int m, int d, float o0, float o1, float top, float sum) {
      // two neighbouring outputs of query row m
      if (whole) {
        const float z = sum == 0.0f ? 0.0f : 1.0f / sum;
        *reinterpret_cast<uint32_t *>(sink.o + sink.row(a, s, row, m) * D + d) = Num<T>::pack(o0 * z, o1 * z);
        if (d == 0) {
          const float y = sum == 0.0f ? -INFINITY : top + log2f(sum);
          sink.put_lse(a, s, row, m, y);
          if (MASS) work.lse2[(long long)row * M + m] = y;
        }
      } else {
        *reinterpret_cast<float2 *>(work.part_o + ((long long)part * M + m) * D + d) = make_float2(o0, o1);
        if (d == 0) work.part_ml[(long long)part * M + m] = make_float2(top, sum);
      }
    };
    // The parts go through shared memory: one is written when the merge before
    // has been read, and read when all are written. All warps take part, or,
    // where the row has a single page here, that page's.
    auto everyone = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(32 * CONSUMERS) : "memory"); };
    auto page_warps = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(2 + pg), "r"(64 * tiles) : "memory"); };
    if (seg > 1 || pending) everyone();
    pending = seg > 1;
    if (seg > 1 || lead == 0) {
      if (seg == 1) page_warps();
      if (active) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (g + 8 * x < tile_rows) {
            float *to = merge + (warp * 16 + g + 8 * x) * C::MERGE_STRIDE + 2 * t;
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
              *reinterpret_cast<float2 *>(to + 8 * c) = make_float2(acc.o[c][2 * x], acc.o[c][2 * x + 1]);
            if (t == 0) merge_ml[warp][g + 8 * x] = make_float2(acc.top[x], acc.sum[x]);
          }
      }
      if (seg == 1)
        page_warps();
      else
        everyone();
      const int from = done % groups, have = min(groups, seg);  // page groups that hold a part
      const int threads = seg == 1 ? 64 * tiles : 32 * CONSUMERS;
      for (int e = seg == 1 ? tid - pg * 64 * tiles : tid; e < M * (D / 2); e += threads) {
        const int m = e / (D / 2), d = e % (D / 2) * 2;
        const int wt = m >> 4, wr = m & 15;
        auto holder = [&](int x) { return ((from + (x >> 1)) % groups * 2 + (x & 1)) * tiles + wt; };
        float top = -INFINITY;
        for (int x = 0; x < 2 * have; ++x) top = fmaxf(top, merge_ml[holder(x)][wr].x);
        const float at = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f, o0 = 0.0f, o1 = 0.0f;
        for (int x = 0; x < 2 * have; ++x) {
          const int w = holder(x);
          const float2 ml = merge_ml[w][wr];
          const float f = tc::ex2(ml.x - at);
          const float2 v = *reinterpret_cast<const float2 *>(merge + (w * 16 + wr) * C::MERGE_STRIDE + d);
          sum += ml.y * f;
          o0 += v.x * f;
          o1 += v.y * f;
        }
        put(m, d, o0, o1, at - Num<T>::SHIFT, sum);
      }
    }
    done += seg;
    u += seg;
    off += seg;
    if (off == n) {
      ++row;
      off = 0;
      if (row >= win.base + 32 && u < u1) win.load(a, s, row, rows);
    }
  }
  if (tid == 0) work.split[blockIdx.x] = split;
}

// grid.x = the CTAs of attend_kernel, grid.y shares out each one's units.
template <int D, typename T, bool MASS>
__global__ void __launch_bounds__(JOIN_THREADS)
join_kernel(const Args a, const Shape s, const Sink<D, T> sink, const Work work) {
  extern __shared__ float factor[];  // [parts][M]
  __shared__ float row_lse[2][MAX_ROWS];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, M = s.group * s.n_q;
  const int cta = blockIdx.x;
  const Split split = work.split[cta];
  for (int x = 0; x < 2; ++x) {
    const int r = split.row[x];
    if (r < 0) continue;
    const int c0 = cache::first_cta(split.start[x], split.chunk);
    const int parts = cache::last_cta(split.start[x], split.n[x], split.chunk) - c0 + 1;
    auto part = [&](int k) { return cache::part_of(c0 + k, k); };
    for (int m = warp; m < M; m += JOIN_THREADS / 32) {
      float top = -INFINITY, z = 0.0f;
      for (int k = lane; k < parts; k += 32)
        if (const float2 ml = work.part_ml[(long long)part(k) * M + m]; ml.y != 0.0f) top = fmaxf(top, ml.x);
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, w));
      const float at = top == -INFINITY ? 0.0f : top;
      for (int k = lane; k < parts; k += 32) {
        const float2 ml = work.part_ml[(long long)part(k) * M + m];
        const float f = ml.y != 0.0f ? tc::ex2(ml.x - at) : 0.0f;
        factor[k * M + m] = f;
        z += ml.y * f;
      }
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, w);
      const float f = z == 0.0f ? 0.0f : 1.0f / z;
      for (int k = lane; k < parts; k += 32) factor[k * M + m] *= f;
      if (lane == 0) {
        const float y = z == 0.0f ? -INFINITY : at + log2f(z);
        row_lse[x][m] = y;
        if (cta == c0 && blockIdx.y == 0) sink.put_lse(a, s, r, m, y);
      }
    }
    __syncthreads();
    // the row's outputs, four at a time, shared out among its CTAs
    const int step = parts * (int)gridDim.y * JOIN_THREADS;
    for (int e = ((cta - c0) * (int)gridDim.y + (int)blockIdx.y) * JOIN_THREADS + tid; e < M * (D / 4); e += step) {
      const int m = e / (D / 4), d = e % (D / 4) * 4;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
      for (int k = 0; k < parts; ++k) {
        const float f = factor[k * M + m];
        const float4 v = *reinterpret_cast<const float4 *>(work.part_o + ((long long)part(k) * M + m) * D + d);
        o.x += v.x * f;
        o.y += v.y * f;
        o.z += v.z * f;
        o.w += v.w * f;
      }
      *reinterpret_cast<uint2 *>(sink.o + sink.row(a, s, r, m) * D + d) =
          make_uint2(Num<T>::pack(o.x, o.y), Num<T>::pack(o.z, o.w));
    }
    __syncthreads();
  }
  if (MASS) {
    const int u1 = cache::chunk_begin(cta + 1, split.chunk, split.units);
    const int j = tid % PAGE;
    for (int u = cache::chunk_begin(cta, split.chunk, split.units) + (int)blockIdx.y * (JOIN_THREADS / PAGE) +
                 tid / PAGE;
         u < u1; u += (int)gridDim.y * (JOIN_THREADS / PAGE)) {
      const int2 at = work.units[u];
      if (at.y < 0) continue;
      const float *lse = at.x == split.row[0] ? row_lse[0] : (at.x == split.row[1] ? row_lse[1] : nullptr);
      float got = 0.0f;
      for (int m = 0; m < M; ++m) {
        const float y = lse != nullptr ? lse[m] : work.lse2[(long long)at.x * M + m];
        const float x = work.scores[((long long)u * M + m) * PAGE + j];
        if (y != -INFINITY) got += tc::ex2(x - y);
      }
      if (got != 0.0f) a.weight[a.slot(at.x, at.y * PAGE + j)] += got;
    }
  }
}

}  // namespace decode
}  // namespace sta
