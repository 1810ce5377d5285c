// Attention of a sequence's newest tokens over its paged key-value cache.
//   row r = (b, h): one key head; its M = n_q * group query rows, row
//   m = i * group + g being token i of query head h * group + g
// Plain form: one CTA per (row, query row), a warp per slot, fp32 throughout.
#pragma once
#include <cuda_fp16.h>

#include "sta_cache.cuh"
#include "sta_tc.cuh"

namespace sta {
namespace decode {

using cache::Args;
using cache::PAGE;

struct Shape {
  int group, n_q;          // query heads per key head, newest tokens
  const int *page_ptr, *page_idx;  // page lists (CSR), or NULL
  long long idx_capacity;
  float scale;
};

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_float(float x, __nv_bfloat16 *y) { *y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_float(float x, __half *y) { *y = __float2half_rn(x); }

// The pages row r attends to: count, and the column of the i-th (-1: left out).
struct PageList {
  int first, n;
  __device__ PageList(const Args &a, const Shape &s, int r, int len) {
    const int filled = len > 0 ? (len + PAGE - 1) / PAGE : 0;
    first = 0;
    n = filled;
    if (s.page_ptr != nullptr) {
      first = s.page_ptr[r];
      n = s.page_ptr[r + 1] - first;
      if (first < 0 || n < 0 || (long long)first + n > s.idx_capacity) {
        record_error(DEV_ERR_BAD_MASK);
        n = 0;
      }
      if (len < 0) n = 0;
    }
  }
  __device__ int column(const Shape &s, int i, int len) const {
    if (s.page_ptr == nullptr) return i;
    const int c = s.page_idx[first + i];
    if (c < 0 || c >= (len + PAGE - 1) / PAGE || (i > 0 && c <= s.page_idx[first + i - 1])) {
      record_error(DEV_ERR_BAD_MASK);
      return -1;
    }
    return c;
  }
};

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;

// grid.x = rows, grid.y = query rows
template <int D, typename T>
__global__ void __launch_bounds__(THREADS)
attend_kernel(Args a, Shape s, const T *__restrict__ q, T *__restrict__ o, float *__restrict__ lse,
              float *__restrict__ lse_rows) {
  constexpr int PER = D / 32;
  __shared__ float sm[WARPS], sl[WARPS], so[WARPS][D];
  const int r = blockIdx.x, b = r / a.H, h = r - b * a.H;
  const int m = blockIdx.y, i = m / s.group, g = m - i * s.group;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = a.H * s.group;
  const long long qrow = ((long long)b * s.n_q + i) * heads + h * s.group + g;
  float qv[PER], acc[PER];
#pragma unroll
  for (int t = 0; t < PER; ++t) {
    qv[t] = to_float(q[qrow * D + t * 32 + lane]) * s.scale;
    acc[t] = 0.0f;
  }
  float top = -INFINITY, sum = 0.0f;
  const int len = a.length(r), seen = len - (s.n_q - 1 - i);
  const PageList list(a, s, r, len);
  const T *k = reinterpret_cast<const T *>(a.k), *v = reinterpret_cast<const T *>(a.v);
  for (int p = 0; p < list.n; ++p) {
    const int c = list.column(s, p, len);
    if (c < 0) continue;
    const int page = a.page(b, c * PAGE);
    if (page < 0) continue;
    for (int j = c * PAGE + warp; j < min(seen, (c + 1) * PAGE); j += WARPS) {
      const long long at = a.row(page, h, j) * D;
      float x = 0.0f;
#pragma unroll
      for (int t = 0; t < PER; ++t) x += qv[t] * to_float(k[at + t * 32 + lane]);
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, w);
      const float up = fmaxf(top, x);
      const float keep = up == -INFINITY ? 1.0f : expf(top - up), e = up == -INFINITY ? 0.0f : expf(x - up);
      top = up;
      sum = sum * keep + e;
#pragma unroll
      for (int t = 0; t < PER; ++t) acc[t] = acc[t] * keep + e * to_float(v[at + t * 32 + lane]);
    }
  }
  if (lane == 0) {
    sm[warp] = top;
    sl[warp] = sum;
  }
#pragma unroll
  for (int t = 0; t < PER; ++t) so[warp][t * 32 + lane] = acc[t];
  __syncthreads();
  float all = -INFINITY, z = 0.0f;
  for (int w = 0; w < WARPS; ++w) all = fmaxf(all, sm[w]);
  const float base = all == -INFINITY ? 0.0f : all;
  for (int w = 0; w < WARPS; ++w) z += sl[w] * expf(sm[w] - base);
  for (int d = threadIdx.x; d < D; d += THREADS) {
    float x = 0.0f;
    for (int w = 0; w < WARPS; ++w) x += so[w][d] * expf(sm[w] - base);
    from_float(z == 0.0f ? 0.0f : x / z, o + qrow * D + d);
  }
  if (threadIdx.x == 0) {
    const float y = z == 0.0f ? -INFINITY : base + logf(z);
    if (lse != nullptr) lse[((long long)b * heads + h * s.group + g) * s.n_q + i] = y;
    if (lse_rows != nullptr) lse_rows[(long long)r * s.group * s.n_q + m] = y;
  }
}

// grid.x = rows, grid.y strides over the row's pages: a thread per slot adds
// what the slot got from every query row, in their order.
template <int D, typename T>
__global__ void __launch_bounds__(PAGE)
weigh_kernel(Args a, Shape s, const T *__restrict__ q, const float *__restrict__ lse_rows) {
  const int r = blockIdx.x, b = r / a.H, h = r - b * a.H;
  const int heads = a.H * s.group;
  const int len = a.length(r);
  const PageList list(a, s, r, len);
  const T *k = reinterpret_cast<const T *>(a.k);
  for (int p = blockIdx.y; p < list.n; p += gridDim.y) {
    const int c = list.column(s, p, len);
    if (c < 0) continue;
    const int page = a.page(b, c * PAGE);
    const int j = c * PAGE + threadIdx.x;
    if (page < 0 || j >= len) continue;
    const long long at = a.row(page, h, j) * D;
    float got = 0.0f;
    for (int m = 0; m < s.group * s.n_q; ++m) {
      const int i = m / s.group, g = m - i * s.group;
      if (j >= len - (s.n_q - 1 - i)) continue;
      const T *qr = q + (((long long)b * s.n_q + i) * heads + h * s.group + g) * D;
      float x = 0.0f;
      for (int d = 0; d < D; ++d) x += to_float(qr[d]) * to_float(k[at + d]);
      got += expf(x * s.scale - lse_rows[(long long)r * s.group * s.n_q + m]);
    }
    a.weight[a.slot(r, j)] += got;
  }
}

}  // namespace decode
}  // namespace sta
