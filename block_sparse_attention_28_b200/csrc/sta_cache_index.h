// Index arithmetic of the paged key-value cache, in plain C++ so that it also
// compiles for the host (tests/test_cache_host.py runs it there): what is in
// bounds, and how the pages of a call are shared out among its CTAs.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define STA_HD __host__ __device__ __forceinline__
#else
#define STA_HD inline
#endif

namespace sta {
namespace cache {

constexpr int PAGE = 64;  // tokens a page holds: the library's tile

STA_HD bool length_ok(int len, int max_pages) { return len >= 0 && len <= PAGE * max_pages; }
STA_HD bool page_ok(int page, int num_pages) { return page >= 0 && page < num_pages; }
STA_HD int filled_pages(int len) { return len > 0 ? (len - 1) / PAGE + 1 : 0; }

// Offsets [first, next) of a row's page list: within the given entries, and
// no more of them than the page table has columns.
STA_HD bool list_ok(int first, int next, long long capacity, int max_pages) {
  return first >= 0 && next >= first && next <= capacity && next - first <= max_pages;
}
// An entry of a list: a filled page, above the largest entry before it (-1:
// none). Comparing with all of them, not with the last one alone, is what keeps
// a list out of order from naming a page twice.
STA_HD bool column_ok(int column, int before, int filled) {
  return column >= 0 && column < filled && column > before;
}

// Work is counted in units, rows one after another: a row of n pages has
// ROW_COST units for itself (its queries, its result) and one for each page; a
// row without pages has none. The units are cut into equal chunks, one per
// worker; a row cut by a chunk border is summed up in parts and joined
// afterwards.
constexpr int ROW_COST = 1;
STA_HD int row_units(int pages) { return pages > 0 ? pages + ROW_COST : 0; }
struct Chunks {
  int units, size;
  STA_HD int begin(int c) const {
    const long long u = (long long)c * size;
    return u < units ? (int)u : units;
  }
  STA_HD int of(int unit) const { return unit / size; }  // the chunk a unit lies in
};
STA_HD Chunks make_chunks(int units, int workers) {
  const int even = (int)(((long long)units + workers - 1) / workers);
  return Chunks{units, even > 1 ? even : 1};
}
// Where a chunk's part of a row lies that it does not hold whole. It has two
// such rows at most: the one it goes on with and the one it begins.
STA_HD int part_of(int chunk, bool begins) { return 2 * chunk + (begins ? 1 : 0); }

}  // namespace cache
}  // namespace sta
