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
// An entry of a list: a filled page, above the entry before it (-1: none).
STA_HD bool column_ok(int column, int before, int filled) {
  return column >= 0 && column < filled && column > before;
}

// The units (pages to be read, rows one after another) are cut into equal
// chunks, one per CTA; a row cut by a chunk border is summed up in parts and
// joined afterwards.
STA_HD int chunk_units(int units, int ctas, int least) {
  const int even = (int)(((long long)units + ctas - 1) / ctas);
  return even > least ? even : least;
}
STA_HD int chunk_begin(int cta, int chunk, int units) {
  const long long u = (long long)cta * chunk;
  return u < units ? (int)u : units;
}
// Where CTA `cta` leaves its part of a row that it does not hold whole: a CTA
// has at most two such rows, the one it goes on with (offset > 0) and the one
// it begins.
STA_HD int part_of(int cta, int offset) { return 2 * cta + (offset == 0 ? 1 : 0); }
// The CTAs that hold parts of the row of `n` units that starts at unit `start`.
STA_HD int first_cta(int start, int chunk) { return start / chunk; }
STA_HD int last_cta(int start, int n, int chunk) { return (int)(((long long)start + n - 1) / chunk); }

}  // namespace cache
}  // namespace sta
