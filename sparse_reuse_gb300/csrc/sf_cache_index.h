// Index arithmetic of the paged-cache operators, plain C++ that the kernels
// and the CPU tests compile alike: which slot of a pool a position lives in,
// and which positions one eviction may choose from.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SF_HD __host__ __device__ __forceinline__
#else
#define SF_HD inline
#endif

namespace sf {

// One page table: entry (s, c) is the page of positions c * page_size ...
struct PageTable {
  const int32_t* pages;
  int64_t ld;       // entries from one sequence's row to the next
  int cols;         // entries of a row that may be read
  int page_size;
  int64_t n_pages;  // pages of the pool
};

// Slot (page * page_size + offset) of position j of sequence s, or -1 when j
// lies outside the table or on a page outside the pool.  s must be in range.
SF_HD int64_t page_slot(const PageTable& t, int s, int j) {
  if (j < 0) return -1;
  const int c = j / t.page_size;
  if (c >= t.cols) return -1;
  const int64_t page = t.pages[(int64_t)s * t.ld + c];
  if (page < 0 || page >= t.n_pages) return -1;
  return page * t.page_size + (j - c * t.page_size);
}

// Longest sequence a call can address.
SF_HD int64_t length_limit(int max_len, int cols, int page_size) {
  const int64_t cap = (int64_t)cols * page_size;
  return cap < max_len ? cap : max_len;
}

// A sequence's length for the kernels: out-of-range lengths count as empty
// and set *bad.
SF_HD int checked_len(int len, int64_t limit, bool* bad) {
  *bad = len < 0 || len > limit;
  return *bad ? 0 : len;
}

}  // namespace sf
