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

constexpr int kMaxLen = 262144;      // positions of a sequence
constexpr int kMaxPageSize = 65536;

// One page table: entry (s, c) is the page of positions c * page_size ...
struct PageTable {
  const int32_t* pages;
  int64_t ld;       // entries from one sequence's row to the next
  int cols;         // entries of a row that may be read
  int page_size;
  int64_t n_pages;  // pages of the pool
  uint64_t inverse;  // ceil(2^40 / page_size)
};

SF_HD PageTable make_page_table(const int32_t* pages, int64_t ld, int cols, int page_size, int64_t n_pages) {
  return PageTable{pages, ld, cols, page_size, n_pages, ((1ull << 40) + page_size - 1) / page_size};
}

// j / page_size for 0 <= j < kMaxLen by one product.  inverse exceeds
// 2^40 / page_size by less than 1, so the product exceeds 2^40 j / page_size by
// less than j < 2^18, while a quotient that is no integer lies at least
// 2^40 / page_size >= 2^24 below the next one.
SF_HD int page_of(const PageTable& t, int j) { return (int)(((uint64_t)(uint32_t)j * t.inverse) >> 40); }

// Entry that holds position j of sequence s, -1 when j lies outside the table.
// s must be in range.
SF_HD int32_t page_entry(const PageTable& t, int s, int j) {
  if (j < 0 || j >= kMaxLen) return -1;
  const int c = page_of(t, j);
  return c < t.cols ? t.pages[(int64_t)s * t.ld + c] : -1;
}

// Slot (page * page_size + offset) of position j on `page`, or -1 for a page
// outside the pool.
SF_HD int64_t entry_slot(const PageTable& t, int32_t page, int j) {
  if (page < 0 || page >= t.n_pages) return -1;
  return (int64_t)page * t.page_size + (j - page_of(t, j) * t.page_size);
}

// The same in 32 bits, ~0 for none: pools have fewer than 2^32 - 1 slots.
SF_HD uint32_t entry_slot32(const PageTable& t, int32_t page, int j) {
  const uint32_t pages = t.n_pages > 0x7fffffff ? 0x80000000u : (uint32_t)t.n_pages;
  if ((uint32_t)page >= pages) return ~0u;
  return (uint32_t)page * (uint32_t)t.page_size + (uint32_t)(j - page_of(t, j) * t.page_size);
}

// Both: -1 when j lies outside the table or on a page outside the pool.
SF_HD int64_t page_slot(const PageTable& t, int s, int j) { return entry_slot(t, page_entry(t, s, j), j); }

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

// ---- the split of a batch's attention over thread blocks ---------------------
//
// The work is a line of units: sequence after sequence, head group after head
// group, tile of kTileKeys keys after tile.  Block k takes units
// [k * per, (k + 1) * per).  A segment (one sequence and head group) that lies
// in one block is finished there.  One that is cut leaves a partial result per
// block; a block is the inside or the end of at most one cut segment (its
// first) and the start of at most one (its last), so two partial slots and one
// arrival counter per block are enough for any batch.

constexpr int kTileKeys = 16;

SF_HD int tiles_of(int len) { return (len + kTileKeys - 1) / kTileKeys; }

// a / b for non-negative a and positive b, in 32 bits where they fit (a 64-bit
// quotient costs a block some 400 cycles, and it is on the critical path).
SF_HD int64_t quotient(int64_t a, int64_t b) {
  if ((((uint64_t)a | (uint64_t)b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// Units per block: all blocks busy, but at least `least` units each.
SF_HD int64_t units_per_block(int64_t units, int blocks, int least) {
  const int64_t per = quotient(units + blocks - 1, blocks);
  return per < least ? least : per;
}

// Blocks that share the segment of `tiles` units starting at unit `first`.
SF_HD int first_block(int64_t first, int64_t per) { return (int)quotient(first, per); }
SF_HD int last_block(int64_t first, int tiles, int64_t per) { return (int)quotient(first + tiles - 1, per); }

// Partial slot of block `block` for the cut segment starting at `first`.
SF_HD int part_slot(int block, int64_t first, int64_t per) { return 2 * block + (first > block * per ? 1 : 0); }

}  // namespace sf
