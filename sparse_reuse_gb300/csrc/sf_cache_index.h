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
// A segment is one sequence and head group, cut into tiles of kTileKeys keys.
// A batch is split in one of two ways:
//
//   chunks  every segment into equal runs of tiles, at most one per block
//           (plan_fits below);
//   line    sequence after sequence, head group after head group, tile after
//           tile: block k takes units [k * per, (k + 1) * per) of that line,
//           but a segment of up to kShort tiles whole, in the block that it
//           starts in.
//
// A segment that lies in one block is finished there.  One that is cut leaves
// a partial result per block; a block is the inside or the end of at most one
// cut segment (its first) and the start of at most one (its last), so two
// partial slots and one arrival counter per block are enough for any batch.

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

// Tiles of a segment that a line does not cut, and that one warp takes alone where several follow one another.  300
// sequences of up to 250 keys, 4 heads: 26 us with 16, 39 with 4; of up to 1,000 keys: 60 with 16, 83 with 64.
constexpr int kShort = 16;
constexpr int kLeast = 8;         // units a block takes at least
constexpr int kInlineParts = 24;  // partial results that the last block to arrive joins itself (at most 32)
// Tiles a block may take beyond an even share to keep to one segment.  8 heads x 128 bf16, us with 0, 64 and no limit:
// 1 x 2,000 keys 12.5, 8.2, 8.2; 3 x 4,096 17.1, 13.5, 13.5; 16 x 4,096 47.5, 43.9, 43.9; 18 x 4,096 52.1, 48.5, 48.5;
// 12 x 4,096 38.1, 38.1, 36.9; 13 x 8,192 73.1, 73.1, 69.5; 12 ragged of up to 8,000 52.9, 52.9, 40.6.
constexpr int kWaste = 64;
constexpr int kPlanTries = 4;     // chunk sizes that are tried

// Blocks of a launch that has `most`: no more than the longest batch of the table could keep busy.
SF_HD int attend_blocks(int64_t longest_units, int most) {
  const int64_t want = (longest_units + kLeast - 1) / kLeast;
  return (int)(want < most ? want : most);
}

// May a segment lie in more than kInlineParts blocks?  One of t tiles lies in
// at most (t - 1) / kLeast + 2, and, having at least 1 / heads of all units, in
// at most blocks / heads + 2.
SF_HD bool may_need_join(int longest_tiles, int heads, int blocks) {
  return (longest_tiles - 1) / kLeast + 2 > kInlineParts && blocks / heads + 2 > kInlineParts;
}

// -- line

// Units in front of a block's work: what is left, from tile t0 on, of a short segment of an earlier block.
SF_HD int skipped(int t0, int tiles) { return t0 > 0 && tiles <= kShort ? tiles - t0 : 0; }

// What the block at unit u, tile t0 of a segment, takes of it: tiles [t0, end), as one of the blocks b0 .. b1.
struct LineTake {
  int end, b0, b1;
};
SF_HD LineTake take_of_line(int block, int64_t u, int64_t u_end, int t0, int tiles, int64_t per) {
  const int64_t first = u - t0;
  const int end = tiles > kShort && u_end - u < tiles - t0 ? t0 + (int)(u_end - u) : tiles;
  return LineTake{end, t0 == 0 ? block : first_block(first, per), end == tiles ? block : last_block(first, tiles, per)};
}

// -- chunks of at most `size` tiles

SF_HD int chunks_of(int tiles, int size) { return (int)(((unsigned)tiles + size - 1) / (unsigned)size); }
// Tiles of each of a segment's n chunks; the last may be short or empty.
SF_HD int chunk_tiles(int tiles, int n) { return (int)((unsigned)(tiles + n - 1) / (unsigned)n); }
// The next size to try where `chunks` are more than there are blocks.
SF_HD int wider_chunks(int size, int chunks, int blocks) {
  return size + (int)quotient((int64_t)size * (chunks - blocks), blocks) + 1;
}
// Is there a block for every chunk, and none of them much longer than an even share?
SF_HD bool plan_fits(int chunks, int longest, int64_t share, int blocks) {
  return chunks <= blocks && longest <= share + kWaste;
}

}  // namespace sf
