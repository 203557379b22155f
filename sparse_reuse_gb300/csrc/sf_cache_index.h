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
constexpr int kMaxCallRows = 1048576;  // rows of a call
constexpr int kMaxGroups = 65536;      // groups of one

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

// Tails of a batch (sf_cache_attend_shared) without a plan: the warps (1, 2 or 4; at most `most`) that each segment gets
// where the table lets a segment have up to `longest` tiles; 0: planned blocks by the real lengths instead.  A block
// takes some 6 us a segment, a warp 0.6 us a tile, and a long segment among short ones is not shared out: so a warp may
// get 16 tiles for every segment of an SM, but never more than kTailMost.  us by warps and by blocks, 8 KV heads x 128
// bf16 (all of the longest length; random ones up to it; one of it, the others 50):
//   8 x 700 keys       16.5, 16.4   16.3, 15.0   16.3, 14.5     128 x 2,048   167, 178   110, 115    45, 23
//   36 x 700           22.4, 30.9   17.9, 25.6   16.9, 20.1     512 x 1,024   324, 343   180, 207    58, 45
//   128 x 700          68.7, 78.2   45.1, 52.5   24.1, 23.0     512 x 4,096  1213, 1290  657, 689   158, 45
//   512 x 700           229, 248     130, 147    48.7, 43.8     1,024, one of 32,768                1115, 90
constexpr int kTailMost = 48, kTailLeast = 4;
SF_HD int tail_warps(int longest, int64_t segments, int most, int sm_count) {
  int w = 1;
  while (w < most && longest > 4 * w && segments * 2 * w <= 16 * (int64_t)sm_count) w *= 2;
  const int64_t share = 16 * segments / sm_count;
  const int64_t tiles = share < kTailLeast ? kTailLeast : share > kTailMost ? kTailMost : share;
  return longest <= tiles * w ? w : 0;
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

// ---- the split of blocks of rows (sf_cache_attend_rows) over thread blocks ------
//
// The rows of a sequence and one KV head are `rows * group` query vectors,
// vector v being row v / group, head v % group of the KV head.  They are taken
// in halves of `half` vectors, `pair` (1 or 2) of them together as a tile (its
// last one may have fewer), over the sequence's keys in blocks of `block`.  The
// batch is a line of units, about equal times: sequence after sequence, KV head
// after KV head, tile after tile, a tile being `fixed` units and then one run of
// cost[halves - 1] for each of its blocks.  Thread block k takes the blocks that
// start in units [k * per, (k + 1) * per) of it.
//
// A tile whose blocks all belong to one thread block is finished there.  One
// that is cut leaves a partial result in each; a thread block is the inside or
// end of at most one cut tile (its first) and the start of at most one (its
// last): two slots each are enough.

// a / b for non-negative a and positive b; small ones, the usual case, by a
// reciprocal of fp32 and one correction: below 2^22 the product is less than 1
// off (two roundings, 3 * 2^-24 of it), a third of the latency of a division.
SF_HD int64_t quick_quotient(int64_t a, int64_t b) {
#ifdef __CUDA_ARCH__
  if ((((uint64_t)a | (uint64_t)b) >> 22) == 0) {
    const unsigned x = (unsigned)a, y = (unsigned)b;
    unsigned q = __float2uint_rz(__uint2float_rn(x) * __frcp_rn(__uint2float_rn(y)));
    const int r = (int)(x - q * y);
    q += r < 0 ? -1 : r >= (int)y ? 1 : 0;
    return q;
  }
#endif
  return quotient(a, b);
}

struct RowsShape {
  int group;  // query heads of a KV head
  int nkv;
  int half, pair, block;
  int fixed, cost[2];
};

SF_HD int row_halves(const RowsShape& a, int rows) {
  return (int)(((unsigned)rows * (unsigned)a.group + a.half - 1) / (unsigned)a.half);
}
SF_HD int row_blocks(const RowsShape& a, int len) { return (int)((unsigned)(len + a.block - 1) / (unsigned)a.block); }
SF_HD int64_t tile_units(const RowsShape& a, int halves, int blocks) {
  return a.fixed + (int64_t)a.cost[halves - 1] * blocks;
}
// Units of one KV head of a sequence.
SF_HD int64_t row_units(const RowsShape& a, int rows, int len) {
  const int halves = row_halves(a, rows), blocks = row_blocks(a, len);
  if (halves == 0 || blocks == 0) return 0;
  const int tiles = a.pair == 2 ? halves >> 1 : halves;
  return tiles * tile_units(a, a.pair, blocks) + (tiles * a.pair < halves ? tile_units(a, 1, blocks) : 0);
}

// What a thread block takes of one tile: blocks [b0, b1) of nb; none where b0 >= b1.
struct RowsPart {
  int kvh;
  int v0, nv;    // the tile's query vectors
  int w;         // its halves
  int nb, b0, b1;
  int cost;
  int64_t u0;    // where its first block starts
};

// The tiles of one sequence, one after the other (quotients only at the start:
// they are on the critical path of a thread block's first loads).
struct RowsTiles {
  int rows, halves, tiles, nb;  // tiles: those of `pair` halves
  int kvh, x, b0;               // the next tile, and the first block to take of it
  int64_t at;                   // where it starts

  // From unit u on of a sequence whose own units start at `first`.
  SF_HD void start(const RowsShape& a, int rows_, int len, int64_t first, int64_t u) {
    rows = rows_;
    halves = row_halves(a, rows);
    tiles = a.pair == 2 ? halves >> 1 : halves;
    nb = row_blocks(a, len);
    kvh = x = b0 = 0;
    at = first;
    if (u <= first) return;
    const int64_t head = row_units(a, rows, len), tile = tile_units(a, a.pair, nb);
    kvh = (int)quick_quotient(u - first, head);
    const int64_t in_head = u - first - kvh * head;
    x = (int)quick_quotient(in_head, tile);
    if (x > tiles) x = tiles;
    at = u - (in_head - x * tile);
    const int cost = a.cost[x < tiles ? a.pair - 1 : 0];
    const int64_t u0 = at + a.fixed;
    b0 = u <= u0 ? 0 : (int)quick_quotient(u - u0 + cost - 1, cost);
  }
  SF_HD bool more(const RowsShape& a) const { return kvh < a.nkv; }
  // What a thread block whose units end at `end` takes of the next tile; then the one after it is next.
  SF_HD RowsPart take(const RowsShape& a, int64_t end) {
    RowsPart p;
    p.kvh = kvh;
    p.w = x < tiles ? a.pair : 1;
    p.cost = a.cost[p.w - 1];
    p.v0 = x * a.pair * a.half;
    p.nv = rows * a.group - p.v0 < p.w * a.half ? rows * a.group - p.v0 : p.w * a.half;
    p.nb = nb;
    p.b0 = b0;
    p.u0 = at + a.fixed;
    at = p.u0 + (int64_t)p.cost * nb;
    p.b1 = at <= end ? nb : end <= p.u0 ? 0 : (int)quick_quotient(end - p.u0 + p.cost - 1, p.cost);
    if (p.b1 > nb) p.b1 = nb;
    b0 = 0;
    if (++x * a.pair >= halves) {
      x = 0;
      ++kvh;
    }
    return p;
  }
};

// Thread blocks share a tile from the one in which its first block starts (whose part begins with block 0) to the one
// in which its last does.
SF_HD int rows_last_cta(const RowsPart& p, int64_t per) { return (int)quotient(p.u0 + (int64_t)p.cost * (p.nb - 1), per); }
// The partial slot of thread block `cta` for a cut tile.
SF_HD int rows_slot(int cta, bool first) { return 2 * cta + (first ? 1 : 0); }

}  // namespace sf
