// Host-side internals of the paged-cache operators: the object and the launch
// functions of every kernel.
#pragma once

#include <cuda_runtime.h>

#include "sf_cache_index.h"
#include "sf_common.cuh"
#include "specfold_cache.h"

namespace sf {
// How positions turn a head: the first `dim` of its dimensions, in pairs
// (j, j + dim / 2), or (2 j, 2 j + 1) where `neighbours`.
struct Rotary {
  int dim;
  bool neighbours;
};

// A cut segment that the join kernel finishes, by its first block.
struct CacheJoin {
  int n;      // partial results; 0 = nothing to do
  int s, h0, nh;
  int first;  // slot of the first one; the others are slots 2 (block + 1), 2 (block + 2), ...
};
}  // namespace sf

namespace sf {
// A tile of query vectors cut over several thread blocks, by the first of them.
struct RowsJoin {
  int n;     // thread blocks that share it; 0 = nothing to do
  int nv;    // its query vectors v0 .. v0 + nv - 1, of the sequence whose rows start at row0
  int row0, kvh, v0;
};
}  // namespace sf

struct sf_cache {
  sf_cache_shapes s{};
  sf_cache_options o{};
  sf::Rotary rotary{};
  int device = 0;
  int sm_count = 148;
  float* rope = nullptr;      // [max_pos][cos half | sin half]
  float* scores = nullptr;    // [max_seqs][n_q_heads][max_len, padded to 4] scaled scores in log2 units (track_weights)
  float2* stats = nullptr;    // [max_seqs][n_q_heads] reference and factor of each softmax (track_weights)
  float* parts = nullptr;     // partial results of sf_cache_attend, two per block
  unsigned* arrived = nullptr;  // [blocks] arrival counters, 0 between calls
  sf::CacheJoin* joins = nullptr;  // [blocks]
  // sf_cache_attend_rows and _shared (max_rows > 0)
  float* row_parts = nullptr;      // partial results of cut tiles, two slots per thread block
  float2* row_ml = nullptr;        // their maxima and denominators
  sf::RowsJoin* row_joins = nullptr;  // [thread blocks]
  float* tail_o = nullptr;         // [max_rows][n_q_heads][head_dim] the sequences' own parts (shared)
  float2* tail_ml = nullptr;       // [max_rows][n_q_heads]
  float* whole_o = nullptr;        // the same of the prefixes
  float2* whole_ml = nullptr;
  int stall = 0;                   // sf_cache_inject_stall
  unsigned* err = nullptr;    // [kCacheErrWords] pinned, written by the kernels through its device address
  unsigned* err_dev = nullptr;
  char last_error[256] = {0};
};

namespace sf {

// Device checks: one word each in pinned host memory, set to 1 by the kernel
// that met the case.  A word per check needs no atomic, costs a clean call
// nothing and no copy back.
enum CacheErr { kCacheBadPage = 0, kCacheBadLength = 1, kCacheBadRow = 2, kCacheStall = 3, kCacheErrWords = 4 };

__device__ __forceinline__ void cache_error(unsigned* err, CacheErr which) {
  *reinterpret_cast<volatile unsigned*>(err + which) = 1u;
}

// The signal between the warps of the rows kernel that sf_cache_inject_stall withholds.
enum CacheStallAt {
  kStallNone, kStallPart, kStallPartRead, kStallQueries, kStallKeys, kStallKeysRead, kStallValues, kStallValuesRead,
  kStallScores, kStallWeights, kStallLateWeights, kStallTurn, kStallOutputs, kStallMeet, kStallEnd
};

struct CacheAppendArgs {
  const void* qkv; int64_t ld_qkv;
  void* q_out; int64_t ld_q;
  const float* q_gain; const float* k_gain;
  const int32_t* index; const int32_t* pos; const int32_t* seq;
  PageTable table;
  void* k; void* v;
  const float* rope;  // [max_pos][cos, sin: rotary.dim / 2 each]
  Rotary rotary;
  int T, S, nq, nkv, hd, max_pos;
  int64_t limit;   // positions a sequence may have
  float eps;
  unsigned* err;
};
cudaError_t launch_cache_append(cudaStream_t st, const CacheAppendArgs& a, int bf16, int sm_count);

struct CacheTurnArgs {
  void* k;
  PageTable table;
  const int32_t* lens;
  const int32_t* from; const int32_t* to; int64_t ld_pos;
  const float* rope;
  Rotary rotary;
  float unscale;   // 1 / the magnitude of the table
  int S, nkv, hd, max_pos;
  int64_t limit;
  unsigned* err;
};
cudaError_t launch_cache_turn(cudaStream_t st, const CacheTurnArgs& a, int bf16, int sm_count);

struct CacheAttendArgs {
  const void* q; int64_t ld_q;
  const void* k; const void* v;
  PageTable table;
  const int32_t* lens;
  int S, nq, nkv, hd;
  int64_t limit;
  float scale_log2;
  void* out; int64_t ld_out;
  const float* w_in; float* w_out; int64_t ld_w;
  float* scores; int64_t ld_scores;
  float2* stats;      // reference and factor of each softmax; with state_o its maximum and denominator
  float* state_o;     // [S][nq][hd] or null: the outputs in fp32 go here instead of `out`
  float* parts;       // two partial results per block: output [heads][hd], max [heads], denominator [heads]
  unsigned* arrived;  // [blocks] arrivals at a cut segment, by its first block; 0 between calls
  CacheJoin* joins;   // [blocks]
  bool join;          // a join kernel follows
  int blocks;         // of the attention kernel
  int group, nsub, heads;  // query heads of a KV head, parts they are taken in, nkv * nsub
  unsigned* err;
};
// Blocks of the largest launch on sm_count SMs, floats of `parts` that each needs, and the kernels' shared-memory limits (once per process and device).
int cache_attend_blocks(int sm_count);
int64_t cache_attend_part_floats(const sf_cache_shapes& s);
cudaError_t prepare_cache_attend();
cudaError_t launch_cache_attend(cudaStream_t st, const CacheAttendArgs& a, int bf16, int sm_count);

struct CacheRowsArgs {
  const void* q; int64_t ld_q; int T;
  const void* k; const void* v;
  PageTable table;
  const int32_t* lens; const int32_t* starts; int S;
  int nq, nkv, group;
  int64_t limit;
  float scale_log2;
  void* out; int64_t ld_out;
  float* lse;              // [T][nq] or null
  const float* tail_o;     // [T][nq][hd] normalised output over other keys, to be joined to every row, or null
  const float2* tail_ml;   // [T][nq] its maximum and denominator
  float* whole_o;          // [T][nq][hd] with a tail: what the tiles gave
  float2* whole_ml;        // [T][nq]
  float* parts; float2* part_ml;
  RowsJoin* joins;         // [ctas]
  int ctas, least;         // thread blocks; units that each takes at least
  uint32_t wait_ns;        // what a wait inside the kernel takes at most
  int stall;               // CacheStallAt
  unsigned* err;
};
int cache_rows_ctas(int sm_count, int bf16);
int cache_rows_slot_rows(int bf16);  // query vectors of a partial slot
constexpr int kTcTileRows = 256;
cudaError_t prepare_cache_rows();
cudaError_t prepare_cache_rows_tc();
// The bf16 tiles (cut ones as partial results).
cudaError_t launch_cache_rows_tc(cudaStream_t st, const CacheRowsArgs& a, int hd);
cudaError_t launch_cache_rows(cudaStream_t st, const CacheRowsArgs& a, int bf16, int hd, int sm_count);

struct CacheEvictArgs {
  const void* k; const void* v;
  PageTable table;
  void* k_out; void* v_out;
  PageTable table_out;
  const int32_t* lens;
  const float* w; float* w_out; int64_t ld_w;
  int32_t* lens_out; int32_t* kept;
  int S, nkv, hd, budget, n_first, n_recent;
  int64_t limit;
  bool in_place;
  unsigned* err;
};
cudaError_t prepare_cache_evict();
cudaError_t launch_cache_evict(cudaStream_t st, const CacheEvictArgs& a, int bf16, int sm_count);

}  // namespace sf
