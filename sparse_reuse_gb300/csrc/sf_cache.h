// Host-side internals of the paged-cache operators: the object and the launch
// functions of every kernel.
#pragma once

#include <cuda_runtime.h>

#include "sf_cache_index.h"
#include "sf_common.cuh"
#include "specfold_cache.h"

namespace sf {
// A cut segment that the join kernel finishes, by its first block.
struct CacheJoin {
  int n;      // partial results; 0 = nothing to do
  int s, h0, nh;
  int first;  // slot of the first one; the others are slots 2 (block + 1), 2 (block + 2), ...
};
}  // namespace sf

struct sf_cache {
  sf_cache_shapes s{};
  int device = 0;
  int sm_count = 148;
  float* rope = nullptr;      // [max_pos][cos half | sin half]
  float* scores = nullptr;    // [max_seqs][n_q_heads][max_len, padded to 4] scaled scores in log2 units (track_weights)
  float2* stats = nullptr;    // [max_seqs][n_q_heads] reference and factor of each softmax (track_weights)
  float* parts = nullptr;     // partial results of sf_cache_attend, two per block
  unsigned* arrived = nullptr;  // [blocks] arrival counters, 0 between calls
  sf::CacheJoin* joins = nullptr;  // [blocks]
  unsigned* err = nullptr;    // [kCacheErrWords] pinned, written by the kernels through its device address
  unsigned* err_dev = nullptr;
  char last_error[256] = {0};
};

namespace sf {

// Device checks: one word each in pinned host memory, set to 1 by the kernel
// that met the case.  A word per check needs no atomic, costs a clean call
// nothing and no copy back.
enum CacheErr { kCacheBadPage = 0, kCacheBadLength = 1, kCacheBadRow = 2, kCacheErrWords = 3 };

__device__ __forceinline__ void cache_error(unsigned* err, CacheErr which) {
  *reinterpret_cast<volatile unsigned*>(err + which) = 1u;
}

struct CacheAppendArgs {
  const void* qkv; int64_t ld_qkv;
  void* q_out; int64_t ld_q;
  const float* q_gain; const float* k_gain;
  const int32_t* index; const int32_t* pos; const int32_t* seq;
  PageTable table;
  void* k; void* v;
  const float* rope;
  int T, S, nq, nkv, hd, max_pos;
  int64_t limit;   // positions a sequence may have
  float eps;
  unsigned* err;
};
cudaError_t launch_cache_append(cudaStream_t st, const CacheAppendArgs& a, int bf16, int sm_count);

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
  float2* stats;
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
