// Eviction from the paged cache by accumulated attention weight
// (specfold_cache.h): choose the kept positions of every (sequence, KV head),
// then move their keys, values and weights to the front.
#include <cmath>

#include "sf_cache.h"

namespace sf {
namespace {

// Order-preserving map of a weight to an unsigned key: NaN 0, then -inf ... -0
// = 0 ... +inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelThreads = 512;

__device__ __forceinline__ int block_count(int v, int* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  int t = 0;
  for (int i = 0; i < kSelThreads / 32; ++i) t += red[i];
  return t;
}

// One CTA per (sequence, KV head).  Candidates are the positions between the
// protected first and last ones; the k-th largest key among them is found bit
// by bit from the top (the largest x with at least k keys >= x), then
// positions are written in order: all keys above it, and the first ones equal
// to it.
__global__ void __launch_bounds__(kSelThreads) cache_select_kernel(const __grid_constant__ CacheEvictArgs a) {
  __shared__ int red[kSelThreads / 32];
  __shared__ int base_sm[2];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x, s = blockIdx.y;
  bool bad;
  const int len = checked_len(a.lens[s], a.limit, &bad);
  if (bad && threadIdx.x == 0) cache_error(a.err, kCacheBadLength);
  int32_t* kept = a.kept + ((int64_t)s * a.nkv + c) * a.budget;
  const float* w = a.w + ((int64_t)s * a.nkv + c) * a.ld_w;
  const int n_keep = min(len, a.budget);
  for (int i = n_keep + threadIdx.x; i < a.budget; i += kSelThreads) kept[i] = -1;
  if (len <= a.budget) {
    for (int i = threadIdx.x; i < len; i += kSelThreads) kept[i] = i;
    return;
  }
  const int lo = a.n_first, hi = len - a.n_recent, need = a.budget - a.n_first - a.n_recent;
  uint32_t thr = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t x = thr | (1u << bit);
    int n = 0;
    for (int j = lo + threadIdx.x; j < hi; j += kSelThreads) n += weight_key(w[j]) >= x;
    if (block_count(n, red) >= need) thr = x;
  }
  int n = 0;
  for (int j = lo + threadIdx.x; j < hi; j += kSelThreads) n += weight_key(w[j]) > thr;
  const int ties = need - block_count(n, red);  // keys equal to thr still to take (need = 0: negative, none)
  if (threadIdx.x == 0) base_sm[0] = base_sm[1] = 0;
  __syncthreads();
  for (int j0 = 0; j0 < len; j0 += kSelThreads) {
    const int j = j0 + threadIdx.x;
    const bool fixed = j < len && (j < lo || j >= hi);
    const uint32_t key = (j >= lo && j < hi) ? weight_key(w[j]) : 0u;
    const bool above = need > 0 && j >= lo && j < hi && key > thr, equal = need > 0 && j >= lo && j < hi && key == thr;
    // ranks of this position among the equal ones and among the kept ones
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned b = __ballot_sync(0xffffffffu, equal);
    __syncthreads();
    if (lane == 0) red[warp] = __popc(b);
    __syncthreads();
    int rank = base_sm[0] + __popc(b & ((1u << lane) - 1u)), total_eq = 0;
    for (int i = 0; i < kSelThreads / 32; ++i) {
      if (i < warp) rank += red[i];
      total_eq += red[i];
    }
    const bool keep = fixed || above || (equal && rank < ties);
    b = __ballot_sync(0xffffffffu, keep);
    __syncthreads();
    if (lane == 0) red[warp] = __popc(b);
    __syncthreads();
    int at = base_sm[1] + __popc(b & ((1u << lane) - 1u)), total = 0;
    for (int i = 0; i < kSelThreads / 32; ++i) {
      if (i < warp) at += red[i];
      total += red[i];
    }
    if (keep && at < a.budget) kept[at] = j;
    __syncthreads();
    if (threadIdx.x == 0) {
      base_sm[0] += total_eq;
      base_sm[1] += total;
    }
    __syncthreads();
  }
}

constexpr int kMoveThreads = 256;

// One CTA per (sequence, KV head) and keys / values / weights.  kept[i] >= i,
// so an in-place chunk of rows [i0, i1) only overwrites rows that this chunk
// or an earlier one reads: read the chunk into registers, meet, write it.
__global__ void __launch_bounds__(kMoveThreads) cache_move_kernel(const __grid_constant__ CacheEvictArgs a, int row16) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x / 3, part = blockIdx.x % 3, s = blockIdx.y;
  bool bad;
  const int len = checked_len(a.lens[s], a.limit, &bad), n_keep = min(len, a.budget);
  const int32_t* kept = a.kept + ((int64_t)s * a.nkv + c) * a.budget;
  if (part == 2) {
    const int64_t at = ((int64_t)s * a.nkv + c) * a.ld_w;
    for (int i0 = 0; i0 < n_keep; i0 += kMoveThreads) {
      const int i = i0 + threadIdx.x;
      float w = 0.f;
      if (i < n_keep) w = a.w[at + kept[i]];
      __syncthreads();
      if (i < n_keep) a.w_out[at + i] = w;
    }
    __syncthreads();
    for (int i = n_keep + threadIdx.x; i < len; i += kMoveThreads) a.w_out[at + i] = 0.f;
    return;
  }
  const uint4* src = static_cast<const uint4*>(part ? a.v : a.k);
  uint4* dst = static_cast<uint4*>(part ? a.v_out : a.k_out);
  const int rows = kMoveThreads / row16, piece = threadIdx.x % row16;
  for (int i0 = 0; i0 < n_keep; i0 += rows) {
    const int i = i0 + threadIdx.x / row16;
    uint4 x;
    int64_t from = -1, to = -1;
    if (i < n_keep) {
      from = page_slot(a.table, s, kept[i]);
      to = page_slot(a.table_out, s, i);
      if ((from < 0 || to < 0) && piece == 0) cache_error(a.err, kCacheBadPage);
      if (from >= 0) x = src[(from * a.nkv + c) * row16 + piece];
    }
    __syncthreads();
    if (from >= 0 && to >= 0) dst[(to * a.nkv + c) * row16 + piece] = x;
  }
}

// Last, so that lens_out may be lens.
__global__ void cache_lens_kernel(const __grid_constant__ CacheEvictArgs a) {
  pdl_wait();
  pdl_trigger();
  for (int s = threadIdx.x; s < a.S; s += blockDim.x) {
    bool bad;
    a.lens_out[s] = min(checked_len(a.lens[s], a.limit, &bad), a.budget);
  }
}

}  // namespace

cudaError_t launch_cache_evict(cudaStream_t st, const CacheEvictArgs& a, int bf16, int) {
  cudaError_t e = launch_pdl(st, dim3(a.nkv, a.S), dim3(kSelThreads), 0, 1, cache_select_kernel, a);
  if (e != cudaSuccess) return e;
  e = launch_pdl(st, dim3(3 * a.nkv, a.S), dim3(kMoveThreads), 0, 1, cache_move_kernel, a, a.hd * (bf16 ? 2 : 4) / 16);
  if (e != cudaSuccess) return e;
  return launch_pdl(st, dim3(1), dim3(256), 0, 1, cache_lens_kernel, a);
}

}  // namespace sf
