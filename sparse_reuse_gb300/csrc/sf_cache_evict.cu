// Eviction from the paged cache by accumulated attention weight
// (specfold_cache.h): choose the kept positions of every (sequence, KV head)
// and move their weights, then move their keys and values to the front.
//
// Bytes: every weight in and out, every kept key and value in and out.  The
// choice is latency (a handful of passes over one head's weights on the SM),
// the move is DRAM bandwidth.
#include <cmath>

#include "sf_cache.h"
#include "sf_tc.cuh"

namespace sf {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// Order-preserving map of a weight to an unsigned key: NaN 0, then -inf ... -0
// = 0 ... +inf (0xff800000).
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2 * kSelThreads;

// A cluster of `cl` blocks per (sequence, KV head); block r holds the r-th
// part of the weights in shared memory.
//
// The need-th largest candidate key is found by narrowing [lo, hi]: the range
// is cut into at most kBins equal bins (keys of positive floats are piecewise
// logarithmic, so weights spread over many bins), the bin that holds it is the
// next range: three passes at most for any 32-bit keys.  The lowest bin is
// never counted (if the others do not reach, it is the one), which keeps the
// usual crowd of zero weights out of the shared-memory atomics.
// Then positions are written in order: all keys above the threshold, and the
// first `ties` equal to it.
__global__ void __launch_bounds__(kSelThreads) cache_select_kernel(const __grid_constant__ CacheEvictArgs a, int cl) {
  extern __shared__ float sw[];
  __shared__ unsigned hist[2][kBins];
  __shared__ unsigned red[2][kSelWarps];
  __shared__ unsigned pub[2][2];  // published to the cluster: (min, max), then (above, equal)
  __shared__ unsigned found[3];   // bin, keys above it, keys in it
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x / cl, s = blockIdx.y;
  const int rank = blockIdx.x % cl;
  auto meet = [&]() {
    if (cl > 1)
      tc::cluster_sync_all();
    else
      __syncthreads();
  };
  auto remote = [&](const unsigned* p, int r) {
    return r == rank ? *p : ld_cluster_u32(tc::map_to_rank(tc::smem_u32(p), r));
  };
  pdl_wait();
  pdl_trigger();
  bool bad;
  const int len = checked_len(a.lens[s], a.limit, &bad);
  if (bad && threadIdx.x == 0) cache_error(a.err, kCacheBadLength);
  const int64_t head = (int64_t)s * a.nkv + c;
  int32_t* kept = a.kept + head * a.budget;
  const float* w = a.w + head * a.ld_w;
  float* w_out = a.w_out + head * a.ld_w;
  const int all = rank * kSelThreads + threadIdx.x, stride = cl * kSelThreads;
  if (len <= a.budget) {  // the same for the whole cluster
    for (int i = all; i < a.budget; i += stride) {
      kept[i] = i < len ? i : -1;
      if (i < len) w_out[i] = w[i];
    }
    return;
  }
  const int chunk = (len + cl - 1) / cl, j0 = min(rank * chunk, len), n = min(chunk, len - j0);
  const int lo_j = a.n_first - j0, hi_j = len - a.n_recent - j0;  // candidates, in this block's indexes
  unsigned kmin = ~0u, kmax = 0u;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kSelThreads) {
    const float x = w[j0 + i];
    sw[i] = x;
    if (i >= lo_j && i < hi_j) {
      const uint32_t k = weight_key(x);
      kmin = min(kmin, k);
      kmax = max(kmax, k);
    }
  }
  kmin = __reduce_min_sync(kFull, kmin);
  kmax = __reduce_max_sync(kFull, kmax);
  if (lane == 0) {
    red[0][warp] = kmin;
    red[1][warp] = kmax;
  }
  for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[0][i] = 0u;
  __syncthreads();
  kmin = __reduce_min_sync(kFull, red[0][lane]);
  kmax = __reduce_max_sync(kFull, red[1][lane]);
  if (threadIdx.x == 0) {
    pub[0][0] = kmin;
    pub[0][1] = kmax;
  }
  meet();  // also: every weight of this head is in shared memory, w_out may be w
  for (int r = 0; r < cl; ++r) {
    kmin = min(kmin, remote(&pub[0][0], r));
    kmax = max(kmax, remote(&pub[0][1], r));
  }
  int need = a.budget - a.n_first - a.n_recent;  // below the number of candidates, since budget < len
  uint32_t thr = ~0u;                            // keys above it are kept (none is above ~0)
  int ties = 0;                                  // and the first `ties` equal to it
  if (need > 0) {
    uint32_t lo = kmin, hi = kmax;
    for (int p = 0;; p ^= 1) {
      const uint32_t range = hi - lo;
      const int bits = 32 - __clz(range), shift = bits > 11 ? bits - 11 : 0;  // kBins = 2^11
#pragma unroll 4
      for (int i = threadIdx.x; i < n; i += kSelThreads) {
        const uint32_t k = weight_key(sw[i]);
        if (i >= lo_j && i < hi_j && k >= lo && k <= hi) {
          const uint32_t b = (k - lo) >> shift;
          if (b) atomicAdd(&hist[p][b], 1u);
        }
      }
      if (threadIdx.x == 0) found[0] = 0u;
      meet();
      // thread t takes bins kBins - 1 - 2 t and the one below it
      const int b1 = kBins - 1 - 2 * threadIdx.x;
      unsigned h1 = 0, h0 = 0;
      for (int r = 0; r < cl; ++r) {
        h1 += remote(&hist[p][b1], r);
        h0 += remote(&hist[p][b1 - 1], r);
      }
      for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[p ^ 1][i] = 0u;
      unsigned sum = h1 + h0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(kFull, sum, o);
        if (lane >= o) sum += y;
      }
      if (lane == 31) red[0][warp] = sum;
      __syncthreads();
      const unsigned others = red[0][lane];
      const unsigned before = __reduce_add_sync(kFull, lane < warp ? others : 0u);
      const unsigned total = __reduce_add_sync(kFull, others);
      const unsigned incl = before + sum, mid = incl - h0, excl = mid - h1;
      if (b1 > 0 && excl < (unsigned)need && mid >= (unsigned)need) {
        found[0] = b1;
        found[1] = excl;
        found[2] = h1;
      } else if (b1 > 1 && mid < (unsigned)need && incl >= (unsigned)need) {
        found[0] = b1 - 1;
        found[1] = mid;
        found[2] = h0;
      }
      __syncthreads();
      const uint32_t bin = found[0];
      const unsigned above = bin ? found[1] : total;
      const bool whole = bin && found[2] == (unsigned)need - above;
      need -= (int)above;
      lo += bin << shift;
      if (whole) {  // the bin's keys are the last ones needed
        thr = lo - 1;
        break;
      }
      hi = min(hi, lo + ((1u << shift) - 1u));
      if (shift == 0 || lo == hi) {
        thr = lo;
        ties = need;
        break;
      }
      __syncthreads();  // found and red are read
    }
  }
  // order: warp w of the block takes a run of its positions
  const int run = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int i0 = min(warp * run, n), i1 = min(i0 + run, n);
  unsigned n_above = 0, n_equal = 0;
  for (int i = i0; i < i1; i += 32) {
    const int x = i + lane;
    const bool in = x < i1, cand = in && x >= lo_j && x < hi_j;
    const uint32_t k = in ? weight_key(sw[x]) : 0u;
    n_above += __popc(__ballot_sync(kFull, (in && !cand) || (cand && k > thr)));
    n_equal += __popc(__ballot_sync(kFull, cand && k == thr));
  }
  __syncthreads();
  if (lane == 0) {
    red[0][warp] = n_above;
    red[1][warp] = n_equal;
  }
  __syncthreads();
  const unsigned ra = red[0][lane], re = red[1][lane];
  unsigned at_above = __reduce_add_sync(kFull, lane < warp ? ra : 0u);
  unsigned at_equal = __reduce_add_sync(kFull, lane < warp ? re : 0u);
  if (cl > 1) {
    const unsigned ta = __reduce_add_sync(kFull, ra), te = __reduce_add_sync(kFull, re);
    if (threadIdx.x == 0) {
      pub[1][0] = ta;
      pub[1][1] = te;
    }
    meet();
    for (int r = 0; r < rank; ++r) {
      at_above += remote(&pub[1][0], r);
      at_equal += remote(&pub[1][1], r);
    }
  }
  for (int i = i0; i < i1; i += 32) {
    const int x = i + lane;
    const bool in = x < i1, cand = in && x >= lo_j && x < hi_j;
    const float v = in ? sw[x] : 0.f;
    const uint32_t k = weight_key(v);
    const bool above = (in && !cand) || (cand && k > thr), equal = cand && k == thr;
    const unsigned ba = __ballot_sync(kFull, above), be = __ballot_sync(kFull, equal);
    const unsigned below = (1u << lane) - 1u;
    const unsigned ia = at_above + __popc(ba & below), ie = at_equal + __popc(be & below);
    const unsigned at = ia + min(ie, (unsigned)ties);
    if ((above || (equal && ie < (unsigned)ties)) && at < (unsigned)a.budget) {
      kept[at] = j0 + x;
      w_out[at] = v;
    }
    at_above += __popc(ba);
    at_equal += __popc(be);
  }
  for (int i = a.budget + all; i < len; i += stride) w_out[i] = 0.f;
  if (cl > 1) tc::cluster_sync_all();  // nobody leaves while its shared memory may be read
}

// ---- keys and values -----------------------------------------------------------

constexpr int kMoveThreads = 256;
constexpr int kMoveItems = 4;  // 16-byte pieces a thread has in flight

// To other pages: every 16-byte piece on its own.  Consecutive threads take
// consecutive pieces of an output position (all heads of it), a thread
// kMoveItems positions of the block's run.
__global__ void __launch_bounds__(kMoveThreads) cache_copy_kernel(const __grid_constant__ CacheEvictArgs a, int row16) {
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.y, part = blockIdx.x & 1;
  const int wide = a.nkv * row16;                       // pieces of a position
  bool bad;
  const int n_keep = min(checked_len(a.lens[s], a.limit, &bad), a.budget);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.lens_out[s] = n_keep;  // lens_out may be lens: n_keep reads back as itself
  const uint4* src = static_cast<const uint4*>(part ? a.v : a.k);
  uint4* dst = static_cast<uint4*>(part ? a.v_out : a.k_out);
  // the block's first piece as (position, piece of it); the rest in 32 bits
  const int64_t base = (int64_t)(blockIdx.x >> 1) * kMoveThreads * kMoveItems;
  const int base_i = (int)(base / wide), base_p = (int)(base - (int64_t)base_i * wide);
  if (base_i >= n_keep) return;
  uint4 x[kMoveItems];
  int64_t to[kMoveItems];
#pragma unroll
  for (int u = 0; u < kMoveItems; ++u) {
    const int e = base_p + (int)threadIdx.x + u * kMoveThreads;
    const int i = base_i + e / wide, hp = e % wide;
    to[u] = -1;
    if (i < n_keep) {
      const int c = hp / row16;
      const int64_t from = page_slot(a.table, s, a.kept[((int64_t)s * a.nkv + c) * a.budget + i]);
      const int64_t dst_slot = page_slot(a.table_out, s, i);
      if (from < 0 || dst_slot < 0) {
        cache_error(a.err, kCacheBadPage);
      } else {
        to[u] = dst_slot * wide + hp;
        x[u] = src[from * wide + hp];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kMoveItems; ++u)
    if (to[u] >= 0) dst[to[u]] = x[u];
}

constexpr int kShiftThreads = 512;

// In place.  kept[i] >= i, so a chunk of rows [i0, i1) only overwrites rows
// that this chunk or an earlier one reads: a block reads the chunk into
// registers, meets, and writes it.  Different bytes of a row never meet, so
// the rows of a (sequence, KV head, keys or values) are cut into slices of
// `pieces` times 16 bytes, a block each.
__global__ void __launch_bounds__(kShiftThreads) cache_shift_kernel(const __grid_constant__ CacheEvictArgs a, int row16,
                                                                    int pieces) {
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.y, slices = row16 / pieces;
  const int slice = blockIdx.x % slices, part = blockIdx.x / slices % 2, c = blockIdx.x / slices / 2;
  bool bad;
  const int n_keep = min(checked_len(a.lens[s], a.limit, &bad), a.budget);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.lens_out[s] = n_keep;  // lens_out may be lens: n_keep reads back as itself
  const int32_t* kept = a.kept + ((int64_t)s * a.nkv + c) * a.budget;
  uint4* pool = static_cast<uint4*>(part ? a.v_out : a.k_out);
  const int rows = kShiftThreads / pieces, piece = threadIdx.x % pieces + slice * pieces;
  for (int i0 = 0; i0 < n_keep; i0 += rows * kMoveItems) {
    uint4 x[kMoveItems];
    int64_t to[kMoveItems];
#pragma unroll
    for (int u = 0; u < kMoveItems; ++u) {
      const int i = i0 + u * rows + (int)threadIdx.x / pieces;
      to[u] = -1;
      if (i < n_keep) {
        const int j = kept[i];
        if (j != i) {
          const int64_t from = page_slot(a.table, s, j), dst = page_slot(a.table_out, s, i);
          if (from < 0 || dst < 0) {
            cache_error(a.err, kCacheBadPage);
          } else {
            to[u] = (dst * a.nkv + c) * row16 + piece;
            x[u] = pool[(from * a.nkv + c) * row16 + piece];
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveItems; ++u)
      if (to[u] >= 0) pool[to[u]] = x[u];
  }
}

// Blocks of a cluster for `heads` (sequence, KV head) pairs of up to `limit`
// weights: kSelCap of them a block at most; more blocks while each keeps
// kSelKeys and the launch stays one wave of two blocks per SM.
constexpr int kSelCap = 32768, kSelKeys = 8192;
int select_cluster(int64_t limit, int64_t heads, int sm_count) {
  int cl = 1;
  while (cl < 8 && (limit > (int64_t)cl * kSelCap ||
                    (limit >= 2 * cl * kSelKeys && heads * cl * 2 <= 2 * sm_count)))
    cl *= 2;
  return cl;
}

}  // namespace

cudaError_t prepare_cache_evict() {
  return cudaFuncSetAttribute(cache_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelCap * 4);
}

cudaError_t launch_cache_evict(cudaStream_t st, const CacheEvictArgs& a, int bf16, int sm_count) {
  const int cl = select_cluster(a.limit, (int64_t)a.S * a.nkv, sm_count);
  const size_t smem = (size_t)((a.limit + cl - 1) / cl) * sizeof(float);
  cudaError_t e = launch_pdl_cluster(st, dim3(cl * a.nkv, a.S), dim3(kSelThreads), smem, dim3(cl), cache_select_kernel,
                                     a, cl);
  if (e != cudaSuccess) return e;
  const int row16 = a.hd * (bf16 ? 2 : 4) / 16;
  if (a.in_place) {
    const int pieces = 2;
    return launch_pdl(st, dim3(a.nkv * 2 * (row16 / pieces), a.S), dim3(kShiftThreads), 0, 1, cache_shift_kernel, a,
                      row16, pieces);
  }
  const int64_t items = (int64_t)a.budget * a.nkv * row16;
  const int64_t runs = (items + kMoveThreads * kMoveItems - 1) / (kMoveThreads * kMoveItems);
  return launch_pdl(st, dim3((unsigned)(2 * runs), a.S), dim3(kMoveThreads), 0, 1, cache_copy_kernel, a, row16);
}

}  // namespace sf
