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
// = 0 ... +inf (0xff800000); and back (-0 comes back as 0).
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_weight(uint32_t k) {
  if (k == 0u) return __uint_as_float(0x7fffffffu);
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void red_cluster_add(uint32_t addr, unsigned v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 4 * kSelThreads;  // 2^11
constexpr int kList = 256;              // keys that are ranked by comparing all pairs
constexpr int kSelCap = 32768;          // weights a block holds at most
static_assert(kSelCap / 32 <= 2 * kSelThreads, "two words of a bitmap a thread");

// A cluster of `cl` blocks per (sequence, KV head); block r holds the keys
// of the r-th part of the weights in shared memory.
//
// The need-th largest candidate key is found by narrowing [lo, hi]: the range
// is cut into at most kBins equal bins (keys of positive floats are piecewise
// logarithmic, so weights spread over many bins), and the bin that holds it is
// the next range, three passes at most for any 32-bit keys.  The lowest bin is
// never counted (if the others do not reach, it is the one), which keeps the
// usual crowd of zero weights out of the shared-memory atomics.  A block that
// is alone ranks the keys of the bin by comparison once they are few, usually
// after one pass.
//
// The choice is two bitmaps, positions certainly kept and positions at the
// threshold, of which the first `ties` are kept; a scan of their populations
// gives every kept position its place.
__global__ void __launch_bounds__(kSelThreads, 2) cache_select_kernel(const __grid_constant__ CacheEvictArgs a, int cl,
                                                                      int cap) {
  extern __shared__ __align__(16) unsigned keys[];               // [cap] of this block's positions
  unsigned* sure = keys + cap;                                   // [cap / 32] kept; later the final choice
  unsigned* tied = sure + cap / 32;                              // [cap / 32] at the threshold; later places
  __shared__ __align__(16) unsigned hist[kBins];
  __shared__ unsigned red[2][32];
  __shared__ unsigned pub[2][2];                                 // to the cluster: (min, max), then (kept, tied)
  __shared__ unsigned found[3];                                  // bin, keys above it, keys in it
  __shared__ uint2 list[kList];                                  // (key, position)
  __shared__ unsigned n_list, s_ties;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x / cl, s = blockIdx.y, rank = blockIdx.x % cl;
  auto meet = [&]() {
    if (cl > 1)
      tc::cluster_sync_all();
    else
      __syncthreads();
  };
  auto of_rank = [&](const unsigned* p, int r) {
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
  // candidates, in this block's indexes
  const int lo_j = min(max(a.n_first - j0, 0), n), hi_j = max(min(len - a.n_recent - j0, n), lo_j);
  const int words = (n + 31) / 32;
  unsigned kmin = ~0u, kmax = 0u;
#pragma unroll 8
  for (int i = threadIdx.x; i < n; i += kSelThreads) {
    const uint32_t k = weight_key(w[j0 + i]);
    keys[i] = k;
    if (i >= lo_j && i < hi_j) {
      kmin = min(kmin, k);
      kmax = max(kmax, k);
    }
  }
  reinterpret_cast<uint4*>(hist)[threadIdx.x] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x == 0) n_list = s_ties = 0u;
  kmin = __reduce_min_sync(kFull, kmin);
  kmax = __reduce_max_sync(kFull, kmax);
  if (lane == 0) {
    red[0][warp] = kmin;
    red[1][warp] = kmax;
  }
  __syncthreads();
  kmin = __reduce_min_sync(kFull, red[0][lane % kSelWarps]);
  kmax = __reduce_max_sync(kFull, red[1][lane % kSelWarps]);
  if (cl > 1) {
    if (threadIdx.x == 0) {
      pub[0][0] = kmin;
      pub[0][1] = kmax;
    }
    meet();  // every weight of this head is read (w_out may be w), every histogram empty
    for (int r = 0; r < cl; ++r) {
      kmin = min(kmin, of_rank(&pub[0][0], r));
      kmax = max(kmax, of_rank(&pub[0][1], r));
    }
  }
  int need = a.budget - a.n_first - a.n_recent;  // below the number of candidates, since budget < len
  uint32_t lo = kmin, hi = kmax;                 // the need-th largest key lies in [lo, hi]
  uint32_t thr = ~0u;                            // keys above it are kept (none is above ~0),
  int ties = 0;                                  // and the first `ties` equal to it
  bool rank_list = false;
  while (need > 0) {
    const uint32_t range = hi - lo;
    const int bits = 32 - __clz(range), shift = bits > 11 ? bits - 11 : 0;
#pragma unroll 8
    for (int i = lo_j + threadIdx.x; i < hi_j; i += kSelThreads) {
      const uint32_t k = keys[i] - lo, b = k >> shift;
      if (k <= range && b) atomicAdd(&hist[b], 1u);
    }
    __syncthreads();
    // thread t holds bins kBins - 1 - 4 t and the three below it
    uint4* mine = reinterpret_cast<uint4*>(hist) + (kSelThreads - 1 - threadIdx.x);
    uint4 h = *mine;
    if (rank != 0) {
      const unsigned v[4] = {h.x, h.y, h.z, h.w};
      const uint32_t to = tc::map_to_rank(tc::smem_u32(mine), 0);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (v[i]) red_cluster_add(to + 4 * i, v[i]);
      *mine = make_uint4(0, 0, 0, 0);
    }
    if (cl > 1) {
      meet();
      h = *mine;
    }
    if (rank == 0) {
      *mine = make_uint4(0, 0, 0, 0);
      unsigned sum = h.x + h.y + h.z + h.w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(kFull, sum, o);
        if (lane >= o) sum += y;
      }
      if (lane == 31) red[0][warp] = sum;
      __syncthreads();
      const unsigned others = lane < kSelWarps ? red[0][lane] : 0u;
      unsigned at = __reduce_add_sync(kFull, lane < warp ? others : 0u) + sum - (h.x + h.y + h.z + h.w);
      const unsigned total = __reduce_add_sync(kFull, others);
      const unsigned v[4] = {h.w, h.z, h.y, h.x};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (at < (unsigned)need && at + v[i] >= (unsigned)need) {
          found[0] = kBins - 1 - 4 * threadIdx.x - i;
          found[1] = at;
          found[2] = v[i];
        }
        at += v[i];
      }
      if (threadIdx.x == 0 && total < (unsigned)need) {  // the lowest bin; how many it holds is not known
        found[0] = 0u;
        found[1] = total;
        found[2] = ~0u;
      }
    }
    meet();
    const uint32_t bin = of_rank(&found[0], 0);
    const unsigned above = of_rank(&found[1], 0), inside = of_rank(&found[2], 0);
    need -= (int)above;
    lo += bin << shift;
    hi = min(hi, lo + ((1u << shift) - 1u));
    if (inside == (unsigned)need) {  // the bin's keys are the last ones needed
      thr = lo - 1;
      break;
    }
    if (lo == hi) {
      thr = lo;
      ties = need;
      break;
    }
    if (cl == 1 && inside <= kList) {
      thr = hi;
      rank_list = true;
      break;
    }
    // found is written again only after everybody has come to the next pass's meeting
  }
  // bitmaps; the keys still to be ranked into the list
  for (int x = warp; x < words; x += kSelWarps) {
    const int i = 32 * x + lane;
    const bool in = i < n, cand = in && i >= lo_j && i < hi_j;
    const uint32_t k = in ? keys[i] : 0u;
    const unsigned b = __ballot_sync(kFull, (in && !cand) || (cand && k > thr));
    const unsigned e = __ballot_sync(kFull, !rank_list && cand && k == thr);
    if (lane == 0) {
      sure[x] = b;
      tied[x] = e;
    }
    if (rank_list && cand && k >= lo && k <= hi) list[atomicAdd(&n_list, 1u)] = make_uint2(k, i);
  }
  __syncthreads();
  if (rank_list) {
    const int m = n_list;  // <= kList: the bin's population
    if (threadIdx.x < m) {
      const uint2 me = list[threadIdx.x];
      int greater = 0, equal = 0;
      for (int x = 0; x < m; ++x) {
        const uint32_t k = list[x].x;
        greater += k > me.x;
        equal += k == me.x;
      }
      const unsigned bit = 1u << (me.y & 31);
      if (greater + equal <= need) {
        atomicOr(&sure[me.y >> 5], bit);
      } else if (greater < need) {
        atomicOr(&tied[me.y >> 5], bit);
        s_ties = need - greater;  // the same from all of them
      }
    }
    __syncthreads();
    ties = s_ties;
  }
  // places: thread t takes words 2 t and 2 t + 1
  unsigned ws[2], we[2], pop = 0;  // populations, kept in the low half, tied in the high one (each <= 2^15)
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int x = 2 * threadIdx.x + i;
    ws[i] = x < words ? sure[x] : 0u;
    we[i] = x < words ? tied[x] : 0u;
    pop += __popc(ws[i]) + (__popc(we[i]) << 16);
  }
  unsigned sum = pop;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(kFull, sum, o);
    if (lane >= o) sum += y;
  }
  if (lane == 31) red[1][warp] = sum;
  __syncthreads();
  const unsigned others = lane < kSelWarps ? red[1][lane] : 0u;
  const unsigned before = __reduce_add_sync(kFull, lane < warp ? others : 0u) + sum - pop;
  unsigned at_sure = before & 0xffffu, at_tied = before >> 16;
  if (cl > 1) {
    const unsigned total = __reduce_add_sync(kFull, others);
    if (threadIdx.x == 0) {
      pub[1][0] = total & 0xffffu;
      pub[1][1] = total >> 16;
    }
    meet();
    for (int r = 0; r < rank; ++r) {
      at_sure += of_rank(&pub[1][0], r);
      at_tied += of_rank(&pub[1][1], r);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int x = 2 * threadIdx.x + i;
    const unsigned pe = __popc(we[i]);
    unsigned take = at_tied >= (unsigned)ties ? 0u : min(pe, (unsigned)ties - at_tied), some = 0u;
    if (take == pe) {
      some = we[i];
    } else {
      for (unsigned left = we[i]; take; --take, left &= left - 1) some |= left & (0u - left);
    }
    if (x < words) {
      sure[x] = ws[i] | some;
      tied[x] = at_sure + min(at_tied, (unsigned)ties);
    }
    at_sure += __popc(ws[i]);
    at_tied += pe;
  }
  __syncthreads();
#pragma unroll 4
  for (int x = warp; x < words; x += kSelWarps) {
    const unsigned keep = sure[x], at = tied[x] + __popc(keep & ((1u << lane) - 1u));
    if ((keep >> lane & 1u) && at < (unsigned)a.budget) {
      kept[at] = j0 + 32 * x + lane;
      w_out[at] = key_weight(keys[32 * x + lane]);
    }
  }
  for (int i = a.budget + all; i < len; i += stride) w_out[i] = 0.f;
  if (cl > 1) tc::cluster_sync_all();  // nobody leaves while its shared memory may be read
}

// ---- keys and values -----------------------------------------------------------

constexpr int kMoveItems = 4;
constexpr int kCopyThreads = 128;
constexpr int kCopyWarps = 16;  // per SM

// To other pages.  A warp takes `rows` output positions of one (sequence, KV
// head): a lane finds where one of them comes from and goes to, then the warp
// moves their keys and values with kMoveItems pieces of each in flight a lane,
// LANES lanes on a row.
template <int LANES>
__global__ void __launch_bounds__(kCopyThreads) cache_copy_kernel(const __grid_constant__ CacheEvictArgs a, int rows) {
  constexpr int RPI = 32 / LANES;  // rows of one load
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.z, c = blockIdx.y, lane = threadIdx.x & 31;
  const int i0 = (blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5)) * rows;
  bool bad;
  const int n_keep = min(checked_len(a.lens[s], a.limit, &bad), a.budget);
  // lens_out may be lens: the blocks that read it later find n_keep, which gives n_keep again
  if (blockIdx.x == 0 && c == 0 && threadIdx.x == 0) a.lens_out[s] = n_keep;
  const int n = min(rows, n_keep - i0);
  if (n <= 0) return;
  uint32_t from = ~0u, to = ~0u;
  if (lane < n) {
    const int64_t f = page_slot(a.table, s, a.kept[((int64_t)s * a.nkv + c) * a.budget + i0 + lane]);
    const int64_t t = page_slot(a.table_out, s, i0 + lane);
    if (f < 0 || t < 0) {
      cache_error(a.err, kCacheBadPage);
    } else {
      from = (uint32_t)f;
      to = (uint32_t)t;
    }
  }
  const int64_t stride = (int64_t)a.nkv * LANES;  // pieces from one position to the next
  const uint4* ks = static_cast<const uint4*>(a.k) + c * LANES + lane % LANES;
  const uint4* vs = static_cast<const uint4*>(a.v) + c * LANES + lane % LANES;
  uint4* kd = static_cast<uint4*>(a.k_out) + c * LANES + lane % LANES;
  uint4* vd = static_cast<uint4*>(a.v_out) + c * LANES + lane % LANES;
  for (int r0 = 0; r0 < n; r0 += RPI * kMoveItems) {
    uint4 k[kMoveItems], v[kMoveItems];
    uint32_t dst[kMoveItems];
#pragma unroll
    for (int u = 0; u < kMoveItems; ++u) {
      const int r = r0 + u * RPI + lane / LANES;  // rows <= 32; behind n: lanes without a slot
      const uint32_t f = __shfl_sync(kFull, from, r & 31);
      dst[u] = __shfl_sync(kFull, to, r & 31);
      if (r >= n) dst[u] = ~0u;
      if (dst[u] != ~0u) {
        k[u] = __ldcs(ks + (int64_t)f * stride);
        v[u] = __ldcs(vs + (int64_t)f * stride);
      }
    }
#pragma unroll
    for (int u = 0; u < kMoveItems; ++u)
      if (dst[u] != ~0u) {
        kd[(int64_t)dst[u] * stride] = k[u];
        vd[(int64_t)dst[u] * stride] = v[u];
      }
  }
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
// weights: as few as hold them, but more, of at least kSelKeys each, while the
// launch leaves SMs idle.
constexpr int kSelKeys = 4096;
int select_cluster(int64_t limit, int64_t heads, int sm_count) {
  int cl = 1;
  while (cl < 8 && (limit > (int64_t)cl * kSelCap || (limit >= 2 * cl * kSelKeys && heads * cl * 2 <= sm_count)))
    cl *= 2;
  return cl;
}

template <int LANES>
cudaError_t copy_rows(cudaStream_t st, const CacheEvictArgs& a, int sm_count) {
  // 32 positions a warp, or 8 where that leaves too few warps to hide the latency of their loads
  const int rows = (int64_t)a.S * a.nkv * ((a.budget + 31) / 32) < kCopyWarps * sm_count ? 8 : 32;
  const int per_block = rows * (kCopyThreads / 32);
  return launch_pdl(st, dim3((a.budget + per_block - 1) / per_block, a.nkv, a.S), dim3(kCopyThreads), 0, 1,
                    cache_copy_kernel<LANES>, a, rows);
}

}  // namespace

cudaError_t prepare_cache_evict() {
  return cudaFuncSetAttribute(cache_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kSelCap * 4 + kSelCap / 4);
}

cudaError_t launch_cache_evict(cudaStream_t st, const CacheEvictArgs& a, int bf16, int sm_count) {
  const int cl = select_cluster(a.limit, (int64_t)a.S * a.nkv, sm_count);
  const int cap = (int)((a.limit + cl - 1) / cl + 31) / 32 * 32;
  cudaError_t e = launch_pdl_cluster(st, dim3(cl * a.nkv, a.S), dim3(kSelThreads), (size_t)cap * 4 + cap / 4, dim3(cl),
                                     cache_select_kernel, a, cl, cap);
  if (e != cudaSuccess) return e;
  const int row16 = a.hd * (bf16 ? 2 : 4) / 16;
  if (a.in_place) {
    const int pieces = 2;
    return launch_pdl(st, dim3(a.nkv * 2 * (row16 / pieces), a.S), dim3(kShiftThreads), 0, 1, cache_shift_kernel, a,
                      row16, pieces);
  }
  if (row16 == 8) return copy_rows<8>(st, a, sm_count);
  return row16 == 16 ? copy_rows<16>(st, a, sm_count) : copy_rows<32>(st, a, sm_count);
}

}  // namespace sf
