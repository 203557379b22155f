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

// The two halves of a cluster barrier: what a thread did before arriving is seen by those that have waited.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, unsigned v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void red_cluster_add(uint32_t addr, unsigned v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ unsigned atom_cluster_add(uint32_t addr, unsigned v) {
  unsigned old;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(addr), "r"(v) : "memory");
  return old;
}

constexpr int kBinBits = 11;
constexpr int kBins = 1 << kBinBits;
constexpr int kList = 256;              // keys that are ranked by comparing all pairs
constexpr int kSelLoads = 8;            // keys a thread handles together
constexpr int kSelWords = 4;            // words of a bitmap a warp handles together
constexpr int kSelCap = 32768;          // weights a block holds at most

// First cut: 2^20 keys a bin from that of 0.0 on, eight bins for every factor
// of two; smaller keys count as the lowest bin.
constexpr uint32_t kFirstKey = 0x80000000u;
constexpr int kFirstShift = 20;
static_assert((0xff800000u - kFirstKey) >> kFirstShift < (uint32_t)kBins, "bins to +inf");

// A cluster of `cl` blocks per (sequence, KV head); block r holds the keys of
// the r-th part of the weights in shared memory.
//
// The need-th largest candidate key is found by counting keys into bins and
// narrowing [lo, hi] to the bin that holds it: first with bins of a fixed size,
// counted while the weights arrive, then, while the bin holds more than kList
// keys, in up to kBins equal parts of it: two such passes at most (shifts 9
// and 0), or three where the first cut's lowest bin is the one, as for a
// threshold among zeros (21, 9, 0) or negative weights (21, 10, 0).  The lowest
// bin is never counted (if the others do not reach, it is the one), which keeps
// the usual crowd of zero weights out of the first cut's shared-memory atomics;
// in later passes equal keys of a warp add once.  The keys of the last bin are
// ranked by comparing all pairs.
//
// The choice is two bitmaps, positions certainly kept and positions at the
// threshold, of which the first `ties` are kept; a scan of their populations
// gives every kept position its place.
template <int kSelThreads>
__global__ void __launch_bounds__(kSelThreads, 1024 / kSelThreads) cache_select_kernel(
    const __grid_constant__ CacheEvictArgs a, int cl, int cap) {
  constexpr int kSelWarps = kSelThreads / 32;
  constexpr int BT = kBins / kSelThreads;          // bins of a thread
  constexpr int WT = kSelCap / 32 / kSelThreads;   // words of a bitmap of a thread
  static_assert(BT * kSelThreads == kBins && WT * kSelThreads * 32 == kSelCap, "shares");
  extern __shared__ __align__(16) unsigned keys[];    // [cap] of this block's positions
  unsigned* sure = keys + cap;                        // [cap / 32] kept; later the final choice
  unsigned* tied = sure + cap / 32;                   // [cap / 32] at the threshold; later places
  __shared__ __align__(16) unsigned hist[kBins];
  __shared__ unsigned red[32];
  __shared__ unsigned pub[3];                         // to the cluster: kept, tied, ties
  __shared__ unsigned found[3];                       // bin, keys above it, keys in it (all ones: not known)
  __shared__ __align__(16) unsigned all_key[kList];   // keys to be ranked, of the whole cluster
  __shared__ unsigned my_key[kList];                  // those of this block
  __shared__ int my_pos[kList];
  __shared__ unsigned n_all, n_mine, s_ties;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x / cl, s = blockIdx.y, rank = blockIdx.x % cl;
  auto meet = [&]() {
    if (cl > 1)
      tc::cluster_sync_all();
    else
      __syncthreads();
  };
  auto remote = [&](const void* p, int r) { return tc::map_to_rank(tc::smem_u32(p), r); };
  auto of_rank = [&](const unsigned* p, int r) { return r == rank ? *p : ld_cluster_u32(remote(p, r)); };
#pragma unroll
  for (int i = 0; i < BT; ++i) hist[threadIdx.x + i * kSelThreads] = 0u;
  if (threadIdx.x == 0) n_all = n_mine = s_ties = 0u;
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
      if (i < len) w_out[i] = key_weight(weight_key(w[i]));  // -0 as 0, as for chosen positions
    }
    return;
  }
  const int chunk = (len + cl - 1) / cl, j0 = min(rank * chunk, len), n = min(chunk, len - j0);
  // candidates, in this block's indexes
  const int lo_j = min(max(a.n_first - j0, 0), n), hi_j = max(min(len - a.n_recent - j0, n), lo_j);
  const int words = (n + 31) / 32;
  __syncthreads();  // this block's histogram and counters are empty;
  if (cl > 1) cluster_arrive();
  for (int i0 = threadIdx.x; i0 < n; i0 += kSelThreads * kSelLoads) {
    float x[kSelLoads];
#pragma unroll
    for (int u = 0; u < kSelLoads; ++u) {
      const int i = i0 + u * kSelThreads;
      if (i < n) x[u] = w[j0 + i];
    }
#pragma unroll
    for (int u = 0; u < kSelLoads; ++u) {
      const int i = i0 + u * kSelThreads;
      if (i < n) {
        const uint32_t k = weight_key(x[u]);
        keys[i] = k;
        if (i >= lo_j && i < hi_j && k >= kFirstKey + (1u << kFirstShift))
          atomicAdd(&hist[(k - kFirstKey) >> kFirstShift], 1u);
      }
    }
  }
  if (cl > 1) cluster_wait();  // so are the cluster's
  int need = a.budget - a.n_first - a.n_recent;  // below the number of candidates, since budget < len
  uint32_t lo = 0u, hi = 0xff800000u;            // the need-th largest key lies in [lo, hi]
  uint32_t base = kFirstKey;                     // bins start here,
  int shift = kFirstShift;                       // of 2^shift keys
  uint32_t thr = ~0u;                            // keys above it are kept (none is above ~0),
  int ties = 0;                                  // and the first `ties` equal to it
  // few candidates: all of them are ranked, nothing is narrowed
  bool rank_list = need > 0 && len - a.n_first - a.n_recent <= kList;
  if (rank_list) thr = hi;
  while (need > 0 && !rank_list) {
    __syncthreads();
    // thread t holds bins kBins - 1 - BT t and those below it
    unsigned* mine = hist + kBins - 1 - BT * threadIdx.x;
    unsigned v[BT], mass = 0;
    if (cl > 1) {
      if (rank != 0) {
#pragma unroll
        for (int i = 0; i < BT; ++i) {
          v[i] = mine[-i];
          if (v[i]) red_cluster_add(remote(mine - i, 0), v[i]);
          mine[-i] = 0u;
        }
      }
      meet();
    }
    if (rank == 0) {
#pragma unroll
      for (int i = 0; i < BT; ++i) {
        v[i] = mine[-i];
        mine[-i] = 0u;
        mass += v[i];
      }
      unsigned sum = mass;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(kFull, sum, o);
        if (lane >= o) sum += y;
      }
      if (lane == 31) red[warp] = sum;
      __syncthreads();
      const unsigned others = lane < kSelWarps ? red[lane] : 0u;
      unsigned at = __reduce_add_sync(kFull, lane < warp ? others : 0u) + sum - mass;
      const unsigned total = __reduce_add_sync(kFull, others);
#pragma unroll
      for (int i = 0; i < BT; ++i) {
        if (at < (unsigned)need && at + v[i] >= (unsigned)need) {
          found[0] = kBins - 1 - BT * threadIdx.x - i;
          found[1] = at;
          found[2] = v[i];
        }
        at += v[i];
      }
      if (threadIdx.x == 0 && total < (unsigned)need) {
        found[0] = 0u;
        found[1] = total;
        found[2] = ~0u;
      }
    }
    meet();
    // found is written again only after everybody has come to the next pass's meeting
    const uint32_t bin = of_rank(&found[0], 0);
    const unsigned above = of_rank(&found[1], 0), inside = of_rank(&found[2], 0);
    need -= (int)above;
    hi = min(hi, base + (bin << shift) + ((1u << shift) - 1u));
    if (bin) lo = base + (bin << shift);
    if (inside == (unsigned)need) {  // the bin's keys are the last ones needed
      thr = lo - 1;
      break;
    }
    if (lo == hi) {
      thr = lo;
      ties = need;
      break;
    }
    if (inside <= kList) {
      thr = hi;
      rank_list = true;
      break;
    }
    const uint32_t range = hi - lo;
    const int bits = 32 - __clz(range);
    base = lo;
    shift = bits > kBinBits ? bits - kBinBits : 0;
    for (int w0 = lo_j + warp * 32; w0 < hi_j; w0 += kSelThreads * kSelLoads) {
      uint32_t k[kSelLoads];
#pragma unroll
      for (int u = 0; u < kSelLoads; ++u) {
        const int i = w0 + lane + u * kSelThreads;
        k[u] = i < hi_j ? keys[i] - lo : ~0u;  // no range is that long
      }
#pragma unroll
      for (int u = 0; u < kSelLoads; ++u) {
        // equal weights crowd here: the lanes that share the first one's bin add once
        const uint32_t b = k[u] <= range ? k[u] >> shift : 0u;
        const unsigned on = __ballot_sync(kFull, b != 0u);
        if (on == 0u) continue;
        const unsigned same = __ballot_sync(kFull, b == __shfl_sync(kFull, b, __ffs(on) - 1));
        if (same >> lane & 1u ? lane == __ffs(on) - 1 : b != 0u)
          atomicAdd(&hist[b], same >> lane & 1u ? __popc(same) : 1u);
      }
    }
  }
  // every key is in place and a.w is read by everybody (w_out may be w); the passes have met for that otherwise
  if (need == 0 || rank_list) meet();
  // bitmaps; the keys still to be ranked into the lists.  kSelWords words at a time, so that their latencies overlap
  for (int x0 = warp * kSelWords; x0 < words; x0 += kSelWarps * kSelWords) {
    uint32_t k[kSelWords];
    unsigned hit[kSelWords], hits = 0;
#pragma unroll
    for (int u = 0; u < kSelWords; ++u) {
      const int i = 32 * (x0 + u) + lane;
      k[u] = i < n ? keys[i] : 0u;
    }
#pragma unroll
    for (int u = 0; u < kSelWords; ++u) {
      const int i = 32 * (x0 + u) + lane;
      const bool cand = i >= lo_j && i < hi_j;
      const unsigned b = __ballot_sync(kFull, (i < n && !cand) || (cand && k[u] > thr));
      const unsigned e = __ballot_sync(kFull, cand && k[u] >= (rank_list ? lo : thr) && k[u] <= thr);
      hit[u] = rank_list ? e : 0u;
      hits += __popc(hit[u]);
      if (lane == 0 && x0 + u < words) {
        sure[x0 + u] = b;
        tied[x0 + u] = rank_list ? 0u : e;
      }
    }
    if (hits) {  // at most kList in the whole cluster: the bin's population
      unsigned at = 0, at_all = 0;
      if (lane == 0) {
        at = atomicAdd(&n_mine, hits);
        at_all = cl > 1 ? atom_cluster_add(remote(&n_all, 0), hits) : at;
      }
      at = __shfl_sync(kFull, at, 0);
      at_all = __shfl_sync(kFull, at_all, 0);
#pragma unroll
      for (int u = 0; u < kSelWords; ++u) {
        if (hit[u] >> lane & 1u) {
          const unsigned below = __popc(hit[u] & ((1u << lane) - 1u));
          my_key[at + below] = k[u];
          my_pos[at + below] = 32 * (x0 + u) + lane;
          if (rank == 0)
            all_key[at_all + below] = k[u];
          else
            st_cluster_u32(remote(all_key + at_all + below, 0), k[u]);
        }
        at += __popc(hit[u]);
        at_all += __popc(hit[u]);
      }
    }
  }
  if (rank_list) {
    meet();
    const int m = cl > 1 ? (int)of_rank(&n_all, 0) : (int)n_mine, mine = (int)n_mine;
    if (rank != 0) {
      for (int x = threadIdx.x; x < m; x += kSelThreads) all_key[x] = ld_cluster_u32(remote(all_key + x, 0));
      __syncthreads();
    }
    // four lanes a key, each a quarter of the list (all of a warp stay for the shuffles)
    const int q = lane & 3;
    for (int t0 = warp * 8; t0 < mine; t0 += kSelWarps * 8) {
      const int t = t0 + (lane >> 2);
      const unsigned me = t < mine ? my_key[t] : 0u;
      int greater = 0, equal = 0, x = 4 * q;
      for (; x + 4 <= m; x += 16) {
        const uint4 k = *reinterpret_cast<const uint4*>(all_key + x);
        greater += (k.x > me) + (k.y > me) + (k.z > me) + (k.w > me);
        equal += (k.x == me) + (k.y == me) + (k.z == me) + (k.w == me);
      }
      for (const int end = min(x + 4, m); x < end; ++x) {  // the list's last, short quarter
        greater += all_key[x] > me;
        equal += all_key[x] == me;
      }
      greater += __shfl_xor_sync(kFull, greater, 1);
      equal += __shfl_xor_sync(kFull, equal, 1);
      greater += __shfl_xor_sync(kFull, greater, 2);
      equal += __shfl_xor_sync(kFull, equal, 2);
      if (t < mine && q == 0) {
        const int i = my_pos[t];
        if (greater + equal <= need) {
          atomicOr(&sure[i >> 5], 1u << (i & 31));
        } else if (greater < need) {
          atomicOr(&tied[i >> 5], 1u << (i & 31));
          s_ties = need - greater;  // the same from all of them
        }
      }
    }
  }
  __syncthreads();
  if (rank_list) ties = s_ties;  // 0 where this block has no tied key; the cluster's largest below
  // places: thread t takes words WT t ...
  unsigned ws[WT], we[WT], pop = 0;  // populations, kept in the low half, tied in the high one (each <= 2^15)
#pragma unroll
  for (int i = 0; i < WT; ++i) {
    const int x = WT * threadIdx.x + i;
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
  if (lane == 31) red[warp] = sum;
  __syncthreads();
  const unsigned others = lane < kSelWarps ? red[lane] : 0u;
  const unsigned before = __reduce_add_sync(kFull, lane < warp ? others : 0u) + sum - pop;
  unsigned at_sure = before & 0xffffu, at_tied = before >> 16;
  if (cl > 1) {
    const unsigned total = __reduce_add_sync(kFull, others);
    if (threadIdx.x == 0) {
      pub[0] = total & 0xffffu;
      pub[1] = total >> 16;
      pub[2] = (unsigned)ties;
    }
    meet();
    for (int r = 0; r < cl; ++r) {
      ties = max(ties, (int)of_rank(&pub[2], r));
      if (r < rank) {
        at_sure += of_rank(&pub[0], r);
        at_tied += of_rank(&pub[1], r);
      }
    }
    cluster_arrive();  // the last reads of other blocks' shared memory are done
  }
#pragma unroll
  for (int i = 0; i < WT; ++i) {
    const int x = WT * threadIdx.x + i;
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
  for (int x0 = warp * kSelWords; x0 < words; x0 += kSelWarps * kSelWords) {
    unsigned keep[kSelWords], at[kSelWords];
    uint32_t k[kSelWords];
#pragma unroll
    for (int u = 0; u < kSelWords; ++u) {
      const bool in = x0 + u < words;
      keep[u] = in ? sure[x0 + u] : 0u;
      at[u] = in ? tied[x0 + u] : 0u;
      k[u] = in ? keys[32 * (x0 + u) + lane] : 0u;  // words are whole in memory
    }
#pragma unroll
    for (int u = 0; u < kSelWords; ++u) {
      const unsigned to = at[u] + __popc(keep[u] & ((1u << lane) - 1u));
      if ((keep[u] >> lane & 1u) && to < (unsigned)a.budget) {
        kept[to] = j0 + 32 * (x0 + u) + lane;
        w_out[to] = key_weight(k[u]);
      }
    }
  }
  for (int i = a.budget + all; i < len; i += stride) w_out[i] = 0.f;
  if (cl > 1) cluster_wait();  // nobody leaves while its shared memory may be read
}

// ---- keys and values -----------------------------------------------------------

constexpr int kCopyItems = 2;
constexpr int kCopyThreads = 128;
constexpr int kCopyWarps = 16;  // per SM

// To other pages.  A warp takes `rows` output positions of one (sequence, KV
// head): a lane finds where one of them comes from and goes to, then the warp
// moves their keys and values with kCopyItems pieces of each in flight a lane,
// LANES lanes on a row.
template <int LANES>
__global__ void __launch_bounds__(kCopyThreads) cache_copy_kernel(const __grid_constant__ CacheEvictArgs a, int rows) {
  constexpr int RPI = 32 / LANES;  // rows of one load
  const int s = blockIdx.z, c = blockIdx.y, lane = threadIdx.x & 31;
  const int i0 = (blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5)) * rows;
  // Behind the selection kernel, which has waited for everything before it and writes neither lengths nor tables:
  // they can be read, through L2, before it is done.
  bool bad;
  const int n_keep = min(checked_len(__ldcg(a.lens + s), a.limit, &bad), a.budget);
  const int n = min(rows, n_keep - i0);
  uint32_t from = ~0u, to = ~0u;
  if (lane < n) {
    const int i = i0 + lane, col = page_of(a.table_out, i);
    to = entry_slot32(a.table_out, col < a.table_out.cols ? __ldcg(a.table_out.pages + s * a.table_out.ld + col) : -1, i);
  }
  pdl_wait();
  pdl_trigger();
  // lens_out may be lens: the blocks that read it later find n_keep, which gives n_keep again
  if (blockIdx.x == 0 && c == 0 && threadIdx.x == 0) a.lens_out[s] = n_keep;
  if (n <= 0) return;
  if (lane < n) {
    const int j = a.kept[((int64_t)s * a.nkv + c) * a.budget + i0 + lane];
    from = entry_slot32(a.table, page_entry(a.table, s, j), j);
    if (from == ~0u || to == ~0u) {
      cache_error(a.err, kCacheBadPage);
      to = ~0u;
    }
  }
  const int64_t stride = (int64_t)a.nkv * LANES;  // pieces from one position to the next
  const uint4* ks = static_cast<const uint4*>(a.k) + c * LANES + lane % LANES;
  const uint4* vs = static_cast<const uint4*>(a.v) + c * LANES + lane % LANES;
  uint4* kd = static_cast<uint4*>(a.k_out) + c * LANES + lane % LANES;
  uint4* vd = static_cast<uint4*>(a.v_out) + c * LANES + lane % LANES;
  for (int r0 = 0; r0 < n; r0 += RPI * kCopyItems) {
    uint4 k[kCopyItems], v[kCopyItems];
    uint32_t dst[kCopyItems];
#pragma unroll
    for (int u = 0; u < kCopyItems; ++u) {
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
    for (int u = 0; u < kCopyItems; ++u)
      if (dst[u] != ~0u) {
        kd[(int64_t)dst[u] * stride] = k[u];
        vd[(int64_t)dst[u] * stride] = v[u];
      }
  }
}

constexpr int kMoveItems = 2;
constexpr int kShiftThreads = 1024;

// In place.  kept[i] >= i, so a chunk of rows [i0, i1) only overwrites rows
// that this chunk or an earlier one reads: a block reads the chunk into
// registers, meets, and writes it.  Different bytes of a row never meet, so
// the rows of a (sequence, KV head, keys or values) are cut into slices of
// 2^log_pieces times 16 bytes, a block each.
__global__ void __launch_bounds__(kShiftThreads) cache_shift_kernel(const __grid_constant__ CacheEvictArgs a, int row16,
                                                                    int log_pieces) {
  const int s = blockIdx.y, slices = row16 >> log_pieces;
  const int slice = blockIdx.x % slices, part = blockIdx.x / slices % 2, c = blockIdx.x / slices / 2;
  bool bad;
  const int n_keep = min(checked_len(__ldcg(a.lens + s), a.limit, &bad), a.budget);  // as in cache_copy_kernel
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) a.lens_out[s] = n_keep;
  const int32_t* kept = a.kept + ((int64_t)s * a.nkv + c) * a.budget;
  const int piece = (threadIdx.x & ((1 << log_pieces) - 1)) + (slice << log_pieces);
  uint4* pool = static_cast<uint4*>(part ? a.v_out : a.k_out) + c * row16 + piece;
  const int64_t stride = (int64_t)a.nkv * row16;
  const int rows = kShiftThreads >> log_pieces, row = threadIdx.x >> log_pieces;
  for (int i0 = 0; i0 < n_keep; i0 += rows * kMoveItems) {
    uint4 x[kMoveItems];
    uint32_t from[kMoveItems], to[kMoveItems];
#pragma unroll
    for (int u = 0; u < kMoveItems; ++u) {
      const int i = i0 + u * rows + row;
      from[u] = to[u] = ~0u;
      if (i < n_keep) {
        const int j = kept[i];
        if (j != i) {
          from[u] = entry_slot32(a.table, page_entry(a.table, s, j), j);
          to[u] = entry_slot32(a.table_out, page_entry(a.table_out, s, i), i);
          if (from[u] == ~0u || to[u] == ~0u) {
            cache_error(a.err, kCacheBadPage);
            to[u] = ~0u;
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kMoveItems; ++u)
      if (to[u] != ~0u) x[u] = pool[from[u] * stride];
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveItems; ++u)
      if (to[u] != ~0u) pool[to[u] * stride] = x[u];
  }
}

// Blocks of a cluster for `heads` (sequence, KV head) pairs of up to `limit`
// weights: as few as hold them, but four, of at least 2,048 weights each, where
// the launch leaves SMs free (32 heads of 16,384 weights: the whole eviction
// takes 35.9 us with four, 37.6 with two or eight, 39.6 with one; two blocks of
// 2,500 weights are slower than one of 5,000, 19.1 against 18.4 us: a pass meets
// the cluster twice, at about 1,500 cycles).
int select_cluster(int64_t limit, int64_t heads, int sm_count) {
  int cl = 1;
  while (cl < 8 && limit > (int64_t)cl * kSelCap) cl *= 2;
  if (cl < 4 && limit >= 4 * 2048 && 4 * heads <= sm_count) cl = 4;
  return cl;
}

// Threads of a selection block: 512, but 1,024 for more than kSelWide weights a
// block while there is an SM for every block: with 66 (sequence, head) pairs the
// whole eviction to 64 positions takes, with 1,024 and 512 threads, 8.9 and 8.9 us
// for 5,001 weights, 9.8 and 10.1 for 8,000, 11.7 and 12.1 for 12,000, 13.1 and
// 14.0 for 16,384, 19.5 and 21.8 for 32,768; with 128 pairs 9.7 and 9.2, 10.6 and
// 10.4, 12.4 and 12.3, 14.0 and 14.3, 23.2 and 27.1; up to 3,500 weights 512 are
// 0.2 to 1 us faster.  And 128 for up to kSelNarrow weights where 512 would not
// all be resident at once (488 heads of 32 weights: 7.3 against 9.6 us; with few
// heads 512 are 0.3 us faster).
constexpr int kSelWide = 4096, kSelNarrow = 512;

template <int LANES>
cudaError_t copy_rows(cudaStream_t st, const CacheEvictArgs& a, int sm_count) {
  // 32 positions a warp, or 8 where that leaves too few warps to hide the latency of their loads (8 heads of 2,048 ->
  // 1,024 positions: 10.3 against 16.5 us for four sequences, 20.3 against 22.1 for eight, 31.0 against 30.3 for 16)
  const int rows = (int64_t)a.S * a.nkv * ((a.budget + 31) / 32) < kCopyWarps * sm_count ? 8 : 32;
  const int per_block = rows * (kCopyThreads / 32);
  return launch_pdl(st, dim3((a.budget + per_block - 1) / per_block, a.nkv, a.S), dim3(kCopyThreads), 0, 1,
                    cache_copy_kernel<LANES>, a, rows);
}

}  // namespace

cudaError_t prepare_cache_evict() {
  const int bytes = kSelCap * 4 + kSelCap / 4;
  cudaError_t e = cudaFuncSetAttribute(cache_select_kernel<512>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(cache_select_kernel<1024>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  return e;
}

cudaError_t launch_cache_evict(cudaStream_t st, const CacheEvictArgs& a, int bf16, int sm_count) {
  const int64_t heads = (int64_t)a.S * a.nkv;
  const int cl = select_cluster(a.limit, heads, sm_count);
  const int cap = (int)((a.limit + cl - 1) / cl + 31) / 32 * 32;
  const bool wide = cap > kSelWide && heads * cl <= sm_count, narrow = cap <= kSelNarrow && heads > 2 * sm_count;
  const int threads = wide ? 1024 : narrow ? 128 : 512;
  cudaError_t e = launch_pdl_cluster(st, dim3(cl * a.nkv, a.S), dim3(threads), (size_t)cap * 4 + cap / 4, dim3(cl),
                                     wide ? cache_select_kernel<1024>
                                          : narrow ? cache_select_kernel<128> : cache_select_kernel<512>,
                                     a, cl, cap);
  if (e != cudaSuccess) return e;
  const int row16 = a.hd * (bf16 ? 2 : 4) / 16;
  if (a.in_place) {
    // slices of 16 bytes at least, until there is a block for every SM
    int log_pieces = row16 == 8 ? 3 : row16 == 16 ? 4 : 5;
    while (log_pieces > 0 && 2 * heads * (row16 >> log_pieces) < sm_count) --log_pieces;
    return launch_pdl(st, dim3(2 * a.nkv * (row16 >> log_pieces), a.S), dim3(kShiftThreads), 0, 1, cache_shift_kernel,
                      a, row16, log_pieces);
  }
  if (row16 == 8) return copy_rows<8>(st, a, sm_count);
  return row16 == 16 ? copy_rows<16>(st, a, sm_count) : copy_rows<32>(st, a, sm_count);
}

}  // namespace sf
