// Keys in the paged cache turned from the positions they were stored for to
// new ones (specfold_cache.h, sf_cache_reposition): rotation by (new - old)
// steps of every pair's frequency, from append's own table.
#include "sf_cache.h"
#include "sf_pairs.cuh"
#include "sf_rotary.cuh"

namespace sf {
namespace {

// 4 x 4,096 places of 8 heads x 128 bf16, and 1,024 of 2 heads: 15.7 to 16.5 and 2.5 us so; 32 places and 256 threads 17.3 and
// 3.1, 16 and 256 17.0 and 2.4, 2 and 128 17.6 and 2.7.
constexpr int kTurnThreads = 128;
constexpr int kTurnPlaces = 4;  // places of a sequence that a block takes at a time

// A group of dim / 2 / VEC lanes turns one key head: each lane holds two
// 16-byte pieces, both members of its rotation pairs.  Bytes bound it: the
// turned part of every key in and out once, and twice as many bytes of the
// table, from L2.  (Not kept, at 16.5 us and half the copy bandwidth: two or
// four keys in flight a group 20 to 29 us, angles as sums of two rows that stay
// in L1 17.4 and of one that stays in registers 19.2, sines and cosines of 64-bit
// phases 16.7.)
template <typename T, int HD, bool NEIGHBOURS>
__global__ void __launch_bounds__(kTurnThreads) cache_turn_kernel(const __grid_constant__ CacheTurnArgs a) {
  using P = Piece<T>;
  constexpr int N = P::PAIRS, VEC = 2 * N;
  const int lanes = a.rotary.dim / 2 / VEC;  // of a key head
  const int s = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  bool bad;
  const int len = checked_len(__ldcg(a.lens + s), a.limit, &bad);
  if (bad && blockIdx.x == 0 && threadIdx.x == 0) cache_error(a.err, kCacheBadLength);
  const int per_place = a.nkv * lanes;
  for (int j0 = blockIdx.x * kTurnPlaces; j0 < len; j0 += gridDim.x * kTurnPlaces) {
    const int places = min(kTurnPlaces, len - j0);
    for (int i = threadIdx.x; i < places * per_place; i += kTurnThreads) {
      const int j = j0 + i / per_place, r = i % per_place, c = r / lanes, lane = r - c * lanes;
      const int64_t at = ((int64_t)s * a.nkv + c) * a.ld_pos + j;
      const int from = a.from[at], to = a.to ? a.to[at] : j;
      if (from < 0 || to < 0) continue;
      if (from >= a.max_pos || to >= a.max_pos) {
        cache_error(a.err, kCacheBadRow);
        continue;
      }
      const int64_t slot = page_slot(a.table, s, j);
      if (slot < 0) {
        cache_error(a.err, kCacheBadPage);
        continue;
      }
      const int steps = to - from;
      if (steps == 0) continue;  // the same key, to the bit
      T* key = static_cast<T*>(a.k) + (slot * a.nkv + c) * HD;
      const int c0 = NEIGHBOURS ? 2 * lane : lane, c1 = NEIGHBOURS ? 2 * lane + 1 : lane + lanes;
      uint4* p0 = reinterpret_cast<uint4*>(key + c0 * VEC);
      uint4* p1 = reinterpret_cast<uint4*>(key + c1 * VEC);
      const uint4 u0 = *p0, u1 = *p1;
      const float* angles = a.rope + (int64_t)(steps < 0 ? -steps : steps) * a.rotary.dim;
      Angles<T, NEIGHBOURS> g;
      g.load(angles, a.rotary.dim / 2, c0, c1);
      g.scale(a.unscale, steps < 0 ? -a.unscale : a.unscale);
      Two x[N], y[N];
      P::load(u0, x);
      P::load(u1, y);
      g.turn(x, y);
      *p0 = P::store(x);
      *p1 = P::store(y);
    }
  }
}

template <typename T, int HD>
cudaError_t turn_t(cudaStream_t st, const CacheTurnArgs& a, int sm_count) {
  // enough blocks for the longest sequence, up to what keeps every SM busy several times over
  const int64_t want = (a.limit + kTurnPlaces - 1) / kTurnPlaces, most = 32 * (int64_t)sm_count;
  const int64_t x = want * a.S <= most ? want : (most + a.S - 1) / a.S;
  const dim3 grid((unsigned)(x < 1 ? 1 : x), a.S);
  return launch_pdl(st, grid, dim3(kTurnThreads), 0, 1,
                    a.rotary.neighbours ? cache_turn_kernel<T, HD, true> : cache_turn_kernel<T, HD, false>, a);
}

}  // namespace

cudaError_t launch_cache_turn(cudaStream_t st, const CacheTurnArgs& a, int bf16, int sm_count) {
  if (bf16) return a.hd == 128 ? turn_t<__nv_bfloat16, 128>(st, a, sm_count) : turn_t<__nv_bfloat16, 64>(st, a, sm_count);
  return a.hd == 128 ? turn_t<float, 128>(st, a, sm_count) : turn_t<float, 64>(st, a, sm_count);
}

}  // namespace sf
