// What the kernels of sf_cache_attend_rows share: the walk over a batch's
// tiles, the end of a row, partial results.
#pragma once

#include "sf_cache.h"

namespace sf {
namespace rows {

constexpr float kRowsRoom = 27.f;
constexpr int kRowsMaxCtas = 512;
constexpr unsigned kFull = 0xffffffffu;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Rows and length of sequence s; bad where its offsets are not ascending within [0, T] or its length is out of range.
struct SeqRows {
  int s, row0, rows, len;
};
__device__ __forceinline__ SeqRows sequence_rows(const CacheRowsArgs& a, int s, bool* bad_rows, bool* bad_len) {
  const int r0 = __ldcg(a.starts + s), r1 = __ldcg(a.starts + s + 1);
  *bad_rows = r0 < 0 || r1 < r0 || r1 > a.T;
  SeqRows q;
  q.s = s;
  q.row0 = r0;
  q.rows = *bad_rows ? 0 : r1 - r0;
  q.len = checked_len(__ldcg(a.lens + s), a.limit, bad_len);
  return q;
}

// Page entry of position j < len of sequence s, through L2: the kernels may run
// before their own wait.
__device__ __forceinline__ int32_t entry_of(const CacheRowsArgs& a, int s, int j) {
  const int c = page_of(a.table, j);
  return c < a.table.cols ? __ldcg(a.table.pages + (int64_t)s * a.table.ld + c) : -1;
}

__device__ __forceinline__ int64_t units_of(const RowsShape& sh, const SeqRows& q) {
  return q.rows > 0 && q.len > 0 ? sh.nkv * row_units(sh, q.rows, q.len) : 0;
}

__device__ __forceinline__ int64_t shfl_up64(int64_t x, int o) {
  return (int64_t)__shfl_up_sync(kFull, (unsigned long long)x, o);
}

// A thread block's share of the line, and the walk along it: start() once, then
// next() for every part, by whole warps.
struct RowsWalk {
  int64_t u, end, per;  // this block's units [u, end)
  int64_t first;        // of seq
  SeqRows seq;
  RowsTiles tiles;

  __device__ __forceinline__ void start(const RowsShape& sh) {
    if (u < end) tiles.start(sh, seq.rows, seq.len, first, u);
    else tiles.at = end;
  }
  __device__ __forceinline__ bool next(const CacheRowsArgs& a, const RowsShape& sh, RowsPart& p, SeqRows& q) {
    while (tiles.at < end) {
      if (!tiles.more(sh)) {  // the next sequence with units: 32 looked at together
        const int lane = threadIdx.x & 31;
        for (int s0 = seq.s + 1;; s0 += 32) {
          bool b0, b1;
          SeqRows x{0, 0, 0, 0};
          if (s0 + lane < a.S) x = sequence_rows(a, s0 + lane, &b0, &b1);
          const unsigned hit = __ballot_sync(kFull, x.rows > 0 && x.len > 0);
          if (hit) {
            const int l = __ffs(hit) - 1;
            seq.s = s0 + l;
            seq.row0 = __shfl_sync(kFull, x.row0, l);
            seq.rows = __shfl_sync(kFull, x.rows, l);
            seq.len = __shfl_sync(kFull, x.len, l);
            break;
          }
          if (s0 + 32 >= a.S) return false;  // not reached: units are left
        }
        tiles.start(sh, seq.rows, seq.len, tiles.at, tiles.at);
      }
      p = tiles.take(sh, end);
      q = seq;
      if (p.b0 < p.b1) return true;
    }
    return false;
  }
};

// By all THREADS of the block: the walk's start.  False where nothing of the
// call may be written (offsets that do not ascend).  *empties: some sequence
// with rows has no keys.  (Who walks calls walk.start() then.)  Batches of up to THREADS sequences are scanned once,
// between two barriers.
template <int THREADS>
__device__ __forceinline__ bool rows_plan(const CacheRowsArgs& a, const RowsShape& sh, RowsWalk& walk, bool* empties) {
  constexpr int WARPS = THREADS / 32;
  __shared__ int64_t sums[WARPS];
  __shared__ int flags_of[WARPS];
  __shared__ RowsWalk found;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto upto_lane = [&](int64_t y) {  // inclusive sum over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t z = shfl_up64(y, o);
      if (lane >= o) y += z;
    }
    return y;
  };
  SeqRows head{0, 0, 0, 0};
  int64_t mine = 0;
  int flags = 0;
  for (int s = threadIdx.x; s < a.S; s += THREADS) {
    bool bad_rows, bad_len;
    const SeqRows q = sequence_rows(a, s, &bad_rows, &bad_len);
    if (s == (int)threadIdx.x) head = q;
    mine += units_of(sh, q);
    flags |= (bad_rows ? 1 : 0) | (bad_len ? 2 : 0) | (q.rows > 0 && q.len == 0 ? 4 : 0);
  }
  const int64_t incl = upto_lane(mine);
  flags = __reduce_or_sync(kFull, flags);
  if (lane == 31) {
    sums[warp] = incl;
    flags_of[warp] = flags;
  }
  __syncthreads();
  int64_t total = 0, before = 0;
  flags = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
    flags |= flags_of[w];
  }
  *empties = flags & 4;
  if (threadIdx.x == 0 && blockIdx.x == 0) {
    if (flags & 1) cache_error(a.err, kCacheBadRow);
    if (flags & 2) cache_error(a.err, kCacheBadLength);
  }
  const int64_t even = quick_quotient(total + a.ctas - 1, a.ctas), per = even < a.least ? a.least : even;
  const int64_t lo = per * blockIdx.x, hi = lo + per < total ? lo + per : total;
  walk.u = walk.end = 0;
  walk.per = per;
  if (flags & 1) return false;
  if (lo >= hi) return true;
  if (a.S <= THREADS) {
    const int64_t at = before + incl - mine;
    if (at <= lo && lo < at + mine) found = RowsWalk{lo, hi, per, at, head, {}};
  } else {
    before = 0;
    for (int s0 = 0; s0 < a.S; s0 += THREADS) {
      const int s = s0 + threadIdx.x;
      bool b0, b1;
      SeqRows q{0, 0, 0, 0};
      if (s < a.S) q = sequence_rows(a, s, &b0, &b1);
      const int64_t x = units_of(sh, q), y = upto_lane(x);
      __syncthreads();
      if (lane == 31) sums[warp] = y;
      __syncthreads();
      int64_t at = before + y - x;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        if (w < warp) at += sums[w];
        before += sums[w];
      }
      if (at <= lo && lo < at + x) found = RowsWalk{lo, hi, per, at, q, {}};
      if (before > lo) break;
    }
  }
  __syncthreads();
  walk = found;
  return true;
}

// One float4 of a finished row of its unnormalised sums (m, l), together with
// the tail's state where the call has one.
template <typename T, int HD>
__device__ __forceinline__ void rows_finish(const CacheRowsArgs& a, int64_t t, int h, int d, float4 o, float m, float l) {
  const int64_t at = t * a.nq + h;
  if (a.tail_ml) {
    const float2 tail = __ldcg(a.tail_ml + at);
    const float4 y = __ldcg(reinterpret_cast<const float4*>(a.tail_o + at * HD + d));
    const float top = fmaxf(m, tail.x), base = top == -INFINITY ? 0.f : top;
    // the tail's output is normalised: its weight is its denominator
    const float f = ex2(m - base), g = tail.y * ex2(tail.x - base);
    o = make_float4(o.x * f + y.x * g, o.y * f + y.y * g, o.z * f + y.z * g, o.w * f + y.w * g);
    l = l * f + g;
    m = top;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;  // no score above -infinity: zeros
  store4<T>(static_cast<T*>(a.out) + t * a.ld_out + (int64_t)h * HD + d,
            make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
  if (a.lse && d == 0) a.lse[at] = l == 0.f ? -INFINITY : kLn2 * (m + kRowsRoom) + logf(l);
}

// With a tail, the kernels of the tiles do not finish rows: the tail's kernel may
// still be running.  A row's own state goes to whole_o and whole_ml; its
// denominator is kRowCut where its tile is cut and the partial results hold it,
// and 0, without an output, where there are no keys.  The join kernel goes
// through all of them.
constexpr float kRowCut = -1.f;

// Rows that no key belongs to: those of sequences without keys, and with a tail
// those of no sequence.  By THREADS threads of every block, each block every
// gridDim.x-th row.
template <typename T, int HD, int THREADS>
__device__ void rows_empties(const CacheRowsArgs& a, bool empties) {
  const int thread = threadIdx.x % THREADS, lane = threadIdx.x & 31;
  auto clear = [&](int t0, int t1) {
    for (int t = t0 + blockIdx.x; t < t1; t += gridDim.x)
      if (a.tail_ml)
        for (int h = thread; h < a.nq; h += THREADS) a.whole_ml[(int64_t)t * a.nq + h] = make_float2(-INFINITY, 0.f);
      else
        for (int i = thread; i < a.nq * (HD / 4); i += THREADS)
          rows_finish<T, HD>(a, t, i / (HD / 4), i % (HD / 4) * 4, make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f);
  };
  if (empties)
    for (int s0 = 0; s0 < a.S; s0 += 32) {  // every warp finds them for itself, 32 sequences at once
      bool b0, b1;
      SeqRows q{0, 0, 0, 1};
      if (s0 + lane < a.S) q = sequence_rows(a, s0 + lane, &b0, &b1);
      unsigned hits = __ballot_sync(kFull, q.len == 0 && q.rows > 0);
      for (; hits; hits &= hits - 1) {
        const int l = __ffs(hits) - 1, t0 = __shfl_sync(kFull, q.row0, l), n = __shfl_sync(kFull, q.rows, l);
        clear(t0, t0 + n);
        __syncwarp();
      }
    }
  if (a.tail_ml) {  // rows in front of the first group and behind the last
    clear(0, __ldcg(a.starts));
    clear(__ldcg(a.starts + a.S), a.T);
  }
}

// Where nothing of the call may be written: with a tail, no row is the join's.
__device__ __forceinline__ void rows_refused(const CacheRowsArgs& a) {
  if (a.tail_ml)
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < (int64_t)a.T * a.nq;
         i += (int64_t)gridDim.x * blockDim.x)
      a.whole_ml[i] = make_float2(0.f, kRowCut);
}

// ---- partial results: per slot ROWS query vectors, [HD / 4][ROWS] float4 and
// (m, l) of each.  Neighbouring rows lie side by side: a thread has one row,
// or a few.
template <int HD, int ROWS>
__device__ __forceinline__ float4* part_at(const CacheRowsArgs& a, int slot, int c4, int row) {
  return reinterpret_cast<float4*>(a.parts) + ((int64_t)slot * (HD / 4) + c4) * ROWS + row;
}
template <int ROWS>
__device__ __forceinline__ float2* part_ml(const CacheRowsArgs& a, int slot, int row) {
  return a.part_ml + (int64_t)slot * ROWS + row;
}

__device__ __forceinline__ bool is_cut(const RowsPart& p) { return p.b0 > 0 || p.b1 < p.nb; }
// By one thread of the block that starts a cut tile.
__device__ __forceinline__ void rows_record(const CacheRowsArgs& a, const RowsPart& p, const SeqRows& q, int64_t per) {
  a.joins[blockIdx.x] = RowsJoin{rows_last_cta(p, per) - (int)blockIdx.x + 1, p.nv, q.row0, p.kvh, p.v0};
}

}  // namespace rows
}  // namespace sf
