// Attention of blocks of rows over the paged cache (specfold_cache.h,
// sf_cache_attend_rows), and the shared prefixes of sf_cache_attend_shared.
//
//   x_j = scale log2(e) q . k_j,  m = max_j x_j,  p_j = 2^(x_j - m - kRowsRoom)
//   out = (sum_j p_j v_j) / (sum_j p_j),  lse = ln 2 (m + kRowsRoom + log2 sum_j p_j)
//
// The rows of a sequence and the query heads of one KV head are query vectors
// of one product: they see the same keys.  Keys are streamed once per tile of
// them with the running maximum and sum of the softmax; how tiles are cut over
// thread blocks is in sf_cache_index.h, and cut ones are joined by
// cache_rows_join_kernel.  kRowsRoom keeps unnormalised sums from overflowing
// where the result does not (2^18 values at most).
#include "sf_cache_rows.cuh"
#include "sf_pairs.cuh"

namespace sf {
namespace {

using namespace rows;

constexpr int kRowsJoinThreads = 256;
constexpr int kRowsJoinWarps = kRowsJoinThreads / 32;
constexpr int kRowsJoinFew = 8;       // parts that one thread joins
constexpr int kRowsJoinCols = 4;      // float4 columns of a block's item of more parts

// A block takes items of 32 rows of one cut tile: of few parts, all columns (HD
// / 32 a warp, lanes on neighbouring rows as the parts lie, then through shared
// memory so that whole rows go out); of more, kRowsJoinCols columns, the warps
// taking the parts in turn.  (Lane by row to the end 20 us, all items by the
// second way 32 us, where most tiles have two parts: 4 requests of 1,440 query
// vectors and 8 KV heads over 4,096 keys; 12 to 19 so, 40 MB of partial results
// out of L2.)
template <typename T, int HD, int ROWS>
__global__ void __launch_bounds__(kRowsJoinThreads) cache_rows_join_kernel(const __grid_constant__ CacheRowsArgs a) {
  __shared__ short list[kRowsMaxCtas];
  __shared__ int upto[kRowsMaxCtas + 1];  // items in front of record i of the list
  __shared__ int sums[2][kRowsJoinWarps];
  __shared__ float4 acc[kRowsJoinWarps][kRowsJoinCols][32];
  __shared__ float2 ml[kRowsJoinWarps][32];
  auto groups = [](int n) { return n <= kRowsJoinFew ? 1 : HD / 4 / kRowsJoinCols; };
  __shared__ float4 rows_[32][HD / 4 + 1];
  __shared__ float2 row_ml[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  // the records in use, in order
  int count = 0, items = 0;
  for (int c0 = 0; c0 < a.ctas; c0 += kRowsJoinThreads) {
    const int c = c0 + threadIdx.x;
    const int n = c < a.ctas ? a.joins[c].n : 0, nv = n > 0 ? a.joins[c].nv : 0;
    int x = nv > 0, y = (nv + 31) / 32 * groups(n);
    const int x0 = x, y0 = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kFull, x, o), v = __shfl_up_sync(kFull, y, o);
      if (lane >= o) {
        x += u;
        y += v;
      }
    }
    if (lane == 31) {
      sums[0][warp] = x;
      sums[1][warp] = y;
    }
    __syncthreads();
    int at = count + x - x0, it = items + y - y0;
#pragma unroll
    for (int w = 0; w < kRowsJoinWarps; ++w) {
      if (w < warp) {
        at += sums[0][w];
        it += sums[1][w];
      }
      count += sums[0][w];
      items += sums[1][w];
    }
    if (nv > 0) {
      list[at] = (short)c;
      upto[at] = it;
    }
    __syncthreads();
  }
  for (int i = blockIdx.x; i < items; i += gridDim.x) {
    int lo = 0, hi = count - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (upto[mid] <= i)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int first = list[lo];
    const RowsJoin j = a.joins[first];
    const int in = i - upto[lo], g = groups(j.n), row = in / g * 32 + lane;
    const bool on = row < j.nv;
    if (j.n <= kRowsJoinFew) {
      float f[kRowsJoinFew], top = -INFINITY, l = 0.f;
      float2 y[kRowsJoinFew];
#pragma unroll
      for (int x = 0; x < kRowsJoinFew; ++x) {
        y[x] = make_float2(-INFINITY, 0.f);
        if (on && x < j.n) y[x] = __ldcg(part_ml<ROWS>(a, rows_slot(first + x, x == 0), row));
      }
      constexpr int CW = HD / 4 / kRowsJoinWarps;  // columns of a warp
      float4 o[CW], z[CW][2];
#pragma unroll
      for (int c = 0; c < CW; ++c) {
        o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < 2; ++x)  // the usual two parts at once
          if (on && x < j.n)
            z[c][x] = __ldcg(part_at<HD, ROWS>(a, rows_slot(first + x, x == 0), c * kRowsJoinWarps + warp, row));
      }
#pragma unroll
      for (int x = 0; x < kRowsJoinFew; ++x) top = fmaxf(top, y[x].x);
      const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int x = 0; x < kRowsJoinFew; ++x) {
        f[x] = ex2(y[x].x - base);
        l += y[x].y * f[x];
      }
      auto add = [](float4& o, const float4& z, float f) {
        o = make_float4(o.x + z.x * f, o.y + z.y * f, o.z + z.z * f, o.w + z.w * f);
      };
      if (on) {
#pragma unroll
        for (int c = 0; c < CW; ++c) {
          add(o[c], z[c][0], f[0]);
          add(o[c], z[c][1], f[1]);
        }
#pragma unroll
        for (int x = 2; x < kRowsJoinFew; ++x)
          if (x < j.n) {
#pragma unroll
            for (int c = 0; c < CW; ++c)
              z[c][0] = __ldcg(part_at<HD, ROWS>(a, rows_slot(first + x, false), c * kRowsJoinWarps + warp, row));
#pragma unroll
            for (int c = 0; c < CW; ++c) add(o[c], z[c][0], f[x]);
          }
      }
#pragma unroll
      for (int c = 0; c < CW; ++c) rows_[lane][c * kRowsJoinWarps + warp] = o[c];
      if (warp == 0) row_ml[lane] = make_float2(top, l);
      __syncthreads();
      for (int x = threadIdx.x; x < 32 * (HD / 4); x += kRowsJoinThreads) {
        const int r = x / (HD / 4), c = x % (HD / 4), rr = in / g * 32 + r;
        if (rr < j.nv) {
          const int v = j.v0 + rr, t = v / a.group;
          rows_finish<T, HD>(a, j.row0 + t, j.kvh * a.group + (v - t * a.group), 4 * c, rows_[r][c], row_ml[r].x,
                             row_ml[r].y);
        }
      }
      __syncthreads();
      continue;
    }
    const int c0 = in % g * kRowsJoinCols;
    float m = -INFINITY, l = 0.f;
    float4 o[kRowsJoinCols];
#pragma unroll
    for (int c = 0; c < kRowsJoinCols; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on)
#pragma unroll 2
      for (int x = warp; x < j.n; x += kRowsJoinWarps) {
        const int slot = rows_slot(first + x, x == 0);
        const float2 y = __ldcg(part_ml<ROWS>(a, slot, row));
        float4 z[kRowsJoinCols];
#pragma unroll
        for (int c = 0; c < kRowsJoinCols; ++c) z[c] = __ldcg(part_at<HD, ROWS>(a, slot, c0 + c, row));
        const float to = fmaxf(m, y.x), base = to == -INFINITY ? 0.f : to;
        const float f = ex2(m - base), g = ex2(y.x - base);
        l = l * f + y.y * g;
        m = to;
#pragma unroll
        for (int c = 0; c < kRowsJoinCols; ++c)
          o[c] = make_float4(o[c].x * f + z[c].x * g, o[c].y * f + z[c].y * g, o[c].z * f + z[c].z * g,
                             o[c].w * f + z[c].w * g);
      }
    ml[warp][lane] = make_float2(m, l);
#pragma unroll
    for (int c = 0; c < kRowsJoinCols; ++c) acc[warp][c][lane] = o[c];
    __syncthreads();
    if (warp < kRowsJoinCols && on) {  // warp c: column c of the rows
      float top = ml[0][lane].x;
#pragma unroll
      for (int w = 1; w < kRowsJoinWarps; ++w) top = fmaxf(top, ml[w][lane].x);
      const float base = top == -INFINITY ? 0.f : top;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kRowsJoinWarps; ++w) {
        const float f = ex2(ml[w][lane].x - base);
        const float4 z = acc[w][warp][lane];
        y = make_float4(y.x + z.x * f, y.y + z.y * f, y.z + z.z * f, y.w + z.w * f);
        sum += ml[w][lane].y * f;
      }
      const int v = j.v0 + row, r = v / a.group;
      rows_finish<T, HD>(a, j.row0 + r, j.kvh * a.group + (v - r * a.group), 4 * (c0 + warp), y, top, sum);
    }
    __syncthreads();
  }
  // with a tail: rows that no cut tile holds
  if (!a.tail_ml) return;
  const int64_t all = (int64_t)a.T * a.nq * (HD / 4);
  for (int64_t i = (int64_t)blockIdx.x * kRowsJoinThreads + threadIdx.x; i < all; i += (int64_t)gridDim.x * kRowsJoinThreads) {
    const int64_t at = i / (HD / 4);
    const int d = (int)(i % (HD / 4)) * 4;
    const float2 y = __ldcg(a.whole_ml + at);
    if (y.y == kRowCut) continue;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (y.y != 0.f) o = __ldcg(reinterpret_cast<const float4*>(a.whole_o + at * HD + d));
    const int64_t r = at / a.nq;
    rows_finish<T, HD>(a, r, (int)(at - r * a.nq), d, o, y.x, y.y);
  }
}

// ---- fp32: CUDA cores --------------------------------------------------------
//
// 64 query vectors and blocks of 64 keys: thread (ty, tx) of 16 x 16 has
// 4 x 4 scores (vectors 4 ty .., keys tx, tx + 16, ...) and
// 4 x HD / 16 outputs (columns 4 tx .., 64 + 4 tx ..), in packed fp32.  The
// scores' operands come 4 dimensions at a time from rows padded by 16 bytes; the
// weights lie over the keys.  Two blocks an SM: one loads while the other
// computes.  The products bound large calls: 36 TFLOP/s of the cores' 74 (27 with
// scalar arithmetic and one block an SM), operands from shared memory being the
// rest; 5 sequences of up to 33 rows over up to 1,999 keys, 4/2 heads x 64, take
// 21.6 us with the join, some 5 us a block of keys and part.  A tile of fewer
// vectors costs as much as a full one: one token over 20,000 keys, 28/4 heads x
// 128, takes 100 us here and 27 by sf_cache_attend.
constexpr int kSimtRows = 64;
constexpr int kSimtThreads = 256;
constexpr int kSimtKeys = 64;
constexpr int kSimtCtasPerSM = 2;

template <int HD>
struct SimtLayout {
  static constexpr int LD = HD + 4, PLD = kSimtKeys + 4;
  static constexpr int Q = 0, K = Q + kSimtRows * LD, V = K + kSimtKeys * LD, SLOTS = V + kSimtKeys * HD;
  static constexpr int BYTES = (SLOTS + 2 * kSimtKeys) * 4;
  static_assert(kSimtRows * PLD <= kSimtKeys * LD, "weights over the keys");
  static_assert(kSimtCtasPerSM * (BYTES + 2048) <= 227 * 1024, "two blocks an SM");
};

template <int HD>
__global__ void __launch_bounds__(kSimtThreads, kSimtCtasPerSM) cache_rows_simt_kernel(const __grid_constant__ CacheRowsArgs a) {
  using Lay = SimtLayout<HD>;
  constexpr int RPT = kSimtRows / 16, KPT = kSimtKeys / 16, CPT = HD / 64, COLS = HD / 4;
  extern __shared__ __align__(16) float sm[];
  float *sq = sm + Lay::Q, *sk = sm + Lay::K, *sv = sm + Lay::V, *sp = sk;
  uint32_t* slots = reinterpret_cast<uint32_t*>(sm + Lay::SLOTS);  // of two blocks in turn
  const RowsShape sh{a.group, a.nkv, kSimtRows, 1, kSimtKeys, 1, {1, 1}};
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  if (!a.tail_ml) pdl_wait();  // beside the tail's kernel, which has waited for everything before it
  pdl_trigger();
  RowsWalk walk;
  bool empties;
  const bool ok = rows_plan<kSimtThreads>(a, sh, walk, &empties);
  if (tid == 0) a.joins[blockIdx.x].n = 0;
  if (ok) rows_empties<float, HD, kSimtThreads>(a, empties);
  else rows_refused(a);
  RowsPart p;
  SeqRows q;
  walk.start(sh);
  while (walk.next(a, sh, p, q)) {
    auto look = [&](int b) {  // slots of block b
      if (tid < kSimtKeys) {
        const int j = b * kSimtKeys + tid;
        uint32_t slot = ~0u;
        if (j < q.len) {
          slot = entry_slot32(a.table, entry_of(a, q.s, j), j);
          if (slot == ~0u) cache_error(a.err, kCacheBadPage);
        }
        slots[(b & 1) * kSimtKeys + tid] = slot;
      }
    };
    __syncthreads();  // the last part's queries and slots are read
    look(p.b0);
    for (int i = tid; i < kSimtRows * COLS; i += kSimtThreads) {
      const int r = i / COLS, d = i % COLS * 4, v = p.v0 + r;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < p.nv)
        x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + (int64_t)(q.row0 + v / a.group) * a.ld_q +
                                             (int64_t)(p.kvh * a.group + v % a.group) * HD + d);
      *reinterpret_cast<float4*>(sq + r * Lay::LD + d) = x;
    }
    Two o[RPT][CPT][2];
    float m[RPT], l[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < CPT; ++c) o[i][c][0] = o[i][c][1] = two(0.f, 0.f);
    }
#pragma unroll 1
    for (int b = p.b0; b < p.b1; ++b) {
      __syncthreads();  // the last block's values and weights are read, this one's slots written
      const uint32_t* slot = slots + (b & 1) * kSimtKeys;
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // keys, then values: so many loads in flight together
        const float* pool = static_cast<const float*>(h ? a.v : a.k) + (int64_t)p.kvh * HD;
        constexpr int PER = kSimtKeys * COLS / kSimtThreads;
        float4 x[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const int i = tid + k * kSimtThreads;
          const uint32_t at = slot[i / COLS];
          x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (at != ~0u) x[k] = *reinterpret_cast<const float4*>(pool + (int64_t)at * a.nkv * HD + i % COLS * 4);
        }
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const int i = tid + k * kSimtThreads;
          *reinterpret_cast<float4*>((h ? sv + i / COLS * HD : sk + i / COLS * Lay::LD) + i % COLS * 4) = x[k];
        }
      }
      if (b + 1 < p.b1) look(b + 1);
      bool live[KPT];
#pragma unroll
      for (int k = 0; k < KPT; ++k) live[k] = slot[tx + 16 * k] != ~0u;
      __syncthreads();
      Two s2[RPT][KPT];
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int k = 0; k < KPT; ++k) s2[i][k] = two(0.f, 0.f);
#pragma unroll 4
      for (int d = 0; d < HD; d += 4) {
        float4 x[RPT], y[KPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i) x[i] = *reinterpret_cast<const float4*>(sq + (ty * RPT + i) * Lay::LD + d);
#pragma unroll
        for (int k = 0; k < KPT; ++k) y[k] = *reinterpret_cast<const float4*>(sk + (tx + 16 * k) * Lay::LD + d);
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
          for (int k = 0; k < KPT; ++k)
            s2[i][k] = fma2(two(x[i].z, x[i].w), two(y[k].z, y[k].w), fma2(two(x[i].x, x[i].y), two(y[k].x, y[k].y), s2[i][k]));
      }
      __syncthreads();  // the keys are read: the weights go over them
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        float s[KPT], top = m[i];
#pragma unroll
        for (int k = 0; k < KPT; ++k) {
          const float2 x = both(s2[i][k]);
          s[k] = live[k] ? (x.x + x.y) * a.scale_log2 : -INFINITY;
          top = fmaxf(top, s[k]);
        }
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, x));
        const float base = top == -INFINITY ? 0.f : top, f = ex2(m[i] - base);
        m[i] = top;
        l[i] *= f;
#pragma unroll
        for (int k = 0; k < KPT; ++k) {
          const float w = ex2((s[k] - base) - kRowsRoom);
          l[i] += w;
          sp[(ty * RPT + i) * Lay::PLD + tx + 16 * k] = w;
        }
        const Two ff = two(f, f);
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
          o[i][c][0] = o[i][c][0] * ff;
          o[i][c][1] = o[i][c][1] * ff;
        }
      }
      __syncwarp();  // a warp's two ty read only their own weights
#pragma unroll 2
      for (int j = 0; j < kSimtKeys; j += 4) {
        float4 w[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i) w[i] = *reinterpret_cast<const float4*>(sp + (ty * RPT + i) * Lay::PLD + j);
#pragma unroll
        for (int c = 0; c < CPT; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 v = *reinterpret_cast<const float4*>(sv + (j + e) * HD + 64 * c + 4 * tx);
            const Two v0 = two(v.x, v.y), v1 = two(v.z, v.w);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
              const float x = e == 0 ? w[i].x : e == 1 ? w[i].y : e == 2 ? w[i].z : w[i].w;
              o[i][c][0] = fma2(two(x, x), v0, o[i][c][0]);
              o[i][c][1] = fma2(two(x, x), v1, o[i][c][1]);
            }
          }
      }
    }
    const bool cut = is_cut(p);
    const int slot = rows_slot(blockIdx.x, p.b0 == 0);
    if (cut && p.b0 == 0 && tid == 0) rows_record(a, p, q, walk.per);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) l[i] += __shfl_xor_sync(kFull, l[i], x);
      const int r = ty * RPT + i, v = p.v0 + r, t = v / a.group, h = p.kvh * a.group + (v - t * a.group);
      const int64_t at = (int64_t)(q.row0 + t) * a.nq + h;
      if (r >= p.nv) continue;
#pragma unroll
      for (int c = 0; c < CPT; ++c) {
        const float2 y0 = both(o[i][c][0]), y1 = both(o[i][c][1]);
        const float4 y = make_float4(y0.x, y0.y, y1.x, y1.y);
        if (cut)
          *part_at<HD, kSimtRows>(a, slot, 16 * c + tx, r) = y;
        else if (a.tail_ml)
          *reinterpret_cast<float4*>(a.whole_o + at * HD + 64 * c + 4 * tx) = y;
        else
          rows_finish<float, HD>(a, q.row0 + t, h, 64 * c + 4 * tx, y, m[i], l[i]);
      }
      if (cut && tx == 0) *part_ml<kSimtRows>(a, slot, r) = make_float2(m[i], l[i]);
      if (a.tail_ml && tx == 0 && p.b0 == 0) a.whole_ml[at] = make_float2(m[i], cut ? kRowCut : l[i]);
    }
  }
  if (a.tail_ml) pdl_wait();  // the join waits for this kernel only
}

template <typename T, int HD, int ROWS>
cudaError_t join_rows(cudaStream_t st, const CacheRowsArgs& a, int sm_count) {
  return launch_pdl(st, dim3(4 * sm_count), dim3(kRowsJoinThreads), 0, 1, cache_rows_join_kernel<T, HD, ROWS>, a);
}

template <int HD>
cudaError_t simt_rows(cudaStream_t st, CacheRowsArgs a, int sm_count) {
  a.least = 1;
  const cudaError_t e = launch_pdl(st, dim3(a.ctas), dim3(kSimtThreads), SimtLayout<HD>::BYTES, 1,
                                   cache_rows_simt_kernel<HD>, a);
  return e == cudaSuccess ? join_rows<float, HD, kSimtRows>(st, a, sm_count) : e;
}

template <int HD>
cudaError_t allow_simt() {
  return cudaFuncSetAttribute(cache_rows_simt_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              SimtLayout<HD>::BYTES);
}

}  // namespace

int cache_rows_ctas(int sm_count, int bf16) {
  const int n = (bf16 ? 1 : kSimtCtasPerSM) * sm_count;
  return n < kRowsMaxCtas ? n : kRowsMaxCtas;
}
int cache_rows_slot_rows(int bf16) { return bf16 ? kTcTileRows : kSimtRows; }

cudaError_t prepare_cache_rows() {
  cudaError_t e = allow_simt<128>();
  if (e == cudaSuccess) e = allow_simt<64>();
  if (e == cudaSuccess) e = prepare_cache_rows_tc();
  return e;
}

cudaError_t launch_cache_rows(cudaStream_t st, const CacheRowsArgs& a, int bf16, int hd, int sm_count) {
  if (!bf16) return hd == 128 ? simt_rows<128>(st, a, sm_count) : simt_rows<64>(st, a, sm_count);
  const cudaError_t e = launch_cache_rows_tc(st, a, hd);
  if (e != cudaSuccess) return e;
  return hd == 128 ? join_rows<__nv_bfloat16, 128, kTcTileRows>(st, a, sm_count)
                   : join_rows<__nv_bfloat16, 64, kTcTileRows>(st, a, sm_count);
}

}  // namespace sf
