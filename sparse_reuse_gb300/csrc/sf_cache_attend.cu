// Attention of one new token per sequence over its paged cache
// (specfold_cache.h).
//
//   score_j = scale log2(e) q . k_j,  m = max_j score_j,  p_j = 2^(score_j - m)
//   out = (sum_j p_j v_j) / (sum_j p_j)
//   weights_j += sum over the KV head's query heads of 2^(score_j - lse),
//   lse = m + log2(sum_j p_j)
//
// The p_j are kept 2^-kRoom times smaller than written (the quotient does not
// change): at most 2^18 of them then sum to less than 1, so the unnormalised
// output stays within the largest value and cannot overflow where the result
// does not.
//
// What bounds it: every cached key and value is read once and used for the
// query heads of its group only (4 G flops for 4 bytes of bf16), so it is
// DRAM bandwidth for all but the smallest batches, where it is the latency of
// one chain table -> keys -> scores -> output and the join.
#include <cmath>

#include "sf_cache.h"
#include "sf_tc.cuh"

namespace sf {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr float kRoom = 19.f;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes global -> shared, zeros if !live.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_bf16(uint32_t x) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x));
}

// Query heads that a block takes together: the 8 columns of one or two
// tensor-core tiles (bf16), 8 (fp32).
template <typename T, int NT>
struct Group {
  static constexpr int kHeads = 8 * NT;
};

// Work of one warp: tiles [t, end) in steps of `step` of one segment.
struct Segment {
  int s, kvh, h0, nh, len;
};

// Slot of key 16 t + (lane & 15), or ~0 where there is none.
__device__ __forceinline__ uint32_t tile_slot(const CacheAttendArgs& a, const Segment& g, int t, int lane) {
  const int j = t * kTileKeys + (lane & 15);
  if (j >= g.len) return ~0u;
  const int64_t slot = page_slot(a.table, g.s, j);
  if (slot < 0) {
    cache_error(a.err, kCacheBadPage);
    return ~0u;
  }
  return (uint32_t)slot;
}

// ---- bf16: tensor cores ------------------------------------------------------
//
// S^T = K Q^T and O^T = V^T P^T with m16n8k16: 16 keys (then 16 dimensions) are
// the rows, the group's query heads the columns, so a group of up to 8 heads
// wastes nothing but columns.  The contraction index may be permuted freely if
// both operands agree, which lets a lane take 16 contiguous bytes of a key row
// (8 dimensions) as its operand of two steps.  For V a lane takes 16 bytes of
// four rows and pairs them by byte permutation: the transpose costs 4 PRMT per
// step.  No operand passes through a shuffle or ldmatrix, and every lane reads
// back exactly the bytes it copied itself: the ring needs no barrier.
//
// P enters as the sum of two bf16 numbers (16 bits of it), twice the PV steps,
// so that the result is as good as fp32 weights; the tensor pipe is idle
// otherwise.
template <int HD, int NT>
struct WarpBf16 {
  static constexpr int kStageBytes = 4 * kTileKeys * HD;      // K and V of a tile
  static constexpr int kStages = HD == 128 ? 3 : 5;
  static constexpr int kRing = kStages * kStageBytes;         // bytes a warp
  static constexpr int KC = HD / 32, VC = HD / 64;            // 16-byte chunks of a lane: per key row, per value row

  float o[4 * VC][NT][4];
  float m[NT][2], l[NT][2];

  __device__ __forceinline__ void issue(const CacheAttendArgs& a, const Segment& g, uint32_t ring, uint32_t slot,
                                        int lane) {
    const int r = lane >> 2, c = lane & 3;
    const __nv_bfloat16* kb = static_cast<const __nv_bfloat16*>(a.k) + (int64_t)g.kvh * HD;
    const __nv_bfloat16* vb = static_cast<const __nv_bfloat16*>(a.v) + (int64_t)g.kvh * HD;
    const int64_t row = (int64_t)a.nkv * HD;
    uint32_t dst = ring + lane * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t sl = __shfl_sync(kFull, slot, r + 8 * i);
      const bool live = sl != ~0u;
      const __nv_bfloat16* p = kb + (live ? sl : 0u) * row + c * 8;
#pragma unroll
      for (int x = 0; x < KC; ++x) cp_async16(dst + (i * KC + x) * 512, p + x * 32, live);
    }
    dst += 2 * KC * 512;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t sl = __shfl_sync(kFull, slot, 2 * c + (i & 1) + 8 * (i >> 1));
      const bool live = sl != ~0u;
      const __nv_bfloat16* p = vb + (live ? sl : 0u) * row + r * 8;
#pragma unroll
      for (int x = 0; x < VC; ++x) cp_async16(dst + (i * VC + x) * 512, p + x * 64, live);
    }
  }

  template <bool TRACK>
  __device__ __forceinline__ void run(const CacheAttendArgs& a, const Segment& g, uint32_t ring, int t, int step,
                                      int end, int lane) {
    const int r = lane >> 2, c = lane & 3;
    // Q as the right operand: column r of a tile is query head h0 + 8 n + r
    uint4 q[NT][KC];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < KC; ++x) {
        const int h = 8 * n + r;
        const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.q) + (int64_t)g.s * a.ld_q +
                                 (int64_t)(g.h0 + h) * HD + x * 32 + c * 8;
        q[n][x] = h < g.nh ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < 4 * VC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][n][e] = 0.f;
    }
    // fill the ring; slots are looked up one tile ahead of their copy
    int ti = t;
    uint32_t slot = ti < end ? tile_slot(a, g, ti, lane) : ~0u;
    uint32_t live_slots[kStages];  // which keys of a stage are there
#pragma unroll
    for (int st = 0; st < kStages; ++st) {
      live_slots[st] = slot;
      if (ti < end) {
        issue(a, g, ring + st * kStageBytes, slot, lane);
        ti += step;
        slot = ti < end ? tile_slot(a, g, ti, lane) : ~0u;
      }
      cp_async_commit();
    }
    for (;;) {
#pragma unroll
      for (int st = 0; st < kStages; ++st) {
        if (t >= end) goto done;
        cp_async_wait<kStages - 1>();
        const uint32_t base = ring + st * kStageBytes + lane * 16;
        float sc[NT][4];
        {
          float s2[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[n][e] = s2[n][e] = 0.f;
#pragma unroll
          for (int x = 0; x < KC; ++x) {
            uint32_t u[4], w[4];
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                         : "r"(base + x * 512));
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(base + (KC + x) * 512));
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816(sc[n], u[0], w[0], u[1], w[1], q[n][x].x, q[n][x].y);
              mma16816(s2[n], u[2], w[2], u[3], w[3], q[n][x].z, q[n][x].w);
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[n][e] = (sc[n][e] + s2[n][e]) * a.scale_log2;
        }
        // keys r and r + 8 of the tile; absent ones weigh nothing
        const bool live0 = __shfl_sync(kFull, live_slots[st], r) != ~0u;
        const bool live1 = __shfl_sync(kFull, live_slots[st], r + 8) != ~0u;
        const int j0 = t * kTileKeys + r;
        uint32_t ph[NT][2], pl[NT][2];
        bool grew = false;
        float f[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (!live0) sc[n][0] = sc[n][1] = -INFINITY;
          if (!live1) sc[n][2] = sc[n][3] = -INFINITY;
          if (TRACK) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int h = 8 * n + 2 * c + (e & 1), j = j0 + 8 * (e >> 1);
              if (h < g.nh && j < g.len) a.scores[((int64_t)g.s * a.nq + g.h0 + h) * a.ld_scores + j] = sc[n][e];
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(sc[n][e], sc[n][2 + e]);
            x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
            x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
            x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
            const float mn = fmaxf(m[n][e], x);
            const float b = mn == -INFINITY ? 0.f : mn;
            grew |= mn > m[n][e];
            f[n][e] = ex2(m[n][e] - b);
            m[n][e] = mn;
            sc[n][e] = ex2((sc[n][e] - b) - kRoom);
            sc[n][2 + e] = ex2((sc[n][2 + e] - b) - kRoom);
            l[n][e] = l[n][e] * f[n][e] + (sc[n][e] + sc[n][2 + e]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t hi = pack_bf16(sc[n][2 * i], sc[n][2 * i + 1]);
            const float2 hf = unpack_bf16(hi);
            ph[n][i] = transpose8x8(hi);
            pl[n][i] = transpose8x8(pack_bf16(sc[n][2 * i] - hf.x, sc[n][2 * i + 1] - hf.y));
          }
        }
        if (__any_sync(kFull, grew)) {
#pragma unroll
          for (int i = 0; i < 4 * VC; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[i][n][e] *= f[n][e & 1];
        }
        const uint32_t vbase = base + 2 * KC * 512;
#pragma unroll
        for (int x = 0; x < VC; ++x) {
          uint32_t v[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(v[i][0]), "=r"(v[i][1]), "=r"(v[i][2]), "=r"(v[i][3])
                         : "r"(vbase + (i * VC + x) * 512));
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a0 = __byte_perm(v[0][w], v[1][w], 0x5410), a1 = __byte_perm(v[0][w], v[1][w], 0x7632);
            const uint32_t a2 = __byte_perm(v[2][w], v[3][w], 0x5410), a3 = __byte_perm(v[2][w], v[3][w], 0x7632);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816(o[4 * x + w][n], a0, a1, a2, a3, ph[n][0], ph[n][1]);
              mma16816(o[4 * x + w][n], a0, a1, a2, a3, pl[n][0], pl[n][1]);
            }
          }
        }
        // the stage's bytes are in registers: refill it
        __syncwarp();
        live_slots[st] = slot;
        if (ti < end) {
          issue(a, g, ring + st * kStageBytes, slot, lane);
          ti += step;
          slot = ti < end ? tile_slot(a, g, ti, lane) : ~0u;
        }
        cp_async_commit();
        t += step;
      }
    }
  done:
    cp_async_wait<0>();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[n][e] += __shfl_xor_sync(kFull, l[n][e], 4);
        l[n][e] += __shfl_xor_sync(kFull, l[n][e], 8);
        l[n][e] += __shfl_xor_sync(kFull, l[n][e], 16);
      }
  }

  // Unnormalised output [head][HD] and (max, denominator) of the warp.
  __device__ __forceinline__ void store(float* so, float2* sml, int lane) const {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 8 * n + 2 * c + e;
        if (r == 0) sml[h] = make_float2(m[n][e], l[n][e]);
#pragma unroll
        for (int x = 0; x < VC; ++x) {
          float* p = so + h * HD + 64 * x + 8 * r;
          *reinterpret_cast<float4*>(p) = make_float4(o[4 * x][n][e], o[4 * x][n][2 + e], o[4 * x + 1][n][e],
                                                      o[4 * x + 1][n][2 + e]);
          *reinterpret_cast<float4*>(p + 4) = make_float4(o[4 * x + 2][n][e], o[4 * x + 2][n][2 + e],
                                                          o[4 * x + 3][n][e], o[4 * x + 3][n][2 + e]);
        }
      }
  }
};

// ---- fp32: CUDA cores --------------------------------------------------------
//
// 8 keys at a time: for the scores lane (r, c) holds a quarter of key r's
// dimensions (queries come from shared memory, the four quarters meet in two
// shuffles); for the output a lane holds 4 dimensions of every key and the
// weights come back through shared memory.
template <int HD>
struct WarpF32 {
  static constexpr int KI = HD / 16;           // 16-byte pieces of a key a lane holds
  static constexpr int LPR = HD / 4;           // lanes on one value row
  static constexpr int RPI = 32 / LPR;         // value rows per load
  static constexpr int kRing = 8 * HD * 4 + 512;  // bytes a warp: output, then weights [8 keys][8 heads]

  float o[8][4];
  float m[8], l[8];

  template <bool TRACK>
  __device__ __forceinline__ void run(const CacheAttendArgs& a, const Segment& g, const float* sq, float* sp, int t,
                                      int step, int end, int lane) {
    const int r = lane >> 2, c = lane & 3;
    const int vr = lane / LPR, vd = lane % LPR;
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[h][e] = 0.f;
    }
    const float* kb = static_cast<const float*>(a.k) + (int64_t)g.kvh * HD;
    const float* vb = static_cast<const float*>(a.v) + (int64_t)g.kvh * HD;
    const int64_t row = (int64_t)a.nkv * HD;
    for (; t < end; t += step) {
      const uint32_t slots = tile_slot(a, g, t, lane);
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int j = t * kTileKeys + 8 * half + r;
        if (t * kTileKeys + 8 * half >= g.len) break;
        float4 k[KI], v[8 / RPI];
        const uint32_t sl = __shfl_sync(kFull, slots, 8 * half + r);
        const bool live = sl != ~0u;
        const float* kp = kb + (live ? sl : 0u) * row + c * 4;
#pragma unroll
        for (int i = 0; i < KI; ++i)
          k[i] = live ? *reinterpret_cast<const float4*>(kp + 16 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8 / RPI; ++i) {
          const uint32_t vs = __shfl_sync(kFull, slots, 8 * half + i * RPI + vr);
          v[i] = vs != ~0u ? *reinterpret_cast<const float4*>(vb + (int64_t)vs * row + vd * 4)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float f[8];
        bool grew = false;
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          float x = 0.f;
#pragma unroll
          for (int i = 0; i < KI; ++i) {
            const float4 q = *reinterpret_cast<const float4*>(sq + h * HD + c * 4 + 16 * i);
            x += q.x * k[i].x + q.y * k[i].y + q.z * k[i].z + q.w * k[i].w;
          }
          x += __shfl_xor_sync(kFull, x, 1);
          x += __shfl_xor_sync(kFull, x, 2);
          x = live ? x * a.scale_log2 : -INFINITY;
          if (TRACK && c == (h & 3) && h < g.nh && j < g.len)
            a.scores[((int64_t)g.s * a.nq + g.h0 + h) * a.ld_scores + j] = x;
          float y = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
          y = fmaxf(y, __shfl_xor_sync(kFull, y, 8));
          y = fmaxf(y, __shfl_xor_sync(kFull, y, 16));
          const float mn = fmaxf(m[h], y);
          const float b = mn == -INFINITY ? 0.f : mn;
          grew |= mn > m[h];
          f[h] = ex2(m[h] - b);
          m[h] = mn;
          const float p = ex2((x - b) - kRoom);
          l[h] = l[h] * f[h] + p;
          if (c == (h & 3)) sp[r * 8 + h] = p;
        }
        __syncwarp();
        if (__any_sync(kFull, grew)) {
#pragma unroll
          for (int h = 0; h < 8; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[h][e] *= f[h];
        }
#pragma unroll
        for (int i = 0; i < 8 / RPI; ++i) {
          const float4 p0 = *reinterpret_cast<const float4*>(sp + (i * RPI + vr) * 8);
          const float4 p1 = *reinterpret_cast<const float4*>(sp + (i * RPI + vr) * 8 + 4);
          const float p[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            o[h][0] += p[h] * v[i].x;
            o[h][1] += p[h] * v[i].y;
            o[h][2] += p[h] * v[i].z;
            o[h][3] += p[h] * v[i].w;
          }
        }
        __syncwarp();
      }
    }
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      l[h] += __shfl_xor_sync(kFull, l[h], 4);
      l[h] += __shfl_xor_sync(kFull, l[h], 8);
      l[h] += __shfl_xor_sync(kFull, l[h], 16);
      if (RPI == 2) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[h][e] += __shfl_xor_sync(kFull, o[h][e], 16);
      }
    }
  }

  __device__ __forceinline__ void store(float* so, float2* sml, int lane) const {
    const int vd = lane % LPR;
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      if (lane == 0) sml[h] = make_float2(m[h], l[h]);
      if (lane < LPR)
        *reinterpret_cast<float4*>(so + h * HD + vd * 4) = make_float4(o[h][0], o[h][1], o[h][2], o[h][3]);
    }
  }
};

// ---- the kernel --------------------------------------------------------------

template <typename T, int HD, int NT>
struct WarpOf {
  using type = WarpBf16<HD, NT>;
};
template <int HD, int NT>
struct WarpOf<float, HD, NT> {
  using type = WarpF32<HD>;
};

// Block-wide exclusive scan of tiles per sequence into first[0..S].
__device__ __forceinline__ void scan_tiles(const CacheAttendArgs& a, int* first, int* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int carry = 0;
  for (int s0 = 0; s0 < a.S; s0 += kThreads) {
    const int s = s0 + threadIdx.x;
    int x = 0;
    if (s < a.S) {
      bool bad;
      x = tiles_of(checked_len(a.lens[s], a.limit, &bad));
      if (bad && blockIdx.x == 0) cache_error(a.err, kCacheBadLength);
    }
    int y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(kFull, y, o);
      if (lane >= o) y += z;
    }
    if (lane == 31) sums[warp] = y;
    __syncthreads();
    int before = carry, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
    if (s < a.S) first[s] = before + y - x;
    carry += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) first[a.S] = carry;
  __syncthreads();
}

// out[s][h] of one segment from its unnormalised sum and denominator.
template <typename T>
__device__ __forceinline__ void write_out(const CacheAttendArgs& a, int s, int h, int hd, int d, float4 o, float l) {
  T* p = static_cast<T*>(a.out) + (int64_t)s * a.ld_out + (int64_t)h * hd + d;
  store4<T>(p, make_float4(o.x / l, o.y / l, o.z / l, o.w / l));
}

// Blocks walk the line of units (sf_cache_index.h).  The 8 warps of a block
// take the tiles of a segment in turn, or, where the next segments are whole
// and short, one segment each.
template <typename T, int HD, int NT, bool TRACK>
__global__ void __launch_bounds__(kThreads, 1) cache_attend_kernel(const __grid_constant__ CacheAttendArgs a) {
  using Warp = typename WarpOf<T, HD, NT>::type;
  constexpr int NH = Group<T, NT>::kHeads;
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int kShort = 4;  // tiles of a segment that one warp takes alone
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float2 sml[kWarps][NH];
  __shared__ float sfac[kWarps][NH];
  __shared__ int s_sums[kWarps];
  __shared__ int s_last;
  __shared__ __align__(16) float sq[F32 ? kWarps : 1][F32 ? 8 * HD : 4];
  int* first = reinterpret_cast<int*>(smem + kWarps * Warp::kRing);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned char* mine = smem + warp * Warp::kRing;
  const uint32_t ring = tc::smem_u32(mine);
  pdl_wait();
  pdl_trigger();
  scan_tiles(a, first, s_sums);
  const int G = a.nq / a.nkv, nsub = (G + NH - 1) / NH, H = a.nkv * nsub;
  // empty sequences have no units: zeros
  for (int s = blockIdx.x; s < a.S; s += gridDim.x)
    if (first[s + 1] == first[s])
      for (int i = threadIdx.x; i < a.nq * HD / 4; i += kThreads)
        store4<T>(static_cast<T*>(a.out) + (int64_t)s * a.ld_out + 4 * i, make_float4(0.f, 0.f, 0.f, 0.f));
  const int64_t units = (int64_t)first[a.S] * H;
  const int64_t per = units_per_block(units, gridDim.x, a.least);
  int64_t u = (int64_t)blockIdx.x * per;
  const int64_t u_end = u + per < units ? u + per : units;
  if (u >= u_end) return;
  int s;
  {
    int lo = 0, hi = a.S - 1;  // last s with first[s] * H <= u, never an empty one: take the last of equals
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)first[mid] * H <= u) lo = mid; else hi = mid - 1;
    }
    s = lo;
  }
  auto segment = [&](int ss, int hs) {
    Segment g;
    g.s = ss;
    g.kvh = hs / nsub;
    const int sub = hs % nsub;
    g.h0 = g.kvh * G + sub * NH;
    g.nh = min(NH, G - sub * NH);
    g.len = a.lens[ss];
    return g;
  };
  auto load_q = [&](const Segment& g, float* to, int i0, int step) {
    if constexpr (F32) {
      for (int i = i0; i < 8 * HD; i += step)
        to[i] = i / HD < g.nh ? static_cast<const float*>(a.q)[(int64_t)g.s * a.ld_q + (int64_t)g.h0 * HD + i] : 0.f;
    }
  };
  Warp w;
  auto walk = [&](const Segment& g, float* q, int t, int step, int end) {
    if constexpr (F32)
      w.template run<TRACK>(a, g, q, reinterpret_cast<float*>(mine) + 8 * HD, t, step, end, lane);
    else
      w.template run<TRACK>(a, g, ring, t, step, end, lane);
  };
  while (u < u_end) {
    int tiles = first[s + 1] - first[s];
    const int in_s = (int)(u - (int64_t)first[s] * H);
    const int hs = in_s / tiles, t0 = in_s % tiles;
    // ---- short whole segments: a warp each
    if (t0 == 0 && tiles <= kShort) {
      int n = 0, my_s = -1, my_hs = 0;
      int64_t v = u;
      int cs = s, ch = hs;
      while (n < kWarps && v < u_end) {
        const int ct = first[cs + 1] - first[cs];
        if (ct > kShort || v + ct > u_end) break;
        if (n == warp) {
          my_s = cs;
          my_hs = ch;
        }
        ++n;
        v += ct;
        if (++ch == H) {
          ch = 0;
          do ++cs;
          while (cs < a.S && first[cs + 1] == first[cs]);
        }
      }
      if (n > 1) {
        if (my_s >= 0) {
          const Segment g = segment(my_s, my_hs);
          if constexpr (F32) {
            load_q(g, sq[warp], lane, 32);
            __syncwarp();
          }
          walk(g, sq[F32 ? warp : 0], 0, 1, tiles_of(g.len));
          __syncwarp();
          w.store(reinterpret_cast<float*>(mine), sml[warp], lane);
          __syncwarp();
          for (int i = lane; i < g.nh * HD / 4; i += 32) {
            const int h = i / (HD / 4), d = i % (HD / 4) * 4;
            write_out<T>(a, g.s, g.h0 + h, HD, d, *reinterpret_cast<const float4*>(mine + (h * HD + d) * 4),
                         sml[warp][h].y);
          }
          if (TRACK && lane < g.nh) {
            const float2 ml = sml[warp][lane];
            a.lse[(int64_t)g.s * a.nq + g.h0 + lane] = (ml.x == -INFINITY ? 0.f : ml.x) + (kRoom + log2f(ml.y));
          }
          __syncwarp();
        }
        __syncthreads();  // the warps' tables are free again
        u = v;
        s = cs;
        continue;
      }
    }
    // ---- one segment by all warps
    const int end = (int)(u_end - u < tiles - t0 ? u_end - u : tiles - t0) + t0;
    const Segment g = segment(s, hs);
    if constexpr (F32) {
      load_q(g, sq[0], threadIdx.x, kThreads);
      __syncthreads();
    }
    walk(g, sq[0], t0 + warp, kWarps, end);
    __syncwarp();
    w.store(reinterpret_cast<float*>(mine), sml[warp], lane);
    __syncthreads();
    const int64_t seg0 = (int64_t)first[s] * H + (int64_t)hs * tiles;
    const int b0 = first_block(seg0, per), b1 = last_block(seg0, tiles, per);
    float* part = a.parts + (int64_t)part_slot(blockIdx.x, seg0, per) * NH * (HD + 2);
    // factors of the warps, by 8 * NH threads; the first NH keep the total
    if (threadIdx.x < kWarps * NH) {
      const int x = threadIdx.x / NH, h = threadIdx.x % NH;
      float mm = sml[0][h].x;
#pragma unroll
      for (int i = 1; i < kWarps; ++i) mm = fmaxf(mm, sml[i][h].x);
      const float b = mm == -INFINITY ? 0.f : mm;
      sfac[x][h] = ex2(sml[x][h].x - b);
    }
    __syncthreads();
    if (threadIdx.x < g.nh) {
      const int h = threadIdx.x;
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        mm = fmaxf(mm, sml[i][h].x);
        ll += sml[i][h].y * sfac[i][h];
      }
      if (b0 != b1) {
        part[NH * HD + h] = mm;
        part[NH * HD + NH + h] = ll;
      } else if (TRACK) {
        a.lse[(int64_t)g.s * a.nq + g.h0 + h] = (mm == -INFINITY ? 0.f : mm) + (kRoom + log2f(ll));
      }
    }
    for (int i = threadIdx.x; i < g.nh * HD / 4; i += kThreads) {
      const int h = i / (HD / 4), d = i % (HD / 4) * 4;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      float ll = 0.f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float4 y = *reinterpret_cast<const float4*>(smem + x * Warp::kRing + (h * HD + d) * 4);
        const float f = sfac[x][h];
        o.x += y.x * f;
        o.y += y.y * f;
        o.z += y.z * f;
        o.w += y.w * f;
        ll += sml[x][h].y * f;
      }
      if (b0 != b1)
        *reinterpret_cast<float4*>(part + h * HD + d) = o;
      else
        write_out<T>(a, g.s, g.h0 + h, HD, d, o, ll);
    }
    if (b0 != b1) {
      // the last block to arrive joins the parts, in block order
      __threadfence();
      __syncthreads();
      const int n = b1 - b0 + 1;
      if (threadIdx.x == 0) s_last = atomicInc(a.arrived + b0, n - 1) == (unsigned)(n - 1);
      __syncthreads();
      if (s_last) {
        __threadfence();
        float* fac = reinterpret_cast<float*>(smem);  // [n][NH], over the rings: nobody uses them now
        float2* tot = &sml[0][0];                      // [NH] (max, denominator)
        for (int h = warp; h < g.nh; h += kWarps) {
          float mm = -INFINITY;
          for (int x = lane; x < n; x += 32)
            mm = fmaxf(mm, __ldcg(a.parts + (int64_t)part_slot(b0 + x, seg0, per) * NH * (HD + 2) + NH * HD + h));
          mm = warp_max(mm);
          const float b = mm == -INFINITY ? 0.f : mm;
          float ll = 0.f;
          for (int x = lane; x < n; x += 32) {
            const float* p = a.parts + (int64_t)part_slot(b0 + x, seg0, per) * NH * (HD + 2) + NH * HD + h;
            const float f = ex2(__ldcg(p) - b);
            fac[x * NH + h] = f;
            ll += __ldcg(p + NH) * f;
          }
          ll = sf::warp_sum(ll);
          if (lane == 0) tot[h] = make_float2(mm, ll);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < g.nh * HD / 4; i += kThreads) {
          const int h = i / (HD / 4), d = i % (HD / 4) * 4;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
          for (int x = 0; x < n; ++x) {
            const float4 y = __ldcg(reinterpret_cast<const float4*>(
                a.parts + (int64_t)part_slot(b0 + x, seg0, per) * NH * (HD + 2) + h * HD + d));
            const float f = fac[x * NH + h];
            o.x += y.x * f;
            o.y += y.y * f;
            o.z += y.z * f;
            o.w += y.w * f;
          }
          write_out<T>(a, g.s, g.h0 + h, HD, d, o, tot[h].y);
        }
        if (TRACK && threadIdx.x < g.nh)
          a.lse[(int64_t)g.s * a.nq + g.h0 + threadIdx.x] =
              (tot[threadIdx.x].x == -INFINITY ? 0.f : tot[threadIdx.x].x) + (kRoom + log2f(tot[threadIdx.x].y));
      }
    }
    __syncthreads();  // rings and tables free for the next segment
    u += end - t0;
    if (end == tiles && hs + 1 == H) {
      do ++s;
      while (s < a.S && first[s + 1] == first[s]);
    }
  }
}

// weights_out[s][c][j] = weights_in + the group's normalised weights of key j.
__global__ void __launch_bounds__(256) cache_weights_kernel(const __grid_constant__ CacheAttendArgs a) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x, s = blockIdx.y, G = a.nq / a.nkv;
  bool bad;
  const int len = checked_len(a.lens[s], a.limit, &bad);
  for (int j = threadIdx.x; j < len; j += 256) {
    const int64_t at = ((int64_t)s * a.nkv + c) * a.ld_w + j;
    float w = 0.f;
    for (int g = 0; g < G; ++g) {
      const int64_t h = (int64_t)s * a.nq + c * G + g;
      const float x = a.scores[h * a.ld_scores + j];
      w += x == -INFINITY ? 0.f : ex2(x - a.lse[h]);
    }
    a.w_out[at] = (a.w_in ? a.w_in[at] : 0.f) + w;
  }
}

template <typename T, int HD, int NT, bool TRACK>
cudaError_t attend_t(cudaStream_t st, const CacheAttendArgs& a, int blocks) {
  using Warp = typename WarpOf<T, HD, NT>::type;
  const size_t smem = (size_t)kWarps * Warp::kRing + ((size_t)a.S + 1) * sizeof(int);
  return launch_pdl(st, dim3(blocks), dim3(kThreads), smem, 1, cache_attend_kernel<T, HD, NT, TRACK>, a);
}

template <typename T, int HD, int NT>
cudaError_t attend_n(cudaStream_t st, const CacheAttendArgs& a, int blocks) {
  cudaError_t e = a.w_out ? attend_t<T, HD, NT, true>(st, a, blocks) : attend_t<T, HD, NT, false>(st, a, blocks);
  if (e == cudaSuccess && a.w_out)
    e = launch_pdl(st, dim3(a.nkv, a.S), dim3(256), 0, 1, cache_weights_kernel, a);
  return e;
}

template <typename T, int HD, int NT>
cudaError_t allow_smem() {
  using Warp = typename WarpOf<T, HD, NT>::type;
  const int bytes = kWarps * Warp::kRing + 4097 * (int)sizeof(int);
  cudaError_t e = cudaFuncSetAttribute(cache_attend_kernel<T, HD, NT, true>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(cache_attend_kernel<T, HD, NT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  return e;
}

}  // namespace

int64_t cache_attend_part_floats(const sf_cache_shapes& s) { return 2 * 16 * (int64_t)(s.head_dim + 2); }

cudaError_t prepare_cache_attend() {
  cudaError_t e = allow_smem<__nv_bfloat16, 128, 1>();
  if (e == cudaSuccess) e = allow_smem<__nv_bfloat16, 128, 2>();
  if (e == cudaSuccess) e = allow_smem<__nv_bfloat16, 64, 1>();
  if (e == cudaSuccess) e = allow_smem<__nv_bfloat16, 64, 2>();
  if (e == cudaSuccess) e = allow_smem<float, 128, 1>();
  if (e == cudaSuccess) e = allow_smem<float, 64, 1>();
  return e;
}

cudaError_t launch_cache_attend(cudaStream_t st, const CacheAttendArgs& args, int bf16, int sm_count) {
  CacheAttendArgs a = args;
  const int G = a.nq / a.nkv;
  const int NH = bf16 && G > 8 ? 16 : 8;
  a.least = 2 * kWarps;
  // no more blocks than the longest batch of this table could keep busy
  const int64_t most = (int64_t)a.S * a.nkv * ((G + NH - 1) / NH) * tiles_of((int)a.limit);
  const int64_t want = (most + a.least - 1) / a.least;
  const int blocks = (int)(want < sm_count ? (want < 1 ? 1 : want) : sm_count);
  if (!bf16) return a.hd == 128 ? attend_n<float, 128, 1>(st, a, blocks) : attend_n<float, 64, 1>(st, a, blocks);
  if (a.hd == 128)
    return NH == 16 ? attend_n<__nv_bfloat16, 128, 2>(st, a, blocks) : attend_n<__nv_bfloat16, 128, 1>(st, a, blocks);
  return NH == 16 ? attend_n<__nv_bfloat16, 64, 2>(st, a, blocks) : attend_n<__nv_bfloat16, 64, 1>(st, a, blocks);
}

}  // namespace sf
