// Attention of one new token per sequence over its paged cache
// (specfold_cache.h).
//
//   score_j = scale log2(e) q . k_j,  m = max_j score_j,  p_j = 2^(score_j - m)
//   out = (sum_j p_j v_j) / (sum_j p_j)
//   weights_j += sum over the KV head's query heads of p_j / (sum_j p_j)
//
// m is not kept exact: a tile whose scores stay below m + kSlack uses the old
// m, so the maximum is reduced and sums are rescaled only while it still grows
// by more than that (a few tiles of a sequence), and a tile costs one vote.
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
constexpr int kBlocksPerSM = 1;
constexpr float kSlack = 8.f;
constexpr float kRoom = 19.f + kSlack;
constexpr float kUnroom = 1.f / (1 << 27);  // 2^-kRoom
static_assert(kRoom == 27.f, "kUnroom");
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes global -> shared, zeros if !live.  FIRST: they leave L2 before what others keep there (4 x 4,096 keys that
// are read again and again, three caches of 67 MB in turn: 16.6 against 17.6 us).  Not for a call that writes scores
// too, where it costs 2 %.
__device__ __forceinline__ uint64_t evict_first() {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
template <bool FIRST>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live, uint64_t policy) {
  if constexpr (FIRST)
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
                 "r"(live ? 16 : 0), "l"(policy)
                 : "memory");
  else
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// One sequence and group of query heads h0 .. h0 + nh - 1 of KV head kvh.
struct Segment {
  int s, kvh, h0, nh, len;
};

// A warp's ring of stages in shared memory: `KEYS` keys, then their values,
// rows of HD * sizeof(T) bytes whose 16-byte chunks are permuted by the row
// (chunk ^ turn(row)) so that the lanes of a load meet no bank twice: eight rows
// at one chunk (bf16, ldmatrix), two rows at four (fp32).
// Only this warp fills and reads it: cp.async groups and __syncwarp order it.
template <typename T, int HD, int KEYS, int STAGES, bool FIRST>
struct Ring {
  static constexpr int kRowBytes = HD * (int)sizeof(T);
  static constexpr int kStageBytes = 2 * KEYS * kRowBytes;
  static constexpr int kBytes = STAGES * kStageBytes;
  static constexpr int CH = kRowBytes / 16;   // chunks of a row
  static constexpr int RPC = CH < 32 ? 32 / CH : 1;  // rows of one copy instruction
  static_assert(CH <= 32 && KEYS * STAGES <= 64, "a row per copy at least; one bit per key of the ring in `live`");

  static __device__ __forceinline__ int turn(int row) { return sizeof(T) == 2 ? row & 7 : (row & 1) << 2; }

  uint32_t base;
  uint64_t policy = FIRST ? evict_first() : 0;
  int fill = 0, use = 0;        // stages
  uint64_t live = 0;            // which keys are there, KEYS bits per stage in use order
  int in_ring = 0;

  // Page entry of this lane's key of the tile at key0.  Asked for a tile before it is pushed: its latency is not
  // waited for.
  static __device__ __forceinline__ int32_t look(const CacheAttendArgs& a, const Segment& g, int key0, int lane) {
    const int j = key0 + lane % KEYS;
    return j < g.len ? page_entry(a.table, g.s, j) : -1;
  }

  // Copy the tile at key0 into the next stage.
  __device__ __forceinline__ void push(const CacheAttendArgs& a, const Segment& g, int key0, int32_t page, int lane) {
    uint32_t sl = ~0u;
    const int j = key0 + lane % KEYS;
    if (j < g.len) {
      sl = entry_slot32(a.table, page, j);
      if (sl == ~0u) cache_error(a.err, kCacheBadPage);
    }
    live |= (uint64_t)(__ballot_sync(kFull, sl != ~0u) & (uint32_t)((1ull << KEYS) - 1)) << (KEYS * in_ring);
    ++in_ring;
    const int ch = lane % CH, r0 = lane / CH;
    const char* kb = static_cast<const char*>(a.k) + (int64_t)g.kvh * kRowBytes + ch * 16;
    const char* vb = static_cast<const char*>(a.v) + (int64_t)g.kvh * kRowBytes + ch * 16;
    const uint32_t stride = a.nkv * kRowBytes;
    const uint32_t dst = base + fill * kStageBytes;
#pragma unroll
    for (int i = 0; i < KEYS / RPC; ++i) {
      const int r = i * RPC + r0;
      const uint32_t x = __shfl_sync(kFull, sl, r);
      const bool on = x != ~0u;
      const uint64_t off = (uint64_t)(on ? x : 0u) * stride;
      const uint32_t to = dst + r * kRowBytes + ((ch ^ turn(r)) << 4);
      cp_async16<FIRST>(to, kb + off, on, policy);
      cp_async16<FIRST>(to + KEYS * kRowBytes, vb + off, on, policy);
    }
    fill = fill + 1 == STAGES ? 0 : fill + 1;
  }

  __device__ __forceinline__ uint32_t front() const { return base + use * kStageBytes; }
  __device__ __forceinline__ uint32_t front_live() const { return (uint32_t)(live & ((1ull << KEYS) - 1)); }
  __device__ __forceinline__ void pop() {
    use = use + 1 == STAGES ? 0 : use + 1;
    live >>= KEYS;
    --in_ring;
  }
};

// ---- bf16: tensor cores ------------------------------------------------------
//
// S^T = K Q^T and O^T = V^T P^T with m16n8k16: 16 keys (then 16 dimensions) are
// the rows, the group's query heads the columns, so a group of up to 8 heads
// wastes nothing but columns.  (tcgen05 tiles have 128 rows and one issuing
// thread per block; here 8 warps each stream their own tiles with no barrier
// between them, and the tensor pipe is busy a tenth of the time at 5.7 TB/s.)
//
// P enters as the sum of two bf16 numbers, twice the PV steps: at most 2^-16 of
// each p_j is lost (with one number 2^-8), up or down, where rounding to bf16
// loses up to 2^-8 of the sum.  The denominator adds the p_j in fp32.  At
// 131,071 keys 6 to 12 of 3,584 outputs are not the nearest bf16 to the exact
// value; with fp32 weights throughout it is 2 to 8.
template <int HD, int NT>
struct WarpBf16 {
  template <bool FIRST>
  using RingOf = Ring<__nv_bfloat16, HD, kTileKeys, HD == 128 ? 3 : 4, FIRST>;
  using R = RingOf<true>;
  static constexpr int kStages = R::kBytes / R::kStageBytes;
  static constexpr int kHeads = 8 * NT;        // query heads a block takes together
  static constexpr int kRow = HD + 4;          // floats of a head's row in store(): no bank conflict
  static constexpr int kBytes = R::kBytes > kHeads * kRow * 4 ? R::kBytes : kHeads * kRow * 4;
  static constexpr int KS = HD / 16;

  float o[KS][NT][4];
  float m[NT][2], l[NT][2];

  // Tiles t, t + step, ... below `end` of one segment.
  template <bool TRACK, typename F>
  __device__ __forceinline__ void run(const CacheAttendArgs& a, const Segment& g, unsigned char* mem, const float*, F,
                                      int t, int step, int end, int lane) {
    const int r = lane >> 2, c = lane & 3;
    // Q as the right operand: column r of a tile is query head h0 + 8 n + r
    uint32_t q[NT][KS][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int h = 8 * n + r;
      const __nv_bfloat16* p =
          static_cast<const __nv_bfloat16*>(a.q) + (int64_t)g.s * a.ld_q + (int64_t)(g.h0 + h) * HD + 2 * c;
#pragma unroll
      for (int x = 0; x < KS; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          q[n][x][y] = h < g.nh ? *reinterpret_cast<const uint32_t*>(p + 16 * x + 8 * y) : 0u;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int x = 0; x < KS; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[x][n][e] = 0.f;
    }
    RingOf<!TRACK> ring;
    ring.base = tc::smem_u32(mem);
    int ti = t;
    int32_t pages[kStages];
#pragma unroll
    for (int i = 0; i < kStages; ++i) pages[i] = R::look(a, g, (t + i * step) * kTileKeys, lane);
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
      if (ti < end) {
        ring.push(a, g, ti * kTileKeys, pages[i], lane);
        ti += step;
      }
      cp_async_commit();
    }
    int32_t page = R::look(a, g, ti * kTileKeys, lane);
    // this lane's row and chunk of the operand loads (chunk 2 x + .. of step x)
    const int krow = lane & 15, kch = lane >> 4;
    const int vrow = (lane & 7) + ((lane >> 4) << 3), vch = (lane >> 3) & 1;
#pragma unroll 1
    for (; t < end; t += step) {
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const uint32_t kbase = ring.front() + krow * R::kRowBytes;
      const uint32_t vbase = ring.front() + kTileKeys * R::kRowBytes + vrow * R::kRowBytes;
      const uint32_t live = ring.front_live();
      float sc[NT][4], s2[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][e] = s2[n][e] = 0.f;
#pragma unroll
      for (int x = 0; x < KS; x += 2) {
        uint32_t k0[4], k1[4];
        ldmatrix4(k0, kbase + (((2 * x + kch) ^ R::turn(krow)) << 4));
        ldmatrix4(k1, kbase + (((2 * x + 2 + kch) ^ R::turn(krow)) << 4));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma16816(sc[n], k0, q[n][x][0], q[n][x][1]);
          mma16816(s2[n], k1, q[n][x + 1][0], q[n][x + 1][1]);
        }
      }
      // keys r and r + 8 of the tile; absent ones weigh nothing
      const bool whole = live == 0xffffu;
      bool grew = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float raw = (sc[n][e] + s2[n][e]) * a.scale_log2;
          sc[n][e] = whole || (live >> (r + 8 * (e >> 1)) & 1) ? raw : -INFINITY;
          if (TRACK) {
            const int h = 8 * n + 2 * c + (e & 1), j = t * kTileKeys + r + 8 * (e >> 1);
            if (h < g.nh && j < g.len) a.scores[((int64_t)g.s * a.nq + g.h0 + h) * a.ld_scores + j] = sc[n][e];
          }
          grew |= !(sc[n][e] <= m[n][e & 1] + kSlack);
        }
      if (__any_sync(kFull, grew)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(sc[n][e], sc[n][2 + e]);
            x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
            x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
            x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
            x = fmaxf(m[n][e], x);
            const float f = m[n][e] == x ? 1.f : ex2(m[n][e] - x);
            m[n][e] = x;
            l[n][e] *= f;
#pragma unroll
            for (int y = 0; y < KS; ++y) {
              o[y][n][e] *= f;
              o[y][n][2 + e] *= f;
            }
          }
      }
      uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float b = m[n][e] == -INFINITY ? 0.f : m[n][e];
          sc[n][e] = ex2((sc[n][e] - b) - kRoom);
          sc[n][2 + e] = ex2((sc[n][2 + e] - b) - kRoom);
          l[n][e] += sc[n][e] + sc[n][2 + e];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t hi = pack_bf16(sc[n][2 * i], sc[n][2 * i + 1]);
          const float2 hf = unpack_bf16(hi);
          ph[n][i] = transpose8x8(hi);
          pl[n][i] = transpose8x8(pack_bf16(sc[n][2 * i] - hf.x, sc[n][2 * i + 1] - hf.y));
        }
      }
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        uint32_t v[4];
        ldmatrix4_trans(v, vbase + (((2 * x + vch) ^ R::turn(vrow)) << 4));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma16816(o[x][n], v, ph[n][0], ph[n][1]);
          mma16816(o[x][n], v, pl[n][0], pl[n][1]);
        }
      }
      __syncwarp();  // the stage is read: refill it
      ring.pop();
      if (ti < end) {
        ring.push(a, g, ti * kTileKeys, page, lane);
        ti += step;
        page = R::look(a, g, ti * kTileKeys, lane);
      }
      cp_async_commit();
    }
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

  // Unnormalised output [head][kRow] and (reference, denominator) of the warp.
  __device__ __forceinline__ void store(float* so, float2* sml, int lane) const {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 8 * n + 2 * c + e;
        if (r == 0) sml[h] = make_float2(m[n][e], l[n][e]);
#pragma unroll
        for (int x = 0; x < KS; ++x) {
          so[h * kRow + 16 * x + r] = o[x][n][e];
          so[h * kRow + 16 * x + 8 + r] = o[x][n][2 + e];
        }
      }
  }
};

// ---- fp32: CUDA cores --------------------------------------------------------
//
// 8 keys a stage: for the scores lane (r, c) takes a quarter of key r's
// dimensions (queries come from shared memory, the four quarters meet in two
// shuffles); for the output a lane holds 4 dimensions of every key and the
// weights come back through shared memory.
template <int HD, int NH>
struct WarpF32 {
  static constexpr int KEYS = 8;
  template <bool FIRST>
  using RingOf = Ring<float, HD, KEYS, HD == 128 ? 2 : 4, FIRST>;
  using R = RingOf<true>;
  static constexpr int kStages = R::kBytes / R::kStageBytes;
  static constexpr int kHeads = NH;      // query heads a block takes together
  static constexpr int kRow = HD;
  static constexpr int kBytes = R::kBytes + KEYS * NH * 4;  // the ring (then the output), weights [keys][heads]
  static constexpr int KI = HD / 16;              // 16-byte pieces of a key a lane takes
  static constexpr int LPR = HD / 4;              // lanes on one value row
  static constexpr int RPI = 32 / LPR;            // value rows per load
  static_assert(kHeads * kRow * 4 <= R::kBytes, "output over the ring");

  float o[NH][4];
  float m[NH], l[NH];

  template <bool TRACK, typename F>
  __device__ __forceinline__ void run(const CacheAttendArgs& a, const Segment& g, unsigned char* mem, const float* sq,
                                      F load_q, int t, int step, int end, int lane) {
    const int r = lane >> 2, c = lane & 3;
    const int vr = lane / LPR, vd = lane % LPR;
    float* sp = reinterpret_cast<float*>(mem + R::kBytes);
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[h][e] = 0.f;
    }
    RingOf<!TRACK> ring;
    ring.base = tc::smem_u32(mem);
    // stages in order: both halves of tile t, then those of t + step, ...; those past the end or the length are
    // left out
    int ki = t * kTileKeys, ku = ki;
    const int stop = min(end * kTileKeys, g.len);
    auto next = [&](int k) { return (k & KEYS) ? k - KEYS + step * kTileKeys : k + KEYS; };
    int32_t pages[kStages];
#pragma unroll
    for (int i = 0, k = ki; i < kStages; ++i, k = next(k)) pages[i] = R::look(a, g, k, lane);
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
      if (ki < stop) {
        ring.push(a, g, ki, pages[i], lane);
        ki = next(ki);
      }
      cp_async_commit();
    }
    int32_t page = R::look(a, g, ki, lane);
    load_q();  // queries to shared memory, behind the first copies
#pragma unroll 1
    for (; ku < stop; ku = next(ku)) {
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const unsigned char* st = mem + (ring.front() - ring.base);
      const bool live = ring.front_live() >> r & 1;
      float4 k[KI];
#pragma unroll
      for (int i = 0; i < KI; ++i)
        k[i] = *reinterpret_cast<const float4*>(st + r * R::kRowBytes + (((c + 4 * i) ^ R::turn(r)) << 4));
      float x[NH];
      bool grew = false;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < KI; ++i) {
          const float4 q = *reinterpret_cast<const float4*>(sq + h * HD + c * 4 + 16 * i);
          y.x += q.x * k[i].x;
          y.y += q.y * k[i].y;
          y.z += q.z * k[i].z;
          y.w += q.w * k[i].w;
        }
        x[h] = (y.x + y.y) + (y.z + y.w);
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        x[h] += __shfl_xor_sync(kFull, x[h], 1);
        x[h] += __shfl_xor_sync(kFull, x[h], 2);
        x[h] = live ? x[h] * a.scale_log2 : -INFINITY;
        if (TRACK && c == (h & 3) && h < g.nh && ku + r < g.len)
          a.scores[((int64_t)g.s * a.nq + g.h0 + h) * a.ld_scores + ku + r] = x[h];
        grew |= !(x[h] <= m[h] + kSlack);
      }
      if (__any_sync(kFull, grew)) {
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          float y = fmaxf(x[h], __shfl_xor_sync(kFull, x[h], 4));
          y = fmaxf(y, __shfl_xor_sync(kFull, y, 8));
          y = fmaxf(y, __shfl_xor_sync(kFull, y, 16));
          y = fmaxf(m[h], y);
          const float f = m[h] == y ? 1.f : ex2(m[h] - y);
          m[h] = y;
          l[h] *= f;
#pragma unroll
          for (int e = 0; e < 4; ++e) o[h][e] *= f;
        }
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const float p = ex2((x[h] - (m[h] == -INFINITY ? 0.f : m[h])) - kRoom);
        l[h] += p;
        if (c == (h & 3)) sp[r * NH + h] = p;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8 / RPI; ++i) {
        const int row = i * RPI + vr;
        const float4 v =
            *reinterpret_cast<const float4*>(st + KEYS * R::kRowBytes + row * R::kRowBytes + ((vd ^ R::turn(row)) << 4));
#pragma unroll
        for (int h = 0; h < NH; h += 2) {
          const float2 p = *reinterpret_cast<const float2*>(sp + row * NH + h);
          o[h][0] += p.x * v.x;
          o[h][1] += p.x * v.y;
          o[h][2] += p.x * v.z;
          o[h][3] += p.x * v.w;
          o[h + 1][0] += p.y * v.x;
          o[h + 1][1] += p.y * v.y;
          o[h + 1][2] += p.y * v.z;
          o[h + 1][3] += p.y * v.w;
        }
      }
      __syncwarp();  // the stage and the weights are read
      ring.pop();
      if (ki < stop) {
        ring.push(a, g, ki, page, lane);
        ki = next(ki);
        page = R::look(a, g, ki, lane);
      }
      cp_async_commit();
    }
    cp_async_wait<0>();
#pragma unroll
    for (int h = 0; h < NH; ++h) {
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
    for (int h = 0; h < NH; ++h) {
      if (lane == 0) sml[h] = make_float2(m[h], l[h]);
      if (lane < LPR)
        *reinterpret_cast<float4*>(so + h * kRow + vd * 4) = make_float4(o[h][0], o[h][1], o[h][2], o[h][3]);
    }
  }
};

// ---- the kernels -------------------------------------------------------------

// NT: column tiles of 8 query heads (bf16), or query heads (fp32).
template <typename T, int HD, int NT>
struct WarpOf {
  using type = WarpBf16<HD, NT>;
};
template <int HD, int NT>
struct WarpOf<float, HD, NT> {
  using type = WarpF32<HD, NT>;
};

// Block-wide exclusive scan of units_of(length) per sequence into
// first[0..S], the lengths themselves into lens[0..S-1]; `sums` one int per
// warp.  Returns the number of sequences that are not empty.
template <int THREADS, typename F>
__device__ __forceinline__ int scan_lens(const CacheAttendArgs& a, int* first, int* lens, int* sums, F units_of) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int carry = 0, filled = 0;
  for (int s0 = 0; s0 < a.S; s0 += THREADS) {
    const int s = s0 + threadIdx.x;
    int x = 0;
    if (s < a.S) {
      bool bad;
      const int len = checked_len(__ldcg(a.lens + s), a.limit, &bad);
      lens[s] = len;
      x = units_of(len);
      if (bad && blockIdx.x == 0) cache_error(a.err, kCacheBadLength);
    }
    int y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(kFull, y, o);
      if (lane >= o) y += z;
    }
    if (lane == 31) sums[warp] = y;
    filled += __syncthreads_count(x > 0);
    int before = carry, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
    if (s < a.S) first[s] = before + y - x;
    carry += total;
    if (s0 + THREADS >= a.S && threadIdx.x == 0) first[a.S] = carry;
    __syncthreads();
  }
  return filled;
}

// The sequence that unit u (of H per entry of first) belongs to: the last one
// that starts at or before it, which is not an empty one.
__device__ __forceinline__ int find_sequence(const int* first, int S, int64_t u, int H) {
  int lo = 0, hi = S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((int64_t)first[mid] * H <= u)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Reciprocal of a denominator; 0 for the denominator 0 of a row without a score above -infinity, which gets zeros
// (its sums are 0, and 0 times the reciprocal's infinity would be NaN).  NaN stays NaN.
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }

// o times the reciprocal of the denominator: one quotient where there were four, for one more rounding of fp32.
template <typename T>
__device__ __forceinline__ void write_out(const CacheAttendArgs& a, int s, int h, int hd, int d, float4 o, float inv) {
  T* p = static_cast<T*>(a.out) + (int64_t)s * a.ld_out + (int64_t)h * hd + d;
  store4<T>(p, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
}

// What the weights kernel needs of a row's softmax: the reference m, and the factor that makes 2^(score - m) a weight.
// Not log2 of the denominator added to m: the sum would be rounded at the size of m (scores around 500 then cost a
// weight 3e-5, with the pair none of that).
__device__ __forceinline__ void write_stats(const CacheAttendArgs& a, int s, int h, float m, float l) {
  a.stats[(int64_t)s * a.nq + h] = make_float2(m == -INFINITY ? 0.f : m, inverse(l) * kUnroom);
}

// ex2(m - top) with an empty part (m = -inf) weighing 0 even where all are.
__device__ __forceinline__ float part_factor(float m, float top) { return ex2(m - (top == -INFINITY ? 0.f : top)); }

// Floats of a partial result: output [NH][HD], reference [NH], denominator [NH].
template <int NH, int HD>
__device__ __forceinline__ float* part_of(const CacheAttendArgs& a, int slot) {
  return a.parts + (int64_t)slot * NH * (HD + 2);
}

// Running sum of partial results: 4 dimensions of one head.
constexpr int kPartLoads = 8;  // parts whose loads are in flight together

struct PartSum {
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float top = -INFINITY, l = 0.f;

  __device__ __forceinline__ void scale(float to) {
    const float f = part_factor(top, to);
    o.x *= f;
    o.y *= f;
    o.z *= f;
    o.w *= f;
    l *= f;
    top = to;
  }
  __device__ __forceinline__ void add_one(float4 y, float m, float ly) {
    const float f = part_factor(m, top);
    o.x += y.x * f;
    o.y += y.y * f;
    o.z += y.z * f;
    o.w += y.w * f;
    l += ly * f;
  }
  // The first min(n, LOADS) of the parts slot(0), slot(1), ...
  template <int NH, int HD, int LOADS, typename F>
  __device__ __forceinline__ void add(const CacheAttendArgs& a, int h, int d, int n, F slot) {
    float4 y[LOADS];
    float m[LOADS], ly[LOADS], to = top;
#pragma unroll
    for (int x = 0; x < LOADS; ++x) {
      m[x] = -INFINITY;
      if (x < n) {
        const float* p = part_of<NH, HD>(a, slot(x));
        y[x] = __ldcg(reinterpret_cast<const float4*>(p + h * HD + d));
        m[x] = __ldcg(p + NH * HD + h);
        ly[x] = __ldcg(p + NH * HD + NH + h);
      }
    }
#pragma unroll
    for (int x = 0; x < LOADS; ++x) to = fmaxf(to, m[x]);
    scale(to);
#pragma unroll
    for (int x = 0; x < LOADS; ++x)
      if (x < n) add_one(y[x], m[x], ly[x]);
  }
};

// The work is cut over the blocks in one of two ways, by the batch's lengths.
//
// Chunks: where there is a block for every segment, every segment is cut into
// equal chunks, as many as give at most one chunk per block.  A block has one
// segment, loads one query, joins once (3 x 4,096 keys of 8 heads: 13.7 against
// 16.9 us on a line).
//
// Line: otherwise, or where a chunk would be more than kWaste tiles longer than
// an even share, blocks walk equal parts of the line of units
// (sf_cache_index.h).  kWaste has measurements on both sides there.
//
// The 8 warps of a block take the tiles of a segment in turn, or, where short
// segments follow one another on a line, one segment each (300 sequences of up
// to 62 keys, 4 heads: 12.6 us; every segment by a block: 43.8).  A segment cut
// over few blocks is joined by the last of them to finish, one cut over many by
// the join kernel.
template <typename T, int HD, int NT, bool TRACK>
__global__ void __launch_bounds__(kThreads, kBlocksPerSM) cache_attend_kernel(const __grid_constant__ CacheAttendArgs a) {
  using Warp = typename WarpOf<T, HD, NT>::type;
  constexpr int NH = Warp::kHeads, ROW = Warp::kRow;
  constexpr bool F32 = sizeof(T) == 4;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float2 sml[kWarps][NH];
  __shared__ float sfac[kWarps][NH];
  __shared__ int sums[kWarps];
  __shared__ int s_last;
  __shared__ __align__(16) float sq[F32 ? kWarps : 1][F32 ? NH * HD : 4];
  int* first = reinterpret_cast<int*>(smem + kWarps * Warp::kBytes);
  int* lens = first + a.S + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, blk = blockIdx.x;
  unsigned char* mine = smem + warp * Warp::kBytes;
  float* my_out = reinterpret_cast<float*>(mine);
  const int H = a.heads;
  pdl_wait();
  pdl_trigger();
  const int filled = scan_lens<kThreads>(a, first, lens, sums, [](int len) { return tiles_of(len); });
  if (a.join && threadIdx.x == 0) a.joins[blk].n = 0;
  // empty sequences have no units: zeros
  if (filled < a.S)
    for (int s = blk; s < a.S; s += gridDim.x)
      if (first[s + 1] == first[s])
        for (int i = threadIdx.x; i < a.nq * HD / 4; i += kThreads)
          store4<T>(static_cast<T*>(a.out) + (int64_t)s * a.ld_out + 4 * i, make_float4(0.f, 0.f, 0.f, 0.f));
  const int64_t units = (int64_t)first[a.S] * H;
  if (units == 0) return;
  const int64_t share = units_per_block(units, gridDim.x, kLeast);

  auto segment = [&](int s, int hs) {
    Segment g;
    g.s = s;
    g.kvh = a.nsub == 1 ? hs : hs / a.nsub;
    const int sub = hs - g.kvh * a.nsub;
    g.h0 = g.kvh * a.group + sub * NH;
    g.nh = min(NH, a.group - sub * NH);
    g.len = lens[s];
    return g;
  };
  auto load_q = [&](const Segment& g, float* to, int i0, int step) {
    if constexpr (F32) {
      for (int i = i0; i < NH * HD; i += step)
        to[i] = i < g.nh * HD ? static_cast<const float*>(a.q)[(int64_t)g.s * a.ld_q + (int64_t)g.h0 * HD + i] : 0.f;
    }
  };
  Warp w;

  // Tiles [t0, end) of a segment by all warps; the segment lies in n blocks from b0 on, whose partial results are
  // in slots `slot0`, 2 (b0 + 1), 2 (b0 + 2), ...; this block's is `slot`.
  auto take = [&](const Segment& g, int t0, int end, int n, int b0, int slot0, int slot) {
    auto queries = [&]() {
      load_q(g, sq[0], threadIdx.x, kThreads);
      __syncthreads();
    };
    w.template run<TRACK>(a, g, mine, sq[0], queries, t0 + warp, kWarps, end, lane);
    __syncwarp();
    w.store(my_out, sml[warp], lane);
    __syncthreads();
    float* part = part_of<NH, HD>(a, slot);
    if (threadIdx.x < kWarps * NH) {
      const int x = threadIdx.x / NH, h = threadIdx.x % NH;
      float top = sml[0][h].x;
#pragma unroll
      for (int i = 1; i < kWarps; ++i) top = fmaxf(top, sml[i][h].x);
      sfac[x][h] = part_factor(sml[x][h].x, top);
    }
    __syncthreads();
    if (threadIdx.x < g.nh && (n > 1 || TRACK)) {
      const int h = threadIdx.x;
      float top = -INFINITY, l = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        top = fmaxf(top, sml[i][h].x);
        l += sml[i][h].y * sfac[i][h];
      }
      if (n > 1) {
        part[NH * HD + h] = top;
        part[NH * HD + NH + h] = l;
      } else {
        write_stats(a, g.s, g.h0 + h, top, l);
      }
    }
    for (int i = threadIdx.x; i < g.nh * HD / 4; i += kThreads) {
      const int h = i / (HD / 4), d = i % (HD / 4) * 4;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      float l = 0.f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float4 y = *reinterpret_cast<const float4*>(smem + x * Warp::kBytes + (h * ROW + d) * 4);
        const float f = sfac[x][h];
        o.x += y.x * f;
        o.y += y.y * f;
        o.z += y.z * f;
        o.w += y.w * f;
        l += sml[x][h].y * f;
      }
      if (n > 1)
        *reinterpret_cast<float4*>(part + h * HD + d) = o;
      else
        write_out<T>(a, g.s, g.h0 + h, HD, d, o, inverse(l));
    }
    if (n > kInlineParts) {
      if (blk == b0 && threadIdx.x == 0) a.joins[b0] = CacheJoin{n, g.s, g.h0, g.nh, slot0};
    } else if (n > 1) {
      // the last block to arrive joins the parts, in block order
      __syncthreads();
      if (threadIdx.x == 0) {
        __threadfence();  // the block's part, which the barrier ordered before this
        s_last = atomicInc(a.arrived + b0, n - 1) == (unsigned)(n - 1);
        __threadfence();
      }
      __syncthreads();
      if (s_last) {
        for (int i = threadIdx.x; i < g.nh * HD / 4; i += kThreads) {
          const int h = i / (HD / 4), d = i % (HD / 4) * 4;
          PartSum sum;
          if (n <= 4)
            sum.add<NH, HD, 4>(a, h, d, n, [&](int x) { return x ? 2 * (b0 + x) : slot0; });
          else
            for (int x0 = 0; x0 < n; x0 += kPartLoads)
              sum.add<NH, HD, kPartLoads>(a, h, d, n - x0, [&](int x) { return x0 + x ? 2 * (b0 + x0 + x) : slot0; });
          const float4 o = sum.o;
          const float top = sum.top, l = sum.l;
          write_out<T>(a, g.s, g.h0 + h, HD, d, o, inverse(l));
          if (TRACK && d == 0) write_stats(a, g.s, g.h0 + h, top, l);
        }
      }
    }
  };

  // ---- chunks.  Every warp works the plan out for itself (no barrier).
  if ((int64_t)filled * H <= gridDim.x && a.S <= kThreads) {
    int size = (int)share, chunks = 0, longest = 0;
    for (int i = 0; i < kPlanTries; ++i) {
      chunks = longest = 0;
      for (int s0 = 0; s0 < a.S; s0 += 32) {
        const int s = s0 + lane;
        const int t = s < a.S ? first[s + 1] - first[s] : 0;
        const int n = chunks_of(t, size), c = n ? chunk_tiles(t, n) : 0;
        chunks += (int)__reduce_add_sync(kFull, (unsigned)n);
        longest = max(longest, (int)__reduce_max_sync(kFull, (unsigned)c));
      }
      if (chunks * H <= (int)gridDim.x) break;
      size = wider_chunks(size, chunks * H, gridDim.x);
    }
    if (plan_fits(chunks * H, longest, share, gridDim.x)) {
      if (blk >= chunks * H) return;
      int before = 0;  // chunks of the sequences in front
      for (int s0 = 0;; s0 += 32) {
        const int s = s0 + lane, t = s < a.S ? first[s + 1] - first[s] : 0;
        const int c = chunks_of(t, size);
        int incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int z = __shfl_up_sync(kFull, incl, o);
          if (lane >= o) incl += z;
        }
        const unsigned hit = __ballot_sync(kFull, blk < (before + incl) * H);
        if (hit) {
          const int l = __ffs(hit) - 1, n = __shfl_sync(kFull, c, l);
          const int r = blk - (before + __shfl_sync(kFull, incl, l) - n) * H;
          const int hs = (unsigned)r / (unsigned)n, x = r - hs * n, tiles = __shfl_sync(kFull, t, l);
          const int each = chunk_tiles(tiles, n);
          take(segment(s0 + l, hs), min(tiles, x * each), min(tiles, (x + 1) * each), n, blk - x, 2 * (blk - x),
               2 * blk);
          return;
        }
        before += __shfl_sync(kFull, incl, 31);
      }
    }
  }

  // ---- line
  int64_t u = blk * share;
  const int64_t u_end = u + share < units ? u + share : units;
  if (u >= u_end) return;
  int s = find_sequence(first, a.S, u, H), hs, t0;
  {
    const int in_s = (int)(u - (int64_t)first[s] * H), tiles = first[s + 1] - first[s];
    hs = (unsigned)in_s / (unsigned)tiles;
    t0 = in_s - hs * tiles;
  }
  auto advance = [&](int& s, int& hs) {  // to the next segment
    if (++hs == H) {
      hs = 0;
      do ++s;
      while (s < a.S && first[s + 1] == first[s]);
    }
  };
  if (const int skip = skipped(t0, first[s + 1] - first[s])) {
    u += skip;
    t0 = 0;
    advance(s, hs);
  }
  while (u < u_end) {
    const int tiles = first[s + 1] - first[s];
    const bool whole = tiles <= kShort;
    // several of them: a warp each (one sequence of 21 keys, 28 heads over 4: 4.2 us of GPU time; with the lengths
    // looked up again for every segment of a sequence and four quotients per float4 of the output 5.1)
    if (whole) {
      int n = 0, my_s = -1, my_hs = 0, cs = s, ch = hs, ct = tiles, taken = 0;
      const int left = (int)(u_end - u < kWarps * kShort ? u_end - u : kWarps * kShort);
      while (n < kWarps && taken < left && ct <= kShort) {
        if (n == warp) {
          my_s = cs;
          my_hs = ch;
        }
        ++n;
        taken += ct;
        if (++ch == H) {
          ch = 0;
          do ++cs;
          while (cs < a.S && first[cs + 1] == first[cs]);
          ct = cs < a.S ? first[cs + 1] - first[cs] : 0;
        }
      }
      if (n > 1) {
        if (my_s >= 0) {
          const Segment g = segment(my_s, my_hs);
          float* q = sq[F32 ? warp : 0];
          auto queries = [&]() {
            load_q(g, q, lane, 32);
            __syncwarp();
          };
          w.template run<TRACK>(a, g, mine, q, queries, 0, 1, tiles_of(g.len), lane);
          __syncwarp();
          w.store(my_out, sml[warp], lane);
          __syncwarp();
          if (lane < g.nh) sfac[warp][lane] = inverse(sml[warp][lane].y);
          __syncwarp();
          for (int i = lane; i < g.nh * HD / 4; i += 32) {
            const int h = i / (HD / 4), d = i % (HD / 4) * 4;
            write_out<T>(a, g.s, g.h0 + h, HD, d, *reinterpret_cast<const float4*>(my_out + h * ROW + d),
                         sfac[warp][h]);
          }
          if (TRACK && lane < g.nh) write_stats(a, g.s, g.h0 + lane, sml[warp][lane].x, sml[warp][lane].y);
        }
        __syncthreads();  // the warps' memory is free again
        u += taken;
        s = cs;
        hs = ch;
        continue;
      }
    }
    const int64_t seg0 = u - t0;
    const LineTake x = take_of_line(blk, u, u_end, t0, tiles, share);
    take(segment(s, hs), t0, x.end, x.b1 - x.b0 + 1, x.b0, part_slot(x.b0, seg0, share), part_slot(blk, seg0, share));
    __syncthreads();  // the warps' memory and tables are free for the next segment
    u += x.end - t0;
    t0 = 0;
    advance(s, hs);
  }
}

// Joins a segment cut over more than kInlineParts blocks: a block per (segment,
// head), the parts dealt over groups of HD / 4 threads.
constexpr int kJoinThreads = 256;
constexpr int kMaxBlocks = 512;  // of the attention kernel

template <typename T, int HD, int NH>
__global__ void __launch_bounds__(kJoinThreads) cache_join_kernel(const __grid_constant__ CacheAttendArgs a) {
  constexpr int COLS = HD / 4, GROUPS = kJoinThreads / COLS;
  __shared__ float4 acc[GROUPS][COLS];
  __shared__ float2 ml[GROUPS];
  pdl_wait();
  pdl_trigger();
  // a joined segment spans more than kInlineParts blocks: at most one starts among kInlineParts neighbours
  const int lane = threadIdx.x & 31, b = blockIdx.x * kInlineParts + lane;
  const unsigned hit = __ballot_sync(kFull, lane < kInlineParts && b < a.blocks && a.joins[b].n > 0);
  if (hit == 0u) return;
  const int b0 = blockIdx.x * kInlineParts + __ffs(hit) - 1;
  const CacheJoin j = a.joins[b0];
  const int h = blockIdx.y;
  if (h >= j.nh) return;
  const int g = threadIdx.x / COLS, col = threadIdx.x % COLS;
  PartSum sum;
  for (int x0 = g; x0 < j.n; x0 += GROUPS * kPartLoads)
    sum.add<NH, HD, kPartLoads>(a, h, 4 * col, (j.n - x0 + GROUPS - 1) / GROUPS, [&](int x) {
      const int p = x0 + x * GROUPS;
      return p ? 2 * (b0 + p) : j.first;
    });
  acc[g][col] = sum.o;
  if (col == 0) ml[g] = make_float2(sum.top, sum.l);
  __syncthreads();
  if (g == 0) {
    float to = ml[0].x;
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) to = fmaxf(to, ml[i].x);
    sum.scale(to);
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) sum.add_one(acc[i][col], ml[i].x, ml[i].y);
    write_out<T>(a, j.s, j.h0 + h, HD, 4 * col, sum.o, inverse(sum.l));
    if (a.w_out && col == 0) write_stats(a, j.s, j.h0 + h, sum.top, sum.l);
  }
}

// weights_out[s][c][j] = weights_in + the group's normalised weights of key j.
// Blocks take units of kWeightKeys keys of one (sequence, KV head) in turn.
constexpr int kWeightThreads = 256;
constexpr int kWeightKeys = 4 * kWeightThreads;

__global__ void __launch_bounds__(kWeightThreads) cache_weights_kernel(const __grid_constant__ CacheAttendArgs a) {
  extern __shared__ int first[];
  __shared__ int sums[kWeightThreads / 32];
  int* lens = first + a.S + 1;
  // Behind the attention kernel, which has waited for everything before it: the lengths, and the weights so far, are
  // there and stay as they are.  Read through L2.
  const int G = a.group;
  scan_lens<kWeightThreads>(a, first, lens, sums, [](int len) { return (len + kWeightKeys - 1) / kWeightKeys; });
  const int64_t units = (int64_t)first[a.S] * a.nkv;
  bool waited = false;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int s = find_sequence(first, a.S, u, a.nkv), n = first[s + 1] - first[s];
    const int in_s = (int)(u - (int64_t)first[s] * a.nkv), c = in_s / n;
    const int j = in_s % n * kWeightKeys + 4 * (int)threadIdx.x, len = lens[s];
    // the rows of scores are padded to 4 floats: behind the length there is something to read, if nothing to use
    const int64_t at = ((int64_t)s * a.nkv + c) * a.ld_w + j;
    const int64_t h = (int64_t)s * a.nq + c * G;
    const float4* sc = reinterpret_cast<const float4*>(a.scores + h * a.ld_scores + j);
    float before[4], w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) before[i] = a.w_in && j + i < len ? __ldcg(a.w_in + at + i) : 0.f;
    if (!waited) {
      pdl_wait();
      pdl_trigger();
      waited = true;
    }
    if (j >= len) continue;
#pragma unroll 4
    for (int g = 0; g < G; ++g) {
      const float2 st = a.stats[h + g];  // its first is finite or +infinity: a score of -infinity weighs 0
      const float4 x = __ldcs(sc + g * (a.ld_scores / 4));
      w[0] += ex2(x.x - st.x) * st.y;
      w[1] += ex2(x.y - st.x) * st.y;
      w[2] += ex2(x.z - st.x) * st.y;
      w[3] += ex2(x.w - st.x) * st.y;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (j + i < len) a.w_out[at + i] = before[i] + w[i];
  }
  if (!waited) pdl_wait();
}

template <typename T, int HD, int NT>
constexpr int ring_bytes() {
  return kWarps * WarpOf<T, HD, NT>::type::kBytes;
}

template <typename T, int HD, int NT>
cudaError_t attend_t(cudaStream_t st, CacheAttendArgs a, int sm_count) {
  const int most_blocks = cache_attend_blocks(sm_count);
  constexpr int NH = WarpOf<T, HD, NT>::type::kHeads;
  const int G = a.nq / a.nkv, longest = tiles_of((int)a.limit);
  a.group = G;
  a.nsub = (G + NH - 1) / NH;
  a.heads = a.nkv * a.nsub;
  const int blocks = attend_blocks((int64_t)a.S * a.heads * longest, most_blocks);
  a.blocks = blocks;
  a.join = may_need_join(longest, a.heads, blocks);
  const size_t table = (2 * (size_t)a.S + 1) * sizeof(int), smem = ring_bytes<T, HD, NT>() + table;
  cudaError_t e = launch_pdl(st, dim3(blocks), dim3(kThreads), smem, 1,
                             a.w_out ? cache_attend_kernel<T, HD, NT, true> : cache_attend_kernel<T, HD, NT, false>, a);
  if (e == cudaSuccess && a.join)
    e = launch_pdl(st, dim3((blocks + kInlineParts - 1) / kInlineParts, NH < G ? NH : G), dim3(kJoinThreads), 0, 1,
                   cache_join_kernel<T, HD, NH>, a);
  if (e == cudaSuccess && a.w_out) {
    const int64_t most = (int64_t)a.S * a.nkv * ((a.limit + kWeightKeys - 1) / kWeightKeys);
    e = launch_pdl(st, dim3((unsigned)(most < 8 * sm_count ? most : 8 * sm_count)), dim3(kWeightThreads), table, 1,
                   cache_weights_kernel, a);
  }
  return e;
}

template <typename T, int HD, int NT>
cudaError_t allow_smem() {
  const int bytes = ring_bytes<T, HD, NT>() + (2 * 4096 + 1) * (int)sizeof(int);
  cudaError_t e = cudaFuncSetAttribute(cache_attend_kernel<T, HD, NT, true>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(cache_attend_kernel<T, HD, NT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  return e;
}

}  // namespace

int64_t cache_attend_part_floats(const sf_cache_shapes& s) { return 2 * 16 * (int64_t)(s.head_dim + 2); }

int cache_attend_blocks(int sm_count) {
  return kBlocksPerSM * sm_count < kMaxBlocks ? kBlocksPerSM * sm_count : kMaxBlocks;
}

cudaError_t prepare_cache_attend() {
  cudaError_t e = allow_smem<__nv_bfloat16, 128, 1>();
  if (e == cudaSuccess) e = allow_smem<__nv_bfloat16, 128, 2>();
  if (e == cudaSuccess) e = allow_smem<__nv_bfloat16, 64, 1>();
  if (e == cudaSuccess) e = allow_smem<__nv_bfloat16, 64, 2>();
  if (e == cudaSuccess) e = allow_smem<float, 128, 2>();
  if (e == cudaSuccess) e = allow_smem<float, 128, 8>();
  if (e == cudaSuccess) e = allow_smem<float, 64, 2>();
  if (e == cudaSuccess) e = allow_smem<float, 64, 8>();
  return e;
}

cudaError_t launch_cache_attend(cudaStream_t st, const CacheAttendArgs& a, int bf16, int sm_count) {
  if (!bf16) {
    const bool few = a.nq / a.nkv <= 2;
    if (a.hd == 128) return few ? attend_t<float, 128, 2>(st, a, sm_count) : attend_t<float, 128, 8>(st, a, sm_count);
    return few ? attend_t<float, 64, 2>(st, a, sm_count) : attend_t<float, 64, 8>(st, a, sm_count);
  }
  const bool wide = a.nq / a.nkv > 8;
  if (a.hd == 128)
    return wide ? attend_t<__nv_bfloat16, 128, 2>(st, a, sm_count) : attend_t<__nv_bfloat16, 128, 1>(st, a, sm_count);
  return wide ? attend_t<__nv_bfloat16, 64, 2>(st, a, sm_count) : attend_t<__nv_bfloat16, 64, 1>(st, a, sm_count);
}

}  // namespace sf
