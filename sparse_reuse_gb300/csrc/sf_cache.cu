// Paged-cache operators: the object, argument checks and the C ABI
// (specfold_cache.h), the rotary table and the append kernel.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "sf_cache.h"

namespace sf {
namespace {

// Rotary table [max_pos][cos half | sin half] in double, rounded once: far
// positions (10^5 radians and more) lose the angle in fp32.  A thread takes one
// frequency over kRopeRun positions: sine and cosine of the first angle and of
// the step, then the addition theorem (double rounding grows by about 2^-53 a
// step, far below fp32's half step); FP64 rates make a sine per entry slow.
constexpr int kRopeRun = 64;

__global__ void rope_table_kernel(float* out, int max_pos, int half, double theta) {
  const int j = threadIdx.x, p0 = blockIdx.x * kRopeRun, p1 = min(p0 + kRopeRun, max_pos);
  const double freq = pow(theta, -(double)j / half);
  double s, c, ds, dc;
  sincos((double)p0 * freq, &s, &c);
  sincos(freq, &ds, &dc);
  for (int p = p0; p < p1; ++p) {
    out[(int64_t)p * 2 * half + j] = (float)c;
    out[(int64_t)p * 2 * half + half + j] = (float)s;
    const double t = c * dc - s * ds;
    s = s * dc + c * ds;
    c = t;
  }
}

// Two fp32 values in a register pair: sm_100's packed arithmetic does both in
// one instruction, each rounded as the scalar one.
struct Two {
  unsigned long long v;
};
__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both(Two a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// 16 bytes of a row as pairs of fp32, and back.
template <typename T>
struct Piece;
template <>
struct Piece<float> {
  static constexpr int PAIRS = 2;
  static __device__ __forceinline__ void load(const uint4& u, Two (&x)[2]) {
    x[0] = two(__uint_as_float(u.x), __uint_as_float(u.y));
    x[1] = two(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ uint4 store(const Two (&x)[2]) {
    const float2 a = both(x[0]), b = both(x[1]);
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  }
};
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int PAIRS = 4;
  static __device__ __forceinline__ void load(const uint4& u, Two (&x)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = two(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 store(const Two (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = both(x[i]);
      const __nv_bfloat162 b = __floats2bfloat162_rn(a.x, a.y);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <int PAIRS>
__device__ __forceinline__ void load_pairs(const float* p, Two (&x)[PAIRS]) {
#pragma unroll
  for (int i = 0; i < PAIRS / 2; ++i) {
    const float4 v = *reinterpret_cast<const float4*>(p + 4 * i);
    x[2 * i] = two(v.x, v.y);
    x[2 * i + 1] = two(v.z, v.w);
  }
}

// 8,188 rows of 40/8 heads x 128 bf16: 43.6 us so (5.4 TB/s in and out); 128 threads 46.6, three or four heads a
// group 51 and 68, the compiler's own 72 registers instead of 56 (18 blocks an SM) 45.3, 48 registers 51.6.
constexpr int kAppendThreads = 64;
constexpr int kAppendHeads = 2;
constexpr int kAppendBlocks = 18;
// (lane, head) pairs per SM from which a group takes several heads.  40/8 heads x 128 bf16, 512 rows (1,509 pairs):
// 4.2 us with one, 4.9 with two; 1,024 rows: 8.6 and 7.8; 4,096 rows: 31.4 and 24.2.
constexpr int kAppendWide = 2048;

// Norm, rotation and store of HPT heads of one row by a group of lanes: a lane
// holds 16 bytes of a head's lower half and the same 16 of its upper half, so
// both members of its rotation pairs are in its registers and the norm needs
// log2(lanes) shuffles.  Bytes bound it (each row in and out once); HPT heads
// keep 2 HPT loads in flight and share the row's angles and its page lookup.
template <typename T, int HD, int HPT>
__global__ void __launch_bounds__(kAppendThreads, kAppendBlocks) cache_append_kernel(const __grid_constant__ CacheAppendArgs a) {
  using P = Piece<T>;
  constexpr int N = P::PAIRS, VEC = 2 * N, LANES = HD / 2 / VEC, GROUPS = kAppendThreads / LANES;
  pdl_wait();
  pdl_trigger();
  const int NH = a.nq + 2 * a.nkv;
  const unsigned NB = (NH + HPT - 1) / HPT;
  const unsigned item = blockIdx.x * GROUPS + threadIdx.x / LANES;  // (row, head block); T * NB < 2^31
  const int lane = threadIdx.x % LANES;
  const int t = item / NB, h0 = (item - t * NB) * HPT;
  if (t >= a.T) return;  // whole groups: the shuffles below stay inside a group
  const unsigned mask = (LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1u)) << ((threadIdx.x & 31) / LANES * LANES);
  // the row itself first: it waits for nothing, its place and angles arrive meanwhile
  const T* src = static_cast<const T*>(a.qkv) + t * a.ld_qkv + h0 * HD + lane * VEC;
  uint4 lo[HPT], hi[HPT];
#pragma unroll
  for (int i = 0; i < HPT; ++i)
    if (h0 + i < NH) {
      lo[i] = *reinterpret_cast<const uint4*>(src + i * HD);
      hi[i] = *reinterpret_cast<const uint4*>(src + i * HD + HD / 2);
    }
  const int idx = a.index[t];
  const int pos = a.pos ? a.pos[t] : idx;
  if (pos < 0) return;
  if (pos >= a.max_pos) {
    if (lane == 0) cache_error(a.err, kCacheBadRow);
    return;
  }
  Two cs[N], sn[N];
  if (h0 < a.nq + a.nkv) {
    const float* p = a.rope + (int64_t)pos * HD + lane * VEC;
    load_pairs(p, cs);
    load_pairs(p + HD / 2, sn);
  }
  int64_t slot = -1;
  if (h0 + HPT > a.nq && idx >= 0) {
    const int s = a.seq ? a.seq[t] : t;
    if (s < 0 || s >= a.S || idx >= a.limit) {
      if (lane == 0) cache_error(a.err, kCacheBadRow);
    } else {
      slot = page_slot(a.table, s, idx);
      if (slot < 0 && lane == 0) cache_error(a.err, kCacheBadPage);
    }
  }
#pragma unroll
  for (int i = 0; i < HPT; ++i) {
    const int head = h0 + i;
    if (head >= NH || (head >= a.nq && slot < 0)) break;  // the rest are keys and values too
    T* dst;
    if (head < a.nq)
      dst = static_cast<T*>(a.q_out) + t * a.ld_q + head * HD;
    else if (head < a.nq + a.nkv)
      dst = static_cast<T*>(a.k) + (slot * a.nkv + (head - a.nq)) * HD;
    else
      dst = static_cast<T*>(a.v) + (slot * a.nkv + (head - a.nq - a.nkv)) * HD;
    dst += lane * VEC;
    if (head < a.nq + a.nkv) {
      const float* gain = head < a.nq ? a.q_gain : a.k_gain;
      Two x[N], y[N];
      P::load(lo[i], x);
      P::load(hi[i], y);
      if (gain) {
        Two s2 = x[0] * x[0];
#pragma unroll
        for (int e = 1; e < N; ++e) s2 = fma2(x[e], x[e], s2);
#pragma unroll
        for (int e = 0; e < N; ++e) s2 = fma2(y[e], y[e], s2);
        float ss = both(s2).x + both(s2).y;
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
        const float r = rsqrtf(ss * (1.f / HD) + a.eps);
        const Two rr = two(r, r);
        Two gl[N], gh[N];
        load_pairs(gain + lane * VEC, gl);
        load_pairs(gain + HD / 2 + lane * VEC, gh);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          x[e] = x[e] * rr * gl[e];
          y[e] = y[e] * rr * gh[e];
        }
      }
      const Two minus = two(-1.f, -1.f);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const Two u = x[e], w = y[e];
        x[e] = fma2(w * minus, sn[e], u * cs[e]);
        y[e] = fma2(u, sn[e], w * cs[e]);
      }
      lo[i] = P::store(x);
      hi[i] = P::store(y);
    }
    *reinterpret_cast<uint4*>(dst) = lo[i];
    *reinterpret_cast<uint4*>(dst + HD / 2) = hi[i];
  }
}

template <typename T, int HD, int HPT>
cudaError_t append_n(cudaStream_t st, const CacheAppendArgs& a) {
  constexpr int LANES = HD / 2 / (16 / (int)sizeof(T));
  const int64_t threads = (int64_t)a.T * ((a.nq + 2 * a.nkv + HPT - 1) / HPT) * LANES;
  return launch_pdl(st, dim3((unsigned)((threads + kAppendThreads - 1) / kAppendThreads)), dim3(kAppendThreads), 0, 1,
                    cache_append_kernel<T, HD, HPT>, a);
}

template <typename T, int HD>
cudaError_t append_t(cudaStream_t st, const CacheAppendArgs& a, int sm_count) {
  constexpr int LANES = HD / 2 / (16 / (int)sizeof(T));
  const int64_t threads = (int64_t)a.T * (a.nq + 2 * a.nkv) * LANES;
  return threads <= (int64_t)sm_count * kAppendWide ? append_n<T, HD, 1>(st, a) : append_n<T, HD, kAppendHeads>(st, a);
}

bool misaligned(const void* p, uintptr_t align) { return p && (reinterpret_cast<uintptr_t>(p) & (align - 1)); }

sf_status fail(sf_cache* c, sf_status st, const char* fmt, ...) __attribute__((format(printf, 3, 4)));
sf_status fail(sf_cache* c, sf_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(c->last_error, sizeof(c->last_error), fmt, ap);
  va_end(ap);
  return st;
}

void free_cache(sf_cache* c) {
  if (!c) return;
  cudaFree(c->rope);
  cudaFree(c->scores);
  cudaFree(c->stats);
  cudaFree(c->parts);
  cudaFree(c->arrived);
  cudaFree(c->joins);
  if (c->err) cudaFreeHost(c->err);
  delete c;
}

// What every call checks after its arguments: the object's device is current
// and no earlier device check waits to be read.
sf_status check_object(sf_cache* c) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != c->device)
    return fail(c, SF_ERR_INVALID_ARG, "the object lives on device %d, the current one is %d", c->device, dev);
  const volatile unsigned* e = c->err;
  if (e[kCacheBadPage] || e[kCacheBadLength] || e[kCacheBadRow])
    return fail(c, SF_ERR_DEVICE_ASSERT, "device check fired:%s%s%s", e[kCacheBadPage] ? " page out of range" : "",
                e[kCacheBadLength] ? " length out of range" : "", e[kCacheBadRow] ? " row out of range" : "");
  return SF_OK;
}

sf_status check_table(sf_cache* c, const void* k, const void* v, int64_t n_pages, const int32_t* table, int S,
                      int cols, int64_t ld) {
  if (!k || !v || !table) return fail(c, SF_ERR_INVALID_ARG, "null pool or page table");
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(table, 4))
    return fail(c, SF_ERR_INVALID_ARG, "pools need 16-byte alignment, page tables 4-byte");
  if (S < 0 || cols < 1 || n_pages < 1 || (S > 1 && ld < cols))
    return fail(c, SF_ERR_INVALID_ARG, "S=%d table_cols=%d ld_table=%lld n_pages=%lld", S, cols, (long long)ld,
                (long long)n_pages);
  // slots are 32-bit in the kernels, the last value meaning none
  if (n_pages > 4294967294ll / c->s.page_size)
    return fail(c, SF_ERR_SHAPE, "n_pages=%lld pages of %d positions", (long long)n_pages, c->s.page_size);
  if (S > c->s.max_seqs) return fail(c, SF_ERR_SHAPE, "S=%d beyond the object's %d sequences", S, c->s.max_seqs);
  return SF_OK;
}

int64_t scores_ld(const sf_cache_shapes& s) { return ((int64_t)s.max_len + 3) / 4 * 4; }

bool bad_row(const sf_cache* c, const void* p, int64_t ld, int64_t width, int rows) {
  const int es = c->s.dtype == SF_BF16 ? 2 : 4;
  return !p || misaligned(p, 16) || (rows > 1 && (ld < width || ld * es % 16 != 0));
}

// Do two arrays of `rows` rows, of wa and wb bytes, lda and ldb bytes apart,
// share memory?  Rows the same distance apart (columns of one wide array) are
// compared column by column, others by the arrays' ends.
bool rows_overlap(const void* a, int64_t lda, int64_t wa, const void* b, int64_t ldb, int64_t wb, int rows) {
  const int64_t pa = (int64_t)reinterpret_cast<uintptr_t>(a), pb = (int64_t)reinterpret_cast<uintptr_t>(b);
  if (pa + (rows - 1) * lda + wa <= pb || pb + (rows - 1) * ldb + wb <= pa) return false;
  if (rows == 1 || lda != ldb) return true;
  const int64_t d = ((pb - pa) % lda + lda) % lda;
  return d < wa || d + wb > lda;
}

// Two arrays of n elements of 4 bytes that are neither the same nor apart.
bool half_the_same(const void* a, const void* b, int64_t n) {
  return a && b && a != b && rows_overlap(a, 0, 4 * n, b, 0, 4 * n, 1);
}

PageTable page_table(const sf_cache* c, const int32_t* table, int cols, int64_t ld, int64_t n_pages) {
  return make_page_table(table, ld, cols, c->s.page_size, n_pages);
}

sf_status launched(sf_cache* c, cudaError_t e) {
  if (e == cudaSuccess) return SF_OK;
  cudaGetLastError();
  return fail(c, SF_ERR_CUDA, "launch failed: %s", cudaGetErrorString(e));
}

}  // namespace

cudaError_t launch_cache_append(cudaStream_t st, const CacheAppendArgs& a, int bf16, int sm_count) {
  if (bf16) return a.hd == 128 ? append_t<__nv_bfloat16, 128>(st, a, sm_count) : append_t<__nv_bfloat16, 64>(st, a, sm_count);
  return a.hd == 128 ? append_t<float, 128>(st, a, sm_count) : append_t<float, 64>(st, a, sm_count);
}

}  // namespace sf

using namespace sf;

extern "C" {

sf_status sf_cache_create(const sf_cache_shapes* shapes, sf_cache** out) {
  if (!out) return SF_ERR_INVALID_ARG;
  *out = nullptr;
  if (!shapes) return SF_ERR_INVALID_ARG;
  const sf_cache_shapes s = *shapes;
  if (s.n_q_heads < 1 || s.n_kv_heads < 1 || s.head_dim < 1 || s.page_size < 1 || s.max_seqs < 1 || s.max_len < 1 ||
      s.max_pos < 1 || !(s.rms_eps >= 0.f) || !std::isfinite(s.rms_eps) || !(s.rope_theta > 0.f) ||
      !std::isfinite(s.rope_theta) || (s.dtype != SF_F32 && s.dtype != SF_BF16))
    return SF_ERR_INVALID_ARG;
  if ((s.head_dim != 64 && s.head_dim != 128) || s.n_q_heads % s.n_kv_heads != 0 || s.n_q_heads > 1024 ||
      s.page_size > kMaxPageSize || s.max_seqs > 4096 || s.max_len > kMaxLen || s.max_pos > 4194304)
    return SF_ERR_UNSUPPORTED;
  sf_cache* c = new (std::nothrow) sf_cache();
  if (!c) return SF_ERR_OOM;
  c->s = s;
  cudaError_t e = cudaGetDevice(&c->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&c->sm_count, cudaDevAttrMultiProcessorCount, c->device);
  const int blocks = cache_attend_blocks(c->sm_count);
  if (e == cudaSuccess) e = cudaMalloc(&c->rope, (size_t)s.max_pos * s.head_dim * sizeof(float));
  if (e == cudaSuccess && s.track_weights)
    e = cudaMalloc(&c->scores, (size_t)s.max_seqs * s.n_q_heads * scores_ld(s) * sizeof(float));
  if (e == cudaSuccess && s.track_weights)
    e = cudaMalloc(&c->stats, (size_t)s.max_seqs * s.n_q_heads * sizeof(float2));
  if (e == cudaSuccess) e = cudaMalloc(&c->parts, (size_t)(blocks * cache_attend_part_floats(s)) * sizeof(float));
  if (e == cudaSuccess) e = cudaMalloc(&c->joins, (size_t)blocks * sizeof(CacheJoin));
  if (e == cudaSuccess) e = cudaMalloc(&c->arrived, (size_t)blocks * sizeof(unsigned));
  if (e == cudaSuccess) e = cudaMemset(c->arrived, 0, (size_t)blocks * sizeof(unsigned));
  if (e == cudaSuccess) e = prepare_cache_attend();
  if (e == cudaSuccess) e = prepare_cache_evict();
  if (e == cudaSuccess) e = cudaHostAlloc(&c->err, kCacheErrWords * sizeof(unsigned), cudaHostAllocMapped);
  if (e == cudaSuccess) e = cudaHostGetDevicePointer(&c->err_dev, c->err, 0);
  if (e == cudaSuccess) {
    for (int i = 0; i < kCacheErrWords; ++i) c->err[i] = 0;
    rope_table_kernel<<<(s.max_pos + kRopeRun - 1) / kRopeRun, s.head_dim / 2>>>(c->rope, s.max_pos, s.head_dim / 2,
                                                                                 (double)s.rope_theta);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    free_cache(c);
    cudaGetLastError();
    return e == cudaErrorMemoryAllocation ? SF_ERR_OOM : SF_ERR_CUDA;
  }
  *out = c;
  return SF_OK;
}

sf_status sf_cache_append(sf_cache* c, void* stream, const void* qkv, int64_t ld_qkv, int T, const float* q_gain,
                          const float* k_gain, const int32_t* index, const int32_t* pos, const int32_t* seq,
                          const int32_t* page_table_, int S, int table_cols, int64_t ld_table, void* k_pages,
                          void* v_pages, int64_t n_pages, void* q_out, int64_t ld_q) {
  if (!c) return SF_ERR_INVALID_ARG;
  const sf_cache_shapes& s = c->s;
  sf_status st = SF_OK;
  if (T == 0) return check_object(c);  // nothing to do, whatever the pointers
  if ((st = check_table(c, k_pages, v_pages, n_pages, page_table_, S, table_cols, ld_table)) != SF_OK) return st;
  if (k_pages == v_pages) return fail(c, SF_ERR_INVALID_ARG, "one pool for keys and values");
  if (T < 0 || !index || misaligned(index, 4) || misaligned(pos, 4) || misaligned(seq, 4) || misaligned(q_gain, 16) ||
      misaligned(k_gain, 16))
    return fail(c, SF_ERR_INVALID_ARG, "T=%d, null index, or index/pos/seq/gain misaligned", T);
  const int64_t wq = (int64_t)s.n_q_heads * s.head_dim, w = wq + 2 * (int64_t)s.n_kv_heads * s.head_dim;
  if (bad_row(c, qkv, ld_qkv, w, T) || bad_row(c, q_out, ld_q, wq, T))
    return fail(c, SF_ERR_INVALID_ARG, "qkv/q_out null, misaligned, or rows closer than their width");
  if (T > 1048576 || (!seq && T > S)) return fail(c, SF_ERR_SHAPE, "T=%d rows for S=%d sequences", T, S);
  const int es = s.dtype == SF_BF16 ? 2 : 4;
  if ((q_out != qkv || (T > 1 && ld_q != ld_qkv)) && rows_overlap(qkv, ld_qkv * es, w * es, q_out, ld_q * es, wq * es, T))
    return fail(c, SF_ERR_INVALID_ARG, "q_out overlaps qkv and is not its query part");
  if ((st = check_object(c)) != SF_OK) return st;
  CacheAppendArgs a{};
  a.qkv = qkv;
  a.ld_qkv = ld_qkv;
  a.q_out = q_out;
  a.ld_q = ld_q;
  a.q_gain = q_gain;
  a.k_gain = k_gain;
  a.index = index;
  a.pos = pos;
  a.seq = seq;
  a.table = page_table(c, page_table_, table_cols, ld_table, n_pages);
  a.k = k_pages;
  a.v = v_pages;
  a.rope = c->rope;
  a.T = T;
  a.S = S;
  a.nq = s.n_q_heads;
  a.nkv = s.n_kv_heads;
  a.hd = s.head_dim;
  a.max_pos = s.max_pos;
  a.limit = length_limit(s.max_len, table_cols, s.page_size);
  a.eps = s.rms_eps;
  a.err = c->err_dev;
  return launched(c, launch_cache_append((cudaStream_t)stream, a, s.dtype == SF_BF16, c->sm_count));
}

sf_status sf_cache_attend(sf_cache* c, void* stream, const void* q, int64_t ld_q, const void* k_pages,
                          const void* v_pages, int64_t n_pages, const int32_t* page_table_, int S, int table_cols,
                          int64_t ld_table, const int32_t* lens, float scale, void* out, int64_t ld_out,
                          const float* weights_in, float* weights_out, int64_t ld_w) {
  if (!c) return SF_ERR_INVALID_ARG;
  const sf_cache_shapes& s = c->s;
  sf_status st = SF_OK;
  if (S == 0) return check_object(c);  // nothing to do, whatever the pointers
  if ((st = check_table(c, k_pages, v_pages, n_pages, page_table_, S, table_cols, ld_table)) != SF_OK) return st;
  if (!lens || misaligned(lens, 4) || misaligned(weights_in, 4) || misaligned(weights_out, 4))
    return fail(c, SF_ERR_INVALID_ARG, "null lens, or lens/weights misaligned");
  const int64_t wq = (int64_t)s.n_q_heads * s.head_dim;
  if (bad_row(c, q, ld_q, wq, S) || bad_row(c, out, ld_out, wq, S))
    return fail(c, SF_ERR_INVALID_ARG, "q/out null, misaligned, or rows closer than their width");
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!std::isfinite(scale_log2))
    return fail(c, SF_ERR_INVALID_ARG, "scale must be finite, and so must scale * log2(e)");
  if (weights_in && !weights_out) return fail(c, SF_ERR_INVALID_ARG, "weights_in without weights_out");
  if (weights_out && !s.track_weights)
    return fail(c, SF_ERR_INVALID_ARG, "the object was created without track_weights");
  const int64_t limit = length_limit(s.max_len, table_cols, s.page_size);
  if (weights_out && ld_w < limit)
    return fail(c, SF_ERR_SHAPE, "ld_w=%lld below the %lld positions of a sequence", (long long)ld_w,
                (long long)limit);
  const int es = s.dtype == SF_BF16 ? 2 : 4;
  if (rows_overlap(q, ld_q * es, wq * es, out, ld_out * es, wq * es, S))
    return fail(c, SF_ERR_INVALID_ARG, "out overlaps q");
  if (half_the_same(weights_in, weights_out, (int64_t)S * s.n_kv_heads * ld_w))
    return fail(c, SF_ERR_INVALID_ARG, "weights_out overlaps weights_in without being the same");
  if ((st = check_object(c)) != SF_OK) return st;
  CacheAttendArgs a{};
  a.q = q;
  a.ld_q = ld_q;
  a.k = k_pages;
  a.v = v_pages;
  a.table = page_table(c, page_table_, table_cols, ld_table, n_pages);
  a.lens = lens;
  a.S = S;
  a.nq = s.n_q_heads;
  a.nkv = s.n_kv_heads;
  a.hd = s.head_dim;
  a.limit = limit;
  a.scale_log2 = scale_log2;
  a.out = out;
  a.ld_out = ld_out;
  a.w_in = weights_in;
  a.w_out = weights_out;
  a.ld_w = ld_w;
  a.scores = c->scores;
  a.ld_scores = scores_ld(s);
  a.stats = c->stats;
  a.parts = c->parts;
  a.arrived = c->arrived;
  a.joins = c->joins;
  a.err = c->err_dev;
  return launched(c, launch_cache_attend((cudaStream_t)stream, a, s.dtype == SF_BF16, c->sm_count));
}

sf_status sf_cache_evict(sf_cache* c, void* stream, const void* k_pages, const void* v_pages, int64_t n_pages,
                         const int32_t* page_table_, int S, int table_cols, int64_t ld_table, const int32_t* lens,
                         const float* weights, int64_t ld_w, int budget, int n_first, int n_recent, void* k_out,
                         void* v_out, int64_t n_pages_out, const int32_t* table_out, int table_out_cols,
                         int64_t ld_table_out, float* weights_out, int32_t* lens_out, int32_t* kept) {
  if (!c) return SF_ERR_INVALID_ARG;
  const sf_cache_shapes& s = c->s;
  sf_status st = SF_OK;
  if (S == 0) return check_object(c);  // nothing to do, whatever the pointers
  if ((st = check_table(c, k_pages, v_pages, n_pages, page_table_, S, table_cols, ld_table)) != SF_OK) return st;
  if ((st = check_table(c, k_out, v_out, n_pages_out, table_out, S, table_out_cols, ld_table_out)) != SF_OK) return st;
  if (!lens || !weights || !weights_out || !lens_out || !kept)
    return fail(c, SF_ERR_INVALID_ARG, "null lens/weights/weights_out/lens_out/kept");
  if (misaligned(lens, 4) || misaligned(weights, 4) || misaligned(weights_out, 4) || misaligned(lens_out, 4) ||
      misaligned(kept, 4))
    return fail(c, SF_ERR_INVALID_ARG, "lens/weights/lens_out/kept need 4-byte alignment");
  if (budget < 1 || n_first < 0 || n_recent < 0 || (int64_t)n_first + n_recent > budget)
    return fail(c, SF_ERR_INVALID_ARG, "budget=%d n_first=%d n_recent=%d", budget, n_first, n_recent);
  const int same = (k_out == k_pages) + (v_out == v_pages) + (table_out == page_table_);
  if ((same != 0 && same != 3) || (same == 3 && (ld_table_out != ld_table || n_pages_out != n_pages)) ||
      k_out == v_out || k_out == v_pages || v_out == k_pages)
    return fail(c, SF_ERR_INVALID_ARG, "output pools and table are the input's in part only");
  const int64_t limit = length_limit(s.max_len, table_cols, s.page_size);
  if (ld_w < limit)
    return fail(c, SF_ERR_SHAPE, "ld_w=%lld below the %lld positions of a sequence", (long long)ld_w,
                (long long)limit);
  if (budget > s.max_len || budget > (int64_t)table_out_cols * s.page_size)
    return fail(c, SF_ERR_SHAPE, "budget=%d beyond max_len=%d or the output table", budget, s.max_len);
  if (half_the_same(weights, weights_out, (int64_t)S * s.n_kv_heads * ld_w) || half_the_same(lens, lens_out, S))
    return fail(c, SF_ERR_INVALID_ARG, "weights_out or lens_out overlaps its input without being the same");
  if ((st = check_object(c)) != SF_OK) return st;
  CacheEvictArgs a{};
  a.k = k_pages;
  a.v = v_pages;
  a.table = page_table(c, page_table_, table_cols, ld_table, n_pages);
  a.k_out = k_out;
  a.v_out = v_out;
  a.table_out = page_table(c, table_out, table_out_cols, ld_table_out, n_pages_out);
  a.lens = lens;
  a.w = weights;
  a.w_out = weights_out;
  a.ld_w = ld_w;
  a.lens_out = lens_out;
  a.kept = kept;
  a.S = S;
  a.nkv = s.n_kv_heads;
  a.hd = s.head_dim;
  a.budget = budget;
  a.n_first = n_first;
  a.n_recent = n_recent;
  a.limit = limit;
  a.in_place = same == 3;
  a.err = c->err_dev;
  return launched(c, launch_cache_evict((cudaStream_t)stream, a, s.dtype == SF_BF16, c->sm_count));
}

sf_status sf_cache_sync_status(sf_cache* c, void* stream) {
  if (!c) return SF_ERR_INVALID_ARG;
  cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e != cudaSuccess) return fail(c, SF_ERR_CUDA, "%s", cudaGetErrorString(e));
  sf_status st = check_object(c);
  if (st == SF_ERR_DEVICE_ASSERT)
    for (int i = 0; i < kCacheErrWords; ++i) c->err[i] = 0;
  return st;
}

const char* sf_cache_last_error(const sf_cache* c) { return c ? c->last_error : ""; }

sf_status sf_cache_destroy(sf_cache* c) {
  if (!c) return SF_ERR_INVALID_ARG;
  cudaError_t e = cudaDeviceSynchronize();
  free_cache(c);
  return e == cudaSuccess ? SF_OK : SF_ERR_CUDA;
}

}  // extern "C"
