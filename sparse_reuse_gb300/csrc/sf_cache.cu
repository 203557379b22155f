// Paged-cache operators: the object, argument checks and the C ABI
// (specfold_cache.h), the rotary table and the append kernel.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "sf_cache.h"
#include "sf_pairs.cuh"
#include "sf_rotary.cuh"

namespace sf {
namespace {

// Rotary table [max_pos][cos half | sin half] in double, rounded once: far
// positions (10^5 radians and more) lose the angle in fp32.  A thread takes one
// frequency over kRopeRun positions: sine and cosine of the first angle and of
// the step, then the addition theorem (double rounding grows by about 2^-53 a
// step, far below fp32's half step); FP64 rates make a sine per entry slow.
constexpr int kRopeRun = 64;

// The frequencies are theta^(-j / half), or the caller's; `magnitude` scales
// every entry.
struct RopeFreqs {
  double f[64];
};
__global__ void rope_table_kernel(float* out, int max_pos, int half, double theta, bool given,
                                  const __grid_constant__ RopeFreqs freqs, double magnitude) {
  const int j = threadIdx.x, p0 = blockIdx.x * kRopeRun, p1 = min(p0 + kRopeRun, max_pos);
  const double freq = given ? freqs.f[j] : pow(theta, -(double)j / half);
  double s, c, ds, dc;
  sincos((double)p0 * freq, &s, &c);
  sincos(freq, &ds, &dc);
  for (int p = p0; p < p1; ++p) {
    out[(int64_t)p * 2 * half + j] = (float)(c * magnitude);
    out[(int64_t)p * 2 * half + half + j] = (float)(s * magnitude);
    const double t = c * dc - s * ds;
    s = s * dc + c * ds;
    c = t;
  }
}

// 8,188 rows of 40/8 heads x 128 bf16: 43.6 us so (5.4 TB/s in and out); 128 threads 46.6, three or four heads a
// group 51 and 68, the compiler's own 72 registers instead of 56 (18 blocks an SM) 45.3, 48 registers 51.6.
constexpr int kAppendThreads = 64;
constexpr int kAppendHeads = 2;
constexpr int kAppendBlocks = 18;
constexpr int kAppendBlocksForms = 16;  // of the other forms, which need more registers
// (lane, head) pairs per SM from which a group takes several heads.  40/8 heads x 128 bf16, 512 rows (1,509 pairs):
// 4.2 us with one, 4.9 with two; 1,024 rows: 8.6 and 7.8; 4,096 rows: 31.4 and 24.2.
constexpr int kAppendWide = 2048;

// Which two 16-byte pieces of a head a lane holds: both members of its rotation
// pairs are in its registers.
//   kHalves      the whole head in halves: piece `lane` of the lower half and
//                the same of the upper
//   kPart        the first rotary.dim dimensions in halves: the lanes of these
//                likewise, the others two neighbouring pieces as they are
//   kNeighbours  pairs of neighbours lie inside a piece: pieces as for kHalves,
//                of which those within the first rotary.dim dimensions turn
enum Form { kHalves, kPart, kNeighbours };

// Norm, rotation and store of HPT heads of one row by a group of lanes, two
// pieces a lane; the norm needs log2(lanes) shuffles.  Bytes bound it (each row
// in and out once); HPT heads keep 2 HPT loads in flight and share the row's
// angles and its page lookup.
template <typename T, int HD, int HPT, Form FORM>
__global__ void __launch_bounds__(kAppendThreads, FORM == kHalves ? kAppendBlocks : kAppendBlocksForms) cache_append_kernel(const __grid_constant__ CacheAppendArgs a) {
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
  const int turned = FORM == kPart ? a.rotary.dim / (2 * VEC) : LANES;  // lanes of the rotated part
  const bool pairs = FORM != kPart || lane < turned;
  const int c0 = pairs ? lane : 2 * lane, c1 = pairs ? lane + turned : 2 * lane + 1;
  // the row itself first: it waits for nothing, its place and angles arrive meanwhile
  const T* src = static_cast<const T*>(a.qkv) + t * a.ld_qkv + h0 * HD;
  uint4 lo[HPT], hi[HPT];
#pragma unroll
  for (int i = 0; i < HPT; ++i)
    if (h0 + i < NH) {
      lo[i] = *reinterpret_cast<const uint4*>(src + i * HD + c0 * VEC);
      hi[i] = *reinterpret_cast<const uint4*>(src + i * HD + c1 * VEC);
    }
  const int idx = a.index[t];
  const int pos = a.pos ? a.pos[t] : idx;
  if (pos < 0) return;
  if (pos >= a.max_pos) {
    if (lane == 0) cache_error(a.err, kCacheBadRow);
    return;
  }
  const int dim = FORM == kHalves ? HD : a.rotary.dim;
  Angles<T, FORM == kNeighbours> angles;
  if (h0 < a.nq + a.nkv && pairs) angles.load(a.rope + (int64_t)pos * dim, dim / 2, c0, c1);
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
        load_pairs(gain + c0 * VEC, gl);
        load_pairs(gain + c1 * VEC, gh);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          x[e] = x[e] * rr * gl[e];
          y[e] = y[e] * rr * gh[e];
        }
      }
      if (pairs) angles.turn(x, y);
      lo[i] = P::store(x);
      hi[i] = P::store(y);
    }
    *reinterpret_cast<uint4*>(dst + c0 * VEC) = lo[i];
    *reinterpret_cast<uint4*>(dst + c1 * VEC) = hi[i];
  }
}

template <typename T, int HD, int HPT, Form FORM>
cudaError_t append_n(cudaStream_t st, const CacheAppendArgs& a) {
  constexpr int LANES = HD / 2 / (16 / (int)sizeof(T));
  const int64_t threads = (int64_t)a.T * ((a.nq + 2 * a.nkv + HPT - 1) / HPT) * LANES;
  return launch_pdl(st, dim3((unsigned)((threads + kAppendThreads - 1) / kAppendThreads)), dim3(kAppendThreads), 0, 1,
                    cache_append_kernel<T, HD, HPT, FORM>, a);
}

template <typename T, int HD, Form FORM>
cudaError_t append_f(cudaStream_t st, const CacheAppendArgs& a, int sm_count) {
  constexpr int LANES = HD / 2 / (16 / (int)sizeof(T));
  const int64_t threads = (int64_t)a.T * (a.nq + 2 * a.nkv) * LANES;
  return threads <= (int64_t)sm_count * kAppendWide ? append_n<T, HD, 1, FORM>(st, a)
                                                       : append_n<T, HD, kAppendHeads, FORM>(st, a);
}

template <typename T, int HD>
cudaError_t append_t(cudaStream_t st, const CacheAppendArgs& a, int sm_count) {
  if (a.rotary.neighbours) return append_f<T, HD, kNeighbours>(st, a, sm_count);
  return a.rotary.dim == HD ? append_f<T, HD, kHalves>(st, a, sm_count) : append_f<T, HD, kPart>(st, a, sm_count);
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
  cudaFree(c->row_parts);
  cudaFree(c->row_ml);
  cudaFree(c->row_joins);
  cudaFree(c->tail_o);
  cudaFree(c->tail_ml);
  cudaFree(c->whole_o);
  cudaFree(c->whole_ml);
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
  if (e[kCacheBadPage] || e[kCacheBadLength] || e[kCacheBadRow] || e[kCacheStall])
    return fail(c, SF_ERR_DEVICE_ASSERT, "device check fired:%s%s%s%s", e[kCacheBadPage] ? " page out of range" : "",
                e[kCacheBadLength] ? " length out of range" : "", e[kCacheBadRow] ? " row out of range" : "",
                e[kCacheStall] ? " a wait inside a kernel ran out" : "");
  return SF_OK;
}

sf_status check_table(sf_cache* c, const void* k, const void* v, int64_t n_pages, const int32_t* table, int S,
                      int cols, int64_t ld, int most) {
  if (!k || !v || !table) return fail(c, SF_ERR_INVALID_ARG, "null pool or page table");
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(table, 4))
    return fail(c, SF_ERR_INVALID_ARG, "pools need 16-byte alignment, page tables 4-byte");
  if (S < 0 || cols < 1 || n_pages < 1 || (S > 1 && ld < cols))
    return fail(c, SF_ERR_INVALID_ARG, "S=%d table_cols=%d ld_table=%lld n_pages=%lld", S, cols, (long long)ld,
                (long long)n_pages);
  // slots are 32-bit in the kernels, the last value meaning none
  if (n_pages > 4294967294ll / c->s.page_size)
    return fail(c, SF_ERR_SHAPE, "n_pages=%lld pages of %d positions", (long long)n_pages, c->s.page_size);
  if (S > most) return fail(c, SF_ERR_SHAPE, "S=%d beyond the object's %d sequences", S, most);
  return SF_OK;
}

sf_status check_table(sf_cache* c, const void* k, const void* v, int64_t n_pages, const int32_t* table, int S,
                      int cols, int64_t ld) {
  return check_table(c, k, v, n_pages, table, S, cols, ld, c->s.max_seqs);
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

constexpr float kLog2e = 1.4426950408889634f;

// What attend_rows and attend_shared check of their rows.
sf_status check_rows(sf_cache* c, const void* q, int64_t ld_q, int T, float scale, const void* out, int64_t ld_out,
                     const float* lse) {
  const sf_cache_shapes& s = c->s;
  if (c->o.max_rows < 1) return fail(c, SF_ERR_INVALID_ARG, "the object was created without max_rows");
  if (T < 0) return fail(c, SF_ERR_INVALID_ARG, "%d rows", T);
  if (T > c->o.max_rows) return fail(c, SF_ERR_SHAPE, "%d rows beyond the object's %d", T, c->o.max_rows);
  const int64_t wq = (int64_t)s.n_q_heads * s.head_dim, es = s.dtype == SF_BF16 ? 2 : 4, w = wq * es;
  const int64_t wl = 4 * (int64_t)s.n_q_heads;
  if (bad_row(c, q, ld_q, wq, T) || bad_row(c, out, ld_out, wq, T))
    return fail(c, SF_ERR_INVALID_ARG, "q/out null, misaligned, or rows closer than their width");
  if (misaligned(lse, 4)) return fail(c, SF_ERR_INVALID_ARG, "lse misaligned");
  if (!std::isfinite(scale * kLog2e))
    return fail(c, SF_ERR_INVALID_ARG, "scale must be finite, and so must scale * log2(e)");
  if (rows_overlap(q, ld_q * es, w, out, ld_out * es, w, T)) return fail(c, SF_ERR_INVALID_ARG, "out overlaps q");
  if (lse && (rows_overlap(q, ld_q * es, w, lse, wl, wl, T) || rows_overlap(out, ld_out * es, w, lse, wl, wl, T)))
    return fail(c, SF_ERR_INVALID_ARG, "lse overlaps q or out");
  return SF_OK;
}

// TMA takes the pool's positions as 31-bit row numbers (and one that is outside).
sf_status check_gather(sf_cache* c, int64_t n_pages) {
  if (c->s.dtype == SF_BF16 && n_pages > 2147483646ll / c->s.page_size)
    return fail(c, SF_ERR_SHAPE, "n_pages=%lld pages of %d positions", (long long)n_pages, c->s.page_size);
  return SF_OK;
}

CacheRowsArgs rows_args(const sf_cache* c, const void* q, int64_t ld_q, int T, float scale, void* out, int64_t ld_out,
                        float* lse) {
  CacheRowsArgs a{};
  a.q = q;
  a.ld_q = ld_q;
  a.T = T;
  a.nq = c->s.n_q_heads;
  a.nkv = c->s.n_kv_heads;
  a.group = a.nq / a.nkv;
  a.scale_log2 = scale * kLog2e;
  a.out = out;
  a.ld_out = ld_out;
  a.lse = lse;
  a.parts = c->row_parts;
  a.part_ml = c->row_ml;
  a.joins = c->row_joins;
  a.ctas = cache_rows_ctas(c->sm_count, c->s.dtype == SF_BF16);
  a.wait_ns = c->stall == kStallNone ? 2000000000u : 50000000u;
  a.stall = c->stall;
  a.err = c->err_dev;
  return a;
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
  return sf_cache_create_with(shapes, nullptr, out);
}

sf_status sf_cache_create_with(const sf_cache_shapes* shapes, const sf_cache_options* options, sf_cache** out) {
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
  sf_cache_options o = options ? *options : sf_cache_options{};
  if (o.rotary_dim == 0) o.rotary_dim = s.head_dim;
  if (o.rotary_magnitude == 0.) o.rotary_magnitude = 1.;
  if (o.max_rows < 0 || o.rotary_dim < 0 || !(o.rotary_magnitude > 0.) || !std::isfinite((float)o.rotary_magnitude) ||
      !std::isfinite((float)(1. / o.rotary_magnitude)) ||
      (o.rotary_layout != SF_ROTARY_HALVES && o.rotary_layout != SF_ROTARY_NEIGHBOURS))
    return SF_ERR_INVALID_ARG;
  if (o.max_rows > kMaxCallRows || o.rotary_dim % 16 != 0 || o.rotary_dim > s.head_dim) return SF_ERR_UNSUPPORTED;
  const int half = o.rotary_dim / 2;
  RopeFreqs freqs{};
  const bool given = o.inv_freq != nullptr;
  for (int j = 0; given && j < half; ++j) {
    freqs.f[j] = o.inv_freq[j];
    if (!std::isfinite(freqs.f[j])) return SF_ERR_INVALID_ARG;
  }
  o.inv_freq = nullptr;  // the caller's array is not kept
  sf_cache* c = new (std::nothrow) sf_cache();
  if (!c) return SF_ERR_OOM;
  c->s = s;
  c->o = o;
  c->rotary = Rotary{o.rotary_dim, o.rotary_layout == SF_ROTARY_NEIGHBOURS};
  cudaError_t e = cudaGetDevice(&c->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&c->sm_count, cudaDevAttrMultiProcessorCount, c->device);
  const int blocks = cache_attend_blocks(c->sm_count);
  if (e == cudaSuccess) e = cudaMalloc(&c->rope, (size_t)s.max_pos * o.rotary_dim * sizeof(float));
  if (e == cudaSuccess && s.track_weights)
    e = cudaMalloc(&c->scores, (size_t)s.max_seqs * s.n_q_heads * scores_ld(s) * sizeof(float));
  if (e == cudaSuccess && s.track_weights)
    e = cudaMalloc(&c->stats, (size_t)s.max_seqs * s.n_q_heads * sizeof(float2));
  if (e == cudaSuccess) e = cudaMalloc(&c->parts, (size_t)(blocks * cache_attend_part_floats(s)) * sizeof(float));
  if (e == cudaSuccess) e = cudaMalloc(&c->joins, (size_t)blocks * sizeof(CacheJoin));
  if (e == cudaSuccess) e = cudaMalloc(&c->arrived, (size_t)blocks * sizeof(unsigned));
  if (e == cudaSuccess) e = cudaMemset(c->arrived, 0, (size_t)blocks * sizeof(unsigned));
  if (o.max_rows > 0) {
    const size_t ctas = (size_t)cache_rows_ctas(c->sm_count, s.dtype == SF_BF16), rows = 2 * ctas * cache_rows_slot_rows(s.dtype == SF_BF16);
    const size_t tails = (size_t)(o.max_rows < s.max_seqs ? o.max_rows : s.max_seqs) * s.n_q_heads;
    if (e == cudaSuccess) e = cudaMalloc(&c->row_parts, rows * s.head_dim * sizeof(float));
    if (e == cudaSuccess) e = cudaMalloc(&c->row_ml, rows * sizeof(float2));
    if (e == cudaSuccess) e = cudaMalloc(&c->row_joins, ctas * sizeof(RowsJoin));
    if (e == cudaSuccess) e = cudaMalloc(&c->tail_o, tails * s.head_dim * sizeof(float));
    if (e == cudaSuccess) e = cudaMalloc(&c->tail_ml, tails * sizeof(float2));
    if (e == cudaSuccess) e = cudaMalloc(&c->whole_o, tails * s.head_dim * sizeof(float));
    if (e == cudaSuccess) e = cudaMalloc(&c->whole_ml, tails * sizeof(float2));
    if (e == cudaSuccess) e = prepare_cache_rows();
  }
  if (e == cudaSuccess) e = prepare_cache_attend();
  if (e == cudaSuccess) e = prepare_cache_evict();
  if (e == cudaSuccess) e = cudaHostAlloc(&c->err, kCacheErrWords * sizeof(unsigned), cudaHostAllocMapped);
  if (e == cudaSuccess) e = cudaHostGetDevicePointer(&c->err_dev, c->err, 0);
  if (e == cudaSuccess) {
    for (int i = 0; i < kCacheErrWords; ++i) c->err[i] = 0;
    rope_table_kernel<<<(s.max_pos + kRopeRun - 1) / kRopeRun, half>>>(c->rope, s.max_pos, half, (double)s.rope_theta,
                                                                       given, freqs, o.rotary_magnitude);
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
  if (T > kMaxCallRows || (!seq && T > S)) return fail(c, SF_ERR_SHAPE, "T=%d rows for S=%d sequences", T, S);
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
  a.rotary = c->rotary;
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

sf_status sf_cache_reposition(sf_cache* c, void* stream, void* k_pages, int64_t n_pages, const int32_t* page_table_, int S,
                              int table_cols, int64_t ld_table, const int32_t* lens, const int32_t* pos_from,
                              const int32_t* pos_to, int64_t ld_pos) {
  if (!c) return SF_ERR_INVALID_ARG;
  const sf_cache_shapes& s = c->s;
  sf_status st = SF_OK;
  if (S == 0) return check_object(c);  // nothing to do, whatever the pointers
  if ((st = check_table(c, k_pages, k_pages, n_pages, page_table_, S, table_cols, ld_table)) != SF_OK) return st;
  if (!lens || !pos_from || misaligned(lens, 4) || misaligned(pos_from, 4) || misaligned(pos_to, 4))
    return fail(c, SF_ERR_INVALID_ARG, "null lens or pos_from, or lens/pos_from/pos_to misaligned");
  if (ld_pos < 1) return fail(c, SF_ERR_INVALID_ARG, "ld_pos=%lld", (long long)ld_pos);
  if ((st = check_object(c)) != SF_OK) return st;
  CacheTurnArgs a{};
  a.k = k_pages;
  a.table = page_table(c, page_table_, table_cols, ld_table, n_pages);
  a.lens = lens;
  a.from = pos_from;
  a.to = pos_to;
  a.ld_pos = ld_pos;
  a.rope = c->rope;
  a.rotary = c->rotary;
  a.unscale = (float)(1. / c->o.rotary_magnitude);
  a.S = S;
  a.nkv = s.n_kv_heads;
  a.hd = s.head_dim;
  a.max_pos = s.max_pos;
  a.limit = length_limit(s.max_len, table_cols, s.page_size);
  if (ld_pos < a.limit) a.limit = ld_pos;
  a.err = c->err_dev;
  return launched(c, launch_cache_turn((cudaStream_t)stream, a, s.dtype == SF_BF16, c->sm_count));
}

sf_status sf_cache_attend_rows(sf_cache* c, void* stream, const void* q, int64_t ld_q, int T, const void* k_pages,
                               const void* v_pages, int64_t n_pages, const int32_t* page_table_, int S, int table_cols,
                               int64_t ld_table, const int32_t* lens, const int32_t* starts, float scale, void* out,
                               int64_t ld_out, float* lse) {
  if (!c) return SF_ERR_INVALID_ARG;
  sf_status st = SF_OK;
  if (S == 0 || T == 0) return check_object(c);  // nothing to do, whatever the pointers
  if ((st = check_rows(c, q, ld_q, T, scale, out, ld_out, lse)) != SF_OK) return st;
  if ((st = check_table(c, k_pages, v_pages, n_pages, page_table_, S, table_cols, ld_table)) != SF_OK) return st;
  if ((st = check_gather(c, n_pages)) != SF_OK) return st;
  if (!lens || !starts || misaligned(lens, 4) || misaligned(starts, 4))
    return fail(c, SF_ERR_INVALID_ARG, "lens or starts null or misaligned");
  if ((st = check_object(c)) != SF_OK) return st;
  CacheRowsArgs a = rows_args(c, q, ld_q, T, scale, out, ld_out, lse);
  a.k = k_pages;
  a.v = v_pages;
  a.table = page_table(c, page_table_, table_cols, ld_table, n_pages);
  a.lens = lens;
  a.starts = starts;
  a.S = S;
  a.limit = length_limit(c->s.max_len, table_cols, c->s.page_size);
  return launched(c, launch_cache_rows((cudaStream_t)stream, a, c->s.dtype == SF_BF16, c->s.head_dim, c->sm_count));
}

sf_status sf_cache_attend_shared(sf_cache* c, void* stream, const void* q, int64_t ld_q, const void* k_pages,
                                 const void* v_pages, int64_t n_pages, const int32_t* page_table_, int S,
                                 int table_cols, int64_t ld_table, const int32_t* lens, const int32_t* prefix_table,
                                 int G, int prefix_cols, int64_t ld_prefix, const int32_t* prefix_lens,
                                 const int32_t* starts, float scale, void* out, int64_t ld_out, float* lse) {
  if (!c) return SF_ERR_INVALID_ARG;
  const sf_cache_shapes& s = c->s;
  sf_status st = SF_OK;
  if (S == 0) return check_object(c);  // nothing to do, whatever the pointers
  if ((st = check_rows(c, q, ld_q, S, scale, out, ld_out, lse)) != SF_OK) return st;
  if ((st = check_table(c, k_pages, v_pages, n_pages, page_table_, S, table_cols, ld_table)) != SF_OK) return st;
  if (G < 1) return fail(c, SF_ERR_INVALID_ARG, "G=%d groups", G);
  if (G > kMaxGroups) return fail(c, SF_ERR_SHAPE, "G=%d groups", G);
  if ((st = check_table(c, k_pages, v_pages, n_pages, prefix_table, G, prefix_cols, ld_prefix, kMaxGroups)) != SF_OK)
    return st;
  if ((st = check_gather(c, n_pages)) != SF_OK) return st;
  if (!lens || !prefix_lens || !starts || misaligned(lens, 4) || misaligned(prefix_lens, 4) || misaligned(starts, 4))
    return fail(c, SF_ERR_INVALID_ARG, "lens, prefix_lens or starts null or misaligned");
  if ((st = check_object(c)) != SF_OK) return st;
  // the sequences' own positions, the prefixes beside them, and what joins both
  CacheAttendArgs t{};
  t.q = q;
  t.ld_q = ld_q;
  t.k = k_pages;
  t.v = v_pages;
  t.table = page_table(c, page_table_, table_cols, ld_table, n_pages);
  t.lens = lens;
  t.S = S;
  t.nq = s.n_q_heads;
  t.nkv = s.n_kv_heads;
  t.hd = s.head_dim;
  t.limit = length_limit(s.max_len, table_cols, s.page_size);
  t.scale_log2 = scale * kLog2e;
  t.state_o = c->tail_o;
  t.stats = c->tail_ml;
  t.parts = c->parts;
  t.arrived = c->arrived;
  t.joins = c->joins;
  t.err = c->err_dev;
  if ((st = launched(c, launch_cache_attend((cudaStream_t)stream, t, s.dtype == SF_BF16, c->sm_count))) != SF_OK)
    return st;
  CacheRowsArgs a = rows_args(c, q, ld_q, S, scale, out, ld_out, lse);
  a.k = k_pages;
  a.v = v_pages;
  a.table = page_table(c, prefix_table, prefix_cols, ld_prefix, n_pages);
  a.lens = prefix_lens;
  a.starts = starts;
  a.S = G;
  a.limit = length_limit(s.max_len, prefix_cols, s.page_size);
  a.tail_o = c->tail_o;
  a.tail_ml = c->tail_ml;
  a.whole_o = c->whole_o;
  a.whole_ml = c->whole_ml;
  return launched(c, launch_cache_rows((cudaStream_t)stream, a, s.dtype == SF_BF16, s.head_dim, c->sm_count));
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

sf_status sf_cache_inject_stall(sf_cache* c, int signal) {
  if (!c) return SF_ERR_INVALID_ARG;
  if (signal < kStallNone || signal >= kStallEnd) return fail(c, SF_ERR_INVALID_ARG, "no signal %d", signal);
  c->stall = signal;
  return SF_OK;
}

const char* sf_cache_last_error(const sf_cache* c) { return c ? c->last_error : ""; }

sf_status sf_cache_destroy(sf_cache* c) {
  if (!c) return SF_ERR_INVALID_ARG;
  cudaError_t e = cudaDeviceSynchronize();
  free_cache(c);
  return e == cudaSuccess ? SF_OK : SF_ERR_CUDA;
}

}  // extern "C"
