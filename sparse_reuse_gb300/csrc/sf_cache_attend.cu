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
#include <cmath>

#include "sf_cache.h"

namespace sf {
namespace {

constexpr int kWarps = 8;
constexpr float kRoom = 19.f;
constexpr int kHeads = 8;  // query heads of one KV head that a CTA takes together

// One CTA per (sequence, KV head, up to 8 of its query heads); a warp takes
// every 8th key, a lane HD / 32 dimensions of it.
template <typename T, int HD>
__global__ void __launch_bounds__(32 * kWarps) cache_attend_kernel(const __grid_constant__ CacheAttendArgs a) {
  constexpr int DL = HD / 32;
  __shared__ float sm_m[kWarps][kHeads], sm_l[kWarps][kHeads];
  __shared__ float sm_o[kWarps][kHeads][HD];
  pdl_wait();
  pdl_trigger();
  const int G = a.nq / a.nkv, nsub = (G + kHeads - 1) / kHeads;
  const int sub = blockIdx.x % nsub, kvh = blockIdx.x / nsub, s = blockIdx.y;
  const int h0 = kvh * G + sub * kHeads;
  const int nh = min(kHeads, G - sub * kHeads);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool bad;
  const int len = checked_len(a.lens[s], a.limit, &bad);
  if (bad && threadIdx.x == 0) cache_error(a.err, kCacheBadLength);
  float q[kHeads][DL], o[kHeads][DL], m[kHeads], l[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int d = 0; d < DL; ++d) {
      o[h][d] = 0.f;
      q[h][d] = h < nh ? to_f32<T>(static_cast<const T*>(a.q)[(int64_t)s * a.ld_q + (int64_t)(h0 + h) * HD + lane * DL + d])
                       : 0.f;
    }
  }
  for (int j = warp; j < len; j += kWarps) {
    const int64_t slot = page_slot(a.table, s, j);
    if (slot < 0) {
      if (lane == 0) cache_error(a.err, kCacheBadPage);
      if (a.w_out && lane < nh) a.scores[((int64_t)s * a.nq + h0 + lane) * a.ld_scores + j] = -INFINITY;
      continue;
    }
    const int64_t at = (slot * a.nkv + kvh) * HD + lane * DL;
    float k[DL], v[DL];
#pragma unroll
    for (int d = 0; d < DL; ++d) {
      k[d] = to_f32<T>(static_cast<const T*>(a.k)[at + d]);
      v[d] = to_f32<T>(static_cast<const T*>(a.v)[at + d]);
    }
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      float x = 0.f;
#pragma unroll
      for (int d = 0; d < DL; ++d) x += q[h][d] * k[d];
      x = warp_sum(x) * a.scale_log2;
      if (a.w_out && lane == 0 && h < nh) a.scores[((int64_t)s * a.nq + h0 + h) * a.ld_scores + j] = x;
      const float mn = fmaxf(m[h], x);
      const float base = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m[h] - base), p = exp2f((x - base) - kRoom);
      m[h] = mn;
      l[h] = l[h] * f + p;
#pragma unroll
      for (int d = 0; d < DL; ++d) o[h][d] = o[h][d] * f + p * v[d];
    }
  }
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    if (lane == 0) {
      sm_m[warp][h] = m[h];
      sm_l[warp][h] = l[h];
    }
#pragma unroll
    for (int d = 0; d < DL; ++d) sm_o[warp][h][lane * DL + d] = o[h][d];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nh * HD; i += 32 * kWarps) {
    const int h = i / HD, d = i % HD;
    float mm = -INFINITY;
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w][h]);
    const float base = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f, oo = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2f(sm_m[w][h] - base);
      ll += sm_l[w][h] * f;
      oo += sm_o[w][h][d] * f;
    }
    static_cast<T*>(a.out)[(int64_t)s * a.ld_out + (int64_t)(h0 + h) * HD + d] = from_f32<T>(len > 0 ? oo / ll : 0.f);
    if (a.w_out && d == 0) a.lse[(int64_t)s * a.nq + h0 + h] = base + kRoom + log2f(ll);
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
      w += exp2f(a.scores[h * a.ld_scores + j] - a.lse[h]);
    }
    a.w_out[at] = (a.w_in ? a.w_in[at] : 0.f) + w;
  }
}

template <typename T, int HD>
cudaError_t attend_t(cudaStream_t st, const CacheAttendArgs& a) {
  const int G = a.nq / a.nkv, nsub = (G + kHeads - 1) / kHeads;
  cudaError_t e = launch_pdl(st, dim3(a.nkv * nsub, a.S), dim3(32 * kWarps), 0, 1, cache_attend_kernel<T, HD>, a);
  if (e == cudaSuccess && a.w_out)
    e = launch_pdl(st, dim3(a.nkv, a.S), dim3(256), 0, 1, cache_weights_kernel, a);
  return e;
}

}  // namespace

cudaError_t launch_cache_attend(cudaStream_t st, const CacheAttendArgs& a, int bf16, int) {
  if (bf16) return a.hd == 128 ? attend_t<__nv_bfloat16, 128>(st, a) : attend_t<__nv_bfloat16, 64>(st, a);
  return a.hd == 128 ? attend_t<float, 128>(st, a) : attend_t<float, 64>(st, a);
}

}  // namespace sf
