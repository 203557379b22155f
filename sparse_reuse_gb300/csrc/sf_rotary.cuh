// Rotation of two 16-byte pieces of a head by table angles, in either pairing.
#pragma once

#include "sf_pairs.cuh"

namespace sf {

// (a, b) -> (a cos - b sin, b cos + a sin).  Halves: piece x holds the a of N
// pairs of pairs, piece y their b, so cosines and sines are packed like them.
// Neighbours: a and b are the two halves of every packed pair, x and y pieces
// of their own; a pair's cosine stands twice, its sine as (-sin, sin).
template <typename T, bool NEIGHBOURS>
struct Angles {
  static_assert(!NEIGHBOURS, "specialised below");
  static constexpr int N = Piece<T>::PAIRS, VEC = 2 * N;
  Two cs[N], sn[N];

  // Angles of pieces c0 and c1 (c0's partner) of a head of `half` pairs.
  __device__ __forceinline__ void load(const float* row, int half, int c0, int) {
    load_pairs(row + c0 * VEC, cs);
    load_pairs(row + half + c0 * VEC, sn);
  }
  __device__ __forceinline__ void scale(float c, float s) {
    const Two cc = two(c, c), ss = two(s, s);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      cs[e] = cs[e] * cc;
      sn[e] = sn[e] * ss;
    }
  }
  __device__ __forceinline__ void turn(Two (&x)[N], Two (&y)[N]) const {
    const Two minus = two(-1.f, -1.f);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const Two u = x[e], w = y[e];
      x[e] = fma2(w * minus, sn[e], u * cs[e]);
      y[e] = fma2(u, sn[e], w * cs[e]);
    }
  }
};

template <typename T>
struct Angles<T, true> {
  static constexpr int N = Piece<T>::PAIRS, VEC = 2 * N;
  float c[2][N], s[2][N];  // of the pairs of both pieces
  bool on[2];              // the piece is of the rotated part

  static __device__ __forceinline__ void load_floats(const float* p, float (&x)[N]) {
    if constexpr (N == 4) {
      const float4 v = *reinterpret_cast<const float4*>(p);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(p);
      x[0] = v.x, x[1] = v.y;
    }
  }
  __device__ __forceinline__ void load(const float* row, int half, int c0, int c1) {
    const int at[2] = {c0 * N, c1 * N};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      on[i] = at[i] < half;
      if (on[i]) {
        load_floats(row + at[i], c[i]);
        load_floats(row + half + at[i], s[i]);
      }
    }
  }
  __device__ __forceinline__ void scale(float fc, float fs) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        c[i][e] *= fc;
        s[i][e] *= fs;
      }
  }
  __device__ __forceinline__ void piece(Two (&x)[N], int i) const {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float2 v = both(x[e]);
      x[e] = fma2(two(v.y, v.x), two(-s[i][e], s[i][e]), x[e] * two(c[i][e], c[i][e]));
    }
  }
  __device__ __forceinline__ void turn(Two (&x)[N], Two (&y)[N]) const {
    if (on[0]) piece(x, 0);
    if (on[1]) piece(y, 1);
  }
};

}  // namespace sf
