// Packed fp32 arithmetic, and 16-byte pieces of rows as pairs of fp32.
#pragma once

#include "sf_common.cuh"

namespace sf {

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
__device__ __forceinline__ Two operator+(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
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

}  // namespace sf
