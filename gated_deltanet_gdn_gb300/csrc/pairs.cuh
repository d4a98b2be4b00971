// Two float32 in one register pair, and the packed arithmetic on them; four consecutive
// elements of a row as loaded (Quad), and the functions of the recurrent mixers' gates.
#pragma once

#include "common.cuh"

namespace gdn {

typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split2(f32x2 r) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(r));
  return f;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// The hardware's approximations: relative error below 2^-22.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float LOG2E = 1.44269504088896341f;

// 1 / (1 + e^-x), relative error below |x| 2^-24 + 2^-21.
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-x * LOG2E)); }

// log(1 + e^x) = max(x, 0) + log1p(e), e = e^-|x| <= 1, with log1p(e) = 2 artanh(s), s = e / (2 + e) <= 1/3, as its
// power series to s^15 (the rest is below 2^-27 of the value): no cancellation at either end, where a plain
// logarithm of 1 + e keeps nothing of a small e. NaN stays NaN.
__device__ __forceinline__ float softplus(float x) {
  const float e = ex2(-fabsf(x) * LOG2E);
  const float s = e * rcp(2.f + e), q = s * s;
  float p = 1.f / 15.f;
  p = fmaf(p, q, 1.f / 13.f);
  p = fmaf(p, q, 1.f / 11.f);
  p = fmaf(p, q, 1.f / 9.f);
  p = fmaf(p, q, 1.f / 7.f);
  p = fmaf(p, q, 1.f / 5.f);
  p = fmaf(p, q, 1.f / 3.f);
  p = fmaf(p, q, 1.f);
  return (x > 0.f ? x : 0.f) + 2.f * s * p;
}

// Four consecutive elements as they lie in memory.
template <class T>
struct Quad;
template <>
struct Quad<bf16> {
  uint2 v;
};
template <>
struct Quad<float> {
  float4 v;
};

// Elements p[0 .. n-1], zeros behind them (n up to 4, 0 or less: none). WIDE: p is aligned to four elements and n is
// 0 or 4.
template <bool WIDE, class T>
__device__ __forceinline__ Quad<T> load_quad(const T* p, int n) {
  Quad<T> q;
  if constexpr (WIDE) {
    memset(&q, 0, sizeof q);
    if (n > 0) q.v = *reinterpret_cast<const decltype(q.v)*>(p);
  } else {
    T e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = i < n ? p[i] : from_f32<T>(0.f);
    memcpy(&q, e, sizeof q);
  }
  return q;
}
template <bool WIDE, class T>
__device__ __forceinline__ void store_quad(T* p, const float (&x)[4], int n) {
  if constexpr (WIDE) {
    if (n > 0) st4(p, x);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = from_f32<T>(x[i]);
  }
}
__device__ __forceinline__ void quad_floats(const Quad<bf16>& q, float (&x)[4]) {
  x[0] = __uint_as_float(q.v.x << 16);
  x[1] = __uint_as_float(q.v.x & 0xffff0000u);
  x[2] = __uint_as_float(q.v.y << 16);
  x[3] = __uint_as_float(q.v.y & 0xffff0000u);
}
__device__ __forceinline__ void quad_floats(const Quad<float>& q, float (&x)[4]) {
  x[0] = q.v.x; x[1] = q.v.y; x[2] = q.v.z; x[3] = q.v.w;
}

}  // namespace gdn
