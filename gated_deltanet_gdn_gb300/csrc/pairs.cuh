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

__device__ __forceinline__ f32x2 both(float x) { return pack2(x, x); }
// One factor for both. (Two scalar products would take the fp32 pipe as long and no copy of the factor, but an issue slot
// more: 154 against 147 us in the forward at B8 T4096 D768.)
__device__ __forceinline__ f32x2 scale2(float s, f32x2 x) { return mul2(both(s), x); }
__device__ __forceinline__ f32x2 fma_by(float s, f32x2 x, f32x2 y) { return fma2(both(s), x, y); }
__device__ __forceinline__ f32x2 ex2_2(f32x2 x) {
  const float2 f = split2(x);
  return pack2(ex2(f.x), ex2(f.y));
}
// 2^x of two factors' exponents s a <= 0 that are multiplied up over many steps. The hardware's result is low on average,
// by 2e-8 of the value between 2^-8 and 1 and by less below, which a slow decay sums up; EX2_SHIFT, added in the same instruction, takes
// most of that (all of it would leave exponents below 2^-9 high): states and gradients came out half as far off.
constexpr float EX2_SHIFT = 2.0e-8f;
__device__ __forceinline__ f32x2 decay2(f32x2 s, f32x2 a) { return ex2_2(fma2(s, a, both(EX2_SHIFT))); }
__device__ __forceinline__ f32x2 rcp_2(f32x2 x) {
  const float2 f = split2(x);
  return pack2(rcp(f.x), rcp(f.y));
}
// sigmoid of two.
__device__ __forceinline__ f32x2 sigmoid2(f32x2 x) { return rcp_2(add2(both(1.f), ex2_2(mul2(x, both(-LOG2E))))); }

// log(1 + e^x) = max(x, 0) + log1p(e) of two, e = e^-|x| <= 1, with log1p(e) = 2 artanh(s), s = e / (2 + e) <= 1/3: no
// cancellation at either end, where a plain logarithm of 1 + e keeps nothing of a small e. artanh(s) / s is taken as the
// polynomial in s^2 that meets it at the five Chebyshev nodes of [0, 1/9] (4e-9 off at most; 3e-7 of the value in
// float32). NaN stays NaN.
// slope: NULL, or where the derivative, sigmoid(x) = 1 / (1 + e) or e / (1 + e), goes.
__device__ __forceinline__ f32x2 softplus2(f32x2 x, f32x2* slope = nullptr) {
  const float2 f = split2(x);
  const f32x2 e = ex2_2(pack2(fabsf(f.x) * -LOG2E, fabsf(f.y) * -LOG2E));
  if (slope) {
    const float2 g = split2(e);
    *slope = mul2(pack2(f.x < 0.f ? g.x : 1.f, f.y < 0.f ? g.y : 1.f), rcp_2(add2(both(1.f), e)));
  }
  const f32x2 s = mul2(e, rcp_2(add2(both(2.f), e))), q = mul2(s, s);
  f32x2 p = fma2(both(0.14078889787197113f), q, both(0.13982579112052917f));
  p = fma2(p, q, both(0.20012298226356506f));
  p = fma2(p, q, both(0.3333316147327423f));
  p = fma2(p, q, both(1.f));
  // (a comparison instead of fmaxf, which would lose a NaN)
  return fma2(add2(s, s), p, pack2(f.x > 0.f ? f.x : 0.f, f.y > 0.f ? f.y : 0.f));
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
__device__ __forceinline__ Quad<T> load_quad(const T* p) {
  Quad<T> q;
  if constexpr (WIDE) {
    q.v = *reinterpret_cast<const decltype(q.v)*>(p);
  } else {
    const T e[4] = {p[0], p[1], p[2], p[3]};
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
// The four as pairs.
__device__ __forceinline__ void quad_pairs(const Quad<bf16>& q, f32x2 (&x)[2]) {
  x[0] = pack2(__uint_as_float(q.v.x << 16), __uint_as_float(q.v.x & 0xffff0000u));
  x[1] = pack2(__uint_as_float(q.v.y << 16), __uint_as_float(q.v.y & 0xffff0000u));
}
__device__ __forceinline__ void quad_pairs(const Quad<float>& q, f32x2 (&x)[2]) {
  x[0] = pack2(q.v.x, q.v.y);
  x[1] = pack2(q.v.z, q.v.w);
}
__device__ __forceinline__ void store_pairs(float* p, const f32x2 (&x)[2]) {
  ulonglong2 v;
  v.x = x[0];
  v.y = x[1];
  *reinterpret_cast<ulonglong2*>(p) = v;
}
__device__ __forceinline__ void load_pairs(f32x2 (&x)[2], const float* p) {
  const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
  x[0] = v.x;
  x[1] = v.y;
}
template <bool WIDE, class T>
__device__ __forceinline__ void store_quad(T* p, const f32x2 (&x)[2], int n) {
  const float2 a = split2(x[0]), b = split2(x[1]);
  const float f[4] = {a.x, a.y, b.x, b.y};
  store_quad<WIDE>(p, f, n);
}

}  // namespace gdn
