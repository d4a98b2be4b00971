// The norms around a block, with its gate and residual scale, forward and backward.
//
// Per row (R rows of G groups, C elements normalised together; every part optional):
//   n = x r1 w_post,  r1 = 1 / sqrt(mean x^2 + eps)     norm after the block
//   m = n act(gate),  act = silu or sigmoid             the block's gate
//   h = residual + res_scale m                          the residual stream
//   y = h r2 w_pre,   r2 = 1 / sqrt(mean h^2 + eps)     norm before the next block
// Everything is fp32 between the loads and the stores: y comes from the unrounded h.
//
// Backward from dh, dy, with the forward's r1, r2 (h is formed again from x, gate and
// residual: the same bytes as reading it, and not rounded):
//   t = dy w_pre;  D = dh + r2 (t - h r2^2 mean(t h));  dresidual = D;  dw_pre = sum dy h r2
//   dres_scale = sum D m;  dm = D res_scale;  dgate = dm n act';  dn = dm act
//   u = dn w_post; dx = r1 (u - x r1^2 mean(u x));  dw_post = sum dn x r1
//
// Every input is read once. Three forms, by the width of a row:
//  * narrow rows (up to 32 vectors of 16 bytes; the norm of a head, which has kernels of its
//    own): a part of a warp per row, reductions by shuffle, the next rows' vectors loaded
//    while this one's are used;
//  * wide rows: persistent CTAs, one row at a time, the inputs of the next rows on their
//    way through a ring in shared memory (bulk copies by a warp of their own);
//  * rows whose width, strides or pointers do not allow 16-byte accesses: element by
//    element, a CTA (or a warp) per row.
// The sums over rows of the weight gradients stay in the registers of the threads that own
// the columns while a CTA walks its rows (a fixed stride, so the order of the sums is
// fixed); one partial row per CTA goes to the workspace and a second kernel adds them.
//
// Bound by memory, less what the reductions and conversions leave uncovered. bf16, all parts,
// 8,192 rows of 6,144: forward 84 us (0.90 of the copy rate on its bytes), backward 144 us
// (0.84). Gated norm of 196,608 heads of 128: forward 29 us (0.78), backward 45 us (0.84).
#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

// VEC elements in one access (16 bytes, or a single element).
template <class T, int VEC>
struct Raw {
  uint4 u;
  __device__ __forceinline__ void load(const T* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void clear() { u = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&x)[VEC]) const {
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = to_f32(e[i]);
  }
  __device__ __forceinline__ void set(const float (&x)[VEC]) {
    T* e = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int i = 0; i < VEC; ++i) e[i] = from_f32<T>(x[i]);
  }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = u; }
};
template <class T>
struct Raw<T, 1> {
  T u;
  __device__ __forceinline__ void load(const T* p) { u = *p; }
  __device__ __forceinline__ void clear() { u = from_f32<T>(0.f); }
  __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = to_f32(u); }
  __device__ __forceinline__ void set(const float (&x)[1]) { u = from_f32<T>(x[0]); }
  __device__ __forceinline__ void store(T* p) const { *p = u; }
};

// Sum over the row's threads: SUB lanes of a warp, or (SUB = 0) the whole CTA. buf: a
// slot per warp; two alternating buffers make one barrier per sum enough.
template <int SUB>
__device__ __forceinline__ float row_sum(float v, float* buf) {
  constexpr int W = SUB ? SUB : 32;
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (SUB) return v;
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  const int nw = (blockDim.x + 31) >> 5;
  float s = 0.f;
  for (int w = 0; w < nw; ++w) s += buf[w];
  return s;
}

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// exp(-g) and 1 / x for the gates of rows of type T. bf16 takes the hardware's approximate
// exponential and reciprocal: relative errors of |g| 2^-24 (the rounded argument) + 2^-22 and
// 2^-23, far below bf16's own 2^-8, and with expf the arithmetic, not memory, bounds the
// kernels. fp32 keeps fp32's accuracy, with twice the bytes per element to cover it: expf, and
// the reciprocal with its subnormals, both within one unit in the last place (4,096 rows of
// 6,144, both directions: 249 us, as with bf16's forms; with a division 271).
template <class T>
__device__ __forceinline__ float exp_neg(float g) {
  if constexpr (sizeof(T) == 2) return ex2_approx(g * -1.4426950408889634f);
  else return expf(-g);
}
template <class T>
__device__ __forceinline__ float inverse(float x) {
  if constexpr (sizeof(T) == 2) return rcp_approx(x);
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// act(g) and act'(g). silu' = s (1 + g (1 - s)) takes 1 - s as it is (an error of |g| 2^-24
// beside the 1); the sigmoid's s (1 - s) takes both sides from exp(-|g|), so that 1 - s keeps its
// relative accuracy where s is near 1. Neither form overflows: exp(-g) = inf gives s = 0.
template <class T, int VEC>
__device__ __forceinline__ void activation(const float (&g)[VEC], int sigmoid, float (&a)[VEC], float (&d)[VEC]) {
  if (!sigmoid) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float s = inverse<T>(1.f + exp_neg<T>(g[e]));
      a[e] = g[e] * s;
      d[e] = s * fmaf(g[e], 1.f - s, 1.f);
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float x = exp_neg<T>(fabsf(g[e])), big = inverse<T>(1.f + x), small = x * big;
      a[e] = g[e] >= 0.f ? big : small;
      d[e] = big * small;
    }
  }
}

constexpr int SUB_THREADS = 256;       // threads of a CTA whose rows take a part of a warp each
constexpr int NORM_THREADS_MAX = 512;  // threads of a CTA that holds one row

// Which row the calling thread starts on, how far apart its rows are and which vector of
// the row it owns first.
template <int SUB>
struct Place {
  unsigned row, step;
  int lane, lanes;
  __device__ __forceinline__ Place() {
    if constexpr (SUB != 0) {
      row = blockIdx.x * (SUB_THREADS / SUB) + threadIdx.x / SUB;
      step = gridDim.x * (SUB_THREADS / SUB);
      lane = threadIdx.x % SUB;
      lanes = SUB;
    } else {
      row = blockIdx.x;
      step = gridDim.x;
      lane = threadIdx.x;
      lanes = blockDim.x;
    }
  }
};

// The inputs of one row, this thread's vectors of them.
template <class T, int VEC, int NV>
struct RowIn {
  Raw<T, VEC> x[NV], gate[NV], res[NV], dh[NV], dy[NV];
};

template <class T, int VEC, int NV, int SUB>
__global__ void __launch_bounds__(SUB ? SUB_THREADS : NORM_THREADS_MAX)
    block_norm_fwd_kernel(NormArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ __align__(16) float buf[2][32];
  const Place<SUB> at;
  const T *wpost = static_cast<const T*>(a.w_post), *rscale = static_cast<const T*>(a.res_scale),
          *wpre = static_cast<const T*>(a.w_pre), *gate = static_cast<const T*>(a.gate),
          *res = static_cast<const T*>(a.residual);
  const float invC = 1.f / (float)a.C;
  // a part-warp's rows end together: the whole warp stays in the loop for the shuffles
  constexpr unsigned PER = SUB ? SUB_THREADS / (SUB ? SUB : 1) : 1;  // rows of a CTA at a time
  const unsigned rows = (unsigned)a.R * (unsigned)a.G, last = (rows + PER - 1) / PER * PER;
  auto fetch = [&](unsigned jj, RowIn<T, VEC, NV>& in) {
    const bool live = jj < rows;
    const long long r = live ? jj / (unsigned)a.G : 0, g = live ? jj % (unsigned)a.G : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (at.lane + i * at.lanes) * VEC;
      in.x[i].clear(); in.gate[i].clear(); in.res[i].clear();
      if (live && c < a.C) {
        in.x[i].load(static_cast<const T*>(a.x) + r * a.x_rs + g * a.x_gs + c);
        if (gate) in.gate[i].load(gate + r * a.gate_rs + g * a.gate_gs + c);
        if (res) in.res[i].load(res + r * a.res_rs + g * a.res_gs + c);
      }
    }
  };
  constexpr bool AHEAD = SUB != 0;  // load the next row while this one is used
  RowIn<T, VEC, NV> in, next;
  if (AHEAD && at.row < last) fetch(at.row, next);
  for (unsigned jj = at.row; jj < last; jj += at.step) {
    const bool live = jj < rows;
    const size_t j = jj;
    if (AHEAD) {
      in = next;
      if (jj + at.step < last) fetch(jj + at.step, next);
    } else {
      fetch(jj, in);
    }
    float v[NV][VEC];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      in.x[i].get(v[i]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) ss = fmaf(v[i][e], v[i][e], ss);
    }
    float r1 = 1.f;
    if (wpost) r1 = rsqrtf(row_sum<SUB>(ss, buf[0]) * invC + a.eps);
    float hh = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (at.lane + i * at.lanes) * VEC;
      if (!live || c >= a.C) continue;
      Raw<T, VEC> raw;
      float w[VEC];
      if (wpost) {
        raw.load(wpost + c);
        raw.get(w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] *= r1 * w[e];
      }
      if (gate) {
        float ac[VEC], ad[VEC];
        in.gate[i].get(w);
        activation<T, VEC>(w, a.sigmoid, ac, ad);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] *= ac[e];
      }
      if (rscale) {
        raw.load(rscale + c);
        raw.get(w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] *= w[e];
      }
      if (res) {
        in.res[i].get(w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] += w[e];
      }
      raw.set(v[i]);
      raw.store(static_cast<T*>(a.h) + j * a.C + c);
#pragma unroll
      for (int e = 0; e < VEC; ++e) hh = fmaf(v[i][e], v[i][e], hh);
    }
    float r2 = 1.f;
    if (wpre) {
      r2 = rsqrtf(row_sum<SUB>(hh, buf[1]) * invC + a.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (at.lane + i * at.lanes) * VEC;
        if (!live || c >= a.C) continue;
        Raw<T, VEC> raw;
        float w[VEC];
        raw.load(wpre + c);
        raw.get(w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] *= v[i][e] * r2;
        raw.set(w);
        raw.store(static_cast<T*>(a.y) + j * a.C + c);
      }
    }
    if (live && at.lane == 0) *reinterpret_cast<float2*>(a.stats + 2 * j) = make_float2(r1, r2);
    // with one sum a row, the next row's write to its buffer must not overtake this one's reads
    if (!SUB && !(wpost && wpre)) __syncthreads();
  }
}

template <class T, int VEC, int NV, int SUB>
__global__ void __launch_bounds__(SUB ? SUB_THREADS : NORM_THREADS_MAX)
    block_norm_bwd_kernel(NormArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ __align__(16) float buf[2][32];
  const Place<SUB> at;
  const T *gate = static_cast<const T*>(a.gate), *res = static_cast<const T*>(a.residual),
          *wpost = static_cast<const T*>(a.w_post), *rscale = static_cast<const T*>(a.res_scale),
          *wpre = static_cast<const T*>(a.w_pre), *dhp = static_cast<const T*>(a.dh),
          *dyp = static_cast<const T*>(a.dy);
  T* dres = static_cast<T*>(a.dresidual);
  const float invC = 1.f / (float)a.C;
  constexpr unsigned PER = SUB ? SUB_THREADS / (SUB ? SUB : 1) : 1;  // rows of a CTA at a time
  const unsigned rows = (unsigned)a.R * (unsigned)a.G, last = (rows + PER - 1) / PER * PER;
  float sw1[NV][VEC], sw2[NV][VEC], ssc[NV][VEC];  // sums of dw_post, dw_pre, dres_scale over this thread's rows
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) sw1[i][e] = sw2[i][e] = ssc[i][e] = 0.f;
  auto fetch = [&](unsigned jj, RowIn<T, VEC, NV>& in, float2& st) {
    const bool live = jj < rows;
    const long long r = live ? jj / (unsigned)a.G : 0, g = live ? jj % (unsigned)a.G : 0;
    st = live ? *reinterpret_cast<const float2*>(a.stats + 2 * (size_t)jj) : make_float2(1.f, 1.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (at.lane + i * at.lanes) * VEC;
      in.x[i].clear(); in.gate[i].clear(); in.res[i].clear(); in.dh[i].clear(); in.dy[i].clear();
      if (live && c < a.C) {
        in.x[i].load(static_cast<const T*>(a.x) + r * a.x_rs + g * a.x_gs + c);
        if (gate) in.gate[i].load(gate + r * a.gate_rs + g * a.gate_gs + c);
        if (res && wpre) in.res[i].load(res + r * a.res_rs + g * a.res_gs + c);
        if (dhp) in.dh[i].load(dhp + r * a.dh_rs + g * a.dh_gs + c);
        if (dyp) in.dy[i].load(dyp + r * a.dy_rs + g * a.dy_gs + c);
      }
    }
  };
  constexpr bool AHEAD = SUB != 0;
  RowIn<T, VEC, NV> in, next;
  float2 st, st_next;
  if (AHEAD && at.row < last) fetch(at.row, next, st_next);
  for (unsigned jj = at.row; jj < last; jj += at.step) {
    const bool live = jj < rows;
    const size_t j = jj;
    if (AHEAD) {
      in = next;
      st = st_next;
      if (jj + at.step < last) fetch(jj + at.step, next, st_next);
    } else {
      fetch(jj, in, st);
    }
    const float r1 = wpost ? st.x : 1.f, r2 = wpre ? st.y : 1.f;
    // n, act(gate), act'(gate) and the residual scale of one vector
    auto forward = [&](int i, int c, const float (&xv)[VEC], float (&n)[VEC], float (&ac)[VEC], float (&ad)[VEC],
                       float (&sc)[VEC]) {
      Raw<T, VEC> raw;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        n[e] = xv[e];
        ac[e] = 1.f;
        ad[e] = 0.f;
        sc[e] = 1.f;
      }
      if (wpost) {
        float w[VEC];
        raw.load(wpost + c);
        raw.get(w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) n[e] *= r1 * w[e];
      }
      if (gate) {
        float w[VEC];
        in.gate[i].get(w);
        activation<T, VEC>(w, a.sigmoid, ac, ad);
      }
      if (rscale) {
        raw.load(rscale + c);
        raw.get(sc);
      }
    };
    float c2 = 0.f;
    if (dyp) {
      float s2 = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (at.lane + i * at.lanes) * VEC;
        if (!live || c >= a.C) continue;
        float xv[VEC], n[VEC], ac[VEC], ad[VEC], sc[VEC], rv[VEC], dyv[VEC], w[VEC];
        in.x[i].get(xv);
        forward(i, c, xv, n, ac, ad, sc);
        in.res[i].get(rv);
        in.dy[i].get(dyv);
        Raw<T, VEC> raw;
        raw.load(wpre + c);
        raw.get(w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float h = rv[e] + sc[e] * (n[e] * ac[e]);
          s2 = fmaf(dyv[e] * w[e], h, s2);
          sw2[i][e] = fmaf(dyv[e] * r2, h, sw2[i][e]);
        }
      }
      c2 = row_sum<SUB>(s2, buf[0]) * invC * r2 * r2;
    }
    float u[NV][VEC], s1 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (at.lane + i * at.lanes) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) u[i][e] = 0.f;
      if (!live || c >= a.C) continue;
      float xv[VEC], n[VEC], ac[VEC], ad[VEC], sc[VEC], D[VEC];
      in.x[i].get(xv);
      forward(i, c, xv, n, ac, ad, sc);
      in.dh[i].get(D);
      Raw<T, VEC> raw;
      if (dyp) {
        float rv[VEC], dyv[VEC], w[VEC];
        in.res[i].get(rv);
        in.dy[i].get(dyv);
        raw.load(wpre + c);
        raw.get(w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float h = rv[e] + sc[e] * (n[e] * ac[e]);
          D[e] += r2 * (dyv[e] * w[e] - h * c2);
        }
      }
      if (dres) {
        raw.set(D);
        raw.store(dres + j * a.C + c);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (rscale) ssc[i][e] = fmaf(D[e], n[e] * ac[e], ssc[i][e]);
        D[e] *= sc[e];
      }
      if (a.dgate) {
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = D[e] * n[e] * ad[e];
        raw.set(o);
        raw.store(static_cast<T*>(a.dgate) + j * a.C + c);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) u[i][e] = D[e] * ac[e];
      if (wpost) {
        float w[VEC];
        raw.load(wpost + c);
        raw.get(w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          sw1[i][e] = fmaf(u[i][e], xv[e] * r1, sw1[i][e]);
          u[i][e] *= w[e];
          s1 = fmaf(u[i][e], xv[e], s1);
        }
      }
    }
    float c1 = 0.f;
    if (wpost) c1 = row_sum<SUB>(s1, buf[1]) * invC * r1 * r1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (at.lane + i * at.lanes) * VEC;
      if (!live || c >= a.C) continue;
      if (wpost) {  // (0 x is not 0 when x is not finite)
        float xv[VEC];
        in.x[i].get(xv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) u[i][e] = r1 * (u[i][e] - xv[e] * c1);
      }
      Raw<T, VEC> raw;
      raw.set(u[i]);
      raw.store(static_cast<T*>(a.dx) + j * a.C + c);
    }
    if (!SUB && !(wpost && dyp)) __syncthreads();
  }
  // this CTA's partial sums: [3][C] of the workspace row blockIdx.x
  float* part = a.partial + (size_t)blockIdx.x * 3 * a.C;
  auto put = [&](int which, float (&s)[NV][VEC]) {
    if constexpr (SUB != 0) {  // add the rows' groups of the CTA column by column, in the order of the groups
      __shared__ float cols[SUB_THREADS * VEC];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VEC; ++e) cols[threadIdx.x * VEC + e] = s[i][e];
        __syncthreads();
        for (int q = threadIdx.x; q < SUB * VEC; q += SUB_THREADS) {
          const int c = i * SUB * VEC + q;
          if (c >= a.C) continue;
          float t = 0.f;
          for (int k = 0; k < SUB_THREADS / SUB; ++k) t += cols[k * SUB * VEC + q];
          part[which * a.C + c] = t;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (at.lane + i * at.lanes) * VEC;
        if (c < a.C)
#pragma unroll
          for (int e = 0; e < VEC; ++e) part[which * a.C + c + e] = s[i][e];
      }
    }
  };
  if (a.dw_post) put(0, sw1);
  if (a.dw_pre) put(1, sw2);
  if (a.dres_scale) put(2, ssc);
}

// ---------------------------------------------------------------- packed arithmetic
// Packed fp32 pairs: one instruction does the fp32 operation on both halves, each rounded
// as the scalar one. The kernels below are close to the issue rate, which this halves for
// most of their arithmetic.
typedef uint64_t f2;
__device__ __forceinline__ f2 pk(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpk(f2 r, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(r)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// 16 bytes as pairs, and back (one rounding).
__device__ __forceinline__ void pairs_of(const uint4& u, f2 (&x)[4], const bf16*) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pk(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void pairs_of(const uint4& u, f2 (&x)[2], const float*) {
  x[0] = pk(__uint_as_float(u.x), __uint_as_float(u.y));
  x[1] = pk(__uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ uint4 rounded(const f2 (&x)[4], const bf16*) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    unpk(x[i], lo, hi);
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 rounded(const f2 (&x)[2], const float*) {
  float a, b, c, d;
  unpk(x[0], a, b);
  unpk(x[1], c, d);
  return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
}
// act(g) and act'(g) of a pair, as `activation`, in one form without a branch: with
// e = exp(-g), s = 1 / (1 + e) and 1 - s = e s (which keeps its accuracy; inf 0 of a
// large -g is 1),
//   silu:  g s, s (1 + g (1 - s))        sigmoid:  s, s (0 + 1 (1 - s))
template <class T>
__device__ __forceinline__ void activation2(f2 g, bool sigmoid, f2& a, f2& d, const T*) {
  const f2 one = pk(1.f, 1.f);
  float t0, t1;
  f2 e;  // exp(-g); bf16's product with log2 e stays packed
  if constexpr (sizeof(T) == 2) {
    unpk(mul2(g, pk(-1.4426950408889634f, -1.4426950408889634f)), t0, t1);
    e = pk(ex2_approx(t0), ex2_approx(t1));
  } else {
    unpk(g, t0, t1);
    e = pk(exp_neg<T>(t0), exp_neg<T>(t1));
  }
  unpk(add2(e, one), t0, t1);
  const f2 s = pk(inverse<T>(t0), inverse<T>(t1));
  unpk(mul2(e, s), t0, t1);
  const f2 rest = pk(fminf(t0, 1.f), fminf(t1, 1.f));
  const f2 f = sigmoid ? one : g;
  a = mul2(f, s);
  d = mul2(s, fma2(f, rest, sigmoid ? pk(0.f, 0.f) : one));
}

// ---------------------------------------------------------------- a head's output
// Rows of up to 32 vectors with w_post and gate alone, the norm of a head's output: SUB
// lanes a row, a weight that is missing is ones. What a row costs beside its arithmetic counts
// here (eight elements a thread): strided places are stepped, not divided. The next two rows
// are on their way while one is used, since the loads of one do not cover the latency:
// 196,608 rows of 128 in bf16 take 71 us in both directions, with one row ahead 80.

// Place of a thread's vector in an input with row and group strides, row after row of its walk.
struct HeadWalk {
  long long at, by, wrap;
  __device__ __forceinline__ HeadWalk(unsigned row, unsigned step, unsigned G, long long rs, long long gs, int c)
      : at((long long)(row / G) * rs + (long long)(row % G) * gs + c),
        by((long long)(step / G) * rs + (long long)(step % G) * gs),
        wrap(rs - (long long)G * gs) {}
  __device__ __forceinline__ void next(bool over) { at += over ? by + wrap : by; }
};
template <int SUB>
__device__ __forceinline__ float head_sum(f2 v2) {
  float v, hi;
  unpk(v2, v, hi);
  v += hi;
#pragma unroll
  for (int off = SUB / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

template <class T, int SUB, bool GATE>
__global__ void __launch_bounds__(SUB_THREADS) block_norm_head_fwd_kernel(NormArgs a) {
  constexpr int VEC = 16 / (int)sizeof(T), NP = VEC / 2, PER = SUB_THREADS / SUB;
  pdl_wait();
  pdl_trigger();
  const Place<SUB> at;
  const T *kind = nullptr, *x = static_cast<const T*>(a.x), *gate = static_cast<const T*>(a.gate);
  const int c = at.lane * VEC;
  const bool mine = c < a.C, post = a.w_post != nullptr;
  const unsigned G = (unsigned)a.G, rows = (unsigned)a.R * G, last = (rows + PER - 1) / PER * PER, dg = at.step % G;
  const float invC = 1.f / (float)a.C;
  HeadWalk wx(at.row, at.step, G, a.x_rs, a.x_gs, c), wg(at.row, at.step, G, a.gate_rs, a.gate_gs, c);
  unsigned g = at.row % G;
  f2 w[NP];
#pragma unroll
  for (int e = 0; e < NP; ++e) w[e] = pk(1.f, 1.f);
  if (post && mine) pairs_of(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.w_post) + c), w, kind);
  struct Row {
    uint4 x, gate;
  } row0, row1;  // the next two rows
  row0.x = row0.gate = row1.x = row1.gate = make_uint4(0u, 0u, 0u, 0u);
  auto fetch = [&](unsigned row, Row& in) {
    if (mine && row < rows) {
      in.x = *reinterpret_cast<const uint4*>(x + wx.at);
      if (GATE) in.gate = *reinterpret_cast<const uint4*>(gate + wg.at);
    }
    g += dg;
    const bool over = g >= G;
    if (over) g -= G;
    wx.next(over);
    if (GATE) wg.next(over);
  };
  auto use = [&](unsigned row, Row& in) {
    f2 v[NP], t[NP], ss = pk(0.f, 0.f);
    pairs_of(in.x, v, kind);
    if (GATE) pairs_of(in.gate, t, kind);
    fetch(row + 2 * at.step, in);
    float r1 = 1.f;
    if (post) {
#pragma unroll
      for (int e = 0; e < NP; ++e) ss = fma2(v[e], v[e], ss);
      r1 = rsqrtf(head_sum<SUB>(ss) * invC + a.eps);
    }
    const f2 r1p = pk(r1, r1);
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      v[e] = mul2(mul2(v[e], r1p), w[e]);
      if (GATE) {
        f2 ac, ad;
        activation2(t[e], a.sigmoid, ac, ad, kind);
        v[e] = mul2(v[e], ac);
      }
    }
    if (row < rows) {
      if (mine) *reinterpret_cast<uint4*>(static_cast<T*>(a.h) + (size_t)row * (unsigned)a.C + c) = rounded(v, kind);
      if (at.lane == 0) *reinterpret_cast<float2*>(a.stats + 2 * (size_t)row) = make_float2(r1, 1.f);
    }
  };
  fetch(at.row, row0);
  fetch(at.row + at.step, row1);
  for (unsigned row = at.row; row < last; row += 2 * at.step) {
    use(row, row0);
    if (row + at.step < last) use(row + at.step, row1);
  }
}

template <class T, int SUB, bool GATE>
__global__ void __launch_bounds__(SUB_THREADS, 2) block_norm_head_bwd_kernel(NormArgs a) {
  constexpr int VEC = 16 / (int)sizeof(T), NP = VEC / 2, PER = SUB_THREADS / SUB;
  pdl_wait();
  pdl_trigger();
  const Place<SUB> at;
  const T *kind = nullptr, *x = static_cast<const T*>(a.x), *gate = static_cast<const T*>(a.gate),
          *dh = static_cast<const T*>(a.dh);
  const int c = at.lane * VEC;
  const bool mine = c < a.C, post = a.w_post != nullptr;
  const unsigned G = (unsigned)a.G, rows = (unsigned)a.R * G, last = (rows + PER - 1) / PER * PER, dg = at.step % G;
  const float invC = 1.f / (float)a.C;
  HeadWalk wx(at.row, at.step, G, a.x_rs, a.x_gs, c), wg(at.row, at.step, G, a.gate_rs, a.gate_gs, c),
      wd(at.row, at.step, G, a.dh_rs, a.dh_gs, c);
  unsigned g = at.row % G;
  const f2 zero2 = pk(0.f, 0.f);
  f2 w[NP], sw[NP];  // the weights, and their gradients' sums over this thread's rows
#pragma unroll
  for (int e = 0; e < NP; ++e) {
    w[e] = pk(1.f, 1.f);
    sw[e] = zero2;
  }
  if (post && mine) pairs_of(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.w_post) + c), w, kind);
  struct Row {
    uint4 x, gate, dh;
    float r1;
  } row0, row1;  // the next two rows
  row0.r1 = row1.r1 = 1.f;
  auto fetch = [&](unsigned row, Row& in) {
    if (mine && row < rows) {
      in.x = *reinterpret_cast<const uint4*>(x + wx.at);
      if (GATE) in.gate = *reinterpret_cast<const uint4*>(gate + wg.at);
      in.dh = dh ? *reinterpret_cast<const uint4*>(dh + wd.at) : make_uint4(0u, 0u, 0u, 0u);
      if (post) in.r1 = a.stats[2 * (size_t)row];
    } else {
      in.x = in.gate = in.dh = make_uint4(0u, 0u, 0u, 0u);  // nothing for the sums
    }
    g += dg;
    const bool over = g >= G;
    if (over) g -= G;
    wx.next(over);
    if (GATE) wg.next(over);
    wd.next(over);
  };
  auto use = [&](unsigned row, Row& in) {
    const size_t out = (size_t)row * (unsigned)a.C + c;
    const bool store = mine && row < rows;
    f2 xv[NP], t[NP], D[NP], s1 = zero2;
    pairs_of(in.x, xv, kind);
    if (GATE) pairs_of(in.gate, t, kind);
    pairs_of(in.dh, D, kind);
    const float r1 = in.r1;
    fetch(row + 2 * at.step, in);
    const f2 r1p = pk(r1, r1);
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      const f2 xr = mul2(xv[e], r1p);
      if (GATE) {
        f2 ac, ad;
        activation2(t[e], a.sigmoid, ac, ad, kind);
        t[e] = mul2(mul2(D[e], mul2(xr, w[e])), ad);  // dgate
        D[e] = mul2(D[e], ac);
      }
      sw[e] = fma2(D[e], xr, sw[e]);
      D[e] = mul2(D[e], w[e]);
      s1 = fma2(D[e], xv[e], s1);
    }
    if (GATE && store && a.dgate) *reinterpret_cast<uint4*>(static_cast<T*>(a.dgate) + out) = rounded(t, kind);
    if (post) {  // without it dx is D (0 x is not 0 when x is not finite)
      const float m = -head_sum<SUB>(s1) * invC * r1 * r1 * r1;
      const f2 c1 = pk(m, m);
#pragma unroll
      for (int e = 0; e < NP; ++e) D[e] = fma2(xv[e], c1, mul2(D[e], r1p));
    }
    if (store) *reinterpret_cast<uint4*>(static_cast<T*>(a.dx) + out) = rounded(D, kind);
  };
  fetch(at.row, row0);
  fetch(at.row + at.step, row1);
  for (unsigned row = at.row; row < last; row += 2 * at.step) {
    use(row, row0);
    if (row + at.step < last) use(row + at.step, row1);
  }
  if (!a.dw_post) return;
  // this CTA's sums: the groups of lanes column by column, in their order
  __shared__ __align__(16) float cols[SUB_THREADS * VEC];
#pragma unroll
  for (int e = 0; e < NP; ++e) *reinterpret_cast<f2*>(cols + threadIdx.x * VEC + 2 * e) = sw[e];
  __syncthreads();
  for (int q = threadIdx.x; q < SUB * VEC; q += SUB_THREADS) {
    if (q >= a.C) continue;
    float t = 0.f;
    for (int k = 0; k < PER; ++k) t += cols[k * SUB * VEC + q];
    a.partial[(size_t)blockIdx.x * 3 * a.C + q] = t;
  }
}

// ---------------------------------------------------------------- wide rows
constexpr int MAX_STAGES = 8;
struct StreamShared {
  float buf[2][32];
  uint64_t full[MAX_STAGES], empty[MAX_STAGES];
};
constexpr int STREAM_HEAD = 512;  // bytes of StreamShared before the ring
static_assert(sizeof(StreamShared) <= STREAM_HEAD, "barriers and sums before the ring");

// A persistent CTA: one warp (the last) fills a ring of `stages` rows, each the row's
// vectors of up to five inputs (bulk copies); the others take a row at a time, NV vectors
// of 16 bytes of it per thread. Two sums over the row each way, a barrier each.
//
// SPLIT: the backward of the widest rows, whose column sums and row values take more
// registers than an equal share: the workers are whole warpgroups and take some of the
// filling warpgroup's (384 of them: 3 * 160 + 32 = 4 * 128; 512: 4 * 112 + 32 = 5 * 96).
constexpr int SPLIT_LOW = 32;
constexpr int split_high(int maxt) { return maxt == 384 ? 160 : 112; }
//
// FULL: the residual and the norm before the next block are there (GATE: the gate too);
// weights that are missing are ones. Nothing in the row's loops branches then, so that the
// loads and conversions of a whole segment are interleaved: a thread beyond the row's end
// works on the first columns and leaves its results out. (With a branch per part the
// 8192 x 6144 backward took 200 us in place of 161.)
//
// The backward keeps only h between its segments and forms act and act' again (6144 wide:
// 144 us, against 156 with all three in registers), except below 2048 columns of bf16,
// where two CTAs per SM have the registers (164 us; formed again 170).
constexpr int stream_ctas(int nv, int maxt, bool bwd, bool full) {  // per SM, of MAXT workers
  return bwd ? (maxt == 256 || (maxt == 384 && nv == 1 && full) ? 2 : 1) : maxt > 384 ? 1 : 2;
}
template <class T, int NV, int MAXT, bool BWD, bool SPLIT, bool FULL, bool GATE>
__global__ void __launch_bounds__(MAXT + (SPLIT ? 128 : 32), stream_ctas(NV, MAXT, BWD, FULL))
    block_norm_stream_kernel(NormArgs a, int stages) {
  constexpr int VEC = 16 / (int)sizeof(T), NP = VEC / 2;
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(128) uint8_t smem[];
  StreamShared* sh = reinterpret_cast<StreamShared*>(smem);
  const bool post = a.w_post, pre = FULL || a.w_pre, gated = FULL ? GATE : a.gate != nullptr;
  const bool weighed = FULL || a.w_post, scaled = FULL || a.res_scale;  // by ones, if need be
  // which tensor of a stage is which input (x is 0)
  int nt = 1;
  const int tg = gated ? nt++ : 0;
  const int tr = FULL || (a.residual && (!BWD || pre)) ? nt++ : 0;
  const int th = BWD && (FULL || a.dh) ? nt++ : 0;
  const int ty = BWD && pre ? nt++ : 0;
  const int workers = blockDim.x - (SPLIT ? 128 : 32);
  const uint32_t bytes = (uint32_t)a.C * sizeof(T);
  constexpr bool KEEP = BWD || (FULL && MAXT == 384);  // weights in shared memory
  const uint32_t ring = STREAM_HEAD + (KEEP ? 3 * bytes : 0);  // offset of the ring
  const unsigned rows = (unsigned)a.R * (unsigned)a.G, grid = gridDim.x;
  const T* kind = nullptr;  // names the type for the packing functions
  for (int i = threadIdx.x; i < 64; i += blockDim.x) (&sh->buf[0][0])[i] = 0.f;
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&sh->full[i], 1);
      mbar_init(&sh->empty[i], workers / 32);
    }
    fence_mbar_init();
  }
  __syncthreads();

  if ((int)threadIdx.x >= workers) {
    if constexpr (SPLIT) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(SPLIT_LOW));
    if ((int)threadIdx.x == workers) {
      int stage = 0, loads = 0;
      for (size_t row = blockIdx.x; row < rows; row += grid, ++loads) {
        if (loads >= stages) mbar_wait(&sh->empty[stage], (uint32_t)(loads / stages - 1) & 1u, a.err);
        mbar_arrive_expect_tx(&sh->full[stage], (uint32_t)nt * bytes);
        uint8_t* dst = smem + ring + (size_t)stage * nt * bytes;
        const long long r = (unsigned)row / (unsigned)a.G, g = (unsigned)row % (unsigned)a.G;
        auto copy = [&](int t, const void* p, long long rs, long long gs) {
          bulk_g2s(dst + (size_t)t * bytes, static_cast<const T*>(p) + r * rs + g * gs, bytes, &sh->full[stage]);
        };
        copy(0, a.x, a.x_rs, a.x_gs);
        if (tg) copy(tg, a.gate, a.gate_rs, a.gate_gs);
        if (tr) copy(tr, a.residual, a.res_rs, a.res_gs);
        if (th) copy(th, a.dh, a.dh_rs, a.dh_gs);
        if (ty) copy(ty, a.dy, a.dy_rs, a.dy_gs);
        if (++stage == stages) stage = 0;
      }
      drain_ring(sh->full, stages, loads);
    }
    return;
  }

  if constexpr (SPLIT) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(split_high(MAXT)));

  // Sum over the workers. Successive sums alternate between two buffers, so that a barrier
  // lies between the reads of one and its next writes; slots of absent warps hold zeros.
  int flip = 0;
  auto total = [&](f2 v2) {
    float v, hi;
    unpk(v2, v, hi);
    v += hi;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    float* buf = sh->buf[flip ^= 1];
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    asm volatile("bar.sync 1, %0;" ::"r"(workers) : "memory");
    float s = 0.f;
    for (int w = 0; w < workers / 32; w += 4) {
      const float4 b = *reinterpret_cast<const float4*>(buf + w);
      s += (b.x + b.y) + (b.z + b.w);
    }
    return s;
  };
  // this thread's columns, and their weights: in registers, or where those are short in
  // shared memory before the ring, each thread its own
  const int col0 = threadIdx.x * VEC, cstep = workers * VEC;
  uint4 wreg[KEEP ? 1 : 3][NV];
  const void* const wsrc[3] = {a.w_post, a.w_pre, a.res_scale};
#pragma unroll
  for (int t = 0; t < 3; ++t)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = col0 + i * cstep;
      f2 ones[NP];
#pragma unroll
      for (int e = 0; e < NP; ++e) ones[e] = pk(1.f, 1.f);
      uint4 u = rounded(ones, kind);
      if (c < a.C && wsrc[t]) u = *reinterpret_cast<const uint4*>(static_cast<const T*>(wsrc[t]) + c);
      if constexpr (!KEEP) wreg[t][i] = u;
      else if (c < a.C) *reinterpret_cast<uint4*>(smem + STREAM_HEAD + (size_t)t * bytes + c * sizeof(T)) = u;
    }
  if constexpr (FULL) asm volatile("bar.sync 1, %0;" ::"r"(workers) : "memory");  // the first columns', for all
  enum { POST = 0, PRE = 1, SCALE = 2 };
  auto weight = [&](int t, int i, int c, f2 (&w)[NP]) {
    if constexpr (!KEEP) pairs_of(wreg[t][i], w, kind);
    else pairs_of(*reinterpret_cast<const uint4*>(smem + STREAM_HEAD + (size_t)t * bytes + c * sizeof(T)), w, kind);
  };
  const f2 zero2 = pk(0.f, 0.f);
  f2 sw1[NV][NP], sw2[NV][NP], ssc[NV][NP];  // backward: sums over this CTA's rows
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < NP; ++e) sw1[i][e] = sw2[i][e] = ssc[i][e] = zero2;
  const float invC = 1.f / (float)a.C;
  int stage = 0;
  uint32_t phase = 0;
  float2 st_next = make_float2(1.f, 1.f);
  if (BWD && blockIdx.x < rows) st_next = *reinterpret_cast<const float2*>(a.stats + 2 * (size_t)blockIdx.x);
  for (size_t row = blockIdx.x; row < rows; row += grid) {
    const float2 st = st_next;
    if (BWD && row + grid < rows) st_next = *reinterpret_cast<const float2*>(a.stats + 2 * (row + grid));
    mbar_wait(&sh->full[stage], phase, a.err);
    const uint8_t* in = smem + ring + (size_t)stage * nt * bytes;
    auto fetch = [&](int t, int c, f2 (&v)[NP]) {
      pairs_of(*reinterpret_cast<const uint4*>(in + (size_t)t * bytes + c * sizeof(T)), v, kind);
    };
    auto release = [&]() {  // the warp has read its part of the stage
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&sh->empty[stage]);
      if (++stage == stages) {
        stage = 0;
        phase ^= 1;
      }
    };
    if constexpr (!BWD) {
      float r1 = 1.f, r2 = 1.f;
      if (post) {
        f2 ss = zero2;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int col = col0 + i * cstep, c = FULL && col >= a.C ? 0 : col;
          const bool in_row = col < a.C;
          if (!FULL && !in_row) continue;
          f2 x[NP], part = ss;
          fetch(0, c, x);
#pragma unroll
          for (int e = 0; e < NP; ++e) part = fma2(x[e], x[e], part);
          if (in_row) ss = part;
        }
        r1 = rsqrtf(total(ss) * invC + a.eps);
      }
      const f2 r1p = pk(r1, r1);
      f2 h[NV][NP], hh = zero2;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = col0 + i * cstep, c = FULL && col >= a.C ? 0 : col;
        const bool in_row = col < a.C;
        if (!FULL && !in_row) continue;
        f2 w[NP];
        fetch(0, c, h[i]);
        if (weighed) {
          weight(POST, i, c, w);
#pragma unroll
          for (int e = 0; e < NP; ++e) h[i][e] = mul2(mul2(h[i][e], r1p), w[e]);
        }
        if (gated) {
          fetch(tg, c, w);
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            f2 ac, ad;
            activation2(w[e], a.sigmoid, ac, ad, kind);
            h[i][e] = mul2(h[i][e], ac);
          }
        }
        if (scaled) {
          weight(SCALE, i, c, w);
#pragma unroll
          for (int e = 0; e < NP; ++e) h[i][e] = mul2(h[i][e], w[e]);
        }
        if (tr) {
          fetch(tr, c, w);
#pragma unroll
          for (int e = 0; e < NP; ++e) h[i][e] = add2(h[i][e], w[e]);
        }
        if (in_row) *reinterpret_cast<uint4*>(static_cast<T*>(a.h) + row * a.C + c) = rounded(h[i], kind);
        f2 part = hh;
#pragma unroll
        for (int e = 0; e < NP; ++e) part = fma2(h[i][e], h[i][e], part);
        if (in_row) hh = part;
      }
      release();
      if (pre) {
        r2 = rsqrtf(total(hh) * invC + a.eps);
        const f2 r2p = pk(r2, r2);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int col = col0 + i * cstep, c = FULL && col >= a.C ? 0 : col;
          const bool in_row = col < a.C;
          if (!FULL && !in_row) continue;
          f2 w[NP];
          weight(PRE, i, c, w);
#pragma unroll
          for (int e = 0; e < NP; ++e) w[e] = mul2(mul2(h[i][e], r2p), w[e]);
          if (in_row) *reinterpret_cast<uint4*>(static_cast<T*>(a.y) + row * a.C + c) = rounded(w, kind);
        }
      }
      if (threadIdx.x == 0) *reinterpret_cast<float2*>(a.stats + 2 * row) = make_float2(r1, r2);
    } else {
      const float r1 = post ? st.x : 1.f, r2 = pre ? st.y : 1.f;
      const f2 r1p = pk(r1, r1), r2p = pk(r2, r2);
      f2 h[NV][NP], ac[NV][NP], nd[NV][NP];  // h, act(gate), n act'(gate)
      // act and act' wait in registers or are formed again from the gate
      constexpr bool AGAIN = FULL && GATE && MAXT > 256;
      f2 s2 = zero2;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = col0 + i * cstep, c = FULL && col >= a.C ? 0 : col;
        const bool in_row = col < a.C;
        if (!FULL && !in_row) continue;
        f2 n[NP], w[NP];
        fetch(0, c, n);
        if (weighed) {
          weight(POST, i, c, w);
#pragma unroll
          for (int e = 0; e < NP; ++e) n[e] = mul2(mul2(n[e], r1p), w[e]);
        }
        if (gated) {
          fetch(tg, c, w);
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            f2 ad;
            activation2(w[e], a.sigmoid, ac[i][e], ad, kind);
            if (!AGAIN) nd[i][e] = mul2(n[e], ad);
            n[e] = mul2(n[e], ac[i][e]);  // m
          }
        }
        if (ty) {
          f2 dy[NP];
          if (scaled) {
            weight(SCALE, i, c, w);
#pragma unroll
            for (int e = 0; e < NP; ++e) n[e] = mul2(n[e], w[e]);
          }
          if (tr) {
            fetch(tr, c, w);
#pragma unroll
            for (int e = 0; e < NP; ++e) n[e] = add2(n[e], w[e]);
          }
          fetch(ty, c, dy);
          weight(PRE, i, c, w);
          f2 part = s2;
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            h[i][e] = n[e];
            part = fma2(mul2(dy[e], w[e]), n[e], part);
            sw2[i][e] = fma2(mul2(dy[e], r2p), n[e], sw2[i][e]);
          }
          if (in_row) s2 = part;
        }
      }
      f2 c2 = zero2;
      if (ty) {
        const float t = -total(s2) * invC * r2 * r2 * r2;
        c2 = pk(t, t);
      }
      f2 s1 = zero2;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = col0 + i * cstep, c = FULL && col >= a.C ? 0 : col;
        const bool in_row = col < a.C;
        if (!FULL && !in_row) continue;
        f2 D[NP], x[NP], w[NP];
        if (th) {
          fetch(th, c, D);
        } else {
#pragma unroll
          for (int e = 0; e < NP; ++e) D[e] = zero2;
        }
        if (ty) {
          f2 dy[NP];
          fetch(ty, c, dy);
          weight(PRE, i, c, w);
#pragma unroll
          for (int e = 0; e < NP; ++e) D[e] = fma2(h[i][e], c2, fma2(mul2(dy[e], w[e]), r2p, D[e]));
        }
        if (in_row && (FULL || a.dresidual)) *reinterpret_cast<uint4*>(static_cast<T*>(a.dresidual) + row * a.C + c) = rounded(D, kind);
        fetch(0, c, x);
        if constexpr (AGAIN) {
          f2 gate[NP];
          fetch(tg, c, gate);
          weight(POST, i, c, w);
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            f2 ad;
            activation2(gate[e], a.sigmoid, ac[i][e], ad, kind);
            nd[i][e] = mul2(mul2(mul2(x[e], r1p), w[e]), ad);
          }
        }
        if (scaled) {
          if (weighed) weight(POST, i, c, w);
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            f2 m = weighed ? mul2(mul2(x[e], r1p), w[e]) : x[e];
            if (gated) m = mul2(m, ac[i][e]);
            ssc[i][e] = fma2(D[e], m, ssc[i][e]);
          }
          weight(SCALE, i, c, w);
#pragma unroll
          for (int e = 0; e < NP; ++e) D[e] = mul2(D[e], w[e]);
        }
        if (gated) {
          if (FULL || a.dgate) {
#pragma unroll
            for (int e = 0; e < NP; ++e) w[e] = mul2(D[e], nd[i][e]);
            if (in_row) *reinterpret_cast<uint4*>(static_cast<T*>(a.dgate) + row * a.C + c) = rounded(w, kind);
          }
#pragma unroll
          for (int e = 0; e < NP; ++e) D[e] = mul2(D[e], ac[i][e]);
        }
        if (weighed) {
          weight(POST, i, c, w);
          f2 part = s1;
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            sw1[i][e] = fma2(D[e], mul2(x[e], r1p), sw1[i][e]);
            D[e] = mul2(D[e], w[e]);
            part = fma2(D[e], x[e], part);
          }
          if (in_row) s1 = part;
        }
#pragma unroll
        for (int e = 0; e < NP; ++e) h[i][e] = D[e];  // now u
      }
      f2 c1 = zero2;
      if (post) {
        const float t = -total(s1) * invC * r1 * r1 * r1;
        c1 = pk(t, t);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = col0 + i * cstep, c = FULL && col >= a.C ? 0 : col;
        const bool in_row = col < a.C;
        if (!FULL && !in_row) continue;
        f2 x[NP];
        fetch(0, c, x);
#pragma unroll
        for (int e = 0; e < NP; ++e) x[e] = fma2(x[e], c1, mul2(h[i][e], r1p));
        if (!FULL && !post) {  // 0 x is not 0 when x is not finite (and with FULL, h and all of its row are not)
#pragma unroll
          for (int e = 0; e < NP; ++e) x[e] = h[i][e];
        }
        if (in_row) *reinterpret_cast<uint4*>(static_cast<T*>(a.dx) + row * a.C + c) = rounded(x, kind);
      }
      release();
    }
  }
  if constexpr (BWD) {
    float* part = a.partial + (size_t)blockIdx.x * 3 * a.C;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = col0 + i * cstep;
      if (c >= a.C) continue;
#pragma unroll
      for (int e = 0; e < NP; ++e) {
        if (a.dw_post) *reinterpret_cast<f2*>(part + c + 2 * e) = sw1[i][e];
        if (a.dw_pre) *reinterpret_cast<f2*>(part + a.C + c + 2 * e) = sw2[i][e];
        if (a.dres_scale) *reinterpret_cast<f2*>(part + 2 * a.C + c + 2 * e) = ssc[i][e];
      }
    }
  }
}

// Adds the CTAs' partial rows: 32 columns per CTA, 32 threads per column over the rows (a
// fixed split, so the order of the sums is fixed).
constexpr int WG_LANES = 32;
template <class T>
__global__ void __launch_bounds__(32 * WG_LANES) block_norm_wgrad_kernel(NormArgs a, int parts) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s[WG_LANES][33];
  T* out = static_cast<T*>(blockIdx.y == 0 ? a.dw_post : blockIdx.y == 1 ? a.dw_pre : a.dres_scale);
  if (!out) return;
  const int l = threadIdx.x & 31, k0 = threadIdx.x >> 5, c = blockIdx.x * 32 + l;
  float t = 0.f;
  if (c < a.C) {
#pragma unroll 8
    for (int k = k0; k < parts; k += WG_LANES) t += a.partial[((size_t)k * 3 + blockIdx.y) * a.C + c];
  }
  s[k0][l] = t;
  __syncthreads();
  t = s[l][k0];  // column k0 of the CTA, its 32 partial sums in the lanes of a warp
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
  if (l == 0 && blockIdx.x * 32 + k0 < a.C) out[blockIdx.x * 32 + k0] = from_f32<T>(t);
}

// The fewest CTAs, `per` rows at a time, that take as many turns as `grid` of them: fewer rows
// of partial sums in the same time (1,021 rows of 1,001 fp32: 511 CTAs in place of 912, 22 us
// for both directions in place of 24).
long long even(long long rows, long long per, long long grid) {
  const long long blocks = (rows + per - 1) / per;
  if (grid < 1 || blocks < 1) return grid;
  const long long turns = (blocks + grid - 1) / grid;
  return (blocks + turns - 1) / turns;
}

// CTAs of a kernel that an SM holds at once (asked for once per kernel).
template <class K>
int resident(K kern, int threads) {
  int n = 0;
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, 0) == cudaSuccess && n > 0 ? n : 1;
}

// SUB lanes per row (0: a CTA); per_sm: CTAs of the forward's and the backward's kernel that
// an SM holds.
template <int SUB, class K>
cudaError_t run_rows(K fwd_kernel, K bwd_kernel, const int* per_sm, const NormArgs& a, int threads, bool bwd, int* parts,
                     cudaStream_t s) {
  const long long rows = (long long)a.R * a.G, per = SUB ? SUB_THREADS / (SUB ? SUB : 1) : 1;
  long long grid = (rows + per - 1) / per, most = grid;
  if (SUB) {
    // part-warp rows: one wave of CTAs, each walking its rows with the next one's loads ahead
    // (with a third of a wave more, the B8 T4096 H6 D128 forward took 34 us in place of 31)
    const int nsm = device_sm_count();
    most = (long long)(nsm > 0 ? nsm : 152) * per_sm[bwd];
  }
  if (bwd && most > norm_bwd_parts(a.C)) most = norm_bwd_parts(a.C);
  if (grid > most) grid = most;
  if (bwd) *parts = (int)(grid = even(rows, per, grid));
  prof_mark(bwd ? K_NORM_BWD : K_NORM_FWD, s, true);
  const cudaError_t e = launch_pdl(bwd ? bwd_kernel : fwd_kernel, dim3((unsigned)grid), dim3(threads), 0, s, a);
  prof_mark(bwd ? K_NORM_BWD : K_NORM_FWD, s, false);
  return e;
}
template <class T, int VEC, int NV, int SUB>
cudaError_t run(const NormArgs& a, int threads, bool bwd, int* parts, cudaStream_t s) {
  const auto fwd = block_norm_fwd_kernel<T, VEC, NV, SUB>, bwd_kernel = block_norm_bwd_kernel<T, VEC, NV, SUB>;
  static const int per_sm[2] = {resident(fwd, SUB_THREADS), resident(bwd_kernel, SUB_THREADS)};
  return run_rows<SUB>(fwd, bwd_kernel, per_sm, a, threads, bwd, parts, s);
}
template <class T, int SUB, bool GATE>
cudaError_t run_head(const NormArgs& a, bool bwd, int* parts, cudaStream_t s) {
  const auto fwd = block_norm_head_fwd_kernel<T, SUB, GATE>, bwd_kernel = block_norm_head_bwd_kernel<T, SUB, GATE>;
  static const int per_sm[2] = {resident(fwd, SUB_THREADS), resident(bwd_kernel, SUB_THREADS)};
  return run_rows<SUB>(fwd, bwd_kernel, per_sm, a, SUB_THREADS, bwd, parts, s);
}
template <class T, int SUB>
cudaError_t run_narrow(const NormArgs& a, bool bwd, int* parts, cudaStream_t s) {
  if (a.residual || a.res_scale || a.w_pre) return run<T, 16 / (int)sizeof(T), 1, SUB>(a, SUB_THREADS, bwd, parts, s);
  return a.gate ? run_head<T, SUB, true>(a, bwd, parts, s) : run_head<T, SUB, false>(a, bwd, parts, s);
}

// Wide rows: persistent CTAs, as many per SM as leave each a ring of two stages or more and
// the SM its registers; the ring takes the rest of the shared memory. *fits: whether one
// stage does.
template <class T, int NV, int MAXT, bool BWD, bool SPLIT, bool FULL = false, bool GATE = false>
cudaError_t run_stream(const NormArgs& a, int* parts, bool* fits, cudaStream_t s) {
  const int nsm = device_sm_count();
  if (nsm < 1) return cudaErrorInvalidDevice;
  constexpr int VEC = 16 / (int)sizeof(T), STEP = SPLIT ? 128 : 32, BUDGET = 226 * 1024;
  const int workers = ((a.C / VEC + NV - 1) / NV + STEP - 1) / STEP * STEP;
  const bool pre = a.w_pre != nullptr;
  if constexpr (!FULL) {
    if (a.residual && pre && (!BWD || (a.dh && a.dresidual && (!a.gate || a.dgate))))
      return a.gate ? run_stream<T, NV, MAXT, BWD, SPLIT, true, true>(a, parts, fits, s)
                    : run_stream<T, NV, MAXT, BWD, SPLIT, true, false>(a, parts, fits, s);
  }
  const int tensors = 1 + (a.gate != nullptr) + (a.residual && (!BWD || pre)) + (BWD && a.dh) + (BWD && pre);
  const int row = a.C * (int)sizeof(T), stage = tensors * row, head = STREAM_HEAD + (BWD || (FULL && MAXT == 384) ? 3 * row : 0);
  *fits = head + stage <= BUDGET;
  if (!*fits) return cudaSuccess;
  int per_sm = stream_ctas(NV, MAXT, BWD, FULL) * MAXT / workers;
  if (per_sm < 1) per_sm = 1;
  if (per_sm > NORM_CTAS_PER_SM) per_sm = NORM_CTAS_PER_SM;
  while (per_sm > 1 && BUDGET / per_sm - 1024 < 2 * stage + head) --per_sm;  // 1 KB of each CTA is the system's
  int stages = (BUDGET / per_sm - (per_sm > 1 ? 1024 : 0) - head) / stage;
  if (stages > MAX_STAGES) stages = MAX_STAGES;
  const int bytes = head + stages * stage;
  auto kern = block_norm_stream_kernel<T, NV, MAXT, BWD, SPLIT, FULL, GATE>;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_shared(reinterpret_cast<const void*>(kern), BUDGET, &allowed);
  if (e != cudaSuccess) return e;
  long long grid = (long long)a.R * a.G;
  if (grid > (long long)nsm * per_sm) grid = (long long)nsm * per_sm;
  if (BWD && grid > norm_bwd_parts(a.C)) grid = norm_bwd_parts(a.C);
  if (BWD) *parts = (int)(grid = even((long long)a.R * a.G, 1, grid));
  prof_mark(BWD ? K_NORM_BWD : K_NORM_FWD, s, true);
  e = launch_pdl(kern, dim3((unsigned)grid), dim3(workers + (SPLIT ? 128 : 32)), bytes, s, a, stages);
  prof_mark(BWD ? K_NORM_BWD : K_NORM_FWD, s, false);
  return e;
}

template <class T>
cudaError_t pick(const NormArgs& a, bool vec, bool bwd, int* parts, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  if (vec) {
    const int n = a.C / V;  // vectors of a row
    if (n <= 8) return run_narrow<T, 8>(a, bwd, parts, s);
    if (n <= 16) return run_narrow<T, 16>(a, bwd, parts, s);
    if (n <= 32) return run_narrow<T, 32>(a, bwd, parts, s);
    bool fits = false;
    cudaError_t e = cudaSuccess;
    if (!bwd) {
      if (n <= 768) e = run_stream<T, 2, 384, false, false>(a, parts, &fits, s);
      else if (n <= 1024) e = run_stream<T, 2, 512, false, false>(a, parts, &fits, s);
      else if constexpr (sizeof(T) == 4) e = run_stream<T, 4, 512, false, false>(a, parts, &fits, s);
    } else if constexpr (sizeof(T) == 2) {
      // eight columns' sums per thread, two CTAs per SM, while those fit in the registers
      // (16,000 rows of 2560: 164 us; one CTA 196), or sixteen with the registers split
      if (n <= 256) e = run_stream<T, 1, 256, true, false>(a, parts, &fits, s);
      else if (n <= 384) e = run_stream<T, 1, 384, true, false>(a, parts, &fits, s);
      else if (n <= 768) e = run_stream<T, 2, 384, true, true>(a, parts, &fits, s);
      else e = run_stream<T, 2, 512, true, true>(a, parts, &fits, s);
    } else {
      if (n <= 512) e = run_stream<T, 2, 256, true, false>(a, parts, &fits, s);
      else if (n <= 1024) e = run_stream<T, 2, 512, true, false>(a, parts, &fits, s);
      else if (n <= 1536) e = run_stream<T, 4, 384, true, true>(a, parts, &fits, s);
      else e = run_stream<T, 4, 512, true, true>(a, parts, &fits, s);
    }
    if (e != cudaSuccess || fits) return e;
    // The backward's inputs of one fp32 row above 28 KB, all parts present, exceed the shared memory
    // beside the weights, and such a row goes element by element below: 4,096 rows of 8,192, both
    // directions, 878 us (of 7,168 through the ring: 284 us).
  }
  if (a.C <= 128) return run<T, 1, 4, 32>(a, SUB_THREADS, bwd, parts, s);
  if (a.C <= 2048) return run<T, 1, 4, 0>(a, ((a.C + 3) / 4 + 31) / 32 * 32, bwd, parts, s);
  return run<T, 1, 16, 0>(a, ((a.C + 15) / 16 + 31) / 32 * 32, bwd, parts, s);
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, bool vec, bool bwd, cudaStream_t s) {
  int parts = 0;
  cudaError_t e = a.bf16 ? pick<bf16>(a, vec, bwd, &parts, s) : pick<float>(a, vec, bwd, &parts, s);
  if (e != cudaSuccess || !bwd || !(a.dw_post || a.dw_pre || a.dres_scale)) return e;
  prof_mark(K_NORM_WGRAD, s, true);
  const dim3 grid((a.C + 31) / 32, 3);
  e = a.bf16 ? launch_pdl(block_norm_wgrad_kernel<bf16>, grid, dim3(32 * WG_LANES), 0, s, a, parts)
             : launch_pdl(block_norm_wgrad_kernel<float>, grid, dim3(32 * WG_LANES), 0, s, a, parts);
  prof_mark(K_NORM_WGRAD, s, false);
  return e;
}

}  // namespace gdn
