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
// A row lies in the registers of a group of threads, so every input is read once. Rows of
// up to 32 vectors of 16 bytes take a part of a warp (reductions by shuffle), longer ones
// a CTA. The sums over rows of the weight gradients stay in the registers of the threads
// that own the columns while a CTA walks its rows (a fixed stride, so the order of the
// sums is fixed); one partial row per CTA goes to the workspace and a second kernel adds
// them.
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

struct Act {
  float a, d;  // act(gate), act'(gate)
};
__device__ __forceinline__ Act activation(float g, int sigmoid) {
  // both sides of the sigmoid from exp(-|g|): neither overflows, and 1 - s keeps its
  // relative accuracy where s is near 1
  const float e = expf(-fabsf(g)), big = 1.f / (1.f + e), small = e * big;
  const float s = g >= 0.f ? big : small, o = g >= 0.f ? small : big;
  Act r;
  if (sigmoid) {
    r.a = s;
    r.d = s * o;
  } else {
    r.a = g * s;
    r.d = s * (1.f + g * o);
  }
  return r;
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

template <class T, int VEC, int NV, int SUB>
__global__ void __launch_bounds__(SUB ? SUB_THREADS : NORM_THREADS_MAX)
    block_norm_fwd_kernel(NormArgs a) {
  pdl_wait();
  __shared__ float buf[2][32];
  const Place<SUB> at;
  const T *x = static_cast<const T*>(a.x), *gate = static_cast<const T*>(a.gate),
          *res = static_cast<const T*>(a.residual), *wpost = static_cast<const T*>(a.w_post),
          *rscale = static_cast<const T*>(a.res_scale), *wpre = static_cast<const T*>(a.w_pre);
  T *hp = static_cast<T*>(a.h), *yp = static_cast<T*>(a.y);
  const float invC = 1.f / (float)a.C;
  // a part-warp's rows end together: the whole warp stays in the loop for the shuffles
  constexpr unsigned PER = SUB ? SUB_THREADS / (SUB ? SUB : 1) : 1;  // rows of a CTA at a time
  const unsigned rows = (unsigned)a.R * (unsigned)a.G, last = (rows + PER - 1) / PER * PER;
  for (unsigned jj = at.row; jj < last; jj += at.step) {
    const bool live = jj < rows;
    const size_t j = jj;
    const long long r = live ? jj / (unsigned)a.G : 0, g = live ? jj % (unsigned)a.G : 0;
    float v[NV][VEC];
    bool on[NV];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (at.lane + i * at.lanes) * VEC;
      on[i] = live && c < a.C;
      Raw<T, VEC> raw;
      if (on[i]) raw.load(x + r * a.x_rs + g * a.x_gs + c);
      else raw.clear();
      raw.get(v[i]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) ss = fmaf(v[i][e], v[i][e], ss);
    }
    float r1 = 1.f;
    if (wpost) r1 = rsqrtf(row_sum<SUB>(ss, buf[0]) * invC + a.eps);
    float hh = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (at.lane + i * at.lanes) * VEC;
      if (!on[i]) continue;
      Raw<T, VEC> raw;
      float w[VEC];
      if (wpost) {
        raw.load(wpost + c);
        raw.get(w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] *= r1 * w[e];
      }
      if (gate) {
        raw.load(gate + r * a.gate_rs + g * a.gate_gs + c);
        raw.get(w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] *= activation(w[e], a.sigmoid).a;
      }
      if (rscale) {
        raw.load(rscale + c);
        raw.get(w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] *= w[e];
      }
      if (res) {
        raw.load(res + r * a.res_rs + g * a.res_gs + c);
        raw.get(w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] += w[e];
      }
      raw.set(v[i]);
      raw.store(hp + j * a.C + c);
#pragma unroll
      for (int e = 0; e < VEC; ++e) hh = fmaf(v[i][e], v[i][e], hh);
    }
    float r2 = 1.f;
    if (wpre) {
      r2 = rsqrtf(row_sum<SUB>(hh, buf[1]) * invC + a.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (at.lane + i * at.lanes) * VEC;
        if (!on[i]) continue;
        Raw<T, VEC> raw;
        float w[VEC];
        raw.load(wpre + c);
        raw.get(w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] *= v[i][e] * r2;
        raw.set(w);
        raw.store(yp + j * a.C + c);
      }
    }
    if (live && at.lane == 0) {
      a.stats[2 * j] = r1;
      a.stats[2 * j + 1] = r2;
    }
    // one sum per row alternates over no second buffer: the next row's write must not
    // overtake this row's reads
    if (!SUB && !(wpost && wpre)) __syncthreads();
  }
}

template <class T, int VEC, int NV, int SUB>
__global__ void __launch_bounds__(SUB ? SUB_THREADS : NORM_THREADS_MAX)
    block_norm_bwd_kernel(NormArgs a) {
  pdl_wait();
  __shared__ float buf[2][32];
  const Place<SUB> at;
  const T *x = static_cast<const T*>(a.x), *gate = static_cast<const T*>(a.gate),
          *res = static_cast<const T*>(a.residual), *wpost = static_cast<const T*>(a.w_post),
          *rscale = static_cast<const T*>(a.res_scale), *wpre = static_cast<const T*>(a.w_pre),
          *dhp = static_cast<const T*>(a.dh), *dyp = static_cast<const T*>(a.dy);
  T *dx = static_cast<T*>(a.dx), *dgate = static_cast<T*>(a.dgate), *dres = static_cast<T*>(a.dresidual);
  const float invC = 1.f / (float)a.C;
  constexpr unsigned PER = SUB ? SUB_THREADS / (SUB ? SUB : 1) : 1;  // rows of a CTA at a time
  const unsigned rows = (unsigned)a.R * (unsigned)a.G, last = (rows + PER - 1) / PER * PER;
  float sw1[NV][VEC], sw2[NV][VEC], ssc[NV][VEC];  // sums of dw_post, dw_pre, dres_scale over this thread's rows
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) sw1[i][e] = sw2[i][e] = ssc[i][e] = 0.f;
  for (unsigned jj = at.row; jj < last; jj += at.step) {
    const bool live = jj < rows;
    const size_t j = jj;
    const long long r = live ? jj / (unsigned)a.G : 0, g = live ? jj % (unsigned)a.G : 0;
    Raw<T, VEC> rx[NV], rg[NV], rr[NV], rh[NV], ry[NV];
    bool on[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (at.lane + i * at.lanes) * VEC;
      on[i] = live && c < a.C;
      rx[i].clear(); rg[i].clear(); rr[i].clear(); rh[i].clear(); ry[i].clear();
      if (on[i]) {
        rx[i].load(x + r * a.x_rs + g * a.x_gs + c);
        if (gate) rg[i].load(gate + r * a.gate_rs + g * a.gate_gs + c);
        if (res && wpre) rr[i].load(res + r * a.res_rs + g * a.res_gs + c);
        if (dhp) rh[i].load(dhp + r * a.dh_rs + g * a.dh_gs + c);
        if (dyp) ry[i].load(dyp + r * a.dy_rs + g * a.dy_gs + c);
      }
    }
    const float r1 = (live && wpost) ? a.stats[2 * j] : 1.f, r2 = (live && wpre) ? a.stats[2 * j + 1] : 1.f;
    // m and h of one vector
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
        rg[i].get(w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const Act q = activation(w[e], a.sigmoid);
          ac[e] = q.a;
          ad[e] = q.d;
        }
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
        if (!on[i]) continue;
        float xv[VEC], n[VEC], ac[VEC], ad[VEC], sc[VEC], rv[VEC], dyv[VEC], w[VEC];
        rx[i].get(xv);
        forward(i, c, xv, n, ac, ad, sc);
        rr[i].get(rv);
        ry[i].get(dyv);
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
      if (!on[i]) continue;
      float xv[VEC], n[VEC], ac[VEC], ad[VEC], sc[VEC], D[VEC];
      rx[i].get(xv);
      forward(i, c, xv, n, ac, ad, sc);
      rh[i].get(D);
      Raw<T, VEC> raw;
      if (dyp) {
        float rv[VEC], dyv[VEC], w[VEC];
        rr[i].get(rv);
        ry[i].get(dyv);
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
        ssc[i][e] = fmaf(D[e], n[e] * ac[e], ssc[i][e]);
        D[e] *= sc[e];
      }
      if (dgate) {
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = D[e] * n[e] * ad[e];
        raw.set(o);
        raw.store(dgate + j * a.C + c);
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
      if (!on[i]) continue;
      float xv[VEC];
      rx[i].get(xv);
#pragma unroll
      for (int e = 0; e < VEC; ++e) u[i][e] = r1 * (u[i][e] - xv[e] * c1);
      Raw<T, VEC> raw;
      raw.set(u[i]);
      raw.store(dx + j * a.C + c);
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
        constexpr int S = SUB ? SUB : 1;
        for (int q = threadIdx.x; q < S * VEC; q += SUB_THREADS) {
          const int c = i * S * VEC + q;
          if (c >= a.C) continue;
          float t = 0.f;
          for (int k = 0; k < SUB_THREADS / S; ++k) t += cols[k * S * VEC + q];
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

// Adds the CTAs' partial rows: 32 columns per CTA, eight threads per column over the rows
// (a fixed split, so the order of the sums is fixed).
template <class T>
__global__ void block_norm_wgrad_kernel(NormArgs a, int parts) {
  pdl_wait();
  __shared__ float s[8][32];
  T* out = static_cast<T*>(blockIdx.y == 0 ? a.dw_post : blockIdx.y == 1 ? a.dw_pre : a.dres_scale);
  if (!out) return;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), k0 = threadIdx.x >> 5;
  float t = 0.f;
  if (c < a.C)
    for (int k = k0; k < parts; k += 8) t += a.partial[((size_t)k * 3 + blockIdx.y) * a.C + c];
  s[k0][threadIdx.x & 31] = t;
  __syncthreads();
  if (k0 == 0 && c < a.C) {
#pragma unroll
    for (int k = 1; k < 8; ++k) t += s[k][threadIdx.x];
    out[c] = from_f32<T>(t);
  }
}

template <class T, int VEC, int NV, int SUB>
cudaError_t run(const NormArgs& a, int threads, bool bwd, int* parts, cudaStream_t s) {
  const long long rows = (long long)a.R * a.G, per = SUB ? SUB_THREADS / (SUB ? SUB : 1) : 1;
  const long long want = (rows + per - 1) / per;
  if (!bwd) {
    prof_mark(K_NORM_FWD, s, true);
    const cudaError_t e = launch_pdl(block_norm_fwd_kernel<T, VEC, NV, SUB>, dim3((unsigned)want), dim3(threads), 0,
                                     s, a);
    prof_mark(K_NORM_FWD, s, false);
    return e;
  }
  *parts = (int)(want < NORM_BWD_PARTS ? want : NORM_BWD_PARTS);
  prof_mark(K_NORM_BWD, s, true);
  const cudaError_t e = launch_pdl(block_norm_bwd_kernel<T, VEC, NV, SUB>, dim3(*parts), dim3(threads), 0, s, a);
  prof_mark(K_NORM_BWD, s, false);
  return e;
}

template <class T>
cudaError_t pick(const NormArgs& a, bool vec, bool bwd, int* parts, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  if (vec) {
    const int n = a.C / V;  // vectors of a row
    if (n <= 8) return run<T, V, 1, 8>(a, SUB_THREADS, bwd, parts, s);
    if (n <= 16) return run<T, V, 1, 16>(a, SUB_THREADS, bwd, parts, s);
    if (n <= 32) return run<T, V, 1, 32>(a, SUB_THREADS, bwd, parts, s);
    if (n <= NORM_THREADS_MAX) return run<T, V, 1, 0>(a, (n + 31) / 32 * 32, bwd, parts, s);
    if (n <= 2 * NORM_THREADS_MAX) return run<T, V, 2, 0>(a, ((n + 1) / 2 + 31) / 32 * 32, bwd, parts, s);
    return run<T, V, 4, 0>(a, ((n + 3) / 4 + 31) / 32 * 32, bwd, parts, s);
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
  e = a.bf16 ? launch_pdl(block_norm_wgrad_kernel<bf16>, grid, dim3(256), 0, s, a, parts)
             : launch_pdl(block_norm_wgrad_kernel<float>, grid, dim3(256), 0, s, a, parts);
  prof_mark(K_NORM_WGRAD, s, false);
  return e;
}

}  // namespace gdn
