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
//  * narrow rows (up to 32 vectors of 16 bytes; the norm of a head): a part of a warp per
//    row, reductions by shuffle, the next row's vectors loaded while this one's are used;
//  * wide rows: persistent CTAs, one row at a time with 16 bytes of it per thread, the
//    inputs of the next rows on their way through a ring in shared memory (bulk copies);
//  * rows whose width, strides or pointers do not allow 16-byte accesses: element by
//    element, a CTA (or a warp) per row.
// The sums over rows of the weight gradients stay in the registers of the threads that own
// the columns while a CTA walks its rows (a fixed stride, so the order of the sums is
// fixed); one partial row per CTA goes to the workspace and a second kernel adds them.
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
// act(g) and act'(g). The hardware's approximate exponential and reciprocal are off by
// |g| 2^-24 and 2^-23; with the exact ones the arithmetic, not memory, bounds the kernels.
// silu' = s (1 + g (1 - s)) takes 1 - s as it is (an error of |g| 2^-24 beside the 1);
// the sigmoid's s (1 - s) takes both sides from exp(-|g|), so that 1 - s keeps its relative
// accuracy where s is near 1. Neither form overflows: exp(-g) = inf gives s = 0.
template <int VEC>
__device__ __forceinline__ void activation(const float (&g)[VEC], int sigmoid, float (&a)[VEC], float (&d)[VEC]) {
  constexpr float L2E = 1.4426950408889634f;
  if (!sigmoid) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float s = rcp_approx(1.f + ex2_approx(g[e] * -L2E));
      a[e] = g[e] * s;
      d[e] = s * fmaf(g[e], 1.f - s, 1.f);
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float x = ex2_approx(fabsf(g[e]) * -L2E), big = rcp_approx(1.f + x), small = x * big;
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

// HEAD: only w_post and gate can be present (the norm of a head's output); the rest is
// compiled out, which halves the registers.
template <class T, int VEC, int NV, int SUB, bool HEAD>
__global__ void __launch_bounds__(SUB ? SUB_THREADS : NORM_THREADS_MAX)
    block_norm_fwd_kernel(NormArgs a) {
  pdl_wait();
  __shared__ __align__(16) float buf[2][32];
  const Place<SUB> at;
  const T *wpost = static_cast<const T*>(a.w_post), *rscale = HEAD ? nullptr : static_cast<const T*>(a.res_scale),
          *wpre = HEAD ? nullptr : static_cast<const T*>(a.w_pre), *gate = static_cast<const T*>(a.gate),
          *res = HEAD ? nullptr : static_cast<const T*>(a.residual);
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
        activation<VEC>(w, a.sigmoid, ac, ad);
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

template <class T, int VEC, int NV, int SUB, bool HEAD>
__global__ void __launch_bounds__(SUB ? SUB_THREADS : NORM_THREADS_MAX, HEAD ? 3 : 1)
    block_norm_bwd_kernel(NormArgs a) {
  pdl_wait();
  __shared__ __align__(16) float buf[2][32];
  const Place<SUB> at;
  const T *gate = static_cast<const T*>(a.gate), *res = HEAD ? nullptr : static_cast<const T*>(a.residual),
          *wpost = static_cast<const T*>(a.w_post), *rscale = HEAD ? nullptr : static_cast<const T*>(a.res_scale),
          *wpre = HEAD ? nullptr : static_cast<const T*>(a.w_pre), *dhp = static_cast<const T*>(a.dh),
          *dyp = HEAD ? nullptr : static_cast<const T*>(a.dy);
  T* dres = HEAD ? nullptr : static_cast<T*>(a.dresidual);
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
        activation<VEC>(w, a.sigmoid, ac, ad);
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
      float xv[VEC];
      in.x[i].get(xv);
#pragma unroll
      for (int e = 0; e < VEC; ++e) u[i][e] = r1 * (u[i][e] - xv[e] * c1);
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
  if (!HEAD && a.dw_pre) put(1, sw2);
  if (!HEAD && a.dres_scale) put(2, ssc);
}

// ---------------------------------------------------------------- wide rows
// Sum over the CTA of one value per thread. buf: 32 floats; successive sums alternate between
// two of them, so that a barrier lies between the reads of one and its next writes.
__device__ __forceinline__ float cta_sum(float v, float* buf) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0, nw = blockDim.x >> 5; w < nw; w += 4) {  // unused slots hold zeros
    const float4 b = *reinterpret_cast<const float4*>(buf + w);
    s += (b.x + b.y) + (b.z + b.w);
  }
  return s;
}

constexpr int MAX_STAGES = 8;
struct StreamShared {
  float buf[2][32];
  uint64_t bar[MAX_STAGES];
};
constexpr int STREAM_HEAD = 512;  // bytes of StreamShared before the ring
static_assert(sizeof(StreamShared) <= STREAM_HEAD, "barriers and sums before the ring");

// The ring of a persistent CTA: stage s holds the inputs of one row, `tensors` rows of
// `bytes` each. Thread 0 issues; a stage is filled again after the first barrier of the row
// after the one that used it, which every thread reaches with that one behind it.
struct Ring {
  uint8_t* base;
  uint64_t* bar;
  const char* src[5];
  long long rs[5], gs[5];  // bytes
  int tensors, stages;
  uint32_t bytes;
  __device__ __forceinline__ void load(unsigned row, unsigned G, int stage) const {
    mbar_arrive_expect_tx(&bar[stage], (uint32_t)tensors * bytes);
    const long long r = row / G, g = row % G;
    for (int t = 0; t < tensors; ++t)
      bulk_g2s(base + ((size_t)stage * tensors + t) * bytes, src[t] + r * rs[t] + g * gs[t], bytes, &bar[stage]);
  }
};

template <class T, int NV, int MAXT, bool BWD>
__global__ void __launch_bounds__(MAXT, BWD || MAXT > 384 ? 1 : 2) block_norm_stream_kernel(NormArgs a, int stages) {
  constexpr int VEC = 16 / (int)sizeof(T);
  pdl_wait();
  extern __shared__ __align__(128) uint8_t smem[];
  StreamShared* sh = reinterpret_cast<StreamShared*>(smem);
  const bool post = a.w_post != nullptr, pre = a.w_pre != nullptr, gated = a.gate != nullptr, scaled = a.res_scale != nullptr;
  // which tensor of a stage is which input (x is 0)
  int nt = 1;
  const int tg = gated ? nt++ : 0;
  const int tr = a.residual && (!BWD || pre) ? nt++ : 0;
  const int th = BWD && a.dh ? nt++ : 0;
  const int ty = BWD && pre ? nt++ : 0;
  Ring ring;
  if (threadIdx.x == 0) {
    ring.base = smem + STREAM_HEAD;
    ring.bar = sh->bar;
    ring.tensors = nt;
    ring.stages = stages;
    ring.bytes = (uint32_t)a.C * sizeof(T);
    auto put = [&](int t, const void* p, long long rs, long long gs) {
      ring.src[t] = static_cast<const char*>(p);
      ring.rs[t] = rs * (long long)sizeof(T);
      ring.gs[t] = gs * (long long)sizeof(T);
    };
    put(0, a.x, a.x_rs, a.x_gs);
    if (tg) put(tg, a.gate, a.gate_rs, a.gate_gs);
    if (tr) put(tr, a.residual, a.res_rs, a.res_gs);
    if (th) put(th, a.dh, a.dh_rs, a.dh_gs);
    if (ty) put(ty, a.dy, a.dy_rs, a.dy_gs);
    for (int i = 0; i < stages; ++i) mbar_init(&sh->bar[i], 1);
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < 64; i += blockDim.x) (&sh->buf[0][0])[i] = 0.f;
  __syncthreads();
  const unsigned rows = (unsigned)a.R * (unsigned)a.G, G = a.G, grid = gridDim.x;
  if (threadIdx.x == 0)
    for (int i = 0; i < stages; ++i)
      if (blockIdx.x + (size_t)i * grid < rows) ring.load(blockIdx.x + i * grid, G, i);

  // this thread's columns, and their weights
  const int col0 = threadIdx.x * VEC, cstep = blockDim.x * VEC;
  Raw<T, VEC> w1[NV], w2[NV], ws[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = col0 + i * cstep;
    w1[i].clear(); w2[i].clear(); ws[i].clear();
    if (c < a.C) {
      if (post) w1[i].load(static_cast<const T*>(a.w_post) + c);
      if (pre) w2[i].load(static_cast<const T*>(a.w_pre) + c);
      if (scaled) ws[i].load(static_cast<const T*>(a.res_scale) + c);
    }
  }
  float sw1[NV][VEC], sw2[NV][VEC], ssc[NV][VEC];  // backward: sums over this CTA's rows
  if (BWD) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) sw1[i][e] = sw2[i][e] = ssc[i][e] = 0.f;
  }
  const float invC = 1.f / (float)a.C;
  int stage = 0, flip = 0;
  uint32_t phase = 0;
  bool first = true;
  float2 st_next = make_float2(1.f, 1.f);
  if (BWD && blockIdx.x < rows) st_next = *reinterpret_cast<const float2*>(a.stats + 2 * (size_t)blockIdx.x);
  for (size_t row = blockIdx.x; row < rows; row += grid) {
    const int used = stage;  // this row's stage
    bool refill = !first;
    first = false;
    auto after_barrier = [&]() {
      if (refill && threadIdx.x == 0) {
        const size_t next = row + (size_t)(stages - 1) * grid;
        if (next < rows) ring.load((unsigned)next, G, used == 0 ? stages - 1 : used - 1);
      }
      refill = false;
    };
    const float2 st = st_next;
    if (BWD && row + grid < rows) st_next = *reinterpret_cast<const float2*>(a.stats + 2 * (row + grid));
    // with one stage the row's data cannot be on its way yet; with no sums there is no other barrier
    if (stages == 1 || !(post || pre)) {
      __syncthreads();
      after_barrier();
    }
    mbar_wait(&sh->bar[stage], phase, a.err);
    const uint8_t* in = smem + STREAM_HEAD + (size_t)stage * nt * a.C * sizeof(T);
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
    auto fetch = [&](int t, int c, float (&v)[VEC]) {
      Raw<T, VEC> r;
      r.load(reinterpret_cast<const T*>(in + (size_t)t * a.C * sizeof(T)) + c);
      r.get(v);
    };
    if constexpr (!BWD) {
      float r1 = 1.f, r2 = 1.f;
      if (post) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = col0 + i * cstep;
          if (c >= a.C) continue;
          float x[VEC];
          fetch(0, c, x);
#pragma unroll
          for (int e = 0; e < VEC; ++e) ss = fmaf(x[e], x[e], ss);
        }
        r1 = rsqrtf(cta_sum(ss, sh->buf[flip ^= 1]) * invC + a.eps);
        after_barrier();
      }
      float h[NV][VEC], hh = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = col0 + i * cstep;
        if (c >= a.C) continue;
        float w[VEC];
        fetch(0, c, h[i]);
        if (post) {
          w1[i].get(w);
#pragma unroll
          for (int e = 0; e < VEC; ++e) h[i][e] *= r1 * w[e];
        }
        if (gated) {
          float ac[VEC], ad[VEC];
          fetch(tg, c, w);
          activation<VEC>(w, a.sigmoid, ac, ad);
#pragma unroll
          for (int e = 0; e < VEC; ++e) h[i][e] *= ac[e];
        }
        if (scaled) {
          ws[i].get(w);
#pragma unroll
          for (int e = 0; e < VEC; ++e) h[i][e] *= w[e];
        }
        if (tr) {
          fetch(tr, c, w);
#pragma unroll
          for (int e = 0; e < VEC; ++e) h[i][e] += w[e];
        }
        Raw<T, VEC> raw;
        raw.set(h[i]);
        raw.store(static_cast<T*>(a.h) + row * a.C + c);
#pragma unroll
        for (int e = 0; e < VEC; ++e) hh = fmaf(h[i][e], h[i][e], hh);
      }
      if (pre) {
        r2 = rsqrtf(cta_sum(hh, sh->buf[flip ^= 1]) * invC + a.eps);
        after_barrier();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = col0 + i * cstep;
          if (c >= a.C) continue;
          float w[VEC];
          w2[i].get(w);
#pragma unroll
          for (int e = 0; e < VEC; ++e) w[e] *= h[i][e] * r2;
          Raw<T, VEC> raw;
          raw.set(w);
          raw.store(static_cast<T*>(a.y) + row * a.C + c);
        }
      }
      if (threadIdx.x == 0) *reinterpret_cast<float2*>(a.stats + 2 * row) = make_float2(r1, r2);
    } else {
      const float r1 = post ? st.x : 1.f, r2 = pre ? st.y : 1.f;
      float h[NV][VEC], ac[NV][VEC], nd[NV][VEC];  // h, act(gate), n act'(gate)
      float c2 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = col0 + i * cstep;
        if (c >= a.C) continue;
        float n[VEC], w[VEC];
        fetch(0, c, n);
        if (post) {
          w1[i].get(w);
#pragma unroll
          for (int e = 0; e < VEC; ++e) n[e] *= r1 * w[e];
        }
        if (gated) {
          fetch(tg, c, w);
          activation<VEC>(w, a.sigmoid, ac[i], nd[i]);
#pragma unroll
          for (int e = 0; e < VEC; ++e) nd[i][e] *= n[e];
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            ac[i][e] = 1.f;
            nd[i][e] = 0.f;
          }
        }
        if (ty) {
          float dy[VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e) h[i][e] = n[e] * ac[i][e];
          if (scaled) {
            ws[i].get(w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) h[i][e] *= w[e];
          }
          if (tr) {
            fetch(tr, c, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) h[i][e] += w[e];
          }
          fetch(ty, c, dy);
          w2[i].get(w);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            s2 = fmaf(dy[e] * w[e], h[i][e], s2);
            sw2[i][e] = fmaf(dy[e] * r2, h[i][e], sw2[i][e]);
          }
        }
      }
      if (ty) {
        c2 = cta_sum(s2, sh->buf[flip ^= 1]) * invC * r2 * r2;
        after_barrier();
      }
      float s1 = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = col0 + i * cstep;
        if (c >= a.C) continue;
        float D[VEC], x[VEC], w[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) D[e] = 0.f;
        if (th) fetch(th, c, D);
        if (ty) {
          float dy[VEC];
          fetch(ty, c, dy);
          w2[i].get(w);
#pragma unroll
          for (int e = 0; e < VEC; ++e) D[e] += r2 * (dy[e] * w[e] - h[i][e] * c2);
        }
        Raw<T, VEC> raw;
        if (a.dresidual) {
          raw.set(D);
          raw.store(static_cast<T*>(a.dresidual) + row * a.C + c);
        }
        fetch(0, c, x);
        if (scaled) {
          w1[i].get(w);
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            ssc[i][e] = fmaf(D[e] * ac[i][e], post ? x[e] * (r1 * w[e]) : x[e], ssc[i][e]);
          ws[i].get(w);
#pragma unroll
          for (int e = 0; e < VEC; ++e) D[e] *= w[e];
        }
        if (a.dgate) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) w[e] = D[e] * nd[i][e];
          raw.set(w);
          raw.store(static_cast<T*>(a.dgate) + row * a.C + c);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[i][e] = D[e] * ac[i][e];  // now dn, then u
        if (post) {
          w1[i].get(w);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            sw1[i][e] = fmaf(h[i][e], x[e] * r1, sw1[i][e]);
            h[i][e] *= w[e];
            s1 = fmaf(h[i][e], x[e], s1);
          }
        }
      }
      float c1 = 0.f;
      if (post) {
        c1 = cta_sum(s1, sh->buf[flip ^= 1]) * invC * r1 * r1;
        after_barrier();
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = col0 + i * cstep;
        if (c >= a.C) continue;
        float x[VEC];
        fetch(0, c, x);
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] = r1 * (h[i][e] - x[e] * c1);
        Raw<T, VEC> raw;
        raw.set(x);
        raw.store(static_cast<T*>(a.dx) + row * a.C + c);
      }
    }
  }
  if constexpr (BWD) {
    float* part = a.partial + (size_t)blockIdx.x * 3 * a.C;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = col0 + i * cstep;
      if (c >= a.C) continue;
#pragma unroll
      for (int e = 0; e < VEC; e += 4) {
        if (a.dw_post) *reinterpret_cast<float4*>(part + c + e) = make_float4(sw1[i][e], sw1[i][e + 1], sw1[i][e + 2], sw1[i][e + 3]);
        if (a.dw_pre) *reinterpret_cast<float4*>(part + a.C + c + e) = make_float4(sw2[i][e], sw2[i][e + 1], sw2[i][e + 2], sw2[i][e + 3]);
        if (a.dres_scale) *reinterpret_cast<float4*>(part + 2 * a.C + c + e) = make_float4(ssc[i][e], ssc[i][e + 1], ssc[i][e + 2], ssc[i][e + 3]);
      }
    }
  }
  if (threadIdx.x == 0)  // after a failed wait copies may still be on their way
    for (int i = 0; i < stages; ++i)
      if (blockIdx.x + (size_t)i * grid < rows) mbar_drain(&sh->bar[i], (uint32_t)(((rows - 1 - blockIdx.x) / grid - i) / stages) & 1u);
}

// Adds the CTAs' partial rows: 32 columns per CTA, 32 threads per column over the rows (a
// fixed split, so the order of the sums is fixed).
constexpr int WG_LANES = 32;
template <class T>
__global__ void __launch_bounds__(32 * WG_LANES) block_norm_wgrad_kernel(NormArgs a, int parts) {
  pdl_wait();
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

template <class T, int VEC, int NV, int SUB, bool HEAD>
cudaError_t run(const NormArgs& a, int threads, bool bwd, int* parts, cudaStream_t s) {
  const long long rows = (long long)a.R * a.G, per = SUB ? SUB_THREADS / (SUB ? SUB : 1) : 1;
  long long grid = (rows + per - 1) / per;
  // part-warp rows: resident CTAs only, each walking its rows with the next one's loads ahead
  const long long most = bwd ? norm_bwd_parts(a.C) : SUB ? 152 * NORM_CTAS_PER_SM : grid;
  if (grid > most) grid = most;
  if (bwd) *parts = (int)grid;
  prof_mark(bwd ? K_NORM_BWD : K_NORM_FWD, s, true);
  const cudaError_t e = launch_pdl(bwd ? block_norm_bwd_kernel<T, VEC, NV, SUB, HEAD> : block_norm_fwd_kernel<T, VEC, NV, SUB, HEAD>,
                                   dim3((unsigned)grid), dim3(threads), 0, s, a);
  prof_mark(bwd ? K_NORM_BWD : K_NORM_FWD, s, false);
  return e;
}
template <class T, int SUB>
cudaError_t run_narrow(const NormArgs& a, bool bwd, int* parts, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const bool head = !a.residual && !a.res_scale && !a.w_pre;
  return head ? run<T, V, 1, SUB, true>(a, SUB_THREADS, bwd, parts, s) : run<T, V, 1, SUB, false>(a, SUB_THREADS, bwd, parts, s);
}

// Wide rows: persistent CTAs of `threads`, as many per SM as leave each a ring of two
// stages or more and the SM its registers; the ring takes the rest of the shared memory.
template <class T, int NV, int MAXT, bool BWD>
cudaError_t run_stream(const NormArgs& a, int threads, int* parts, cudaStream_t s) {
  const int nsm = device_sm_count();
  if (nsm < 1) return cudaErrorInvalidDevice;
  const bool pre = a.w_pre != nullptr;
  const int tensors = 1 + (a.gate != nullptr) + (a.residual && (!BWD || pre)) + (BWD && a.dh) + (BWD && pre);
  const int stage = tensors * a.C * (int)sizeof(T), budget = 216 * 1024;
  int per_sm = (BWD ? 384 : 768) / threads;
  if (per_sm < 1) per_sm = 1;
  if (per_sm > NORM_CTAS_PER_SM) per_sm = NORM_CTAS_PER_SM;
  while (per_sm > 1 && budget / per_sm < 2 * stage + STREAM_HEAD) --per_sm;
  int stages = (budget / per_sm - STREAM_HEAD) / stage;
  stages = stages < 1 ? 1 : stages > MAX_STAGES ? MAX_STAGES : stages;
  const int bytes = STREAM_HEAD + stages * stage;
  auto kern = block_norm_stream_kernel<T, NV, MAXT, BWD>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  long long grid = (long long)a.R * a.G;
  if (grid > (long long)nsm * per_sm) grid = (long long)nsm * per_sm;
  if (BWD && grid > norm_bwd_parts(a.C)) grid = norm_bwd_parts(a.C);
  if (BWD) *parts = (int)grid;
  prof_mark(BWD ? K_NORM_BWD : K_NORM_FWD, s, true);
  e = launch_pdl(kern, dim3((unsigned)grid), dim3(threads), bytes, s, a, stages);
  prof_mark(BWD ? K_NORM_BWD : K_NORM_FWD, s, false);
  return e;
}
template <class T, int NV, int MAXT>
cudaError_t run_stream(const NormArgs& a, int threads, bool bwd, int* parts, cudaStream_t s) {
  return bwd ? run_stream<T, NV, MAXT, true>(a, threads, parts, s) : run_stream<T, NV, MAXT, false>(a, threads, parts, s);
}

template <class T>
cudaError_t pick(const NormArgs& a, bool vec, bool bwd, int* parts, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  if (vec) {
    const int n = a.C / V;  // vectors of a row
    if (n <= 8) return run_narrow<T, 8>(a, bwd, parts, s);
    if (n <= 16) return run_narrow<T, 16>(a, bwd, parts, s);
    if (n <= 32) return run_narrow<T, 32>(a, bwd, parts, s);
    // two vectors per thread (four of fp32 in the widest rows): as many columns' sums as the
    // backward's registers hold without spilling at 384 threads
    if (n <= 768) return run_stream<T, 2, 384>(a, ((n + 1) / 2 + 31) / 32 * 32, bwd, parts, s);
    if constexpr (sizeof(T) == 2) {
      return run_stream<T, 2, 512>(a, ((n + 1) / 2 + 31) / 32 * 32, bwd, parts, s);
    } else {
      if (n <= 1536) return run_stream<T, 4, 384>(a, ((n + 3) / 4 + 31) / 32 * 32, bwd, parts, s);
      return run_stream<T, 4, 512>(a, ((n + 3) / 4 + 31) / 32 * 32, bwd, parts, s);
    }
  }
  if (a.C <= 128) return run<T, 1, 4, 32, false>(a, SUB_THREADS, bwd, parts, s);
  if (a.C <= 2048) return run<T, 1, 4, 0, false>(a, ((a.C + 3) / 4 + 31) / 32 * 32, bwd, parts, s);
  return run<T, 1, 16, 0, false>(a, ((a.C + 15) / 16 + 31) / 32 * 32, bwd, parts, s);
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
