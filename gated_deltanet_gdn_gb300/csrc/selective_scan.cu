// Selective state space scan, forward: prompts, training and single tokens (selective_scan.cuh has
// the mathematics, the tiling and the split of long sequences).
#include "selective_scan.cuh"

namespace gdn {
namespace {

constexpr int WARPS = 4;

template <class Shape>
struct WarpShared {
  float delta[Shape::TT * Shape::CW], du[Shape::TT * Shape::CW], y[Shape::TT * Shape::CW];
  float B[Shape::TT * Shape::NS], C[Shape::TT * Shape::NS];
};

// SUM: what a chunk adds to the state (from zeros) and the sum of its delta, no outputs.
// start: [chunks][D][NS] states at the chunks' starts (SUM: written as the chunks' own ends), sums: [chunks][D].
template <class T, int NS, bool WIDE, bool SUM>
__global__ void __launch_bounds__(32 * WARPS) selective_scan_kernel(ScanArgs a, int L, int tiles, long long warps, float* start,
                                                                    float* sums) {
  using Shape = ScanShape<NS>;
  constexpr int S = Shape::S, P = Shape::P, CW = Shape::CW, TT = Shape::TT;
  __shared__ __align__(16) WarpShared<Shape> shared[WARPS];
  pdl_wait();
  pdl_trigger();
  const long long at = (long long)blockIdx.x * WARPS + threadIdx.x / 32;
  if (at >= warps) return;
  WarpShared<Shape>& sm = shared[threadIdx.x / 32];
  const long long number = at / tiles;
  const ScanPlace<Shape> w(a, (int)(at - number * tiles));
  Chunk k;
  if (!packed_chunk(a.q, number, L, &k)) return;
  const int t0 = k.j * L, t1 = k.len - t0 < L ? k.len : t0 + L;
  if (k.b == a.q.B) {  // rows behind the last sequence
    if (!SUM && a.q.zero_tail) {
      const float none[4] = {};
      for (int t = t0 + w.s; t < t1; t += S)
        store_quad<WIDE>(static_cast<T*>(a.y) + (k.first + (long long)t) * a.y_ts + w.c, none, w.n);
    }
    return;
  }
  if (SUM && t1 == k.len) return;  // nothing comes after it

  f32x2 A[2][4], h[2][4];
  load_states<Shape>(a.A, w, A);
  const f32x2 log2e = pack2(LOG2E, LOG2E);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    A[0][i] = mul2(A[0][i], log2e);
    A[1][i] = mul2(A[1][i], log2e);
    h[0][i] = h[1][i] = pack2(0.f, 0.f);
  }
  const int slot = SUM || (start && t1 != k.len) ? -1 : packed_slot(a.q, k.b);
  const long long row = (long long)a.D * NS;
  if constexpr (!SUM) {
    if (start) load_states<Shape>(start + number * row, w, h);
    else if (slot >= 0 && a.h0 && packed_goes_on(a.q, k.b, k.len)) load_states<Shape>(a.h0 + slot * row, w, h);
  }
  float bias[4] = {}, skip[4] = {}, total[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < w.n) {
      if (a.bias) bias[i] = a.bias[w.c + i];
      if (!SUM && a.skip) skip[i] = a.skip[w.c + i];
    }
  float* kept = nullptr;
  if (!SUM && a.kept) kept = a.kept + (packed_number(a.q, k.b, k.first, TT) + t0 / TT) * row;

  ScanRows<Shape, WIDE, T> ru, rd, rz;
  ScanMix<Shape, WIDE, T> rb, rc;
  auto fetch = [&](int t) {
    const int rows = t1 - t;
    ru.load(a.u, k.first + (long long)t, a.u_ts, rows, w);
    rd.load(a.dt, k.first + (long long)t, a.dt_ts, rows, w);
    rb.load(a.B, k.first + (long long)t, a.b_ts, a.b_gs, rows, w);
    if (!SUM) rc.load(a.C, k.first + (long long)t, a.c_ts, a.c_gs, rows, w);
  };
  if (t0 < t1) fetch(t0);
  for (int t = t0; t < t1; t += TT) {
    const int rows = t1 - t < TT ? t1 - t : TT;
    const ScanRows<Shape, WIDE, T> cu = ru;
    __syncwarp();
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int r = p * S + w.s;
      float d[4], u[4];
      quad_floats(rd.v[p], d);
      quad_floats(cu.v[p], u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        d[i] += bias[i];
        if (a.softplus) d[i] = softplus(d[i]);
        if (r >= rows) d[i] = 0.f;  // leaves the state as it is
        if (SUM) total[i] += d[i];
        u[i] *= d[i];
      }
      *reinterpret_cast<float4*>(sm.delta + r * CW + 4 * w.q) = make_float4(d[0], d[1], d[2], d[3]);
      *reinterpret_cast<float4*>(sm.du + r * CW + 4 * w.q) = make_float4(u[0], u[1], u[2], u[3]);
    }
    rb.store(sm.B, w);
    if (!SUM) rc.store(sm.C, w);
    __syncwarp();
    if (kept) {
      store_states<Shape>(kept, w, h);
      kept += row;
    }
    if (!SUM && a.z) rz.load(a.z, k.first + (long long)t, a.z_ts, rows, w);
    if (t + TT < t1) fetch(t + TT);
    for (int r0 = 0; r0 < rows; r0 += 4) {
      float out[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + i;
        const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(sm.delta + r * CW + 4 * w.q);
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(sm.du + r * CW + 4 * w.q);
        const float4 bq = *reinterpret_cast<const float4*>(sm.B + r * NS + 4 * w.s);
        const float bn[4] = {bq.x, bq.y, bq.z, bq.w};
        float cn[4];
        if constexpr (!SUM) {
          const float4 cq = *reinterpret_cast<const float4*>(sm.C + r * NS + 4 * w.s);
          cn[0] = cq.x; cn[1] = cq.y; cn[2] = cq.z; cn[3] = cq.w;
        }
        f32x2 y[2];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const f32x2 b2 = pack2(bn[n], bn[n]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 arg = split2(mul2(e ? d.y : d.x, A[e][n]));
            h[e][n] = fma2(pack2(ex2(arg.x), ex2(arg.y)), h[e][n], mul2(e ? x.y : x.x, b2));
            if constexpr (!SUM) {
              const f32x2 c2 = pack2(cn[n], cn[n]);
              y[e] = n == 0 ? mul2(h[e][n], c2) : fma2(h[e][n], c2, y[e]);
            }
          }
        }
        if constexpr (!SUM) {
          const float2 y0 = split2(y[0]), y1 = split2(y[1]);
          const float v[4] = {y0.x, y0.y, y1.x, y1.y};
          sum_quad<S>(v, w.s, out[i]);
        }
      }
      if constexpr (!SUM) {
#pragma unroll
        for (int i = 0; i < 4; ++i) put_quad<S>(sm.y + (r0 + i) * CW + 4 * w.q, w.s, out[i]);
      }
    }
    if constexpr (!SUM) {
      __syncwarp();
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int r = p * S + w.s;
        if (r >= rows) continue;
        float y[4], u[4];
        ld4(y, sm.y + r * CW + 4 * w.q);
        quad_floats(cu.v[p], u);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = fmaf(skip[i], u[i], y[i]);
        if (a.z) {
          float z[4];
          quad_floats(rz.v[p], z);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] *= z[i] * sigmoid(z[i]);
        }
        store_quad<WIDE>(static_cast<T*>(a.y) + (k.first + (long long)t + r) * a.y_ts + w.c, y, w.n);
      }
    }
  }
  if constexpr (SUM) {
    store_states<Shape>(start + number * row, w, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int d = 1; d < S; d *= 2) total[i] += __shfl_xor_sync(0xffffffffu, total[i], d);
      if (w.s == 0 && i < w.n) sums[number * a.D + w.c + i] = total[i];
    }
  } else if (t1 == k.len && slot >= 0 && a.h_final) {
    store_states<Shape>(a.h_final + slot * row, w, h);
  }
}

// The states at the chunks' starts, in place of what each chunk adds: a thread per sequence, channel and state. The
// loads of CARRY chunks are in flight while the chain waits for them.
constexpr int CARRY = 8;
__global__ void __launch_bounds__(128) selective_scan_carry_kernel(ScanArgs a, int L, float* start, const float* sums) {
  pdl_wait();
  pdl_trigger();
  const long long row = (long long)a.D * a.NS, at = (long long)blockIdx.x * 128 + threadIdx.x;
  if (at >= a.q.B * row) return;
  const int b = (int)(at / row), i = (int)(at - b * row), c = i / a.NS;
  int first, len;
  packed_bounds(a.q, b, &first, &len);
  const int chunks = packed_per(len, L);
  const long long number = packed_number(a.q, b, first, L);
  const int slot = packed_slot(a.q, b);
  const float rate = a.A[i] * LOG2E;
  float h = slot >= 0 && a.h0 && packed_goes_on(a.q, b, len) ? a.h0[slot * row + i] : 0.f;
  float* p = start + number * row + i;
  const float* d = sums + number * a.D + c;
  for (int j = 0; j < chunks; j += CARRY) {
    float own[CARRY], sum[CARRY];
#pragma unroll
    for (int e = 0; e < CARRY; ++e)
      if (j + e < chunks - 1) {
        own[e] = p[(j + e) * row];
        sum[e] = d[(long long)(j + e) * a.D];
      }
#pragma unroll
    for (int e = 0; e < CARRY; ++e) {
      if (j + e < chunks) p[(j + e) * row] = h;
      if (j + e < chunks - 1) h = fmaf(ex2(rate * sum[e]), h, own[e]);
    }
  }
}

int split_of(const ScanArgs& a) { return scan_split(a, ScanCost{90, 130, 60, 12}); }

template <class T, int NS, bool WIDE>
cudaError_t run(const ScanArgs& a, cudaStream_t s) {
  const int L = split_of(a), tiles = scan_tiles(a.D, a.G, NS);
  const long long numbers = packed_numbers(a.q, L), warps = numbers * tiles, blocks = (warps + WARPS - 1) / WARPS;
  if (blocks > 0x7fffffff) return cudaErrorNotSupported;
  const dim3 grid((unsigned)blocks), block(32 * WARPS);
  float* start = nullptr;
  if (L != SCAN_WHOLE) {
    start = static_cast<float*>(a.ws);
    float* sums = start + numbers * a.D * NS;
    prof_mark(K_SCAN_SUM, s, true);
    cudaError_t e = launch_pdl(selective_scan_kernel<T, NS, WIDE, true>, grid, block, 0, s, a, L, tiles, warps, start, sums);
    prof_mark(K_SCAN_SUM, s, false);
    if (e != cudaSuccess) return e;
    const long long threads = (long long)a.q.B * a.D * NS;
    prof_mark(K_SCAN_CARRY, s, true);
    e = launch_pdl(selective_scan_carry_kernel, dim3((unsigned)((threads + 127) / 128)), dim3(128), 0, s, a, L, start,
                   (const float*)sums);
    prof_mark(K_SCAN_CARRY, s, false);
    if (e != cudaSuccess) return e;
  }
  prof_mark(K_SSCAN, s, true);
  const cudaError_t e =
      launch_pdl(selective_scan_kernel<T, NS, WIDE, false>, grid, block, 0, s, a, L, tiles, warps, start, (float*)nullptr);
  prof_mark(K_SSCAN, s, false);
  return e;
}
template <class T, bool WIDE>
cudaError_t pick(const ScanArgs& a, cudaStream_t s) {
  switch (a.NS) {
    case 8: return run<T, 8, WIDE>(a, s);
    case 16: return run<T, 16, WIDE>(a, s);
    case 32: return run<T, 32, WIDE>(a, s);
    default: return run<T, 64, WIDE>(a, s);
  }
}

}  // namespace

size_t selective_scan_workspace(const ScanArgs& a) {
  const int L = split_of(a);
  if (L == SCAN_WHOLE) return 0;
  return (size_t)packed_numbers(a.q, L) * a.D * (a.NS + 1) * sizeof(float);
}
cudaError_t launch_selective_scan(const ScanArgs& a, bool wide, cudaStream_t s) {
  if (a.bf16) return wide ? pick<bf16, true>(a, s) : pick<bf16, false>(a, s);
  return wide ? pick<float, true>(a, s) : pick<float, false>(a, s);
}

}  // namespace gdn
