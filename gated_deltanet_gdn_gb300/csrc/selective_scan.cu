// Selective state space scan, forward: prompts, training and single tokens (selective_scan.cuh has
// the mathematics, the tiling and the split of long sequences).
#include "selective_scan.cuh"

namespace gdn {
namespace {

constexpr int WARPS = 4;
constexpr int STATES = 8, CTAS = 3;  // states of a lane, CTAs of an SM

template <class Shape>
struct WarpShared {
  float delta[Shape::TT * Shape::LD], du[Shape::TT * Shape::LD], y[Shape::TT * Shape::LD];
  float B[Shape::TT * Shape::NS], C[Shape::TT * Shape::NS];
};

// SUM: what a chunk adds to the state (from zeros) and the sum of its delta, no outputs.
// start: [chunks][D][NS] states at the chunks' starts (SUM: written as the chunks' own ends), sums: [chunks][D].
template <class T, int NS, bool WIDE, bool SUM>
__global__ void __launch_bounds__(32 * WARPS, CTAS) selective_scan_kernel(ScanArgs a, int L, int tiles, long long warps, float* start,
                                                                       float* sums) {
  using Shape = ScanShape<NS, STATES>;
  constexpr int S = Shape::S, P = Shape::P, LD = Shape::LD, TT = Shape::TT, N = STATES / 2;
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

  f32x2 A[4][N], h[4][N];
  load_states<Shape>(a.A, w, A);
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      A[c][i] = mul2(A[c][i], both(LOG2E));
      h[c][i] = both(0.f);
    }
  const int slot = SUM || (start && t1 != k.len) ? -1 : packed_slot(a.q, k.b);
  const long long row = (long long)a.D * NS;
  if constexpr (!SUM) {
    if (start) load_states<Shape>(start + number * row, w, h);
    else if (slot >= 0 && a.h0 && packed_goes_on(a.q, k.b, k.len)) load_states<Shape>(a.h0 + slot * row, w, h);
  }
  f32x2 bias[2], skip[2], total[2] = {both(0.f), both(0.f)};
  load_channels(a.bias, w, bias);
  load_channels(SUM ? nullptr : a.skip, w, skip);
  float* kept = nullptr;
  if (!SUM && a.kept) kept = a.kept + (packed_number(a.q, k.b, k.first, SCAN_KEEP) + t0 / SCAN_KEEP) * row;

  ScanRows<Shape, WIDE, T> ru, rd, rz;
  ScanMix<Shape, WIDE, T> rb, rc;
  RowPtr<T> pu, pd, pz, py;
  MixPtr<T> pb, pc;
  {
    const long long row0 = k.first + (long long)t0;
    pu.set(a.u, row0, a.u_ts, w);
    pd.set(a.dt, row0, a.dt_ts, w);
    pb.set(a.B, row0, a.b_ts, a.b_gs, w);
    pc.set(a.C, row0, a.c_ts, a.c_gs, w);
    pz.set(a.z, row0, a.z_ts, w);
    py.set(a.y, row0, a.y_ts, w);
  }
  const bool whole = __all_sync(0xffffffffu, w.n == 4);  // every lane has its channels
  auto fetch = [&](int rows) {
    if (whole && rows >= TT) {
      ru.template load<true>(pu, rows, w);
      rd.template load<true>(pd, rows, w);
      rb.template load<true>(pb, rows, w);
      if (!SUM) rc.template load<true>(pc, rows, w);
    } else {
      ru.template load<false>(pu, rows, w);
      rd.template load<false>(pd, rows, w);
      rb.template load<false>(pb, rows, w);
      if (!SUM) rc.template load<false>(pc, rows, w);
    }
    pu.p += pu.tile;
    pd.p += pd.tile;
    pb.p += pb.tile;
    pc.p += pc.tile;
  };
  fetch(t1 - t0);
  for (int t = t0; t < t1; t += TT) {
    const int rows = t1 - t < TT ? t1 - t : TT;
    const bool full = whole && rows == TT;
    const ScanRows<Shape, WIDE, T> cu = ru;
    __syncwarp();
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int r = p * S + w.s;
      f32x2 d[2], u[2];
      quad_pairs(rd.v[p], d);
      quad_pairs(cu.v[p], u);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        d[i] = add2(d[i], bias[i]);
        if (a.softplus) d[i] = softplus2(d[i]);
        if (!full && r >= rows) d[i] = both(0.f);  // leaves the state as it is
        if (SUM) total[i] = add2(total[i], d[i]);
        u[i] = mul2(u[i], d[i]);
      }
      store_pairs(sm.delta + r * LD + 4 * w.q, d);
      store_pairs(sm.du + r * LD + 4 * w.q, u);
    }
    rb.store(sm.B, w);
    if (!SUM) rc.store(sm.C, w);
    __syncwarp();
    if (kept && (t - t0) % SCAN_KEEP == 0) {
      store_states<Shape>(kept, w, h);
      kept += row;
    }
    if (!SUM) {
      if (full && a.z) rz.template load<true>(pz, rows, w);
      else rz.template load<false>(pz, a.z ? rows : 0, w);
      pz.p += pz.tile;
    }
    fetch(t1 - t - TT);  // no rows are left behind the last tile
    for (int r0 = 0; r0 < rows; r0 += 4) {
      float out[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + i;
        const float4 dq = *reinterpret_cast<const float4*>(sm.delta + r * LD + 4 * w.q);
        const float4 xq = *reinterpret_cast<const float4*>(sm.du + r * LD + 4 * w.q);
        const float d[4] = {dq.x, dq.y, dq.z, dq.w}, x[4] = {xq.x, xq.y, xq.z, xq.w};
        f32x2 b[N], c[N];
        load_row(b, sm.B + r * NS + STATES * w.s);
        if constexpr (!SUM) load_row(c, sm.C + r * NS + STATES * w.s);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f32x2 y;
#pragma unroll
          for (int n = 0; n < N; ++n) {
            h[e][n] = fma2(ex2_2(scale2(d[e], A[e][n])), h[e][n], scale2(x[e], b[n]));
            if constexpr (!SUM) y = n == 0 ? mul2(h[e][n], c[n]) : fma2(h[e][n], c[n], y);
          }
          if constexpr (!SUM) {
            const float2 f = split2(y);
            out[i][e] = f.x + f.y;
          }
        }
        if constexpr (!SUM) sum_quad<S>(out[i], w.s);
      }
      if constexpr (!SUM) {
#pragma unroll
        for (int i = 0; i < 4; ++i) put_quad<S>(sm.y + (r0 + i) * LD + 4 * w.q, w.s, out[i]);
      }
    }
    if constexpr (!SUM) {
      __syncwarp();
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int r = p * S + w.s;
        if (!full && r >= rows) continue;
        f32x2 y[2], u[2];
        load_pairs(y, sm.y + r * LD + 4 * w.q);
        quad_pairs(cu.v[p], u);
#pragma unroll
        for (int i = 0; i < 2; ++i) y[i] = fma2(skip[i], u[i], y[i]);
        if (a.z) {
          f32x2 z[2];
          quad_pairs(rz.v[p], z);
#pragma unroll
          for (int i = 0; i < 2; ++i) y[i] = mul2(y[i], mul2(z[i], sigmoid2(z[i])));
        }
        store_quad<WIDE>(const_cast<T*>(py.p) + p * py.step, y, w.n);
      }
      py.p += py.tile;
    }
  }
  if constexpr (SUM) {
    store_states<Shape>(start + number * row, w, h);
    const float2 s0 = split2(total[0]), s1 = split2(total[1]);
    float v[4] = {s0.x, s0.y, s1.x, s1.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int d = 1; d < S; d *= 2) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
      if (w.s == 0 && i < w.n) sums[number * a.D + w.c + i] = v[i];
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

// One token a sequence, or few: a warp per sequence and 512 / NS channels, nothing staged. Bound by the states, which are
// read and written once (32 sequences x 6144 channels x 16 states: 25 MB), so registers are kept low for
// many warps, and everything a token needs is on its way before the first result is used.
template <class T, int NS, bool WIDE>
__global__ void __launch_bounds__(32 * WARPS, 5) selective_step_kernel(ScanArgs a, int tiles, int warps) {
  using Shape = ScanShape<NS, 4>;
  constexpr int S = Shape::S;
  pdl_wait();
  pdl_trigger();
  const int at = blockIdx.x * WARPS + threadIdx.x / 32;
  if (at >= warps) return;
  const int b = at / tiles;
  const ScanPlace<Shape> w(a, at - b * tiles);
  int first, len;
  packed_bounds(a.q, b, &first, &len);
  if (b == a.q.B) {  // rows behind the last sequence
    const float none[4] = {};
    if (a.q.zero_tail)
      for (int t = w.s; t < len; t += S)
        store_quad<WIDE>(static_cast<T*>(a.y) + (first + (long long)t) * a.y_ts + w.c, none, w.n);
    return;
  }
  const int slot = packed_slot(a.q, b);
  const long long row = (long long)a.D * NS;
  f32x2 A[4][2], h[4][2], bias[2], skip[2];
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e][0] = h[e][1] = both(0.f);
  if (slot >= 0 && a.h0 && packed_goes_on(a.q, b, len)) load_states<Shape>(a.h0 + slot * row, w, h);
  load_states<Shape>(a.A, w, A);
  load_channels(a.bias, w, bias);
  load_channels(a.skip, w, skip);
  for (int t = 0; t < len; ++t) {
    const long long r = first + (long long)t;
    const Quad<T> qu = load_quad<WIDE>(static_cast<const T*>(a.u) + r * a.u_ts + w.c, w.n);
    const Quad<T> qd = load_quad<WIDE>(static_cast<const T*>(a.dt) + r * a.dt_ts + w.c, w.n);
    const Quad<T> qz = load_quad<WIDE>(static_cast<const T*>(a.z) + r * a.z_ts + w.c, a.z ? w.n : 0);
    const Quad<T> qb = load_quad<WIDE>(static_cast<const T*>(a.B) + r * a.b_ts + w.g * a.b_gs + 4 * w.s, 4);
    const Quad<T> qc = load_quad<WIDE>(static_cast<const T*>(a.C) + r * a.c_ts + w.g * a.c_gs + 4 * w.s, 4);
    f32x2 d[2], u[2], bn[2], cn[2];
    float v[4];
    quad_pairs(qd, d);
    quad_pairs(qu, u);
    quad_pairs(qb, bn);
    quad_pairs(qc, cn);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      d[i] = add2(d[i], bias[i]);
      if (a.softplus) d[i] = softplus2(d[i]);
      const float2 df = split2(d[i]), xf = split2(mul2(d[i], u[i]));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int e = 2 * i + j;
        const float de = j ? df.y : df.x, xe = j ? xf.y : xf.x;
#pragma unroll
        for (int n = 0; n < 2; ++n)
          h[e][n] = fma2(ex2_2(mul2(scale2(de, A[e][n]), both(LOG2E))), h[e][n], scale2(xe, bn[n]));
        const float2 f = split2(fma2(h[e][1], cn[1], mul2(h[e][0], cn[0])));
        v[e] = f.x + f.y;
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int f = 1; f < S; f *= 2) v[e] += __shfl_xor_sync(0xffffffffu, v[e], f);
    if (w.s == 0) {
      f32x2 y[2] = {fma2(skip[0], u[0], pack2(v[0], v[1])), fma2(skip[1], u[1], pack2(v[2], v[3]))};
      if (a.z) {
        f32x2 z[2];
        quad_pairs(qz, z);
#pragma unroll
        for (int i = 0; i < 2; ++i) y[i] = mul2(y[i], mul2(z[i], sigmoid2(z[i])));
      }
      store_quad<WIDE>(static_cast<T*>(a.y) + r * a.y_ts + w.c, y, w.n);
    }
  }
  if (slot >= 0 && a.h_final) store_states<Shape>(a.h_final + slot * row, w, h);
}
constexpr int FEW = 2;  // tokens of a sequence up to which the step kernel is taken

int split_of(const ScanArgs& a) { return scan_split(a, ScanCost{190, 260, 120, 4 * CTAS, STATES}); }

template <class T, int NS, bool WIDE>
cudaError_t run(const ScanArgs& a, cudaStream_t s) {
  if (a.max_q <= FEW && !a.kept) {
    const int tiles = scan_tiles(a.D, a.G, NS, 4);
    const long long warps = packed_numbers(a.q, SCAN_WHOLE) * tiles;
    if (warps > 0x7fffffff) return cudaErrorNotSupported;
    prof_mark(K_SSTEP, s, true);
    const cudaError_t e = launch_pdl(selective_step_kernel<T, NS, WIDE>, dim3((unsigned)((warps + WARPS - 1) / WARPS)),
                                     dim3(32 * WARPS), 0, s, a, tiles, (int)warps);
    prof_mark(K_SSTEP, s, false);
    return e;
  }
  const int L = split_of(a), tiles = scan_tiles(a.D, a.G, NS, STATES);
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

size_t selective_scan_workspace(const ScanArgs& a) {  // that of the split, which few tokens never need
  const int L = split_of(a);
  if (L == SCAN_WHOLE) return 0;
  return (size_t)packed_numbers(a.q, L) * a.D * (a.NS + 1) * sizeof(float);
}
cudaError_t launch_selective_scan(const ScanArgs& a, bool wide, cudaStream_t s) {
  if (a.bf16) return wide ? pick<bf16, true>(a, s) : pick<bf16, false>(a, s);
  return wide ? pick<float, true>(a, s) : pick<float, false>(a, s);
}

}  // namespace gdn
