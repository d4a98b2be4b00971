// Selective state space scan, backward (selective_scan.cuh has the tiling and the split).
//
// With dy' = dy silu(z) and the adjoint of the states running backwards,
//   G_t = C_t dy'_t + a_{t+1} G_{t+1},   a_t = exp(delta_t A),   G behind the last token = dh_final
//   dC_t = sum_d dy' h_t          dB_t = sum_d G delta u          d(delta u) = sum_n G B
//   ddelta = sum_n (G a h_{t-1}) A + u d(delta u)                 dA = sum_t (G a h_{t-1}) delta
//   du = delta d(delta u) + dy' skip    ddt = ddelta softplus'    dz = dy (C.h + skip u) silu'(z)    dh0 = a_0 G_0
//
// Bound by arithmetic, 15 products and two exponentials per token, channel and state. The states are not
// kept for every token but for every tile: a tile is scanned forward once from its kept state, which leaves
// the states before each group of GROUP tokens in shared memory, then group by group from the
// last: a group's states and factors are formed again into registers and read by the reverse steps. (All 16
// states of a tile in shared memory instead would leave room for 5 warps an SM.)
//
// A CTA's warps work on the same tokens of neighbouring channels, so their sums over channels (dB, dC) are added in
// shared memory before they leave the SM; what is left per CTA, and the sums over the tokens
// of a chunk (dA, dskip, ddt_bias), are added in a fixed order by a last kernel.
#include "selective_scan.cuh"

namespace gdn {
namespace {

constexpr int WARPS = 4;
constexpr int GROUP = 4;  // tokens whose states are in registers at a time

template <class Shape>
struct BwdShared {
  static constexpr int GROUPS = Shape::TT / GROUP;
  float delta[Shape::TT * Shape::CW];
  float du[Shape::TT * Shape::CW];   // delta u; then d(delta u)
  float dy[Shape::TT * Shape::CW];   // dy'; then C.h
  float gd[Shape::TT * Shape::CW];   // sum_n (G a h) A log2 e
  float B[Shape::TT * Shape::NS], C[Shape::TT * Shape::NS];
  float4 h[GROUPS * 4 * 32];         // states before each group, four vectors a lane
  float mix[Shape::TT * 2 * Shape::NS];  // dB, dC over the warp's channels
};

// Partial sums in the workspace.
struct BwdParts {
  float* start;  // [chunks][D][NS] adjoints entering the chunks from behind (split only)
  float* sums;   // [chunks][D] sums of delta (split only)
  float* mix;    // [CTAs' channel tiles][N][2 NS]
  float* dA;     // [chunks][D][NS]
  float* vec;    // [chunks][2][D]: dskip, ddt_bias
};
struct BwdPlan {
  int L, tiles;      // chunk length; CTAs' channel tiles of all groups
  long long numbers; // chunks
  size_t start, sums, mix, dA, vec, total;  // bytes
};
int cta_tiles(const ScanArgs& a) {
  const int cw = 512 / a.NS * WARPS, dg = a.D / a.G;
  return a.G * ((dg + cw - 1) / cw);
}
BwdPlan plan_of(const ScanArgs& a) {
  BwdPlan p;
  p.L = scan_split(a, ScanCost{330, 420, 75, 8});
  p.tiles = cta_tiles(a);
  p.numbers = packed_numbers(a.q, p.L);
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const size_t states = up((size_t)p.numbers * a.D * a.NS * sizeof(float)), rows = up((size_t)p.numbers * a.D * sizeof(float));
  p.start = 0;
  p.sums = p.start + (p.L == SCAN_WHOLE ? 0 : states);
  p.mix = p.sums + (p.L == SCAN_WHOLE ? 0 : rows);
  p.dA = p.mix + up((size_t)p.tiles * a.q.N * 2 * a.NS * sizeof(float));
  p.vec = p.dA + states;
  p.total = p.vec + 2 * rows;
  return p;
}

template <bool WIDE, class T>
__device__ __forceinline__ Quad<T> row_quad(const void* base, long long row, long long ts, int c, int n) {
  return load_quad<WIDE>(static_cast<const T*>(base) + row * ts + c, n);
}

// What a chunk hands to the one before it when nothing comes in from behind, and the sum of its delta.
template <class T, int NS, bool WIDE>
__global__ void __launch_bounds__(32 * WARPS) selective_scan_bwd_sum_kernel(ScanArgs a, int L, int tiles, long long warps, float* start,
                                                                            float* sums) {
  using Shape = ScanShape<NS>;
  constexpr int S = Shape::S, P = Shape::P, CW = Shape::CW, TT = Shape::TT;
  struct Mine {
    float delta[TT * CW], dy[TT * CW], C[TT * NS];
  };
  __shared__ __align__(16) Mine shared[WARPS];
  pdl_wait();
  pdl_trigger();
  const long long at = (long long)blockIdx.x * WARPS + threadIdx.x / 32;
  if (at >= warps) return;
  Mine& sm = shared[threadIdx.x / 32];
  const long long number = at / tiles;
  const ScanPlace<Shape> w(a, (int)(at - number * tiles));
  Chunk k;
  if (!packed_chunk(a.q, number, L, &k) || k.b == a.q.B || k.j == 0) return;
  const int t0 = k.j * L, t1 = k.len - t0 < L ? k.len : t0 + L;
  f32x2 A[2][4], G[2][4];
  load_states<Shape>(a.A, w, A);
  const f32x2 log2e = pack2(LOG2E, LOG2E);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    A[0][i] = mul2(A[0][i], log2e);
    A[1][i] = mul2(A[1][i], log2e);
    G[0][i] = G[1][i] = pack2(0.f, 0.f);
  }
  float bias[4] = {}, total[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (a.bias && i < w.n) bias[i] = a.bias[w.c + i];
  ScanRows<Shape, WIDE, T> rd, ry, rz;
  ScanMix<Shape, WIDE, T> rc;
  auto fetch = [&](int t) {
    const int rows = t1 - t;
    rd.load(a.dt, k.first + (long long)t, a.dt_ts, rows, w);
    ry.load(a.dy, k.first + (long long)t, a.dy_ts, rows, w);
    if (a.z) rz.load(a.z, k.first + (long long)t, a.z_ts, rows, w);
    rc.load(a.C, k.first + (long long)t, a.c_ts, a.c_gs, rows, w);
  };
  const int last = t0 + (t1 - 1 - t0) / TT * TT;
  fetch(last);
  for (int t = last; t >= t0; t -= TT) {
    const int rows = t1 - t < TT ? t1 - t : TT;
    __syncwarp();
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int r = p * S + w.s;
      float d[4], y[4], z[4];
      quad_floats(rd.v[p], d);
      quad_floats(ry.v[p], y);
      if (a.z) quad_floats(rz.v[p], z);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        d[i] += bias[i];
        if (a.softplus) d[i] = softplus(d[i]);
        if (r >= rows) d[i] = 0.f;
        total[i] += d[i];
        if (a.z) y[i] *= z[i] * sigmoid(z[i]);
      }
      *reinterpret_cast<float4*>(sm.delta + r * CW + 4 * w.q) = make_float4(d[0], d[1], d[2], d[3]);
      *reinterpret_cast<float4*>(sm.dy + r * CW + 4 * w.q) = make_float4(y[0], y[1], y[2], y[3]);
    }
    rc.store(sm.C, w);
    __syncwarp();
    if (t > t0) fetch(t - TT);
#pragma unroll 4
    for (int r = TT - 1; r >= 0; --r) {
      const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(sm.delta + r * CW + 4 * w.q);
      const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(sm.dy + r * CW + 4 * w.q);
      const float4 cq = *reinterpret_cast<const float4*>(sm.C + r * NS + 4 * w.s);
      const float cn[4] = {cq.x, cq.y, cq.z, cq.w};
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const f32x2 c2 = pack2(cn[n], cn[n]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 arg = split2(mul2(e ? d.y : d.x, A[e][n]));
          G[e][n] = mul2(pack2(ex2(arg.x), ex2(arg.y)), fma2(c2, e ? y.y : y.x, G[e][n]));
        }
      }
    }
  }
  store_states<Shape>(start + number * a.D * NS, w, G);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int d = 1; d < S; d *= 2) total[i] += __shfl_xor_sync(0xffffffffu, total[i], d);
    if (w.s == 0 && i < w.n) sums[number * a.D + w.c + i] = total[i];
  }
}

// The adjoints that enter the chunks from behind, in place of what each hands on.
constexpr int CARRY = 8;
__global__ void __launch_bounds__(128) selective_scan_bwd_carry_kernel(ScanArgs a, int L, float* start, const float* sums) {
  pdl_wait();
  pdl_trigger();
  const long long row = (long long)a.D * a.NS, at = (long long)blockIdx.x * 128 + threadIdx.x;
  if (at >= a.q.B * row) return;
  const int b = (int)(at / row), i = (int)(at - b * row), c = i / a.NS;
  int first, len;
  packed_bounds(a.q, b, &first, &len);
  const int chunks = packed_per(len, L);
  const long long number = packed_number(a.q, b, first, L);
  const float rate = a.A[i] * LOG2E;
  float g = a.dh_final ? a.dh_final[at] : 0.f;
  float* p = start + number * row + i;
  const float* d = sums + number * a.D + c;
  for (int j = chunks - 1; j >= 0; j -= CARRY) {
    float own[CARRY], sum[CARRY];
#pragma unroll
    for (int e = 0; e < CARRY; ++e)
      if (j - e > 0) {
        own[e] = p[(j - e) * row];
        sum[e] = d[(long long)(j - e) * a.D];
      }
#pragma unroll
    for (int e = 0; e < CARRY; ++e) {
      if (j - e >= 0) p[(j - e) * row] = g;
      if (j - e > 0) g = fmaf(ex2(rate * sum[e]), g, own[e]);
    }
  }
}

// Sums of eight values (dB and dC of the lane's states) over the warp's quads. A lane ends with 8 / min(Q, 8) of
// them, from `base` on.
template <class Shape>
__device__ __forceinline__ int sum_mix(float (&v)[8], int q) {
  int base = 0;
#pragma unroll
  for (int lvl = 0, n = 8; (1 << lvl) < Shape::Q; ++lvl) {
    const int far = Shape::S << lvl;
    if (n > 1) {
      n /= 2;
      const bool up = (q >> lvl) & 1;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float keep = up ? v[i + n] : v[i], send = up ? v[i] : v[i + n];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, far);
      }
      base += up ? n : 0;
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], far);
    }
  }
  return base;
}

template <class T, int NS, bool WIDE>
__global__ void __launch_bounds__(32 * WARPS) selective_scan_bwd_kernel(ScanArgs a, int L, int tiles, BwdParts parts) {
  using Shape = ScanShape<NS>;
  using Shared = BwdShared<Shape>;
  constexpr int S = Shape::S, P = Shape::P, CW = Shape::CW, TT = Shape::TT, Q = Shape::Q;
  constexpr int LEFT = 8 / (Q < 8 ? Q : 8);  // sums over quads that a lane ends with
  extern __shared__ __align__(16) unsigned char raw_shared[];
  Shared* const all = reinterpret_cast<Shared*>(raw_shared);
  pdl_wait();
  pdl_trigger();
  Shared& sm = all[threadIdx.x / 32];
  const long long number = blockIdx.x / tiles;
  const int tile = (int)(blockIdx.x - number * tiles);
  // the CTA's channels belong to one group; a warp of its end may have none
  const int dg = a.D / a.G, per = (dg + CW * WARPS - 1) / (CW * WARPS), g = tile / per;
  ScanPlace<Shape> w(a, 0);
  w.g = g;
  w.c = g * dg + ((tile - g * per) * WARPS + (int)threadIdx.x / 32) * CW + 4 * w.q;
  w.n = min(max((g + 1) * dg - w.c, 0), 4);
  const long long row = (long long)a.D * NS;
  f32x2 A[2][4], G[2][4], dA[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dA[0][i] = dA[1][i] = G[0][i] = G[1][i] = pack2(0.f, 0.f);
  float dskip[4] = {}, dbias[4] = {};

  Chunk k;
  const bool used = packed_chunk(a.q, number, L, &k);
  if (used && k.b == a.q.B) {  // rows behind the last sequence
    const int t0 = k.j * L, t1 = k.len - t0 < L ? k.len : t0 + L;
    const float none[4] = {};
    for (int t = t0 + w.s; t < t1; t += S) {
      const long long to = (k.first + (long long)t) * a.D + w.c;
      store_quad<WIDE>(static_cast<T*>(a.du) + to, none, w.n);
      store_quad<WIDE>(static_cast<T*>(a.ddt) + to, none, w.n);
      if (a.dz) store_quad<WIDE>(static_cast<T*>(a.dz) + to, none, w.n);
    }
  } else if (used) {
    const int t0 = k.j * L, t1 = k.len - t0 < L ? k.len : t0 + L;
    load_states<Shape>(a.A, w, A);
    const f32x2 log2e = pack2(LOG2E, LOG2E);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      A[0][i] = mul2(A[0][i], log2e);
      A[1][i] = mul2(A[1][i], log2e);
    }
    if (parts.start) load_states<Shape>(parts.start + number * row, w, G);
    else if (a.dh_final) load_states<Shape>(a.dh_final + k.b * row, w, G);
    float bias[4] = {}, skip[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < w.n) {
        if (a.bias) bias[i] = a.bias[w.c + i];
        if (a.skip) skip[i] = a.skip[w.c + i];
      }
    const float* kept = a.kept + packed_number(a.q, k.b, k.first, TT) * row;
    const int last = t1 > t0 ? t0 + (t1 - 1 - t0) / TT * TT : t0 - TT;
    for (int t = last; t >= t0; t -= TT) {
      const int rows = t1 - t < TT ? t1 - t : TT;
      const long long row0 = k.first + (long long)t;
      {
        ScanRows<Shape, WIDE, T> ru, rd, ry, rz;
        ScanMix<Shape, WIDE, T> rb, rc;
        ru.load(a.u, row0, a.u_ts, rows, w);
        rd.load(a.dt, row0, a.dt_ts, rows, w);
        ry.load(a.dy, row0, a.dy_ts, rows, w);
        if (a.z) rz.load(a.z, row0, a.z_ts, rows, w);
        rb.load(a.B, row0, a.b_ts, a.b_gs, rows, w);
        rc.load(a.C, row0, a.c_ts, a.c_gs, rows, w);
        __syncwarp();
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const int r = p * S + w.s;
          float d[4], u[4], y[4], z[4];
          quad_floats(rd.v[p], d);
          quad_floats(ru.v[p], u);
          quad_floats(ry.v[p], y);
          if (a.z) quad_floats(rz.v[p], z);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            d[i] += bias[i];
            if (a.softplus) d[i] = softplus(d[i]);
            if (r >= rows) d[i] = 0.f;  // a step that changes nothing
            u[i] *= d[i];
            if (a.z) y[i] *= z[i] * sigmoid(z[i]);
          }
          *reinterpret_cast<float4*>(sm.delta + r * CW + 4 * w.q) = make_float4(d[0], d[1], d[2], d[3]);
          *reinterpret_cast<float4*>(sm.du + r * CW + 4 * w.q) = make_float4(u[0], u[1], u[2], u[3]);
          *reinterpret_cast<float4*>(sm.dy + r * CW + 4 * w.q) = make_float4(y[0], y[1], y[2], y[3]);
        }
        rb.store(sm.B, w);
        rc.store(sm.C, w);
        __syncwarp();
      }
      const int groups = (rows + GROUP - 1) / GROUP;
      f32x2 h[2][4];
      load_states<Shape>(kept + (long long)(t / TT) * row, w, h);
      auto keep = [&](int i) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            ulonglong2 v;
            v.x = h[e][2 * n];
            v.y = h[e][2 * n + 1];
            reinterpret_cast<ulonglong2*>(sm.h)[(i * 4 + 2 * e + n) * 32 + w.lane] = v;
          }
      };
      for (int i = 0; i + 1 < groups; ++i) {
        keep(i);
#pragma unroll
        for (int r0 = 0; r0 < GROUP; ++r0) {
          const int r = i * GROUP + r0;
          const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(sm.delta + r * CW + 4 * w.q);
          const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(sm.du + r * CW + 4 * w.q);
          const float4 bq = *reinterpret_cast<const float4*>(sm.B + r * NS + 4 * w.s);
          const float bn[4] = {bq.x, bq.y, bq.z, bq.w};
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const f32x2 b2 = pack2(bn[n], bn[n]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 arg = split2(mul2(e ? d.y : d.x, A[e][n]));
              h[e][n] = fma2(pack2(ex2(arg.x), ex2(arg.y)), h[e][n], mul2(e ? x.y : x.x, b2));
            }
          }
        }
      }
      for (int i = groups - 1; i >= 0; --i) {
        f32x2 hs[GROUP + 1][2][4], f[GROUP][2][4];  // states before and after the tokens, factors
        if (i == groups - 1) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < 4; ++n) hs[0][e][n] = h[e][n];
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const ulonglong2 v = reinterpret_cast<const ulonglong2*>(sm.h)[(i * 4 + 2 * e + n) * 32 + w.lane];
              hs[0][e][2 * n] = v.x;
              hs[0][e][2 * n + 1] = v.y;
            }
        }
#pragma unroll
        for (int r0 = 0; r0 < GROUP; ++r0) {
          const int r = i * GROUP + r0;
          const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(sm.delta + r * CW + 4 * w.q);
          const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(sm.du + r * CW + 4 * w.q);
          const float4 bq = *reinterpret_cast<const float4*>(sm.B + r * NS + 4 * w.s);
          const float bn[4] = {bq.x, bq.y, bq.z, bq.w};
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const f32x2 b2 = pack2(bn[n], bn[n]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 arg = split2(mul2(e ? d.y : d.x, A[e][n]));
              f[r0][e][n] = pack2(ex2(arg.x), ex2(arg.y));
              hs[r0 + 1][e][n] = fma2(f[r0][e][n], hs[r0][e][n], mul2(e ? x.y : x.x, b2));
            }
          }
        }
        float own[GROUP][3][2];
#pragma unroll
        for (int r0 = GROUP - 1; r0 >= 0; --r0) {
          const int r = i * GROUP + r0;
          const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(sm.delta + r * CW + 4 * w.q);
          const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(sm.du + r * CW + 4 * w.q);
          const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(sm.dy + r * CW + 4 * w.q);
          const float4 bq = *reinterpret_cast<const float4*>(sm.B + r * NS + 4 * w.s);
          const float4 cq = *reinterpret_cast<const float4*>(sm.C + r * NS + 4 * w.s);
          const float bn[4] = {bq.x, bq.y, bq.z, bq.w}, cn[4] = {cq.x, cq.y, cq.z, cq.w};
          f32x2 gx[2], gd[2], ch[2];
          float mix[8];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const f32x2 b2 = pack2(bn[n], bn[n]), c2 = pack2(cn[n], cn[n]);
            f32x2 db, dc;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              G[e][n] = fma2(c2, e ? y.y : y.x, G[e][n]);
              dc = e ? fma2(hs[r0 + 1][e][n], y.y, dc) : mul2(hs[r0 + 1][e][n], y.x);
              db = e ? fma2(G[e][n], x.y, db) : mul2(G[e][n], x.x);
              gx[e] = n ? fma2(G[e][n], b2, gx[e]) : mul2(G[e][n], b2);
              ch[e] = n ? fma2(hs[r0 + 1][e][n], c2, ch[e]) : mul2(hs[r0 + 1][e][n], c2);
              G[e][n] = mul2(G[e][n], f[r0][e][n]);
              const f32x2 ga = mul2(G[e][n], hs[r0][e][n]);
              gd[e] = n ? fma2(ga, A[e][n], gd[e]) : mul2(ga, A[e][n]);
              dA[e][n] = fma2(ga, e ? d.y : d.x, dA[e][n]);
            }
            const float2 b = split2(db), c = split2(dc);
            mix[n] = b.x + b.y;
            mix[4 + n] = c.x + c.y;
          }
          const f32x2* const sums[3] = {gx, gd, ch};
#pragma unroll
          for (int m = 0; m < 3; ++m) {
            if (m == 2 && !a.z) break;
            const float2 v0 = split2(sums[m][0]), v1 = split2(sums[m][1]);
            const float v[4] = {v0.x, v0.y, v1.x, v1.y};
            sum_quad<S>(v, w.s, own[r0][m]);
          }
          const int base = sum_mix<Shape>(mix, w.q);
          if (Q <= 8 || w.q < 8) {
#pragma unroll
            for (int m = 0; m < LEFT; ++m) {
              const int v = base + m;
              sm.mix[r * 2 * NS + (v < 4 ? 0 : NS - 4) + 4 * w.s + v] = mix[m];
            }
          }
        }
        __syncwarp();
#pragma unroll
        for (int r0 = 0; r0 < GROUP; ++r0) {
          const int to = (i * GROUP + r0) * CW + 4 * w.q;
          put_quad<S>(sm.du + to, w.s, own[r0][0]);
          put_quad<S>(sm.gd + to, w.s, own[r0][1]);
          if (a.z) put_quad<S>(sm.dy + to, w.s, own[r0][2]);
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < rows * 2 * NS; i += 32 * WARPS) {
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < WARPS; ++j) v += all[j].mix[i];
        parts.mix[((long long)tile * a.q.N + row0) * 2 * NS + i] = v;
      }
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int r = p * S + w.s;
        if (r >= rows) continue;
        float d[4], u[4], y[4], raw[4], gx[4], gd[4], du[4], ddt[4];
        quad_floats(row_quad<WIDE, T>(a.u, row0 + r, a.u_ts, w.c, w.n), u);
        quad_floats(row_quad<WIDE, T>(a.dt, row0 + r, a.dt_ts, w.c, w.n), raw);
        quad_floats(row_quad<WIDE, T>(a.dy, row0 + r, a.dy_ts, w.c, w.n), y);
        ld4(d, sm.delta + r * CW + 4 * w.q);
        ld4(gx, sm.du + r * CW + 4 * w.q);
        ld4(gd, sm.gd + r * CW + 4 * w.q);
        const long long to = (row0 + r) * a.D + w.c;
        if (a.z) {
          float z[4], ch[4], dz[4];
          quad_floats(row_quad<WIDE, T>(a.z, row0 + r, a.z_ts, w.c, w.n), z);
          ld4(ch, sm.dy + r * CW + 4 * w.q);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float s = sigmoid(z[e]);
            dz[e] = y[e] * fmaf(skip[e], u[e], ch[e]) * fmaf(z[e] * s, 1.f - s, s);
            y[e] *= z[e] * s;
          }
          store_quad<WIDE>(static_cast<T*>(a.dz) + to, dz, w.n);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          du[e] = fmaf(gx[e], d[e], y[e] * skip[e]);
          ddt[e] = fmaf(gx[e], u[e], gd[e] * 0.693147180559945309f);
          if (a.softplus) ddt[e] *= sigmoid(raw[e] + bias[e]);
          dskip[e] = fmaf(y[e], u[e], dskip[e]);
          dbias[e] += ddt[e];
        }
        store_quad<WIDE>(static_cast<T*>(a.du) + to, du, w.n);
        store_quad<WIDE>(static_cast<T*>(a.ddt) + to, ddt, w.n);
      }
      __syncthreads();  // the sums over channels have been read
    }
    if (k.j == 0 && a.dh0) store_states<Shape>(a.dh0 + k.b * row, w, G);
  }
  store_states<Shape>(parts.dA + number * row, w, dA);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int d = 1; d < S; d *= 2) {
      dskip[i] += __shfl_xor_sync(0xffffffffu, dskip[i], d);
      dbias[i] += __shfl_xor_sync(0xffffffffu, dbias[i], d);
    }
    if (w.s == 0 && i < w.n) {
      parts.vec[(2 * number) * a.D + w.c + i] = dskip[i];
      parts.vec[(2 * number + 1) * a.D + w.c + i] = dbias[i];
    }
  }
}

// Adds the partial sums: CTAs of 256 threads take dB and dC (a thread four values of a row), then 32 columns of dA, dskip
// and ddt_bias each (8 warps over every eighth chunk).
template <class T>
__global__ void __launch_bounds__(256) selective_scan_join_kernel(ScanArgs a, BwdParts parts, int tiles, long long numbers,
                                                                  int mix_blocks) {
  __shared__ float sum[8][32];
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x < mix_blocks) {
    const int vecs = a.NS / 2;  // of a row and group, dB and dC
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, per = (long long)a.G * vecs, r = i / per;
    if (r >= a.q.N) return;
    const int left = (int)(i - r * per), g = left / vecs, n = left % vecs * 4, each = tiles / a.G;
    const int end = packed_start(a.q, a.q.B);
    float v[4] = {};
    if (!a.q.cu || r < end) {
      const float* p = parts.mix + ((long long)g * each * a.q.N + r) * 2 * a.NS + n;
#pragma unroll 4
      for (int t = 0; t < each; ++t) {
        float x[4];
        ld4(x, p + (long long)t * a.q.N * 2 * a.NS);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += x[e];
      }
    }
    T* const out = static_cast<T*>(n < a.NS ? a.dB : a.dC) + (r * a.G + g) * a.NS + (n < a.NS ? n : n - a.NS);
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = from_f32<T>(v[e]);
    return;
  }
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const long long row = (long long)a.D * a.NS, col = ((long long)blockIdx.x - mix_blocks) * 32 + lane;
  const bool in = col < row + 2 * a.D;
  float s = 0.f;
  if (in) {
    const float* p = col < row ? parts.dA + col : parts.vec + (col - row);
    const long long step = col < row ? row : 2 * (long long)a.D;
#pragma unroll 4
    for (long long j = warp; j < numbers; j += 8) s += p[j * step];
  }
  sum[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || !in) return;
  for (int i = 1; i < 8; ++i) s += sum[i][lane];
  if (col < row) a.dA[col] = s;
  else if (col < row + a.D) {
    if (a.dskip) a.dskip[col - row] = s;
  } else if (a.dbias) {
    a.dbias[col - row - a.D] = s;
  }
}

template <class T, int NS, bool WIDE>
cudaError_t run(const ScanArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const BwdPlan p = plan_of(a);
  char* const ws = static_cast<char*>(a.ws);
  BwdParts parts;
  parts.start = p.L == SCAN_WHOLE ? nullptr : reinterpret_cast<float*>(ws + p.start);
  parts.sums = reinterpret_cast<float*>(ws + p.sums);
  parts.mix = reinterpret_cast<float*>(ws + p.mix);
  parts.dA = reinterpret_cast<float*>(ws + p.dA);
  parts.vec = reinterpret_cast<float*>(ws + p.vec);
  const long long blocks = p.numbers * p.tiles;
  const long long per = (long long)a.G * (a.NS / 2), mix_blocks = (a.q.N * per + 255) / 256;
  const long long join_blocks = mix_blocks + ((long long)a.D * (a.NS + 2) + 31) / 32;
  if (blocks > 0x7fffffff || join_blocks > 0x7fffffff) return cudaErrorNotSupported;
  cudaError_t e;
  if (parts.start) {
    const int tiles = scan_tiles(a.D, a.G, NS);
    const long long warps = p.numbers * tiles, sum_blocks = (warps + WARPS - 1) / WARPS;
    if (sum_blocks > 0x7fffffff) return cudaErrorNotSupported;
    prof_mark(K_SSCAN_RSUM, s, true);
    e = launch_pdl(selective_scan_bwd_sum_kernel<T, NS, WIDE>, dim3((unsigned)sum_blocks), dim3(32 * WARPS), 0, s, a, p.L, tiles,
                   warps, parts.start, parts.sums);
    prof_mark(K_SSCAN_RSUM, s, false);
    if (e != cudaSuccess) return e;
    const long long threads = (long long)a.q.B * a.D * NS;
    prof_mark(K_SCAN_CARRY, s, true);
    e = launch_pdl(selective_scan_bwd_carry_kernel, dim3((unsigned)((threads + 127) / 128)), dim3(128), 0, s, a, p.L, parts.start,
                   (const float*)parts.sums);
    prof_mark(K_SCAN_CARRY, s, false);
    if (e != cudaSuccess) return e;
  }
  const int bytes = (int)sizeof(BwdShared<ScanShape<NS>>) * WARPS;
  e = allow_shared(reinterpret_cast<const void*>(selective_scan_bwd_kernel<T, NS, WIDE>), bytes, &done);
  if (e != cudaSuccess) return e;
  prof_mark(K_SSCAN_BWD, s, true);
  e = launch_pdl(selective_scan_bwd_kernel<T, NS, WIDE>, dim3((unsigned)blocks), dim3(32 * WARPS), bytes, s, a, p.L, p.tiles, parts);
  prof_mark(K_SSCAN_BWD, s, false);
  if (e != cudaSuccess) return e;
  prof_mark(K_SSCAN_JOIN, s, true);
  e = launch_pdl(selective_scan_join_kernel<T>, dim3((unsigned)join_blocks), dim3(256), 0, s, a, parts, p.tiles, p.numbers,
                 (int)mix_blocks);
  prof_mark(K_SSCAN_JOIN, s, false);
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

size_t selective_scan_bwd_workspace(const ScanArgs& a) { return plan_of(a).total; }
cudaError_t launch_selective_scan_bwd(const ScanArgs& a, bool wide, cudaStream_t s) {
  if (a.bf16) return wide ? pick<bf16, true>(a, s) : pick<bf16, false>(a, s);
  return wide ? pick<float, true>(a, s) : pick<float, false>(a, s);
}

}  // namespace gdn
