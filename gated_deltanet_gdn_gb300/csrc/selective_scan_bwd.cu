// Selective state space scan, backward (selective_scan.cuh has the tiling and the split).
//
// With dy' = dy silu(z) and the adjoint of the states running backwards,
//   G_t = C_t dy'_t + a_{t+1} G_{t+1},   a_t = exp(delta_t A),   G behind the last token = dh_final
//   dC_t = sum_d dy' h_t          dB_t = sum_d G delta u          d(delta u) = sum_n G B
//   ddelta = sum_n (G a h_{t-1}) A + u d(delta u)                 dA = sum_t (G a h_{t-1}) delta
//   du = delta d(delta u) + dy' skip    ddt = ddelta softplus'    dz = dy (C.h + skip u) silu'(z)    dh0 = a_0 G_0
//
// Bound by arithmetic, 14 products and 2.5 exponentials per token, channel and state. The states are not
// kept for every token but for every tile of SCAN_KEEP: a tile is scanned forward once from its kept state, which leaves
// the state before every second token in shared memory, then pair by pair from the last: the state between a pair's
// tokens is formed again, and a token's factors where they are used. So three states and one token's factors
// are in registers at a time, 12 warps fit an SM, and the arithmetic's latency is hidden. (Four tokens' states and factors,
// 255 registers and 8 warps: 607 against 463 us at B8 T4096 D768, 16 states.)
//
// A CTA's warps work on the same tokens of neighbouring channels, so their sums over channels (dB, dC) are added in
// shared memory before they leave the SM; what is left per CTA, and the sums over the tokens
// of a chunk (dA, dskip, ddt_bias), are added in a fixed order by a last kernel.
#include "selective_scan.cuh"

namespace gdn {
namespace {

constexpr int WARPS = 4;
constexpr int SUM_STATES = 8;

template <class Shape>
struct BwdShared {
  static constexpr int TILE = Shape::TT * Shape::LD;
  float delta[TILE];
  float du[TILE];     // delta u; then d(delta u)
  float dy[TILE];     // dy'
  float u[TILE];
  float slope[TILE];  // softplus'
  float dz[TILE];     // dy silu'(z)
  float B[Shape::TT * Shape::NS], C[Shape::TT * Shape::NS];
  float mix[Shape::TT * 2 * Shape::NS];  // dB, dC over the warp's channels
  // States before every second token, four vectors a lane. Once a pair's are in registers, its place
  // takes two rows of sum_n (G a h) A log2 e, then two of C.h.
  float4 h[Shape::TT / 2][4 * 32];
  static_assert(4 * Shape::LD <= 4 * 4 * 32, "four rows fit a pair's states");
};

// Partial sums in the workspace.
struct BwdParts {
  float* start;  // [half chunks][D][NS] adjoints entering the half chunks from behind (split only)
  float* sums;   // [half chunks][D] sums of delta (split only)
  float* mix;    // [CTAs' channel tiles][N][2 NS]
  float* dA;     // [chunks][D][NS]
  float* vec;    // [chunks][2][D]: dskip, ddt_bias
};
struct BwdPlan {
  int L, tiles;             // chunk length; CTAs' channel tiles of all groups
  int half;                 // of it: the launches before the chunks' own work on twice as many (130 against 88 us)
  long long numbers, halves;
  size_t start, sums, mix, dA, vec, total;  // bytes
};
int cta_tiles(const ScanArgs& a) {
  const int cw = 512 / a.NS * WARPS, dg = a.D / a.G;
  return a.G * ((dg + cw - 1) / cw);
}
BwdPlan plan_of(const ScanArgs& a) {
  BwdPlan p;
  p.tiles = cta_tiles(a);
  p.L = scan_split(a, p.tiles * WARPS, ScanCost{710, 1600, 130, 140, ctas_of(!a.bf16, a.NS), 16});
  p.half = p.L / 2;
  p.numbers = packed_numbers(a.q, p.L);
  p.halves = packed_numbers(a.q, p.half);
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const size_t states = up((size_t)p.numbers * a.D * a.NS * sizeof(float)), rows = up((size_t)p.numbers * a.D * sizeof(float));
  p.start = 0;
  p.sums = p.start + (p.L == PACKED_WHOLE ? 0 : up((size_t)p.halves * a.D * a.NS * sizeof(float)));
  p.mix = p.sums + (p.L == PACKED_WHOLE ? 0 : up((size_t)p.halves * a.D * sizeof(float)));
  p.dA = p.mix + up((size_t)p.tiles * a.q.N * 2 * a.NS * sizeof(float));
  p.vec = p.dA + states;
  p.total = p.vec + 2 * rows;
  return p;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// What a chunk hands to the one before it when nothing comes in from behind, and the sum of its delta.
template <class T, int NS, bool WIDE>
__global__ void __launch_bounds__(32 * WARPS, ctas_of(sizeof(T) == 4, NS))
    selective_scan_bwd_sum_kernel(ScanArgs a, int L, int tiles, long long warps, float* start, float* sums) {
  using Shape = ScanShape<NS, SUM_STATES, SCAN_KEEP>;
  constexpr int S = Shape::S, P = Shape::P, LD = Shape::LD, TT = Shape::TT, N = Shape::SP / 2;
  struct Mine {
    float delta[TT * LD], dy[TT * LD], C[TT * NS];
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
  if (!packed_chunk(a.q, number, L, &k) || k.j == 0) return;
  const int t0 = k.j * L, t1 = k.len - t0 < L ? k.len : t0 + L;
  f32x2 A[4][N], G[4][N];
  load_states<Shape>(a.A, w, A);
  finite_rates(A);
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      A[c][i] = mul2(A[c][i], both(LOG2E));
      G[c][i] = both(0.f);
    }
  f32x2 bias[2], total[2] = {both(0.f), both(0.f)};
  load_channels(a.bias, w, bias);
  ScanRows<Shape, WIDE, T> rd, ry, rz;
  ScanMix<Shape, WIDE, T> rc;
  const int last = t0 + (t1 - 1 - t0) / TT * TT;
  RowPtr<T> pd, py, pz;
  MixPtr<T> pc;
  {
    const long long row0 = k.first + (long long)last;
    pd.set(a.dt, row0, a.dt_ts, w);
    py.set(a.dy, row0, a.dy_ts, w);
    pz.set(a.z, row0, a.z_ts, w);
    pc.set(a.C, row0, a.c_ts, a.c_gs, w);
  }
  const bool whole = __all_sync(0xffffffffu, w.n == 4);
  auto fetch = [&](int rows) {
    if (whole && rows >= TT) {
      rd.template load<true>(pd, rows, w);
      ry.template load<true>(py, rows, w);
      if (a.z) rz.template load<true>(pz, rows, w);
      rc.template load<true>(pc, rows, w);
    } else {
      rd.template load<false>(pd, rows, w);
      ry.template load<false>(py, rows, w);
      rz.template load<false>(pz, a.z ? rows : 0, w);
      rc.template load<false>(pc, rows, w);
    }
    pd.p -= pd.tile;
    py.p -= py.tile;
    pz.p -= pz.tile;
    pc.p -= pc.tile;
  };
  fetch(t1 - last);
  for (int t = last; t >= t0; t -= TT) {
    const int rows = t1 - t < TT ? t1 - t : TT;
    __syncwarp();
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int r = p * S + w.s;
      f32x2 d[2], y[2], z[2];
      quad_pairs(rd.v[p], d);
      quad_pairs(ry.v[p], y);
      quad_pairs(rz.v[p], z);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        d[i] = add2(d[i], bias[i]);
        if (a.softplus) d[i] = softplus2(d[i]);
        if (r >= rows) d[i] = both(0.f);
        total[i] = add2(total[i], d[i]);
        if (a.z) y[i] = mul2(y[i], mul2(z[i], sigmoid2(z[i])));
      }
      store_pairs(sm.delta + r * LD + 4 * w.q, d);
      store_pairs(sm.dy + r * LD + 4 * w.q, y);
    }
    rc.store(sm.C, w);
    __syncwarp();
    fetch(t > t0 ? TT : 0);
#pragma unroll 4
    for (int r = TT - 1; r >= 0; --r) {
      const float4 dq = *reinterpret_cast<const float4*>(sm.delta + r * LD + 4 * w.q);
      const float4 yq = *reinterpret_cast<const float4*>(sm.dy + r * LD + 4 * w.q);
      const float d[4] = {dq.x, dq.y, dq.z, dq.w}, y[4] = {yq.x, yq.y, yq.z, yq.w};
      f32x2 c[N];
      load_row(c, sm.C + r * NS + Shape::SP * w.s);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int n = 0; n < N; ++n) G[e][n] = mul2(decay2(both(d[e]), A[e][n]), fma_by(y[e], c[n], G[e][n]));
    }
  }
  store_states<Shape>(start + number * a.D * NS, w, G);
  const float2 s0 = split2(total[0]), s1 = split2(total[1]);
  float v[4] = {s0.x, s0.y, s1.x, s1.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int d = 1; d < S; d *= 2) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
    if (w.s == 0 && i < w.n) sums[number * a.D + w.c + i] = v[i];
  }
}

template <int SEG>
__global__ void __launch_bounds__(32 * CARRY_WARPS) selective_scan_bwd_carry_kernel(ScanArgs a, int L, float* start, const float* sums) {
  pdl_wait();
  pdl_trigger();
  scan_carry<true, SEG>(a, L, start, sums);
}

// Whether lane s of a quad takes the channels' second pair first: the one whose sums it ends with.
template <int S>
__device__ __forceinline__ int pair_flip(int s) {
  return S == 2 ? s & 1 : (s >> 1) & 1;
}
// Sums of four values (channels of the quad in each lane's order, x[0] those it ends with) over its S lanes: S = 2 leaves
// two channels a lane, from 4 on the first of the two is channel s % 4.
template <int S>
__device__ __forceinline__ f32x2 sum_pairs(const f32x2 (&x)[2], int s) {
  constexpr unsigned ALL = 0xffffffffu;
  constexpr int FAR = S == 2 ? 1 : 2;
  const float2 keep = split2(x[0]), give = split2(x[1]);
  float a = keep.x + __shfl_xor_sync(ALL, give.x, FAR), b = keep.y + __shfl_xor_sync(ALL, give.y, FAR);
  if constexpr (S >= 4) {
    const bool odd = s & 1;
    a = (odd ? b : a) + __shfl_xor_sync(ALL, odd ? a : b, 1);
#pragma unroll
    for (int d = 4; d < S; d *= 2) a += __shfl_xor_sync(ALL, a, d);
    b = 0.f;
  }
  return pack2(a, b);
}
// Sums of eight values over the warp's quads: dB of the lane's four states in its order, then dC. The first step keeps the
// lane's first two states, the next one state, the third dB or dC.
template <class Shape>
__device__ __forceinline__ void put_mix(float* to, float (&v)[8], const ScanPlace<Shape>& w) {
  constexpr unsigned ALL = 0xffffffffu;
  constexpr int S = Shape::S, Q = Shape::Q;
  float x[4] = {v[0], v[1], v[4], v[5]};  // dB, dB, dC, dC
  {
    const float give[4] = {v[2], v[3], v[6], v[7]};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] += __shfl_xor_sync(ALL, give[i], S);
  }
  if constexpr (Q == 2) {
    to[0] = x[0]; to[1] = x[1]; to[Shape::NS] = x[2]; to[Shape::NS + 1] = x[3];
  } else {
    const bool second = w.q & 2;
    float b = (second ? x[1] : x[0]) + __shfl_xor_sync(ALL, second ? x[0] : x[1], 2 * S);
    float c = (second ? x[3] : x[2]) + __shfl_xor_sync(ALL, second ? x[2] : x[3], 2 * S);
    if constexpr (Q == 4) {
      to[0] = b;
      to[Shape::NS] = c;
    } else {
      const bool last = w.q & 4;
      b = (last ? c : b) + __shfl_xor_sync(ALL, last ? b : c, 4 * S);
      if constexpr (Q == 16) b += __shfl_xor_sync(ALL, b, 8 * S);
      if (Q == 8 || w.q < 8) to[0] = b;
    }
  }
}
// Where in a row of dB and dC put_mix's first result goes.
template <class Shape>
__device__ __forceinline__ int mix_place(const ScanPlace<Shape>& w) {
  return 4 * w.s + 2 * (w.q & 1) + (Shape::Q > 2 ? (w.q >> 1) & 1 : 0) + (Shape::Q > 4 ? ((w.q >> 2) & 1) * Shape::NS : 0);
}

template <class T, int NS, bool WIDE>
__global__ void __launch_bounds__(32 * WARPS, ctas_of(sizeof(T) == 4, NS)) selective_scan_bwd_kernel(ScanArgs a, int L, int tiles, BwdParts parts, unsigned ctas) {
  using Shape = ScanShape<NS, 4, SCAN_KEEP>;
  using Shared = BwdShared<Shape>;
  constexpr int S = Shape::S, P = Shape::P, CW = Shape::CW, LD = Shape::LD, TT = Shape::TT;
  static_assert(TT == SCAN_KEEP, "a kept state for every tile");
  extern __shared__ __align__(16) unsigned char raw_shared[];
  Shared* const all = reinterpret_cast<Shared*>(raw_shared);
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x >= ctas) {
    zero_padding<WIDE, 32 * WARPS, T>(a, ctas, a.du, a.D);
    zero_padding<WIDE, 32 * WARPS, T>(a, ctas, a.ddt, a.D);
    if (a.dz) zero_padding<WIDE, 32 * WARPS, T>(a, ctas, a.dz, a.D);
    return;
  }
  Shared& sm = all[threadIdx.x / 32];
  const long long number = blockIdx.x / tiles;
  const int tile = (int)(blockIdx.x - number * tiles);
  // the CTA's channels belong to one group; a warp of its end may have none
  const int dg = a.D / a.G, per = (dg + CW * WARPS - 1) / (CW * WARPS), g = tile / per;
  ScanPlace<Shape> w(a, 0);
  w.g = g;
  w.c = g * dg + ((tile - g * per) * WARPS + (int)threadIdx.x / 32) * CW + 4 * w.q;
  w.n = min(max((g + 1) * dg - w.c, 0), 4);
  const int flip_c = pair_flip<S>(w.s), flip_n = w.q & 1;  // the lane's order of channels and states
  const long long row = (long long)a.D * NS;
  f32x2 A[2][4], G[2][4], dA[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dA[0][i] = dA[1][i] = G[0][i] = G[1][i] = both(0.f);
  f32x2 dskip[2] = {both(0.f), both(0.f)}, dbias[2] = {both(0.f), both(0.f)};

  Chunk k;
  if (packed_chunk(a.q, number, L, &k)) {
    const int t0 = k.j * L, t1 = k.len - t0 < L ? k.len : t0 + L;
    load_columns<Shape>(a.A, w, flip_c, flip_n, A);
    finite_rates(A);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      A[0][i] = mul2(A[0][i], both(LOG2E));
      A[1][i] = mul2(A[1][i], both(LOG2E));
    }
    if (parts.start) {
      const long long behind = packed_number(a.q, k.b, k.first, L / 2) + min(2 * k.j + 1, packed_per(k.len, L / 2) - 1);
      load_columns<Shape>(parts.start + behind * row, w, flip_c, flip_n, G);
    } else if (a.dh_final) {
      load_columns<Shape>(a.dh_final + k.b * row, w, flip_c, flip_n, G);
    }
    f32x2 bias[2], skip[2];
    load_channels(a.bias, w, bias);
    load_channels(a.skip, w, skip);
    const int last = t1 > t0 ? t0 + (t1 - 1 - t0) / TT * TT : t0 - TT;
    const long long kept_channel = kept_step<NS>(a), kept_row = 8 * kept_channel;
    const float* kept = a.kept + (packed_number(a.q, k.b, k.first, TT) + last / TT) * kept_row + kept_place(a, w, w.s);
    RowPtr<T> pu, pd, py, pz;
    MixPtr<T> pb, pc;
    {
      const long long row0 = k.first + (long long)last;
      pu.set(a.u, row0, a.u_ts, w);
      pd.set(a.dt, row0, a.dt_ts, w);
      py.set(a.dy, row0, a.dy_ts, w);
      pz.set(a.z, row0, a.z_ts, w);
      pb.set(a.B, row0, a.b_ts, a.b_gs, w);
      pc.set(a.C, row0, a.c_ts, a.c_gs, w);
    }
    long long to = ((long long)k.first + last + w.s) * a.D + w.c;  // the contiguous gradients' place
    float* mix_to = parts.mix + ((long long)tile * a.q.N + k.first + last) * 2 * NS;
    const bool whole = __all_sync(0xffffffffu, w.n == 4);
    const int at = 4 * w.q, mix_at = mix_place<Shape>(w);
    // pairs of the quad's values in the lane's order
    auto load_quad_pairs = [&](f32x2 (&x)[2], const float* p) {
      x[0] = *reinterpret_cast<const f32x2*>(p + 2 * flip_c);
      x[1] = *reinterpret_cast<const f32x2*>(p + 2 - 2 * flip_c);
    };
    auto load_four = [&](float (&x)[4], const float* p) {
      const float2 a0 = *reinterpret_cast<const float2*>(p + 2 * flip_n), a1 = *reinterpret_cast<const float2*>(p + 2 - 2 * flip_n);
      x[0] = a0.x; x[1] = a0.y; x[2] = a1.x; x[3] = a1.y;
    };
    // token r of the tile forwards: the state before it, and after
    auto step = [&](int r, const f32x2 (&before)[2][4], f32x2 (&after)[2][4]) {
      f32x2 d[2], x[2];
      float bn[4];
      load_quad_pairs(d, sm.delta + r * LD + at);
      load_quad_pairs(x, sm.du + r * LD + at);
      load_four(bn, sm.B + r * NS + 4 * w.s);
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) after[e][n] = fma2(decay2(d[e], A[e][n]), before[e][n], scale2(bn[n], x[e]));
    };
    // and backwards, its factors formed again: own gets the lane's part of the quad's d(delta u), sum_n (G a h) A log2 e and
    // C.h, summed over the lanes
    auto back = [&](int r, const f32x2 (&before)[2][4], const f32x2 (&after)[2][4], f32x2 (&own)[3]) {
      f32x2 d[2], x[2], y[2], sums[3][2];
      float bn[4], cn[4], mix[8];
      load_quad_pairs(d, sm.delta + r * LD + at);
      load_quad_pairs(x, sm.du + r * LD + at);
      load_quad_pairs(y, sm.dy + r * LD + at);
      load_four(bn, sm.B + r * NS + 4 * w.s);
      load_four(cn, sm.C + r * NS + 4 * w.s);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        f32x2 db, dc;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          G[e][n] = fma_by(cn[n], y[e], G[e][n]);
          dc = e ? fma2(after[e][n], y[e], dc) : mul2(after[e][n], y[e]);
          db = e ? fma2(G[e][n], x[e], db) : mul2(G[e][n], x[e]);
          sums[0][e] = n ? fma_by(bn[n], G[e][n], sums[0][e]) : scale2(bn[n], G[e][n]);
          sums[2][e] = n ? fma_by(cn[n], after[e][n], sums[2][e]) : scale2(cn[n], after[e][n]);
          G[e][n] = mul2(G[e][n], decay2(d[e], A[e][n]));
          const f32x2 ga = mul2(G[e][n], before[e][n]);
          sums[1][e] = n ? fma2(ga, A[e][n], sums[1][e]) : mul2(ga, A[e][n]);
          dA[e][n] = fma2(ga, d[e], dA[e][n]);
        }
        const float2 b = split2(db), c = split2(dc);
        mix[n] = b.x + b.y;
        mix[4 + n] = c.x + c.y;
      }
#pragma unroll
      for (int m = 0; m < 3; ++m)
        if (m < 2 || a.z) own[m] = sum_pairs<S>(sums[m], w.s);
      put_mix<Shape>(sm.mix + r * 2 * NS + mix_at, mix, w);
    };
    auto put = [&](float* row_quad, f32x2 v) {
      const float2 f = split2(v);
      if constexpr (S == 2) *reinterpret_cast<float2*>(row_quad + 2 * w.s) = f;
      else if (S == 4 || w.s < 4) row_quad[w.s % 4] = f.x;
    };
    for (int t = last; t >= t0; t -= TT) {
      const int rows = t1 - t < TT ? t1 - t : TT;
      const bool full = whole && rows == TT;
      f32x2 h[2][4];
      {
        ScanRows<Shape, WIDE, T> ru, rd, ry, rz;
        ScanMix<Shape, WIDE, T> rb, rc;
        rd.load(pd, rows, w);
        ru.load(pu, rows, w);
        ry.load(py, rows, w);
        rz.load(pz, a.z ? rows : 0, w);
        rb.load(pb, rows, w);
        rc.load(pc, rows, w);
        load_columns<Shape>(kept, kept_channel, w, flip_c, flip_n, h);
        if (full && t > t0) {  // the next tile's rows and state to L2
#pragma unroll
          for (int p = 0; p < P; ++p) {
            prefetch_l2(pu.p - pu.tile + p * pu.step);
            prefetch_l2(pd.p - pd.tile + p * pd.step);
            prefetch_l2(py.p - py.tile + p * py.step);
            if (a.z) prefetch_l2(pz.p - pz.tile + p * pz.step);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) prefetch_l2(kept - kept_row + c * kept_channel);
        }
        __syncwarp();
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const int r = p * S + w.s;
          if (S > TT && r >= TT) continue;
          f32x2 d[2], u[2], y[2], z[2];
          quad_pairs(rd.v[p], d);
          quad_pairs(ru.v[p], u);
          quad_pairs(ry.v[p], y);
          store_pairs(sm.u + r * LD + at, u);
          if (a.softplus) {
            f32x2 s[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) d[i] = softplus2(add2(d[i], bias[i]), &s[i]);
            store_pairs(sm.slope + r * LD + at, s);
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) d[i] = add2(d[i], bias[i]);
          }
          if (!full && r >= rows) d[0] = d[1] = both(0.f);  // a step that changes nothing
#pragma unroll
          for (int i = 0; i < 2; ++i) u[i] = mul2(u[i], d[i]);
          if (a.z) {
            quad_pairs(rz.v[p], z);
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // silu' = s + z s (1 - s)
              const f32x2 s = sigmoid2(z[i]), zs = mul2(z[i], s);
              z[i] = mul2(y[i], fma2(zs, fma2(s, both(-1.f), both(1.f)), s));
              y[i] = mul2(y[i], zs);
            }
            store_pairs(sm.dz + r * LD + at, z);
          }
          store_pairs(sm.delta + r * LD + at, d);
          store_pairs(sm.du + r * LD + at, u);
          store_pairs(sm.dy + r * LD + at, y);
        }
        rb.store(sm.B, w);
        rc.store(sm.C, w);
        __syncwarp();
      }
      // forward through the tile: the state before every second token is kept, the last one stays in registers
      const int pairs = (rows + 1) / 2;
#pragma unroll
      for (int i = 0; i < TT / 2; ++i) {
        if (i >= pairs) break;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int n = 0; n < 2; ++n)
            reinterpret_cast<ulonglong2*>(sm.h[i])[(2 * e + n) * 32 + w.lane] = make_ulonglong2(h[e][2 * n], h[e][2 * n + 1]);
#pragma unroll
        for (int r0 = 0; r0 < 2; ++r0) step(2 * i + r0, h, h);
      }
#pragma unroll 2
      for (int i = pairs - 1; i >= 0; --i) {
        f32x2 h0[2][4], h1[2][4], own[2][3];  // states before the pair and between its tokens
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const ulonglong2 v = reinterpret_cast<const ulonglong2*>(sm.h[i])[(2 * e + n) * 32 + w.lane];
            h0[e][2 * n] = v.x;
            h0[e][2 * n + 1] = v.y;
          }
        step(2 * i, h0, h1);
        back(2 * i + 1, h1, h, own[1]);
        back(2 * i, h0, h1, own[0]);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int n = 0; n < 4; ++n) h[e][n] = h0[e][n];
        __syncwarp();  // every lane has read the pair's values and states
        float* place = reinterpret_cast<float*>(sm.h[i]) + at;
#pragma unroll
        for (int r0 = 0; r0 < 2; ++r0) {
          put(sm.du + (2 * i + r0) * LD + at, own[r0][0]);
          put(place + r0 * LD, own[r0][1]);
          if (a.z) put(place + (2 + r0) * LD, own[r0][2]);
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < rows * 2 * NS; i += 32 * WARPS) {
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < WARPS; ++j) v += all[j].mix[i];
        mix_to[i] = v;
      }
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int r = p * S + w.s;
        if ((S > TT || !full) && r >= rows) continue;  // (S above TT: lanes without a row)
        f32x2 d[2], u[2], y[2], gx[2], gd[2];
        const float* place = reinterpret_cast<const float*>(sm.h[r / 2]) + r % 2 * LD + at;
        load_pairs(d, sm.delta + r * LD + at);
        load_pairs(u, sm.u + r * LD + at);
        load_pairs(y, sm.dy + r * LD + at);
        load_pairs(gx, sm.du + r * LD + at);
        load_pairs(gd, place);
        const long long off = to + p * S * a.D;
        if (a.z) {
          f32x2 dz[2], ch[2];
          load_pairs(dz, sm.dz + r * LD + at);
          load_pairs(ch, place + 2 * LD);
#pragma unroll
          for (int e = 0; e < 2; ++e) dz[e] = mul2(dz[e], fma2(skip[e], u[e], ch[e]));
          store_quad<WIDE>(static_cast<T*>(a.dz) + off, dz, w.n);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          gd[e] = fma2(gx[e], u[e], mul2(gd[e], both(0.693147180559945309f)));
          gx[e] = fma2(gx[e], d[e], mul2(y[e], skip[e]));
          dskip[e] = fma2(y[e], u[e], dskip[e]);
        }
        if (a.softplus) {
          f32x2 s[2];
          load_pairs(s, sm.slope + r * LD + at);
#pragma unroll
          for (int e = 0; e < 2; ++e) gd[e] = mul2(gd[e], s[e]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) dbias[e] = add2(dbias[e], gd[e]);
        store_quad<WIDE>(static_cast<T*>(a.du) + off, gx, w.n);
        store_quad<WIDE>(static_cast<T*>(a.ddt) + off, gd, w.n);
      }
      __syncthreads();  // the sums over channels have been read
      pu.p -= pu.tile;
      pd.p -= pd.tile;
      py.p -= py.tile;
      pz.p -= pz.tile;
      to -= TT * a.D;
      pb.p -= pb.tile;
      pc.p -= pc.tile;
      kept -= kept_row;
      mix_to -= TT * 2 * NS;
    }
    if (k.j == 0 && a.dh0) store_columns<Shape>(a.dh0 + k.b * row, w, flip_c, flip_n, G);
  }
  store_columns<Shape>(parts.dA + number * row, w, flip_c, flip_n, dA);
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const float2 v0 = split2(m ? dbias[0] : dskip[0]), v1 = split2(m ? dbias[1] : dskip[1]);
    float v[4] = {v0.x, v0.y, v1.x, v1.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int d = 1; d < S; d *= 2) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
      if (w.s == 0 && i < w.n) parts.vec[(2 * number + m) * a.D + w.c + i] = v[i];
    }
  }
}

// Adds the partial sums: CTAs of 256 threads take 32 columns of dA, dskip and ddt_bias each (8 warps over every eighth
// chunk), then dB and dC: four values of a row a thread, or, where a group has JOIN_TILES CTAs' sums or more, 8 threads of
// different warps (1024 tokens, 4096 channels, 64 states, 128 sums: 55 against 25 us; 16 sums: 1 to 2 us either way).
constexpr int JOIN_TILES = 32;
template <class T>
__global__ void __launch_bounds__(256) selective_scan_join_kernel(ScanArgs a, BwdParts parts, int tiles, long long numbers,
                                                                  int sum_blocks) {
  __shared__ float4 sum4[8][32];
  float(*const sum)[32] = reinterpret_cast<float(*)[32]>(sum4);
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  if ((int)blockIdx.x >= sum_blocks) {
    const int vecs = a.NS / 2, each = tiles / a.G;  // of a row and group, dB and dC
    const bool shared = each >= JOIN_TILES;
    const long long block = blockIdx.x - sum_blocks, i = shared ? block * 32 + lane : block * 256 + threadIdx.x;
    const long long per = (long long)a.G * vecs, r = i / per;
    const int left = (int)(i - r * per), g = left / vecs, n = left % vecs * 4;
    const int first = packed_start(a.q, 0), end = packed_start(a.q, a.q.B);
    float v[4] = {};
    if (r < a.q.N && (!a.q.cu || (r >= first && r < end))) {
      const float* p = parts.mix + ((long long)g * each * a.q.N + r) * 2 * a.NS + n;
      const int step = shared ? 8 : 1;
#pragma unroll 8
      for (int t = shared ? warp : 0; t < each; t += step) {
        float x[4];
        ld4(x, p + (long long)t * a.q.N * 2 * a.NS);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += x[e];
      }
    }
    if (shared) {
      sum4[warp][lane] = make_float4(v[0], v[1], v[2], v[3]);
      __syncthreads();
      if (warp != 0) return;
      for (int w = 1; w < 8; ++w) {
        const float4 x = sum4[w][lane];
        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
      }
    }
    if (r >= a.q.N) return;
    T* const out = static_cast<T*>(n < a.NS ? a.dB : a.dC) + (r * a.G + g) * a.NS + (n < a.NS ? n : n - a.NS);
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = from_f32<T>(v[e]);
    return;
  }
  const long long row = (long long)a.D * a.NS, col = (long long)blockIdx.x * 32 + lane;
  const bool in = col < row + 2 * a.D;
  float s = 0.f;
  if (in) {
    const float* p = col < row ? parts.dA + col : parts.vec + (col - row);
    const long long step = col < row ? row : 2 * (long long)a.D;
#pragma unroll 8
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
  parts.start = p.L == PACKED_WHOLE ? nullptr : reinterpret_cast<float*>(ws + p.start);
  parts.sums = reinterpret_cast<float*>(ws + p.sums);
  parts.mix = reinterpret_cast<float*>(ws + p.mix);
  parts.dA = reinterpret_cast<float*>(ws + p.dA);
  parts.vec = reinterpret_cast<float*>(ws + p.vec);
  const long long blocks = p.numbers * p.tiles;
  const long long per = (long long)a.G * (a.NS / 2), items = p.tiles / a.G >= JOIN_TILES ? 32 : 256;
  const long long mix_blocks = (a.q.N * per + items - 1) / items;
  const long long column_blocks = ((long long)a.D * (a.NS + 2) + 31) / 32, join_blocks = mix_blocks + column_blocks;
  const unsigned pad = packed_pad_ctas(a.q, true, (a.D + 3) / 4, 32 * WARPS);
  if (blocks + pad > 0x7fffffff || join_blocks > 0x7fffffff) return cudaErrorNotSupported;
  cudaError_t e;
  if (parts.start) {
    const int tiles = scan_tiles(a.D, a.G, NS, SUM_STATES);
    const long long warps = p.halves * tiles, sum_blocks = (warps + WARPS - 1) / WARPS;
    if (sum_blocks > 0x7fffffff) return cudaErrorNotSupported;
    prof_mark(K_SSCAN_RSUM, s, true);
    e = launch_pdl(selective_scan_bwd_sum_kernel<T, NS, WIDE>, dim3((unsigned)sum_blocks), dim3(32 * WARPS), 0, s, a, p.half, tiles,
                   warps, parts.start, parts.sums);
    prof_mark(K_SSCAN_RSUM, s, false);
    if (e != cudaSuccess) return e;
    const bool shared = carry_shared(a, p.half);
    prof_mark(K_SCAN_CARRY, s, true);
    e = launch_pdl(shared ? selective_scan_bwd_carry_kernel<CARRY_WARPS> : selective_scan_bwd_carry_kernel<1>,
                   dim3(carry_blocks(a, shared)), dim3(32 * CARRY_WARPS), 0, s, a, p.half, parts.start, (const float*)parts.sums);
    prof_mark(K_SCAN_CARRY, s, false);
    if (e != cudaSuccess) return e;
  }
  const int bytes = (int)sizeof(BwdShared<ScanShape<NS, 4, SCAN_KEEP>>) * WARPS;
  e = allow_shared(reinterpret_cast<const void*>(selective_scan_bwd_kernel<T, NS, WIDE>), bytes, &done);
  if (e != cudaSuccess) return e;
  prof_mark(K_SSCAN_BWD, s, true);
  e = launch_pdl(selective_scan_bwd_kernel<T, NS, WIDE>, dim3((unsigned)blocks + pad), dim3(32 * WARPS), bytes, s, a, p.L, p.tiles, parts,
                 (unsigned)blocks);
  prof_mark(K_SSCAN_BWD, s, false);
  if (e != cudaSuccess) return e;
  prof_mark(K_SSCAN_JOIN, s, true);
  e = launch_pdl(selective_scan_join_kernel<T>, dim3((unsigned)join_blocks), dim3(256), 0, s, a, parts, p.tiles, p.numbers,
                 (int)column_blocks);
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
