// Selective state space scan, forward: prompts, training and single tokens (selective_scan.cuh has
// the mathematics, the tiling and the split of long sequences).
#include "selective_scan.cuh"

namespace gdn {
namespace {

constexpr int WARPS = 4;
// States of a lane. (16 states need more registers than there are: 249 against 141 us at B8 T4096 D768,
// 16 states; 4 states: 144 us, and the chunks' ends 91 against 85 us.)
constexpr int STATES = 8;

// Stores the first n of a lane's OWN channels.
template <bool WIDE, int OWN, class T>
__device__ __forceinline__ void put_own(T* p, const float (&x)[4], int n) {
  if constexpr (WIDE && OWN == 4) {
    if (n > 0) st4(p, x);
  } else if constexpr (WIDE && OWN == 2) {
    if (n > 0) store2(p, x[0], x[1]);
  } else {
#pragma unroll
    for (int i = 0; i < OWN; ++i)
      if (i < n) p[i] = from_f32<T>(x[i]);
  }
}

constexpr int TILE = 4;  // tokens

template <class Shape>
struct WarpTile {
  float delta[Shape::TT * Shape::LD], du[Shape::TT * Shape::LD];
  float skip[Shape::TT * Shape::LD], gate[Shape::TT * Shape::LD];  // D u and silu(z)
  float B[Shape::TT * Shape::NS], C[Shape::TT * Shape::NS];
};
template <class Shape>
struct SumTile {
  float delta[Shape::TT * Shape::LD], du[Shape::TT * Shape::LD], B[Shape::TT * Shape::NS];
};

// SUM: what a chunk adds to the state (from zeros) and the sum of its delta, no outputs.
// start: [chunks][D][NS] states at the chunks' starts (SUM: written as the chunks' own ends), sums: [chunks][D].
template <class T, int NS, bool WIDE, bool SUM>
__global__ void __launch_bounds__(32 * WARPS, SUM ? 3 : ctas_of(sizeof(T) == 4, NS))
    selective_scan_kernel(ScanArgs a, int L, int tiles, long long warps, float* start, float* sums, unsigned ctas) {
  using Shape = ScanShape<NS, STATES, TILE>;
  constexpr int S = Shape::S, P = Shape::P, LD = Shape::LD, TT = Shape::TT, N = STATES / 2;
  constexpr int OWN = S == 1 ? 4 : S == 2 ? 2 : 1;  // channels whose sums a lane ends with
  using Tile = std::conditional_t<SUM, SumTile<Shape>, WarpTile<Shape>>;
  __shared__ __align__(16) Tile shared[WARPS][2];
  pdl_wait();
  pdl_trigger();
  if constexpr (!SUM) {
    if (blockIdx.x >= ctas) {
      zero_padding<WIDE, 32 * WARPS, T>(a, ctas, a.y, a.y_ts);
      return;
    }
  }
  const long long at = (long long)blockIdx.x * WARPS + threadIdx.x / 32;
  if (at >= warps) return;
  Tile(&sm)[2] = shared[threadIdx.x / 32];
  const long long number = at / tiles;
  const ScanPlace<Shape> w(a, (int)(at - number * tiles));
  Chunk k;
  if (!packed_chunk(a.q, number, L, &k)) return;
  const int t0 = k.j * L, t1 = k.len - t0 < L ? k.len : t0 + L;
  if (SUM && t1 == k.len) return;  // nothing comes after it

  f32x2 A[4][N], h[4][N];
  load_states<Shape>(a.A, w, A);
  finite_rates(A);
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
  long long kept_channel = 0, kept_row = 0;
  if (!SUM && a.kept) {
    kept_channel = kept_step<NS>(a);
    kept_row = kept_channel * 8;
    kept = a.kept + (packed_number(a.q, k.b, k.first, SCAN_KEEP) + t0 / SCAN_KEEP) * kept_row + kept_place(a, w, 2 * w.s);
  }
  // the lane's channels of the sums, and how many of them there are
  const int own = S == 1 ? 0 : S == 2 ? 2 * w.s : w.s % 4, own_n = S > 4 && w.s >= 4 ? 0 : w.n - own;
  T* y = static_cast<T*>(a.y) + (k.first + (long long)t0) * a.y_ts + w.c + own;

  ScanRows<Shape, WIDE, T> ru, rd, rz;
  ScanMix<Shape, WIDE, T> rb, rc;
  RowPtr<T> pu, pd, pz;
  MixPtr<T> pb, pc;
  {
    const long long row0 = k.first + (long long)t0;
    pu.set(a.u, row0, a.u_ts, w);
    pd.set(a.dt, row0, a.dt_ts, w);
    pz.set(a.z, row0, a.z_ts, w);
    pb.set(a.B, row0, a.b_ts, a.b_gs, w);
    pc.set(a.C, row0, a.c_ts, a.c_gs, w);
  }
  const bool whole = __all_sync(0xffffffffu, w.n == 4);  // every lane has its channels
  // The next tile's loads; no rows are left behind the last one.
  auto fetch = [&](int rows) {
    if (whole && rows >= TT) {
      ru.template load<true>(pu, rows, w);
      rd.template load<true>(pd, rows, w);
      rb.template load<true>(pb, rows, w);
      if constexpr (!SUM) {
        if (a.z) rz.template load<true>(pz, rows, w);
        rc.template load<true>(pc, rows, w);
      }
    } else {
      ru.template load<false>(pu, rows, w);
      rd.template load<false>(pd, rows, w);
      rb.template load<false>(pb, rows, w);
      if constexpr (!SUM) {
        rz.template load<false>(pz, a.z ? rows : 0, w);
        rc.template load<false>(pc, rows, w);
      }
    }
    pu.p += pu.tile;
    pd.p += pd.tile;
    pb.p += pb.tile;
    if constexpr (!SUM) {
      pz.p += pz.tile;
      pc.p += pc.tile;
    }
  };
  // What was loaded, as the values that the steps read.
  auto form = [&](Tile& to, int rows) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int r = p * S + w.s;
      f32x2 d[2], u[2], z[2], x[2];
      quad_pairs(rd.v[p], d);
      quad_pairs(ru.v[p], u);
      if constexpr (!SUM) quad_pairs(rz.v[p], z);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        d[i] = add2(d[i], bias[i]);
        if (a.softplus) d[i] = softplus2(d[i]);
        if (r >= rows) d[i] = both(0.f);  // leaves the state as it is
        x[i] = mul2(u[i], d[i]);
        if constexpr (SUM) {
          if (S <= TT || r < TT) total[i] = add2(total[i], d[i]);
        } else {
          u[i] = mul2(u[i], skip[i]);
          z[i] = a.z ? mul2(z[i], sigmoid2(z[i])) : both(1.f);
        }
      }
      if (S <= TT || r < TT) {
        store_pairs(to.delta + r * LD + 4 * w.q, d);
        store_pairs(to.du + r * LD + 4 * w.q, x);
        if constexpr (!SUM) {
          store_pairs(to.skip + r * LD + 4 * w.q, u);
          store_pairs(to.gate + r * LD + 4 * w.q, z);
        }
      }
    }
    rb.store(to.B, w);
    if constexpr (!SUM) rc.store(to.C, w);
  };
  auto steps = [&](const Tile& tile, int rows) {
#pragma unroll
    for (int r = 0; r < TT; ++r) {
      const float4 dq = *reinterpret_cast<const float4*>(tile.delta + r * LD + 4 * w.q);
      const float4 xq = *reinterpret_cast<const float4*>(tile.du + r * LD + 4 * w.q);
      const float d[4] = {dq.x, dq.y, dq.z, dq.w}, x[4] = {xq.x, xq.y, xq.z, xq.w};
      f32x2 b[N], c[N];
      float out[4];
      load_row(b, tile.B + r * NS + STATES * w.s);
      if constexpr (!SUM) load_row(c, tile.C + r * NS + STATES * w.s);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f32x2 v;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          h[e][n] = fma2(decay2(both(d[e]), A[e][n]), h[e][n], scale2(x[e], b[n]));
          if constexpr (!SUM) v = n == 0 ? mul2(h[e][n], c[n]) : fma2(h[e][n], c[n], v);
        }
        if constexpr (!SUM) {
          const float2 f = split2(v);
          out[e] = f.x + f.y;
        }
      }
      if constexpr (!SUM) {
        sum_quad<S>(out, w.s);
        float more[OWN], gate[OWN];
        memcpy(more, __builtin_assume_aligned(tile.skip + r * LD + 4 * w.q + own, 4 * OWN), 4 * OWN);
        memcpy(gate, __builtin_assume_aligned(tile.gate + r * LD + 4 * w.q + own, 4 * OWN), 4 * OWN);
#pragma unroll
        for (int e = 0; e < OWN; ++e) out[e] = (out[e] + more[e]) * gate[e];
        put_own<WIDE, OWN>(y, out, r < rows ? own_n : 0);
        y += a.y_ts;
      }
    }
  };
  auto keep = [&](int t) {
    if (!SUM && kept && t < t1 && w.n > 0) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int n = 0; n < 2; ++n)
          *reinterpret_cast<ulonglong2*>(kept + c * kept_channel + n * 4 * kept_channel) = make_ulonglong2(h[c][2 * n], h[c][2 * n + 1]);
      kept += kept_row;
    }
  };
  static_assert(SCAN_KEEP == 2 * TT, "a kept state for every two tiles");
  fetch(t1 - t0);
  form(sm[0], t1 - t0);
  fetch(t1 - t0 - TT);
  for (int t = t0; t < t1; t += 2 * TT) {  // two tiles, so that their places are known when the steps are scheduled
    const int rows = t1 - t;
    keep(t);
    __syncwarp();
    steps(sm[0], rows);
    form(sm[1], rows - TT);
    fetch(rows - 2 * TT);
    __syncwarp();
    steps(sm[1], rows - TT);
    form(sm[0], rows - 2 * TT);
    fetch(rows - 3 * TT);
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

template <int SEG>
__global__ void __launch_bounds__(32 * CARRY_WARPS) selective_scan_carry_kernel(ScanArgs a, int L, float* start, const float* sums) {
  pdl_wait();
  pdl_trigger();
  scan_carry<false, SEG>(a, L, start, sums);
}

// One token a sequence, or few: a warp per 512 / NS channels of SEQS sequences, nothing staged. Bound by the states, which are
// read and written once (32 sequences x 6144 channels x 16 states: 25 MB), and by latency: everything that the first tokens
// need is on its way before the first result is used, and a sequence's next token while one is worked on. Where there is one
// token each and more than STEP_FULL warps, a warp takes two sequences and reads A once for both: 32 sequences 6.8 against 7.5 us,
// 64 11.0 against 13.7 (16: 4.8 against 4.6). STEP_CTAS an SM leave 128 registers: with 96 and the next token's loads, 8 sequences
// of 4 tokens x 2048 channels take 4.3 in place of 3.7 us; with 112, two sequences a warp spill (8.4 us).
constexpr int STEP_CTAS = 16;
constexpr long long STEP_FULL = 152 * STEP_CTAS;
template <class T, int NS, bool WIDE, int SEQS>
__global__ void __launch_bounds__(32, STEP_CTAS) selective_step_kernel(ScanArgs a, int tiles, unsigned ctas) {
  using Shape = ScanShape<NS, 4, TILE>;
  constexpr int S = Shape::S;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x >= ctas) {
    zero_padding<WIDE, 32, T>(a, ctas, a.y, a.y_ts);
    return;
  }
  const int at = blockIdx.x / tiles * SEQS;  // the first sequence
  const ScanPlace<Shape> w(a, blockIdx.x % tiles);
  f32x2 A[4][2], h[SEQS][4][2], bias[2], skip[2];
  load_states<Shape>(a.A, w, A);
  finite_rates(A);
  load_channels(a.bias, w, bias);
  load_channels(a.skip, w, skip);
  int first[SEQS], len[SEQS], slot[SEQS];
  const long long row = (long long)a.D * NS;
  struct Token {
    Quad<T> u, d, z, B, C;
  } token[SEQS];
  auto load = [&](Token& q, long long r, bool on) {
    const int n = on ? w.n : 0;
    q.u = load_quad<WIDE>(static_cast<const T*>(a.u) + r * a.u_ts + w.c, n);
    q.d = load_quad<WIDE>(static_cast<const T*>(a.dt) + r * a.dt_ts + w.c, n);
    q.z = load_quad<WIDE>(static_cast<const T*>(a.z) + r * a.z_ts + w.c, a.z ? n : 0);
    q.B = load_quad<WIDE>(static_cast<const T*>(a.B) + r * a.b_ts + w.g * a.b_gs + 4 * w.s, on ? 4 : 0);
    q.C = load_quad<WIDE>(static_cast<const T*>(a.C) + r * a.c_ts + w.g * a.c_gs + 4 * w.s, on ? 4 : 0);
  };
#pragma unroll
  for (int i = 0; i < SEQS; ++i) {
    const int b = at + i;
    slot[i] = -1;
    first[i] = len[i] = 0;
    if (b < a.q.B) {
      packed_bounds(a.q, b, &first[i], &len[i]);
      slot[i] = packed_slot(a.q, b);
    }
  }
#pragma unroll
  for (int i = 0; i < SEQS; ++i) {
    load(token[i], first[i], len[i] > 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[i][e][0] = h[i][e][1] = both(0.f);
    if (slot[i] >= 0 && a.h0 && packed_goes_on(a.q, at + i, len[i])) load_states<Shape>(a.h0 + slot[i] * row, w, h[i]);
  }
#pragma unroll
  for (int i = 0; i < SEQS; ++i) {
    for (int t = 0; t < len[i]; ++t) {
      const long long r = first[i] + (long long)t;
      if (SEQS > 1 && t > 0) load(token[i], r, true);
      const Token now = token[i];
      if (SEQS == 1) load(token[i], r + 1, t + 1 < len[i]);  // on its way while this one is worked on
      f32x2 d[2], u[2], bn[2], cn[2];
      float v[4];
      quad_pairs(now.d, d);
      quad_pairs(now.u, u);
      quad_pairs(now.B, bn);
      quad_pairs(now.C, cn);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        d[m] = add2(d[m], bias[m]);
        if (a.softplus) d[m] = softplus2(d[m]);
        const float2 df = split2(d[m]), xf = split2(mul2(d[m], u[m]));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int e = 2 * m + j;
          const float de = j ? df.y : df.x, xe = j ? xf.y : xf.x;
#pragma unroll
          for (int n = 0; n < 2; ++n)
            h[i][e][n] = fma2(decay2(both(de), mul2(A[e][n], both(LOG2E))), h[i][e][n], scale2(xe, bn[n]));
          const float2 f = split2(fma2(h[i][e][1], cn[1], mul2(h[i][e][0], cn[0])));
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
          quad_pairs(now.z, z);
#pragma unroll
          for (int m = 0; m < 2; ++m) y[m] = mul2(y[m], mul2(z[m], sigmoid2(z[m])));
        }
        store_quad<WIDE>(static_cast<T*>(a.y) + r * a.y_ts + w.c, y, w.n);
      }
    }
    if (slot[i] >= 0 && a.h_final) store_states<Shape>(a.h_final + slot[i] * row, w, h[i]);
  }
}
// Whether it is taken: it goes token by token where the other kernel's tiles of eight cost the same for one as for eight. In us,
// it against the other: 32 sequences x 6144 channels, of 4 tokens 12.5 and 18.2, of 6 16.1 and 18.4, of 8 19.7 and 18.5; of at most
// STEP_FULL warps also more tokens: 12 x 6144, of 8 8.4 and 10.7, of 16 14.2 and 14.6; 2 x 6144 of 16 7.6 and 10.5.
bool few(int tokens, long long warps) { return tokens <= 6 || (tokens <= 16 && warps <= STEP_FULL); }

int split_of(const ScanArgs& a) {
  const int warps = scan_tiles(a.D, a.G, a.NS, STATES);
  return scan_split(a, warps, ScanCost{400, 670, 250, 70, ctas_of(!a.bf16, a.NS), 8});
}

template <class T, int NS, bool WIDE>
cudaError_t run(const ScanArgs& a, cudaStream_t s) {
  const int step_tiles = scan_tiles(a.D, a.G, NS, 4);
  const long long sequences = a.q.B;
  if (!a.kept && few(a.max_q, sequences * step_tiles)) {
    const bool two = a.max_q == 1 && sequences * step_tiles > STEP_FULL;
    const long long blocks = (two ? (sequences + 1) / 2 : sequences) * step_tiles;
    const unsigned pad = packed_pad_ctas(a.q, a.q.zero_tail, (a.D + 3) / 4, 32);
    if (blocks + pad > 0x7fffffff) return cudaErrorNotSupported;
    if (blocks + pad == 0) return cudaSuccess;  // rows of no sequence, left alone
    prof_mark(K_SSTEP, s, true);
    const cudaError_t e = launch_pdl(two ? selective_step_kernel<T, NS, WIDE, 2> : selective_step_kernel<T, NS, WIDE, 1>,
                                     dim3((unsigned)blocks + pad), dim3(32), 0, s, a, step_tiles, (unsigned)blocks);
    prof_mark(K_SSTEP, s, false);
    return e;
  }
  const int L = split_of(a), tiles = scan_tiles(a.D, a.G, NS, STATES);
  const long long numbers = packed_numbers(a.q, L), warps = numbers * tiles, blocks = (warps + WARPS - 1) / WARPS;
  const unsigned pad = packed_pad_ctas(a.q, a.q.zero_tail, (a.D + 3) / 4, 32 * WARPS), own = (unsigned)blocks;
  if (blocks + pad > 0x7fffffff) return cudaErrorNotSupported;
  const dim3 grid(own), block(32 * WARPS);
  float* start = nullptr;
  if (L != PACKED_WHOLE) {
    start = static_cast<float*>(a.ws);
    float* sums = start + numbers * a.D * NS;
    prof_mark(K_SCAN_SUM, s, true);
    cudaError_t e = launch_pdl(selective_scan_kernel<T, NS, WIDE, true>, grid, block, 0, s, a, L, tiles, warps, start, sums, own);
    prof_mark(K_SCAN_SUM, s, false);
    if (e != cudaSuccess) return e;
    const bool shared = carry_shared(a, L);
    prof_mark(K_SCAN_CARRY, s, true);
    e = launch_pdl(shared ? selective_scan_carry_kernel<CARRY_WARPS> : selective_scan_carry_kernel<1>, dim3(carry_blocks(a, shared)),
                   dim3(32 * CARRY_WARPS), 0, s, a, L, start, (const float*)sums);
    prof_mark(K_SCAN_CARRY, s, false);
    if (e != cudaSuccess) return e;
  }
  prof_mark(K_SSCAN, s, true);
  const cudaError_t e =
      launch_pdl(selective_scan_kernel<T, NS, WIDE, false>, dim3(own + pad), block, 0, s, a, L, tiles, warps, start, (float*)nullptr, own);
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
  if (L == PACKED_WHOLE) return 0;
  return (size_t)packed_numbers(a.q, L) * a.D * (a.NS + 1) * sizeof(float);
}
cudaError_t launch_selective_scan(const ScanArgs& a, bool wide, cudaStream_t s) {
  if (a.bf16) return wide ? pick<bf16, true>(a, s) : pick<bf16, false>(a, s);
  return wide ? pick<float, true>(a, s) : pick<float, false>(a, s);
}

}  // namespace gdn
