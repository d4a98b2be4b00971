// Shared by the selective scan's forward and backward (selective_scan.cu, selective_scan_bwd.cu):
// the tiling, the loads of a tile and the split of long sequences.
//
// Per channel d and state n, with delta_t = softplus(dt_t + bias):
//   h_t = exp(delta_t A) h_{t-1} + delta_t u_t B_t,   y_t = (sum_n C_t h_t + D u_t) z_t sigmoid(z_t)
//
// Bound by arithmetic: one exponential and four products per token, channel and state (32 and 128 a
// clock and SM: 16 states x 768 channels x 32,768 tokens cannot take less than 44 us, their
// bytes 30 us), so the layout is made to keep everything else off the inner loop:
//  * a lane holds 4 channels x SP states (8 forward, 4 backward, whose registers hold several tokens' states). NS / SP
//    lanes share four channels (a quad). What a step reads from shared memory grows with the sides of this tile and its
//    products with the area: with 4 x 4 the reads alone took as long as the exponentials;
//  * what is per token and channel only (softplus, delta u, the gate, conversions) is done once for a tile of
//    TT tokens, spread over all lanes, and passed through shared memory;
//  * a warp owns its tile and its shared memory: no barrier of a CTA in the forward. It forms the next tile's values
//    between the steps of this one (their chains of latency are as long as a step), with the loads of the one
//    after that in flight;
//  * two values go through each fp32 instruction (fma.rn.f32x2), which halves the issue slots.
//
// Few channels and long sequences do not fill the SMs: a chunk per warp then, in three launches. The first
// scans every chunk but the last from zeros and keeps its last state and the sum of its delta, since a
// state decays over a chunk by exp(A sum delta); the second carries the states over the chunks;
// the third scans the chunks from their true starts. scan_split() weighs the arithmetic done twice
// against the time of one warp over the longest sequence.
#pragma once

#include "packed.cuh"
#include "pairs.cuh"

namespace gdn {

template <int NS_, int SP_, int TT_>
struct ScanShape {
  static constexpr int NS = NS_, SP = SP_, S = NS / SP, Q = 32 / S, CW = 4 * Q, TT = TT_, P = TT > S ? TT / S : 1;
  static constexpr int BV = (TT * NS / 4 + 31) / 32;  // quads of B (and of C) a lane loads for a tile
  // Row length of a tile in shared memory: eight lanes' vectors, of 8 / S quads and S rows, on different banks.
  static constexpr int LD = CW + (S == 1 ? 0 : S < 8 ? 32 / S : 4);
  static_assert(P * S >= TT && SCAN_KEEP % TT == 0, "whole tiles between kept states");
};

// CTAs of four warps that an SM holds: three, with 168 registers. Eight states in fp32 (a lane loads all of a tile's rows
// then) would spill a third of them: B4 T4096 D2048 forward 156 against 122 us, B8 T4096 D768 backward 466 against 334 us;
// in bf16 the third CTA gives more (117 against 127 us).
constexpr int ctas_of(bool f32, int ns) { return f32 && ns == 8 ? 2 : 3; }

// Warps for the channels of all groups (a warp's channels belong to one group).
inline int scan_tiles(int D, int G, int NS, int SP) {
  const int cw = 128 * SP / NS, dg = D / G;
  return G * ((dg + cw - 1) / cw);
}

// Clocks of a warp's step that weigh a split against whole sequences, as measured: in a full SM sub-partition; of a warp
// with no other beside it; and (beside a full one) in the launch before that gives the chunks' ends; then clocks to carry a
// state over a chunk. CTAs of four warps that an SM holds, and the multiple of tokens that a chunk has.
struct ScanCost {
  int full, alone, ends, carry, resident, unit;
};
// Chunk length: PACKED_WHOLE, or the length of the least time by these clocks, among those whose chunks fill the SMs one to
// four times and their shorter and longer multiples of two (a warp's start counts as START tokens; sequences of unknown
// lengths end in the middle of a chunk). warps: of one chunk.
inline int scan_split(const ScanArgs& a, int warps, ScanCost cost) {
  constexpr int START = 12, LAUNCHES = 12000;  // clocks of two more launches
  const long long parts = 152 * 4, tokens = a.q.cu ? a.q.N : a.q.T;
  if (a.q.B == 0) return PACKED_WHOLE;
  auto step = [&](long long n) {  // clocks of a token where every SM sub-partition has n warps
    return n * cost.full > cost.alone ? n * cost.full : (long long)cost.alone;
  };
  const long long busy = (long long)a.q.N * warps * cost.full / parts, one = (long long)a.max_q * cost.alone;
  long long best = busy > one ? busy : one;
  int length = PACKED_WHOLE;
  auto weigh = [&](long long L) {
    if (L < cost.unit) L = cost.unit;
    if (L >= a.max_q) return;
    const long long chunks = a.q.cu ? (tokens + L - 1) / L + a.q.B / 2 : (tokens + L - 1) / L * a.q.B;
    const long long each = (chunks * warps + parts - 1) / parts;  // warps of a sub-partition
    const long long waves = (each + cost.resident - 1) / cost.resident;
    const long long clocks = step(waves > 1 ? cost.resident : each) * (cost.full + cost.ends) / cost.full;
    const long long time = waves * (L + START) * clocks + (a.max_q + L - 1) / L * cost.carry + LAUNCHES;
    if (time < best) {
      best = time;
      length = (int)L;
    }
  };
  for (int waves = 1; waves <= 4; ++waves) {
    const long long room = waves * parts * cost.resident / warps;  // chunks
    const long long each = a.q.cu ? room - a.q.B / 2 : room / a.q.B;
    if (each >= 1) weigh(((tokens + each - 1) / each + cost.unit - 1) / cost.unit * cost.unit);
  }
  for (int L = cost.unit; L <= 1024; L *= 2) weigh(L);
  return length;
}

// A state carried over a chunk whose delta sum to `sum` (in units of 1 / log2 e). Where the factor leaves float32's range the
// carried state need not (1e-20 that grows by 1e39), so half of the exponent goes into the state and half comes after it. A zero
// stays zero where even that overflows, as it does step by step.
__device__ __forceinline__ float carried(float rate, float sum, float state, float own) {
  const float x = rate * sum;
  const bool far = fabsf(x) > 126.f;
  const float f = ex2(far ? 0.5f * x : x);
  return state == 0.f ? own : fmaf(f, far ? f * state : state, own);
}

// A warp's place: its channels and the chunk it works on.
template <class Shape>
struct ScanPlace {
  int lane, s, q, g, c, n;  // states SP s .. SP s + SP - 1 of channels c .. c + n - 1 (n up to 4) of group g
  __device__ __forceinline__ ScanPlace(const ScanArgs& a, int tile) {
    lane = threadIdx.x % 32;
    s = lane % Shape::S;
    q = lane / Shape::S;
    const int dg = a.D / a.G, per = (dg + Shape::CW - 1) / Shape::CW;
    g = tile / per;
    c = g * dg + (tile - g * per) * Shape::CW + 4 * q;
    const int left = (g + 1) * dg - c;
    n = left < 0 ? 0 : left > 4 ? 4 : left;
  }
};

// [channel][state] rows of fp32: pairs of neighbouring states of each channel.
template <class Shape>
__device__ __forceinline__ void load_states(const float* p, const ScanPlace<Shape>& w, f32x2 (&x)[4][Shape::SP / 2]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int n = 0; n < Shape::SP / 4; ++n) {
      ulonglong2 v = {0ull, 0ull};
      if (i < w.n) v = *reinterpret_cast<const ulonglong2*>(p + (long long)(w.c + i) * Shape::NS + Shape::SP * w.s + 4 * n);
      x[i][2 * n] = v.x;
      x[i][2 * n + 1] = v.y;
    }
}
// Rates A, where -infinity becomes a finite value whose products with a step decay to zero all the same: the tokens that fill
// up a tile have steps of zero and are to leave the states as they are. NaN stays NaN.
__device__ __forceinline__ float finite_rate(float a) { return a < -2e38f ? -2e38f : a; }
template <int N, int M>
__device__ __forceinline__ void finite_rates(f32x2 (&A)[N][M]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int n = 0; n < M; ++n) {
      const float2 f = split2(A[i][n]);
      A[i][n] = pack2(finite_rate(f.x), finite_rate(f.y));
    }
}
template <class Shape>
__device__ __forceinline__ void store_states(float* p, const ScanPlace<Shape>& w, const f32x2 (&x)[4][Shape::SP / 2]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < w.n) {
#pragma unroll
      for (int n = 0; n < Shape::SP / 4; ++n)
        *reinterpret_cast<ulonglong2*>(p + (long long)(w.c + i) * Shape::NS + Shape::SP * w.s + 4 * n) =
            make_ulonglong2(x[i][2 * n], x[i][2 * n + 1]);
    }
}
// Kept states: 16-byte vectors of four states, [parity of the vector][channel of the quad][quad][vector / 2], so that the
// forward's stores (two vectors a lane) and the backward's loads (one) both run over consecutive addresses.
template <class Shape>
__device__ __forceinline__ long long kept_place(const ScanArgs& a, const ScanPlace<Shape>& w, int vector) {
  const int dg = a.D / a.G, quad = w.g * ((dg + 3) / 4) + (w.c - w.g * dg) / 4;
  return ((long long)(vector % 2) * 4 * scan_quads(a.D, a.G) + quad) * (Shape::NS / 2) + vector / 2 * 4;
}
// Floats between two channels of a quad there.
template <int NS>
__device__ __forceinline__ long long kept_step(const ScanArgs& a) {
  return (long long)scan_quads(a.D, a.G) * (NS / 2);
}
// SP consecutive floats as pairs.
template <int N>
__device__ __forceinline__ void load_row(f32x2 (&x)[N], const float* p) {
#pragma unroll
  for (int n = 0; n < N / 2; ++n) {
    const ulonglong2 v = reinterpret_cast<const ulonglong2*>(p)[n];
    x[2 * n] = v.x;
    x[2 * n + 1] = v.y;
  }
}
// The other way about, for four states a lane: x[e][i] holds channels 2 e' and 2 e' + 1, e' = e ^ flip_c, of state
// i' = i ^ 2 flip_n. (Lanes that take their channels or states in another order exchange sums without selecting.)
template <class Shape>
__device__ __forceinline__ void load_columns(const float* p, long long channel, const ScanPlace<Shape>& w, int flip_c, int flip_n,
                                             f32x2 (&x)[2][4]) {
  static_assert(Shape::SP == 4, "four states a lane");
  float2 f[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = i ^ (2 * flip_c);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      f[i][n] = make_float2(0.f, 0.f);
      if (c < w.n) f[i][n] = *reinterpret_cast<const float2*>(p + c * channel + 2 * (n ^ flip_n));
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      x[e][2 * n] = pack2(f[2 * e][n].x, f[2 * e + 1][n].x);
      x[e][2 * n + 1] = pack2(f[2 * e][n].y, f[2 * e + 1][n].y);
    }
}
template <class Shape>
__device__ __forceinline__ void load_columns(const float* p, const ScanPlace<Shape>& w, int flip_c, int flip_n, f32x2 (&x)[2][4]) {
  load_columns<Shape>(p + (long long)w.c * Shape::NS + 4 * w.s, Shape::NS, w, flip_c, flip_n, x);
}
template <class Shape>
__device__ __forceinline__ void store_columns(float* p, const ScanPlace<Shape>& w, int flip_c, int flip_n, const f32x2 (&x)[2][4]) {
  p += (long long)w.c * Shape::NS + 4 * w.s;
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const float2 a = split2(x[e][2 * n]), b = split2(x[e][2 * n + 1]);
      const int c = 2 * (e ^ flip_c);
      float2* to = reinterpret_cast<float2*>(p + c * Shape::NS + 2 * (n ^ flip_n));
      if (c < w.n) to[0] = make_float2(a.x, b.x);
      if (c + 1 < w.n) to[Shape::NS / 2] = make_float2(a.y, b.y);
    }
}
// Four floats of channels c .. c + 3, zeros where there are none.
template <class Shape>
__device__ __forceinline__ void load_channels(const float* p, const ScanPlace<Shape>& w, f32x2 (&x)[2]) {
  float f[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (p && i < w.n) f[i] = p[w.c + i];
  x[0] = pack2(f[0], f[1]);
  x[1] = pack2(f[2], f[3]);
}

// A lane's place in a [rows, channels] tensor: rows s, S + s, ... of a tile. The pointer moves with the tiles, since
// 64-bit products of rows and strides cost as much as a tile's arithmetic on them.
template <class T>
struct RowPtr {
  const T* p;
  long long step, tile;  // elements between a lane's rows, and between tiles
  template <class Shape>
  __device__ __forceinline__ void set(const void* base, long long row, long long ts, const ScanPlace<Shape>& w) {
    p = static_cast<const T*>(base) + (row + w.s) * ts + w.c;
    step = Shape::S * ts;
    tile = Shape::TT * ts;
  }
};
// Rows p S + s of a tile, as loaded: rows [0, rows) are real, the others become zeros. (S above TT: some lanes have no
// row.) FULL: all of them are, and the warp's channels too.
template <class Shape, bool WIDE, class T>
struct ScanRows {
  Quad<T> v[Shape::P];
  template <bool FULL = false>
  __device__ __forceinline__ void load(const RowPtr<T>& from, int rows, const ScanPlace<Shape>& w) {
#pragma unroll
    for (int p = 0; p < Shape::P; ++p) {
      const T* at = from.p + p * from.step;
      if constexpr (FULL && Shape::S <= Shape::TT) v[p] = load_quad<WIDE>(at);
      else v[p] = load_quad<WIDE>(at, p * Shape::S + w.s < rows ? w.n : 0);
    }
  }
};
// B or C of a tile: [TT][NS] of the warp's group.
template <class T>
struct MixPtr {
  const T* p;
  long long step, tile;
  template <class Shape>
  __device__ __forceinline__ void set(const void* base, long long row, long long ts, long long gs, const ScanPlace<Shape>& w) {
    p = static_cast<const T*>(base) + (row + w.lane / (Shape::NS / 4)) * ts + w.g * gs + w.lane % (Shape::NS / 4) * 4;
    step = 128 / Shape::NS * ts;
    tile = Shape::TT * ts;
  }
};
template <class Shape, bool WIDE, class T>
struct ScanMix {
  static constexpr int QUADS = Shape::TT * Shape::NS / 4;
  Quad<T> v[Shape::BV];
  template <bool FULL = false>
  __device__ __forceinline__ void load(const MixPtr<T>& from, int rows, const ScanPlace<Shape>& w) {
#pragma unroll
    for (int i = 0; i < Shape::BV; ++i) {
      const int k = w.lane + 32 * i;
      const T* at = from.p + i * from.step;
      if constexpr (FULL && QUADS % 32 == 0) v[i] = load_quad<WIDE>(at);
      else v[i] = load_quad<WIDE>(at, k / (Shape::NS / 4) < rows && k < QUADS ? 4 : 0);
    }
  }
  __device__ __forceinline__ void store(float* sm, const ScanPlace<Shape>& w) const {
#pragma unroll
    for (int i = 0; i < Shape::BV; ++i) {
      f32x2 f[2];
      quad_pairs(v[i], f);
      if (QUADS % 32 == 0 || w.lane + 32 * i < QUADS) store_pairs(sm + 4 * (w.lane + 32 * i), f);
    }
  }
};

// Zeros in the padding's rows of y or a gradient, by CTAs of THREADS.
template <bool WIDE, int THREADS, class T>
__device__ __forceinline__ void zero_padding(const ScanArgs& a, unsigned from, void* p, long long ts) {
  packed_padding<THREADS>(a.q, from, (a.D + 3) / 4, [&](long long r, int v) {
    const float none[4] = {};
    store_quad<WIDE>(static_cast<T*>(p) + r * ts + 4 * v, none, a.D - 4 * v);
  });
}

// Sums of four values (channels of the quad) over its S lanes: every lane ends with channels 4 s / S .. of them in front
// (S = 1 all, S = 2 two; from 4 on channel s % 4).
template <int S>
__device__ __forceinline__ void sum_quad(float (&v)[4], int s) {
  constexpr unsigned ALL = 0xffffffffu;
  if constexpr (S >= 2) {
    constexpr int FAR = S == 2 ? 1 : 2;
    const bool up = s & FAR;
    const float a = up ? v[0] : v[2], b = up ? v[1] : v[3];
    v[0] = (up ? v[2] : v[0]) + __shfl_xor_sync(ALL, a, FAR);
    v[1] = (up ? v[3] : v[1]) + __shfl_xor_sync(ALL, b, FAR);
  }
  if constexpr (S >= 4) {
    const bool odd = s & 1;
    v[0] = (odd ? v[1] : v[0]) + __shfl_xor_sync(ALL, odd ? v[0] : v[1], 1);
#pragma unroll
    for (int d = 4; d < S; d *= 2) v[0] += __shfl_xor_sync(ALL, v[0], d);
  }
}
// The states at the chunks' starts, in place of what each chunk adds (BACK: the adjoints that enter them from behind, in place
// of what each hands on). A lane has four states of a sequence's channel and takes CARRY chunks at once, whose loads are in flight
// together. SEG warps share a long sequence, each with the CARRY chunks behind the warp before it: it adds up its own from zeros,
// and what the warps before it give is carried over them.
constexpr int CARRY = 8, CARRY_WARPS = 8;
template <bool BACK, int SEG>
__device__ __forceinline__ void scan_carry(const ScanArgs& a, int L, float* start, const float* sums) {
  constexpr int LANES = 32 * CARRY_WARPS / SEG;
  static_assert(SEG == 1 || SEG == CARRY_WARPS, "a CTA's warps share their lanes' sequences, or none does");
  __shared__ float4 ends[SEG == 1 ? 1 : 2][SEG][32];
  __shared__ float spans[SEG == 1 ? 1 : 2][SEG][32];
  const int part = SEG == 1 ? 0 : threadIdx.x / 32, lane = SEG == 1 ? threadIdx.x : threadIdx.x % 32;
  const long long row = (long long)a.D * a.NS, at = ((long long)blockIdx.x * LANES + lane) * 4;
  const bool live = at < a.q.B * row;
  const int b = live ? (int)(at / row) : 0, i = live ? (int)(at - b * row) : 0;
  int first, len;
  packed_bounds(a.q, b, &first, &len);
  const int chunks = live ? packed_per(len, L) : 0;
  float rate[4], h[4] = {};
  ld4(rate, a.A + i);
#pragma unroll
  for (int n = 0; n < 4; ++n) rate[n] = finite_rate(rate[n]);
  if constexpr (BACK) {
    if (live && a.dh_final) ld4(h, a.dh_final + at);
  } else {
    const int slot = live ? packed_slot(a.q, b) : -1;
    if (slot >= 0 && a.h0 && packed_goes_on(a.q, b, len)) ld4(h, a.h0 + slot * row + i);
  }
  // A lane behind the last state loads chunk 0 of the first sequence with the others of its warp, and stores nothing.
  const int last = chunks > 0 ? chunks - 1 : 0;
  const long long number = packed_number(a.q, b, first, L) + (BACK ? last : 0);
  const long long step = BACK ? -row : row, down = BACK ? -a.D : a.D;
  float* p = start + number * row + i;
  const float* d = sums + number * a.D + i / a.NS;
  const int most = SEG == 1 ? chunks : __reduce_max_sync(0xffffffffu, chunks);
  for (int j = 0, side = 0; j < most; j += SEG * CARRY, side ^= 1) {
    const int j0 = j + part * CARRY;
    // Loads without a condition (of a place that is there), so that they are on their way together.
    float own[CARRY][4], sum[CARRY];
#pragma unroll
    for (int e = 0; e < CARRY; ++e) {
      const int at = j0 + e < last ? j0 + e : last;
      ld4(own[e], p + at * step);
      sum[e] = d[at * down];
    }
    auto pass = [&](int e, float (&g)[4]) {  // chunk j0 + e, if another comes after it
      const bool on = j0 + e < chunks - 1;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float x = carried(rate[n], sum[e] * LOG2E, g[n], own[e][n]);
        g[n] = on ? x : g[n];
      }
    };
    float g[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) g[n] = h[n];
    if constexpr (SEG > 1) {
      float end[4] = {}, span = 0.f;
#pragma unroll
      for (int e = 0; e < CARRY; ++e) {
        span += j0 + e < chunks - 1 ? sum[e] : 0.f;
        pass(e, end);
      }
      ends[side][part][lane] = make_float4(end[0], end[1], end[2], end[3]);
      spans[side][part][lane] = span * LOG2E;
      __syncthreads();  // one a round: the other side is written next
#pragma unroll
      for (int v = 0; v < SEG; ++v) {
        const float4 o = ends[side][v][lane];
        const float x[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          g[n] = v == part ? h[n] : g[n];
          h[n] = carried(rate[n], spans[side][v][lane], h[n], x[n]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < CARRY; ++e) {
      if (j0 + e < chunks) st4(p + (j0 + e) * step, g);
      pass(e, g);
    }
    if constexpr (SEG == 1) {
#pragma unroll
      for (int n = 0; n < 4; ++n) h[n] = g[n];
    }
  }
}
// Whether the warps of a CTA share sequences: from half a round of them on (64 channels x 16 states, 398 chunks: 20 against
// 57 us; 1024 x 16, 13 chunks: 8 both, but the two launches of a training step of 2 x 200 tokens take 80 against 58 us), and
// where there are SMs to spare (6144 channels x 16 states of six sequences: 62 against 13 us).
inline bool carry_shared(const ScanArgs& a, int L) {
  return a.max_q > (long long)CARRY * CARRY_WARPS / 2 * L && (long long)a.q.B * a.D * a.NS <= 1 << 16;
}
inline unsigned carry_blocks(const ScanArgs& a, bool shared) {
  const int lanes = shared ? 32 : 32 * CARRY_WARPS;
  return (unsigned)(((long long)a.q.B * a.D * a.NS / 4 + lanes - 1) / lanes);
}

}  // namespace gdn
