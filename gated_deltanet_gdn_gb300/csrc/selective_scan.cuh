// Shared by the selective scan's forward and backward (selective_scan.cu, selective_scan_bwd.cu):
// the tiling, the loads of a tile and the split of long sequences.
//
// Per channel d and state n, with delta_t = softplus(dt_t + bias):
//   h_t = exp(delta_t A) h_{t-1} + delta_t u_t B_t,   y_t = (sum_n C_t h_t + D u_t) z_t sigmoid(z_t)
//
// Bound by arithmetic: one exponential and four products per token, channel and state (32 and 128 a
// clock and SM: 16 states x 768 channels x 32,768 tokens cannot take less than 44 us, their
// bytes 30 us), so the layout is made to keep everything else off the inner loop:
//  * a lane holds 4 channels x 4 states. NS / 4 lanes share four channels (a quad), so a step's values are read from
//    shared memory in four 16-byte loads and the sum over states takes 3 (NS = 16) shuffles for 16 states;
//    a lane per channel with all its states would take 32 shuffles in the backward's sums over channels;
//  * what is per token and channel only (softplus, delta u, the gate, conversions) is done once for a tile of
//    scan_tile(NS) tokens, spread over all lanes, and passed through shared memory;
//  * a warp owns its tile and its shared memory: no barrier of a CTA anywhere, loads of the next
//    tile are in flight during the steps;
//  * two channels go through each fp32 instruction (fma.rn.f32x2), which halves the issue slots.
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

template <int NS_>
struct ScanShape {
  static constexpr int NS = NS_, S = NS / 4, Q = 32 / S, CW = 4 * Q, TT = scan_tile(NS), P = TT / S;
  static constexpr int BV = (TT * NS / 4 + 31) / 32;  // quads of B (and of C) a lane loads for a tile
  static_assert(P >= 1 && P * S == TT, "whole passes");
};

// Tiles of channels of all groups (a warp's channels belong to one group).
inline int scan_tiles(int D, int G, int NS) {
  const int cw = 512 / NS, dg = D / G;
  return G * ((dg + cw - 1) / cw);
}

constexpr int SCAN_WHOLE = 0x40000000;  // chunk length where sequences are not split

// Clocks of a warp's step (512 products of channel and state) that weigh a split against whole sequences: in a full SM
// sub-partition; of a warp with no other beside it; in the launch before that gives the chunks' ends; and the warps an
// SM holds.
struct ScanCost {
  int full, alone, ends, resident;
};
// Chunk length, a multiple of the tile: SCAN_WHOLE, or as many chunks as fill the SMs once.
inline int scan_split(const ScanArgs& a, ScanCost cost) {
  const long long tiles = scan_tiles(a.D, a.G, a.NS), steps = a.q.N * tiles, parts = 152 * 4;
  const long long busy = steps * cost.full / parts, one = (long long)a.max_q * cost.alone;
  const long long whole = busy > one ? busy : one;
  const long long split = steps * (cost.full + cost.ends) / parts + 12000;  // and two more launches
  if (split >= whole) return SCAN_WHOLE;
  // sequences of max_q tokens, were they all as long
  const long long warps = (long long)152 * cost.resident * a.max_q, each = steps > 0 ? warps / steps : 0;
  if (each < 2) return SCAN_WHOLE;
  const int L = (int)((a.max_q + each - 1) / each);
  return L < 64 ? 64 : (L + 15) / 16 * 16;
}

// A warp's place: its channels and the chunk it works on.
template <class Shape>
struct ScanPlace {
  int lane, s, q, g, c, n;  // states 4 s .. 4 s + 3 of channels c .. c + n - 1 (n up to 4) of group g
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

// [channel][state] rows of fp32 as pairs of channels: x[0][i] channels 0, 1 and x[1][i] channels 2, 3 of state i.
template <class Shape>
__device__ __forceinline__ void load_states(const float* p, const ScanPlace<Shape>& w, f32x2 (&x)[2][4]) {
  float f[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < w.n) v = *reinterpret_cast<const float4*>(p + (long long)(w.c + i) * Shape::NS + 4 * w.s);
    f[i][0] = v.x; f[i][1] = v.y; f[i][2] = v.z; f[i][3] = v.w;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[0][i] = pack2(f[0][i], f[1][i]);
    x[1][i] = pack2(f[2][i], f[3][i]);
  }
}
template <class Shape>
__device__ __forceinline__ void store_states(float* p, const ScanPlace<Shape>& w, const f32x2 (&x)[2][4]) {
  float2 f[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[0][i] = split2(x[0][i]);
    f[1][i] = split2(x[1][i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < w.n) {
      const float4 v = i % 2 == 0 ? make_float4(f[i / 2][0].x, f[i / 2][1].x, f[i / 2][2].x, f[i / 2][3].x)
                                  : make_float4(f[i / 2][0].y, f[i / 2][1].y, f[i / 2][2].y, f[i / 2][3].y);
      *reinterpret_cast<float4*>(p + (long long)(w.c + i) * Shape::NS + 4 * w.s) = v;
    }
}

// Rows p S + s of a tile (rows [0, rows) of it are real), as loaded.
template <class Shape, bool WIDE, class T>
struct ScanRows {
  Quad<T> v[Shape::P];
  __device__ __forceinline__ void load(const void* base, long long row0, long long ts, int rows, const ScanPlace<Shape>& w) {
#pragma unroll
    for (int p = 0; p < Shape::P; ++p) {
      const int r = p * Shape::S + w.s;
      v[p] = load_quad<WIDE>(static_cast<const T*>(base) + (row0 + r) * ts + w.c, r < rows ? w.n : 0);
    }
  }
};
// B or C of a tile: [TT][NS] of the warp's group.
template <class Shape, bool WIDE, class T>
struct ScanMix {
  Quad<T> v[Shape::BV];
  __device__ __forceinline__ void load(const void* base, long long row0, long long ts, long long gs, int rows,
                                       const ScanPlace<Shape>& w) {
#pragma unroll
    for (int i = 0; i < Shape::BV; ++i) {
      const int k = w.lane + 32 * i, r = k / (Shape::NS / 4), n = k % (Shape::NS / 4) * 4;
      v[i] = load_quad<WIDE>(static_cast<const T*>(base) + (row0 + r) * ts + w.g * gs + n, r < rows ? 4 : 0);
    }
  }
  __device__ __forceinline__ void store(float* sm, const ScanPlace<Shape>& w) const {
#pragma unroll
    for (int i = 0; i < Shape::BV; ++i) {
      const int k = w.lane + 32 * i;
      float f[4];
      quad_floats(v[i], f);
      if (k < Shape::TT * Shape::NS / 4) *reinterpret_cast<float4*>(sm + 4 * k) = make_float4(f[0], f[1], f[2], f[3]);
    }
  }
};

// Sums of four values (channels of the quad) over its S lanes: lane s ends with channel s % 4 in out[0] (S >= 4),
// or with channels 2 s, 2 s + 1 (S = 2).
template <int S>
__device__ __forceinline__ void sum_quad(const float (&v)[4], int s, float (&out)[2]) {
  constexpr unsigned ALL = 0xffffffffu;
  constexpr int FAR = S == 2 ? 1 : 2;
  const bool up = s & FAR;
  float a = up ? v[2] : v[0], b = up ? v[3] : v[1];
  a += __shfl_xor_sync(ALL, up ? v[0] : v[2], FAR);
  b += __shfl_xor_sync(ALL, up ? v[1] : v[3], FAR);
  if constexpr (S == 2) {
    out[0] = a;
    out[1] = b;
  } else {
    const bool odd = s & 1;
    float r = odd ? b : a;
    r += __shfl_xor_sync(ALL, odd ? a : b, 1);
#pragma unroll
    for (int d = 4; d < S; d *= 2) r += __shfl_xor_sync(ALL, r, d);
    out[0] = r;
    out[1] = 0.f;
  }
}
// Stores sum_quad's result in the quad's place of a row.
template <int S>
__device__ __forceinline__ void put_quad(float* row_quad, int s, const float (&v)[2]) {
  if constexpr (S == 2) *reinterpret_cast<float2*>(row_quad + 2 * s) = make_float2(v[0], v[1]);
  else if (S == 4 || s < 4) row_quad[s % 4] = v[0];
}

}  // namespace gdn
