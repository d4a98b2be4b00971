// Attention of new tokens over a paged key/value cache, for few query rows per KV head
// (single tokens, drafts) and for fp32.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - m),  j <= the token's position
//
// One pass over the keys with the running maximum m and sum (fp32, base 2). Every key and
// value is used for 16 query rows, so HBM bounds it: 4 D bytes per key in bf16 against
// 64 D flop. What matters is a deep, even stream of loads:
//  * the keys of all items are cut into units of 16 (inside one page, page sizes being
//    multiples of 16) and numbered through, with units for an item's start and end in front;
//    each CTA takes an equal run of them, whatever the lengths of the sequences, and its
//    warps take every WARPS-th unit of the run;
//  * each warp streams its units through a ring of its own (cp.async, 16 bytes a lane)
//    that runs ahead across item boundaries, with no barrier between warps;
//  * at an item's end the warps' (m, sum, o) are merged through shared memory. An item
//    that a CTA holds whole is written at once; the parts of one cut between CTAs go to
//    the workspace and a second kernel joins them in the order of the CTAs.
// The products run on mma.sync: a 16-row tile would leave seven eighths of a 128-row
// tcgen05 tile empty, and the tensor rate is not what bounds this kernel. In bf16 the
// probabilities are rounded to bf16 for the second product (their sum is not); fp32 uses
// three-term TF32 products for both.
//
// 32 sequences of one token, up to 32k keys (48 query and 8 KV heads of 128, bf16): 364-373 us,
// 6.6-6.8 TB/s, the measured copy rate. One sequence over 2k keys: 10 us, the latency
// of two launches. fp32, 3 x 200 tokens over 1.3k keys (6 and 2 heads of 64): 47 us, and 512
// tokens over 8k keys (64 and 8 heads of 128): 4.1 ms, bound by the products and the splits.
#include "paged_attn.cuh"

namespace gdn {
namespace {

constexpr int ROWS = 16, UNIT = 16;

// x = hi + lo for the split products, by cutting the mantissa: hi keeps tf32's 11 bits, lo
// the other 13, of which the tensor core takes 11 (off by at most 2^-22 of x). Two plain
// instructions, for keys and values; rounding conversions, at a quarter of the rate, took
// much of the kernel's time. Queries and probabilities, split rarely, are rounded
// (tf32_split): their lo has either sign, so the lo lo terms that the three-term products
// leave out do not bias the sums, as they would between two cut operands.
__device__ __forceinline__ void tf32_cut(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}

// As many warps as the rings leave room for: eight of three stages, or with fp32 rows of 128
// (16 KB a stage), where the arithmetic bounds it, six of two.
constexpr int warps_of(int D, int bytes) { return D * bytes <= 256 ? 8 : 6; }
// An item's start and end take about as long as one or two units of each warp: so many units
// without keys stand in front of its keys, and every warp passes over its share of them. bf16,
// 48 query and 8 KV heads of 128, one token each: 32 sequences of 20 keys 28 us without, 15
// with one unit a warp and with two; 128 of up to 500 keys 106, 65 and 54 us (with three and
// four 54). fp32, 3 x 200 tokens over 1.3k keys: 50, 48 and 49 us. Calls of fewer items than
// SMs have none: there an item is cut into parts, each with a start and an end of its own (one
// sequence over 2k keys: 9.5 us, with such units 10.2).
constexpr int units_over(int warps, int bytes) { return bytes == 2 ? 2 * warps : warps; }

template <class T, int D>
struct Lay {
  static constexpr int WARPS = warps_of(D, sizeof(T));
  static constexpr int THREADS = WARPS * 32;
  static constexpr int TILE = UNIT * D * (int)sizeof(T);  // bytes of one K or V unit
  static constexpr int STAGES = D * sizeof(T) <= 256 ? 3 : 2;
  static constexpr int Q = 0;                              // [16][D] T, swizzled; fp32: hi, then lo
  static constexpr int RING = (sizeof(T) == 2 ? 1 : 2) * ROWS * D * (int)sizeof(T);
  static constexpr int MROWS = 4096 / (WARPS * D);         // rows merged at a time
  static constexpr int MERGE = RING + WARPS * STAGES * 2 * TILE;
  static constexpr int ML = MERGE + WARPS * MROWS * D * 4;  // float m[WARPS][16], l[WARPS][16]
  static constexpr int TOT = ML + 2 * WARPS * ROWS * 4;        // float m[16], l[16] of the CTA
  static constexpr int BYTES = TOT + 2 * ROWS * 4;
  static_assert(BYTES + 1024 <= 227 * 1024, "one CTA per SM");
};

// What a part's sum and output count for beside the maximum M of all parts. A maximum of
// -inf alone does not say that a part is empty: maxima pass over NaN, which then stands in
// the sum and the output, and reaches the row's through the factor 0. Empty is a sum of 0.
__device__ __forceinline__ float part_factor(float m, float M) { return m == -INFINITY ? 0.f : exp2f(m - M); }

template <class T, int D, int OVER>
__global__ void __launch_bounds__(Lay<T, D>::THREADS, 1) paged_attn_kernel(AttnArgs a, int least) {
  pdl_wait();
  pdl_trigger();
  typedef Lay<T, D> L;
  typedef Numbering<ROWS, UNIT, OVER> Num;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  const PagedArgs& p = a.p;
  const int G = p.Hq / p.Hk;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  Tile<T, ROWS, D> Qs{reinterpret_cast<T*>(sm + L::Q)};
  uint8_t* ring = sm + L::RING + warp * L::STAGES * 2 * L::TILE;
  float* merge = reinterpret_cast<float*>(sm + L::MERGE);
  float* sml = reinterpret_cast<float*>(sm + L::ML);
  float* tot = reinterpret_cast<float*>(sm + L::TOT);

  PartHead* head = part_heads<ROWS, D>(a.ws, gridDim.x) + blockIdx.x;
  typename Num::Run run;
  if (!Num::plan(p, G, lane, blockIdx.x, gridDim.x, least, run)) {
    if (tid == 0) head->more = 0;
    return;
  }
  const long long lo = run.lo, hi = run.hi;
  Item cur = run.first;
  // The loads run ahead of the item in work. A unit's page is looked up one unit before its
  // loads are issued, so that they do not wait for it.
  Item ahead = cur;
  long long nextf = lo + warp;  // the next unit to look up
  struct Ref {
    int entry, row0, h;  // h < 0: nothing to load
  };
  auto look_up = [&]() {
    Ref r{0, 0, -1};
    while (nextf < hi) {
      while (nextf >= ahead.end) Num::next_item(p, G, ahead);
      if (nextf >= ahead.start + OVER) break;
      nextf += L::WARPS;
    }
    if (nextf < hi) {
      const int key0 = (int)(nextf - ahead.start - OVER) * UNIT;
      if (key0 < ahead.s.len) r = Ref{page_entry(p, ahead.b, key0), key0 % p.page_size, ahead.h};
    }
    nextf += L::WARPS;
    return r;
  };
  int st_load = 0;
  auto load_unit = [&](const Ref& u) {
    if (u.h >= 0) {
      const long long page = checked_page(p, u.entry);
      const T* kp = static_cast<const T*>(p.kc) + page * p.k_ps + u.h * p.k_hs + u.row0 * p.k_rs;
      const T* vp = static_cast<const T*>(p.vc) + page * p.v_ps + u.h * p.v_hs + u.row0 * p.v_rs;
      constexpr int V = 16 / (int)sizeof(T), CH = D / V;  // 16-byte chunks of a row
      Tile<T, UNIT, D> Kt{reinterpret_cast<T*>(ring + st_load * 2 * L::TILE)};
      Tile<T, UNIT, D> Vt{reinterpret_cast<T*>(ring + (st_load * 2 + 1) * L::TILE)};
#pragma unroll
      for (int q = 0; q < UNIT * CH / 32; ++q) {
        const int r = (q * 32 + lane) / CH, c = (q * 32 + lane) % CH * V;
        cp_async16(Kt.ptr(r, c), kp + r * p.k_rs + c);
      }
#pragma unroll
      for (int q = 0; q < UNIT * CH / 32; ++q) {
        const int r = (q * 32 + lane) / CH, c = (q * 32 + lane) % CH * V;
        cp_async16(Vt.ptr(r, c), vp + r * p.v_rs + c);
      }
    }
    cp_async_commit();
    st_load = st_load + 1 == L::STAGES ? 0 : st_load + 1;
  };
  // the queries of an item, this thread's 16-byte pieces (rows past the end are zero)
  constexpr int QV = 16 / (int)sizeof(T), QCH = D / QV, QN = (ROWS * QCH + L::THREADS - 1) / L::THREADS;
  uint4 qr[QN];
  auto load_q = [&](const Item& it) {
#pragma unroll
    for (int i = 0; i < QN; ++i) {
      const int q = tid + i * L::THREADS, r = it.i * ROWS + q / QCH;
      qr[i] = make_uint4(0u, 0u, 0u, 0u);
      if (q < ROWS * QCH && r < it.s.n * G)
        qr[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (it.s.first + r / G) * a.q_ts +
                                                (long long)(it.h * G + r % G) * a.q_hs + q % QCH * QV);
    }
  };
  auto store_q = [&]() {
#pragma unroll
    for (int i = 0; i < QN; ++i) {
      const int q = tid + i * L::THREADS;
      if (q >= ROWS * QCH) continue;
      T* at = Qs.ptr(q / QCH, q % QCH * QV);
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(at) = qr[i];
      } else {  // split once for the item
        uint4 h, l;
        tf32_split(__uint_as_float(qr[i].x), h.x, l.x);
        tf32_split(__uint_as_float(qr[i].y), h.y, l.y);
        tf32_split(__uint_as_float(qr[i].z), h.z, l.z);
        tf32_split(__uint_as_float(qr[i].w), h.w, l.w);
        *reinterpret_cast<uint4*>(at) = h;
        *reinterpret_cast<uint4*>(at + ROWS * D) = l;
      }
    }
  };
  load_q(cur);
  Ref ref;
  {
    Ref first[L::STAGES - 1];
#pragma unroll
    for (int i = 0; i < L::STAGES - 1; ++i) first[i] = look_up();
    ref = look_up();
#pragma unroll
    for (int i = 0; i < L::STAGES - 1; ++i) load_unit(first[i]);
  }
  store_q();

  int st = 0;
  long long f = lo + warp;  // the next unit to use
  const float c = a.scale * LOG2E;
  while (true) {
    const int row0 = cur.i * ROWS, rows = min(ROWS, cur.s.n * G - row0);
    __syncthreads();  // the item's queries are in place
    uint32_t qf[sizeof(T) == 2 ? D / 16 : 1][4];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) load_a(qf[ks], aview<false>(Qs), 0, ks * 16, lane);
    }
    // last key each of this thread's two rows sees
    const int p0 = cur.s.len - cur.s.n;
    int lim[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) lim[e] = g + 8 * e < rows ? p0 + (row0 + g + 8 * e) / G : -1;
    const int lim_min = p0 + row0 / G;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;

    const long long end = cur.end < hi ? cur.end : hi;
    while (f < cur.start + OVER) f += L::WARPS;
    for (; f < end; f += L::WARPS) {
      load_unit(ref);
      ref = look_up();
      cp_async_wait<L::STAGES - 1>();
      __syncwarp();
      const int key0 = (int)(f - cur.start - OVER) * UNIT;
      Tile<T, UNIT, D> Kt{reinterpret_cast<T*>(ring + st * 2 * L::TILE)};
      Tile<T, UNIT, D> Vt{reinterpret_cast<T*>(ring + (st * 2 + 1) * L::TILE)};
      st = st + 1 == L::STAGES ? 0 : st + 1;
      if (key0 + UNIT > cur.s.len) {  // rows of the page past the length hold anything: 0 * NaN is not 0
        constexpr int V = 16 / (int)sizeof(T), CH = D / V;
        const int keep = max(cur.s.len - key0, 0);
        for (int q = lane; q < (UNIT - keep) * CH; q += 32)
          *reinterpret_cast<uint4*>(Vt.ptr(keep + q / CH, q % CH * V)) = make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
      }
      float s[1][2][4];
      zero<1, 2>(s);
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t b[4];
          load_b2(b, bview<false>(Kt), 0, ks * 16, lane);
          mma_bf16(s[0][0], qf[ks], b);
          mma_bf16(s[0][1], qf[ks], b + 2);
        }
      } else {
        // each step of eight channels starts from zero and is added in fp32: the tensor core's own
        // accumulation truncates, which over D channels costs a digit. Two steps at a time, so
        // that four chains of dependent products overlap.
#pragma unroll
        for (int k0 = 0; k0 < D; k0 += 16) {
          uint32_t ah[2][4], al[2][4], bh[2][2][2], bl[2][2][2];
          float x[2][2][4];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int k = k0 + 8 * u + t;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const T* at = Qs.ptr(g + 8 * (e & 1), k + 4 * (e >> 1));
              ah[u][e] = __float_as_uint(at[0]);
              al[u][e] = __float_as_uint(at[ROWS * D]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              tf32_cut(Kt.at(8 * j + g, k), bh[u][j][0], bl[u][j][0]);
              tf32_cut(Kt.at(8 * j + g, k + 4), bh[u][j][1], bl[u][j][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) x[u][j][e] = 0.f;
            }
          }
#pragma unroll
          for (int term = 0; term < 3; ++term)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int j = 0; j < 2; ++j) mma_tf32(x[u][j], term == 0 ? al[u] : ah[u], term == 1 ? bl[u][j] : bh[u][j]);
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[0][j][e] += x[u][j][e];
        }
      }
      // scores in base 2; hidden keys are -inf
      const bool mask = key0 + UNIT - 1 > lim_min;
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = s[0][j][e] * c;
          if (mask && key0 + j * 8 + frag_col(lane, e) > lim[e >> 1]) x = -INFINITY;
          s[0][j][e] = x;
          top[e >> 1] = fmaxf(top[e >> 1], x);
        }
      float ref[2];
      bool moved = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
        moved |= top[e] > m[e];
      }
      if (__any_sync(0xffffffffu, moved)) {
        float fac[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float nm = fmaxf(m[e], top[e]);
          fac[e] = m[e] == nm ? 1.f : exp2f(m[e] - nm);  // m = -inf: 0
          m[e] = nm;
          l[e] *= fac[e];
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] *= fac[e >> 1];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) ref[e] = m[e] == -INFINITY ? 0.f : m[e];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[0][j][e] = exp2f(s[0][j][e] - ref[e >> 1]);
          l[e >> 1] += s[0][j][e];
        }
      // the score fragment is the second product's A fragment
      if constexpr (sizeof(T) == 2) {
        uint32_t pa[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(s[0][q >> 1][(q & 1) * 2], s[0][q >> 1][(q & 1) * 2 + 1]);
          pa[q] = *reinterpret_cast<const uint32_t*>(&h);
        }
#pragma unroll
        for (int n0 = 0; n0 < D; n0 += 16) {
          uint32_t b[4];
          load_b2(b, bview<true>(Vt), n0, 0, lane);
          mma_bf16(o[n0 / 8], pa, b);
          mma_bf16(o[n0 / 8 + 1], pa, b + 2);
        }
      } else {
        // keys 2t and 2t + 1 of each eight stand at k = t and t + 4, in both operands
        uint32_t ah[2][4], al[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          tf32_split(s[0][j][0], ah[j][0], al[j][0]);
          tf32_split(s[0][j][2], ah[j][1], al[j][1]);
          tf32_split(s[0][j][1], ah[j][2], al[j][2]);
          tf32_split(s[0][j][3], ah[j][3], al[j][3]);
        }
#pragma unroll
        for (int n0 = 0; n0 < D / 8; n0 += 4) {  // four chains of dependent products
          uint32_t bh[4][2][2], bl[4][2][2];
          float x[4][4];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              tf32_cut(Vt.at(j * 8 + 2 * t, (n0 + n) * 8 + g), bh[n][j][0], bl[n][j][0]);
              tf32_cut(Vt.at(j * 8 + 2 * t + 1, (n0 + n) * 8 + g), bh[n][j][1], bl[n][j][1]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int term = 0; term < 3; ++term)
#pragma unroll
              for (int n = 0; n < 4; ++n) mma_tf32(x[n], term == 0 ? al[j] : ah[j], term == 1 ? bl[n][j] : bh[n][j]);
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n0 + n][e] += x[n][e];
        }
      }
      __syncwarp();  // the stage is loaded again by other lanes
    }
    // the next item's queries are on their way while the warps are merged
    const bool more = cur.end < hi;
    Item nxt = cur;
    if (more) {
      Num::next_item(p, G, nxt);
      load_q(nxt);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      if (t == 0) {
        sml[warp * ROWS + g + 8 * e] = m[e];
        sml[(L::WARPS + warp) * ROWS + g + 8 * e] = l[e];
      }
    }
    __syncthreads();
    const bool whole = cur.start >= lo && cur.end <= hi;
    float* part = Parts<ROWS, D>::slot(a.ws, blockIdx.x, cur.start < lo ? 0 : 1);
    if (tid < ROWS) {
      float M = -INFINITY, lt = 0.f;
#pragma unroll
      for (int w = 0; w < L::WARPS; ++w) M = fmaxf(M, sml[w * ROWS + tid]);
#pragma unroll
      for (int w = 0; w < L::WARPS; ++w)
        lt += sml[(L::WARPS + w) * ROWS + tid] * part_factor(sml[w * ROWS + tid], M);
      tot[tid] = M;
      tot[ROWS + tid] = lt;
      if (tid < rows) {
        if (!whole) {
          part[ROWS * D + tid] = M;
          part[ROWS * D + ROWS + tid] = lt;
        } else if (a.lse) {
          const int qr = row0 + tid;
          a.lse[(size_t)(cur.s.first + qr / G) * p.Hq + cur.h * G + qr % G] = lt == 0.f ? -INFINITY : (M + log2f(lt)) * LN2;
        }
      }
    }
    float fac[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float M = -INFINITY;
      for (int w = 0; w < L::WARPS; ++w) M = fmaxf(M, sml[w * ROWS + g + 8 * e]);
      fac[e] = part_factor(m[e], M);
    }
    for (int r0 = 0; r0 < rows; r0 += L::MROWS) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = g + 8 * e - r0;
        if (r >= 0 && r < L::MROWS) {
          float* d = merge + ((size_t)warp * L::MROWS + r) * D + 2 * t;
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            *reinterpret_cast<float2*>(d + j * 8) = make_float2(o[j][2 * e] * fac[e], o[j][2 * e + 1] * fac[e]);
        }
      }
      __syncthreads();
      for (int q = tid; q < L::MROWS * (D / 4); q += L::THREADS) {
        const int r = r0 + q / (D / 4), col = q % (D / 4) * 4;
        if (r >= rows) continue;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < L::WARPS; ++w) {
          const float4 v = *reinterpret_cast<const float4*>(merge + (w * L::MROWS + r - r0) * D + col);
          sum[0] += v.x; sum[1] += v.y; sum[2] += v.z; sum[3] += v.w;
        }
        if (whole) {
          const int qr = row0 + r, tok = cur.s.first + qr / G, head_ = cur.h * G + qr % G;
          const float inv = tot[ROWS + r] == 0.f ? 0.f : 1.f / tot[ROWS + r];
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] *= inv;
          st4(static_cast<T*>(a.out) + tok * a.o_ts + head_ * a.o_hs + col, sum);
        } else {
          st4(part + r * D + col, sum);
        }
      }
      __syncthreads();
    }
    if (!more) {
      if (tid == 0) {
        int more = 0;
        if (cur.start >= lo && cur.end > hi) more = holder(run.total, run.ncta, cur.end - 1) - blockIdx.x;
        *head = PartHead{more, row0, rows, cur.s.first, cur.h, {0, 0, 0}};
      }
      break;
    }
    cur = nxt;
    store_q();
  }
  cp_async_wait<0>();
}

// Joins the parts of the item that begins in CTA blockIdx.x and goes on in the next ones:
// o = sum_c o_c 2^(m_c - m), in the order of the CTAs. A thread per row and four columns.
template <class T, int D>
__global__ void __launch_bounds__(ROWS * D / 4) paged_attn_join_kernel(AttnArgs a) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x;
  const int r = threadIdx.x / (D / 4), col = threadIdx.x % (D / 4) * 4;
  constexpr size_t STEP = 2 * Parts<ROWS, D>::SLOT;  // from one CTA's slot to the next CTA's
  constexpr int BATCH = 8;
  const float *first = Parts<ROWS, D>::slot(a.ws, c, 1), *rest = Parts<ROWS, D>::slot(a.ws, c + 1, 0);
  float M = -INFINITY, o[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
  const PartHead h = part_heads<ROWS, D>(a.ws, gridDim.x)[c];
  if (h.more == 0 || r >= h.rows) return;
  for (int q0 = 0; q0 <= h.more; q0 += BATCH) {  // parts in batches, all of a batch's loads in flight
    float m[BATCH], s[BATCH];
    float4 v[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int q = q0 + i;  // part 0 is this CTA's
      const float* part = q == 0 ? first : rest + (size_t)(min(q, h.more) - 1) * STEP;
      m[i] = part[ROWS * D + r];
      s[i] = part[ROWS * D + ROWS + r];
      v[i] = *reinterpret_cast<const float4*>(part + r * D + col);
    }
    float top = M;
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (q0 + i <= h.more) top = fmaxf(top, m[i]);
    const float f = part_factor(M, top);
    M = top;
    l *= f;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] *= f;
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (q0 + i <= h.more) {
        const float w = part_factor(m[i], M);
        o[0] += v[i].x * w; o[1] += v[i].y * w; o[2] += v[i].z * w; o[3] += v[i].w * w;
        l += s[i] * w;
      }
  }
  const int G = a.p.Hq / a.p.Hk, qr = h.row0 + r, tok = h.first + qr / G, head = h.h * G + qr % G;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] *= inv;
  st4(static_cast<T*>(a.out) + tok * a.o_ts + head * a.o_hs + col, o);
  if (a.lse && col == 0) a.lse[(size_t)tok * a.p.Hq + head] = l == 0.f ? -INFINITY : (M + log2f(l)) * LN2;
}

// Units that make a CTA take part: one for each warp, or an item of the longest length.
int units_least(const AttnArgs& a, int warps) {
  const int most = (a.max_kv - 1) / UNIT + 1;
  return most < 1 ? 1 : most < warps ? most : warps;
}

template <class T, int D, int OVER>
cudaError_t run(const AttnArgs& a, cudaStream_t s) {
  typedef Lay<T, D> L;
  const int bytes = L::BYTES + 1024;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_shared(reinterpret_cast<const void*>(paged_attn_kernel<T, D, OVER>), bytes, &allowed);
  if (e != cudaSuccess) return e;
  const int least = units_least(a, L::WARPS), grid = launch_ctas(a, ROWS, UNIT, 0, least);
  prof_mark(K_ATTN, s, true);
  e = launch_pdl(paged_attn_kernel<T, D, OVER>, dim3(grid), dim3(L::THREADS), bytes, s, a, least);
  prof_mark(K_ATTN, s, false);
  if (e != cudaSuccess) return e;
  prof_mark(K_ATTN_JOIN, s, true);
  e = launch_pdl(paged_attn_join_kernel<T, D>, dim3(grid), dim3(ROWS * D / 4), 0, s, a);
  prof_mark(K_ATTN_JOIN, s, false);
  return e;
}

template <class T, int D>
cudaError_t pick(const AttnArgs& a, cudaStream_t s) {
  const int nsm = device_sm_count() > 0 ? device_sm_count() : 152;
  return launch_items(a, ROWS) < nsm ? run<T, D, 0>(a, s) : run<T, D, units_over(warps_of(D, sizeof(T)), sizeof(T))>(a, s);
}

}  // namespace

size_t paged_attn_workspace(const AttnArgs& a) {
  const int warps = warps_of(a.p.D, a.p.bf16 ? 2 : 4);
  const int grid = launch_ctas(a, ROWS, UNIT, 0, units_least(a, warps));
  const size_t own = a.p.D == 64 ? Parts<ROWS, 64>::bytes(grid) : Parts<ROWS, 128>::bytes(grid);
  const size_t tc = paged_attn_tc_applies(a) ? paged_attn_tc_workspace(a) : 0;
  return own > tc ? own : tc;
}

cudaError_t launch_paged_attn(const AttnArgs& a, cudaStream_t s) {
  if (paged_attn_tc_applies(a)) {
    bool done = false;
    const cudaError_t e = launch_paged_attn_tc(a, s, &done);
    if (done || e != cudaSuccess) return e;
  }
  if (a.p.bf16) return a.p.D == 64 ? pick<bf16, 64>(a, s) : pick<bf16, 128>(a, s);
  return a.p.D == 64 ? pick<float, 64>(a, s) : pick<float, 128>(a, s);
}

}  // namespace gdn
