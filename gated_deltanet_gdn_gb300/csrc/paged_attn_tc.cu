// Attention of new tokens over a paged key/value cache on the 5th-generation tensor cores
// (bf16), for chunks and prompts: items of up to 256 query rows of one (sequence, KV head),
// two tiles of 128 rows that share every key tile.
//
// Per tile of 128 keys and 128 rows: S = Q K^T (tcgen05, fp32 in tensor memory), the
// softmax of a row in the registers of one thread, P (bf16) back into tensor memory as the
// A operand of O += P V. One pass with a running maximum: O is only rescaled when a row's
// maximum has grown by more than 2^8 over the one in use, so nearly never after the first
// tiles (the sums stay exact: P, its sum and O refer to the same maximum).
//
// Two warpgroups of softmax threads (one row tile each, a thread per row), and in a third
// one warp that issues every MMA and one that feeds a ring of key and value tiles by TMA, a box
// per run of rows inside one page. The tensor pipe works on one row tile's products while
// the other tile's softmax runs:
//   ... PV0(j) QK0(j+1) | PV1(j) QK1(j+1) | PV0(j+1) ...
// P takes the first half of its tile's S columns at D = 128 (MMAs of one shape execute in
// issue order, so QK(j+1) cannot overtake the PV(j) that reads P); at D = 64 it has columns
// of its own.
//
// Few items are split over the keys (a fixed number of splits per call, equal runs of
// tiles per item); the parts go to the workspace and a second kernel joins them in order.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "paged_attn.cuh"
#include "umma.cuh"

namespace gdn {
namespace {

constexpr int ROWS = 256, HALF = 128, KT = 128;  // query rows of an item, of a tile; keys of a tile
constexpr int THREADS = 384;  // three warpgroups: two of softmax, and one with the two warps below
constexpr int MMA_WARP = 8, LOAD_WARP = 9;
// Registers a thread, moved from the third warpgroup to the softmax (which holds 128 scores):
// the launch has 168 each, 2 * 224 + 56 = 3 * 168.
constexpr int SOFTMAX_REGS = 224, OTHER_REGS = 56;
constexpr float RESCALE = 8.f;  // growth of the maximum (base 2) that rescales O

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int D>
struct TcLay {
  static constexpr int SLOT = KT * D * 2;                // one K or V tile
  static constexpr int SLOTS = D == 128 ? 5 : 8;
  static constexpr int Q = 0;                            // two [128][D] tiles
  static constexpr int RING = 2 * HALF * D * 2;
  static constexpr int BAR = RING + SLOTS * SLOT;
  // barriers: full[SLOTS], empty[SLOTS], q[2], s[2], p[2], o[2], drained
  static constexpr int NBAR = 2 * SLOTS + 9;
  static constexpr int TSLOT = BAR + NBAR * 8;
  static constexpr int BYTES = TSLOT + 16;
  // tensor memory columns
  static constexpr int S = 0, O = 256, P = D == 128 ? 0 : 256 + 2 * D;
  static constexpr int P_STEP = D == 128 ? 128 : 64;     // between the two tiles' P
};

// Four MMAs along K (64 channels of Q and K, or 64 keys of P and V), called by a whole warp
// and issued by the lane that elect.sync names, the same one every time. The descriptors'
// steps are added inside: kept outside, the compiler holds every step of every tile in
// registers, and the warp spends more time on them than the tensor cores on the products.
__device__ __forceinline__ void umma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 x, y;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n setp.eq.b32 p, 0, 0;\n"
      " add.s64 x, %1, 2;\n add.s64 y, %2, 2;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n"
      " add.s64 x, %1, 4;\n add.s64 y, %2, 4;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n"
      " add.s64 x, %1, 6;\n add.s64 y, %2, 6;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A[tmem]: 16-bit pairs in 32-bit columns; B MN-major, 2048 bytes a step.
__device__ __forceinline__ void umma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b32 x;\n .reg .b64 y;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n setp.eq.b32 p, 0, 0;\n"
      " add.u32 x, %1, 8;\n add.s64 y, %2, 128;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, p;\n"
      " add.u32 x, %1, 16;\n add.s64 y, %2, 256;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, p;\n"
      " add.u32 x, %1, 24;\n add.s64 y, %2, 384;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// umma_commit by the elected lane.
__device__ __forceinline__ void commit_elected(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const void* map, int c0, int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];\n" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// An item of one CTA: rows row0 .. row0 + rows - 1 of (sequence, KV head), key tiles
// [t0, t1) of the item's `tiles`, and the tiles each row half needs.
struct TcItem {
  int b, h, row0, rows, p0;
  Seq s;
  int tiles, t0, t1, splits, need[2];
};

__device__ __forceinline__ int tile_count(const Seq& s, int G, int last_row) {
  const int limit = s.len - s.n + last_row / G;
  return limit < 0 ? 0 : limit / KT + 1;
}
// Item `idx` (one warp, all lanes). Sequences and the items of a sequence are numbered from
// the last, the one with the most keys first, and the KV heads of a run of rows side by
// side. False when there are fewer items.
__device__ __forceinline__ bool find_item(const PagedArgs& p, int G, int lane, int idx, int split, int splits, TcItem& it) {
  int run = idx / p.Hk;
  it.h = idx % p.Hk;
  it.b = -1;
  for (int b0 = p.B - 1; b0 >= 0; b0 -= 32) {
    const int b = b0 - lane;
    const Seq s = b >= 0 ? load_seq(p, b, false) : Seq{0, 0, 0};
    const int n = (s.n * G + ROWS - 1) / ROWS;
    int inc = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += o;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, inc > run);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const int before = __shfl_sync(0xffffffffu, inc - n, l), count = __shfl_sync(0xffffffffu, n, l);
      it.b = b0 - l;
      it.s.n = __shfl_sync(0xffffffffu, s.n, l);
      it.s.first = __shfl_sync(0xffffffffu, s.first, l);
      it.s.len = __shfl_sync(0xffffffffu, s.len, l);
      it.row0 = (count - 1 - (run - before)) * ROWS;
      break;
    }
    run -= __shfl_sync(0xffffffffu, inc, 31);
  }
  if (it.b < 0) return false;
  it.rows = min(ROWS, it.s.n * G - it.row0);
  it.p0 = it.s.len - it.s.n;
  it.tiles = tile_count(it.s, G, it.row0 + it.rows - 1);
  const int per = max((it.tiles + splits - 1) / splits, 1);
  it.splits = max((it.tiles + per - 1) / per, 1);
  it.t0 = min(split * per, it.tiles);
  it.t1 = min(it.t0 + per, it.tiles);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int last = min(it.rows, (w + 1) * HALF) - 1;
    const int t = last >= w * HALF ? tile_count(it.s, G, it.row0 + last) : 0;
    it.need[w] = max(min(t, it.t1) - it.t0, 0);
  }
  return true;
}

// Part of item-split c: o [256][D] relative to m, then m [256] (base 2), l [256].
template <int D>
__device__ __forceinline__ float* tc_part(float* ws, size_t c) {
  return ws + c * (ROWS * (D + 2));
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    paged_attn_tc_kernel(AttnArgs a, int splits, int box_rows, const __grid_constant__ CUtensorMap k_map,
                         const __grid_constant__ CUtensorMap v_map) {
  pdl_wait();
  pdl_trigger();
  typedef TcLay<D> L;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  const PagedArgs& p = a.p;
  const int G = p.Hq / p.Hk;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  TcItem it;
  if (!find_item(p, G, lane, blockIdx.x / splits, blockIdx.x % splits, splits, it)) return;
  if (p.err && warp == 0 && lane == 0 && p.lens[it.b] > (long long)p.max_pages * p.page_size) atomicOr(p.err, ERR_PAGE);
  if ((int)(blockIdx.x % splits) >= it.splits) return;

  if (warp < MMA_WARP && it.need[warp >> 2] > 0) {
    // The queries of a row tile, rows past the end zero: a thread takes 16 bytes of every
    // STEP-th row, all in flight at once (cp.async), while the CTA sets itself up.
    constexpr int CH = D / 8, STEP = HALF / CH;
    const int w = warp >> 2, r = tid & (HALF - 1), col = r % CH * 8;
    Tile<bf16, HALF, D> Qs{reinterpret_cast<bf16*>(sm + L::Q + w * HALF * D * 2)};
    int row = r / CH, g = it.row0 + w * HALF + row, tok = it.s.first + g / G, sub = g % G;
    const int dt = STEP / G, ds = STEP % G;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (w * HALF + row < it.rows)
        cp_async16(Qs.ptr(row, col),
                   static_cast<const bf16*>(a.q) + tok * a.q_ts + (long long)(it.h * G + sub) * a.q_hs + col);
      else
        *reinterpret_cast<uint4*>(Qs.ptr(row, col)) = make_uint4(0u, 0u, 0u, 0u);
      row += STEP;
      tok += dt;
      sub += ds;
      if (sub >= G) {
        sub -= G;
        ++tok;
      }
    }
    cp_async_commit();
  }

  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint64_t *full = bars, *empty = bars + L::SLOTS, *qbar = bars + 2 * L::SLOTS, *sbar = qbar + 2, *pbar = sbar + 2,
           *obar = pbar + 2, *drained = obar + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + L::TSLOT);
  if (tid == 0) {
    for (int i = 0; i < 2 * L::SLOTS; ++i) mbar_init(&bars[i], 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&qbar[w], HALF);
      mbar_init(&sbar[w], 1);
      mbar_init(&pbar[w], HALF);
      mbar_init(&obar[w], 1);
    }
    mbar_init(drained, 1);
    fence_mbar_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *tslot;
  const int n = max(it.need[0], it.need[1]);  // key tiles of this CTA

  if (warp < MMA_WARP) {
    // ---------------------------------------------------------------- softmax
    more_registers<SOFTMAX_REGS>();
    const int w = warp >> 2, r = tid & (HALF - 1);  // row tile, row of it
    const int row = w * HALF + r;                   // row of the item
    Tile<bf16, HALF, D> Qs{reinterpret_cast<bf16*>(sm + L::Q + w * HALF * D * 2)};
    const int need = it.need[w];
    if (need > 0) {  // the queries, on their way since before the barrier
      cp_async_wait<0>();
      fence_proxy_async();
      mbar_arrive(&qbar[w]);
    }
    const int lim = row < it.rows ? it.p0 + (it.row0 + row) / G : -1;
    const int lim_min = it.p0 + (it.row0 + w * HALF) / G;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's quarter of tensor memory
    const uint32_t ts = tm + lanes + L::S + w * 128, tp = tm + lanes + L::P + w * L::P_STEP, to = tm + lanes + L::O + w * D;
    const float c = a.scale * LOG2E;
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < need; ++j) {
      mbar_wait(&sbar[w], j & 1, p.err);
      tc_fence_after();
      uint32_t s[4][32];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld32_nowait(ts + 32 * i, s[i]);
      tmem_wait_ld();
      const int key0 = (it.t0 + j) * KT;
      if (key0 + KT - 1 > lim_min) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (key0 + 32 * i + e > lim) s[i][e] = 0xff800000u;
      }
      float top[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        top[i] = __uint_as_float(s[i][0]);
#pragma unroll
        for (int e = 1; e < 32; ++e) top[i] = fmaxf(top[i], __uint_as_float(s[i][e]));
      }
      const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
      const bool grow = mx > m + RESCALE;  // also the first finite maximum
      if (j == 0) {
        m = mx;
      } else if (__any_sync(0xffffffffu, grow)) {
        const float nm = grow ? mx : m;
        const float f = grow ? ex2(m - nm) : 1.f;  // m = -inf: 0
        m = nm;
        l *= f;
        mbar_wait(&obar[w], (j - 1) & 1, p.err);  // the last PV has completed
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t o[32];
          tmem_ld32_nowait(to + 32 * i, o);
          tmem_wait_ld();
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(o[e]) * f;
          tmem_st32(to + 32 * i, v);
        }
        tmem_wait_st();
      }
      const float ref = m == -INFINITY ? 0.f : -m;
      const uint64_t c2 = pair(c, c), r2 = pair(ref, ref);
      uint64_t sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t o[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float x0, x1;
          unpair(fma2(pair(__uint_as_float(s[i][2 * e]), __uint_as_float(s[i][2 * e + 1])), c2, r2), x0, x1);
          x0 = ex2(x0);
          x1 = ex2(x1);
          sum[e & 1] = add2(sum[e & 1], pair(x0, x1));
          const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
          o[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
        tmem_st16(tp + 16 * i, o);
      }
      float s0, s1;
      unpair(add2(sum[0], sum[1]), s0, s1);
      l += s0 + s1;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&pbar[w]);
    }
    // the tile's output, or its part
    if (need > 0) {
      mbar_wait(&obar[w], (need - 1) & 1, p.err);
      tc_fence_after();
    }
    const bool live = row < it.rows;
    const bool none = need == 0 || m == -INFINITY;
    if (it.splits == 1) {
      // Through shared memory (the tile's queries are done with), so that a warp stores whole
      // rows: a row per lane would touch 32 lines with every store.
      const float inv = none ? 0.f : 1.f / l;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t o[32];
        if (need > 0) {
          tmem_ld32_nowait(to + 32 * i, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint32_t u[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float v0 = none ? 0.f : __uint_as_float(o[e + 2 * x]) * inv;
            const float v1 = none ? 0.f : __uint_as_float(o[e + 2 * x + 1]) * inv;
            const __nv_bfloat162 h = __floats2bfloat162_rn(v0, v1);
            u[x] = *reinterpret_cast<const uint32_t*>(&h);
          }
          *reinterpret_cast<uint4*>(Qs.ptr(r, 32 * i + e)) = make_uint4(u[0], u[1], u[2], u[3]);
        }
      }
      if (live && a.lse) {
        const int g = it.row0 + row;
        a.lse[(size_t)(it.s.first + g / G) * p.Hq + it.h * G + g % G] = none ? -INFINITY : (m + log2f(l)) * LN2;
      }
      __syncwarp();
      constexpr int CH = D / 8, STEP = 32 / CH;  // rows of one store
#pragma unroll 4
      for (int i = 0; i < CH; ++i) {
        const int rr = (warp & 3) * 32 + i * STEP + lane / CH, col = lane % CH * 8, g = it.row0 + w * HALF + rr;
        if (w * HALF + rr < it.rows)
          *reinterpret_cast<uint4*>(static_cast<bf16*>(a.out) + (it.s.first + g / G) * a.o_ts +
                                    (long long)(it.h * G + g % G) * a.o_hs + col) =
              *reinterpret_cast<const uint4*>(Qs.ptr(rr, col));
      }
    } else {
      float* part = tc_part<D>(a.ws, blockIdx.x);
      if (live) {
        part[ROWS * D + row] = none ? -INFINITY : m;
        part[ROWS * D + ROWS + row] = l;
      }
      if (need > 0) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t o[32];
          tmem_ld32_nowait(to + 32 * i, o);
          tmem_wait_ld();
          if (live)
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(part + (size_t)row * D + 32 * i + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
    }
    tc_fence_before();
  } else {
    fewer_registers<OTHER_REGS>();
  }
  if (warp == MMA_WARP) {
    // ---------------------------------------------------------------- products
    constexpr uint32_t id_s = umma_idesc_bf16(HALF, KT), id_o = umma_idesc_bf16(HALF, D, false, true);
    constexpr int PANEL = KT * 128;
    // warp-uniform by construction, and known to be to the compiler
    const int need[2] = {__shfl_sync(0xffffffffu, it.need[0], 0), __shfl_sync(0xffffffffu, it.need[1], 0)};
    const int tiles = max(need[0], need[1]), keys = __shfl_sync(0xffffffffu, it.s.len - it.t0 * KT, 0);
    const uint32_t acc = __shfl_sync(0xffffffffu, tm, 0);
    const uint64_t dq = desc_kmajor(sm + L::Q), dring = desc_kmajor(sm + L::RING),
                   dvring = desc_mnmajor(sm + L::RING, PANEL);
    int slot = 0;
    uint32_t phase = 0;
    auto next_slot = [&]() {
      if (++slot == L::SLOTS) {
        slot = 0;
        phase ^= 1;
      }
    };
    auto scores = [&](int w, int kslot) {
      const uint64_t q = dq + (uint64_t)(w * (HALF * D * 2 / 16)), k = dring + (uint64_t)(kslot * (L::SLOT / 16));
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
        umma4_ss(acc + L::S + w * 128, q + h * (PANEL / 16), k + h * (PANEL / 16), id_s, h > 0);
      commit_elected(&sbar[w]);
    };
    for (int w = 0; w < 2; ++w)
      if (need[w] > 0) mbar_wait(&qbar[w], 0, p.err);
    tc_fence_after();
    if (tiles > 0) {
      mbar_wait(&full[slot], phase, p.err);
      for (int w = 0; w < 2; ++w)
        if (need[w] > 0) scores(w, slot);
      commit_elected(&empty[slot]);
      next_slot();
    }
    for (int j = 0; j < tiles; ++j) {
      const int vslot = slot;
      mbar_wait(&full[vslot], phase, p.err);
      next_slot();
      const int kslot = slot;
      const uint32_t kphase = phase;
      const bool more = j + 1 < tiles;
      if (more) next_slot();
      const int keep = keys - j * KT;
      if (keep < KT) {  // rows past the length hold anything: 0 * NaN is not 0
        Tile<bf16, KT, D> Vs{reinterpret_cast<bf16*>(sm + L::RING + vslot * L::SLOT)};
        for (int q = lane; q < (KT - keep) * (D / 8); q += 32)
          *reinterpret_cast<uint4*>(Vs.ptr(keep + q / (D / 8), q % (D / 8) * 8)) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async();
        __syncwarp();
      }
      bool kready = false;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if (j < need[w]) {
          mbar_wait(&pbar[w], j & 1, p.err);
          tc_fence_after();
          const uint64_t v = dvring + (uint64_t)(vslot * (L::SLOT / 16));
#pragma unroll
          for (int h = 0; h < 2; ++h)
            umma4_ts(acc + L::O + w * D, acc + L::P + w * L::P_STEP + 32 * h, v + h * 512, id_o, (j > 0 || h > 0) ? 1u : 0u);
          commit_elected(&obar[w]);
        }
        if (j + 1 < need[w]) {
          if (!kready) {
            mbar_wait(&full[kslot], kphase, p.err);
            kready = true;
          }
          scores(w, kslot);
        }
      }
      commit_elected(&empty[vslot]);
      if (more) commit_elected(&empty[kslot]);
    }
    commit_elected(drained);
    mbar_drain(drained, 0);
    tc_fence_before();
  } else if (warp == LOAD_WARP) {
    // ---------------------------------------------------------------- key and value tiles
    const int pieces = KT / box_rows;
    constexpr int PANELS = D / 64;
    int slot = 0, uses = 0;  // uses: loads issued
    for (int j = 0; j < n; ++j) {
      const int key0 = (it.t0 + j) * KT;
      const int have = min(pieces, (it.s.len - key0 + box_rows - 1) / box_rows);  // pieces with cached rows
      int page = 0, prow = 0;
      if (lane < have) {
        const int key = key0 + lane * box_rows;
        page = checked_page(p, page_entry(p, it.b, key));
        prow = key % p.page_size;
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (uses >= L::SLOTS) mbar_wait(&empty[slot], ((uses / L::SLOTS) - 1) & 1, p.err);
        if (lane == 0) mbar_arrive_expect_tx(&full[slot], (uint32_t)(have * box_rows * D * 2));
        __syncwarp();
        if (lane < have) {
          uint8_t* dst = sm + L::RING + slot * L::SLOT + lane * box_rows * 128;
#pragma unroll
          for (int c = 0; c < PANELS; ++c)
            tma_load_4d(dst + c * KT * 128, kv ? &v_map : &k_map, 64 * c, prow, it.h, page, &full[slot]);
        }
        ++uses;
        if (++slot == L::SLOTS) slot = 0;
      }
    }
    if (lane == 0) drain_ring(full, L::SLOTS, uses);
    __syncwarp();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == MMA_WARP) tmem_dealloc(tm, 512);
}

// Joins the parts of the split items: eight rows per CTA, a thread per four columns.
constexpr int JOIN_ROWS = 8;
template <int D>
__global__ void __launch_bounds__(JOIN_ROWS * D / 4) paged_attn_tc_join_kernel(AttnArgs a, int splits) {
  pdl_wait();
  const PagedArgs& p = a.p;
  const int G = p.Hq / p.Hk, lane = threadIdx.x & 31;
  TcItem it;
  if (!find_item(p, G, lane, blockIdx.x, 0, splits, it) || it.splits == 1) return;
  const int row = blockIdx.y * JOIN_ROWS + threadIdx.x / (D / 4), col = threadIdx.x % (D / 4) * 4;
  if (row >= it.rows) return;
  const float* first = tc_part<D>(a.ws, (size_t)blockIdx.x * splits);
  constexpr size_t STEP = ROWS * (D + 2);
  float M = -INFINITY;
  for (int s = 0; s < it.splits; ++s) M = fmaxf(M, first[s * STEP + ROWS * D + row]);
  float o[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
  for (int s = 0; s < it.splits; ++s) {
    const float m = first[s * STEP + ROWS * D + row];
    if (m == -INFINITY) continue;
    const float f = ex2(m - M);
    const float4 v = *reinterpret_cast<const float4*>(first + s * STEP + (size_t)row * D + col);
    o[0] += v.x * f; o[1] += v.y * f; o[2] += v.z * f; o[3] += v.w * f;
    l += first[s * STEP + ROWS * D + ROWS + row] * f;
  }
  const int g = it.row0 + row, tok = it.s.first + g / G, head = it.h * G + g % G;
  const float inv = M == -INFINITY ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] *= inv;
  st4(static_cast<bf16*>(a.out) + tok * a.o_ts + head * a.o_hs + col, o);
  if (a.lse && col == 0) a.lse[(size_t)tok * p.Hq + head] = M == -INFINITY ? -INFINITY : (M + log2f(l)) * LN2;
}

// Most items a call can have: full ones, and one that is not full per sequence.
long long item_bound(const AttnArgs& a) {
  const long long G = a.p.Hq / a.p.Hk, rows = (long long)a.p.N * G, seqs = a.p.B < a.p.N ? a.p.B : a.p.N;
  return (rows / ROWS + seqs) * a.p.Hk;
}
// Splits per item: the fewest SM-waves of key tiles, with a few tiles' time for an item's
// start and end, and for reading the parts again.
int split_count(const AttnArgs& a, int nsm) {
  const long long G = a.p.Hq / a.p.Hk;
  const long long per_seq = ((a.max_q < a.p.N ? a.max_q : a.p.N) * G + ROWS - 1) / ROWS;
  long long items = per_seq * a.p.B * a.p.Hk;
  if (item_bound(a) < items) items = item_bound(a);
  const long long tiles = ((long long)a.max_kv + KT - 1) / KT;
  long long best = 1, cost = 0;
  for (long long ns = 1; ns <= 64 && (ns == 1 || (items * ns <= TC_SPLIT_ITEMS && 2 * ns <= tiles)); ++ns) {
    const long long waves = (items * ns + nsm - 1) / nsm;
    const long long c = waves * ((tiles + ns - 1) / ns + 4) + (ns > 1 ? 4 + ns / 4 : 0);
    if (ns == 1 || c < cost) {
      best = ns;
      cost = c;
    }
  }
  return (int)best;
}

// [pages][heads][rows][D] bf16 with the cache's strides; box: 64 channels of `box` rows.
bool cache_map(CUtensorMap* map, void* base, const PagedArgs& p, long long ps, long long hs, long long rs, int box) {
  auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_fn());
  if (!encode) return false;
  // a dimension of one element has no stride of its own
  const auto step = [](long long s, int n) { return (cuuint64_t)(n > 1 ? s * 2 : 16); };
  const cuuint64_t dims[4] = {(cuuint64_t)p.D, (cuuint64_t)p.page_size, (cuuint64_t)p.Hk, (cuuint64_t)p.num_pages};
  const cuuint64_t strides[3] = {step(rs, p.page_size), step(hs, p.Hk), step(ps, p.num_pages)};
  const cuuint32_t b[4] = {64, (cuuint32_t)box, 1, 1}, one[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t run(const AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, int box, int nsm, cudaStream_t s) {
  const int bytes = TcLay<D>::BYTES + 1024;
  cudaError_t e = cudaFuncSetAttribute(paged_attn_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const int splits = split_count(a, nsm);
  const long long items = item_bound(a);
  prof_mark(K_ATTN_TC, s, true);
  e = launch_pdl(paged_attn_tc_kernel<D>, dim3((unsigned)(items * splits)), dim3(THREADS), bytes, s, a, splits, box, km, vm);
  prof_mark(K_ATTN_TC, s, false);
  if (e != cudaSuccess || splits == 1) return e;
  prof_mark(K_ATTN_TC_JOIN, s, true);
  e = launch_pdl(paged_attn_tc_join_kernel<D>, dim3((unsigned)items, ROWS / JOIN_ROWS), dim3(JOIN_ROWS * D / 4), 0, s, a, splits);
  prof_mark(K_ATTN_TC_JOIN, s, false);
  return e;
}

}  // namespace

bool paged_attn_tc_applies(const AttnArgs& a) {
  const long long G = a.p.Hq / a.p.Hk;
  return a.p.bf16 && (a.max_q < a.p.N ? a.max_q : a.p.N) * G > 16;
}

size_t paged_attn_tc_workspace(const AttnArgs& a) {
  const int nsm = device_sm_count();
  const int splits = split_count(a, nsm > 0 ? nsm : 152);
  return splits == 1 ? 0 : (size_t)item_bound(a) * splits * ROWS * (a.p.D + 2) * sizeof(float);
}

cudaError_t launch_paged_attn_tc(const AttnArgs& a, cudaStream_t s, bool* done) {
  *done = false;
  const int nsm = device_sm_count();
  if (nsm < 1) return cudaErrorInvalidDevice;
  int box = KT;  // rows of a box: a run inside one page and inside one tile
  while (a.p.page_size % box != 0) box >>= 1;
  CUtensorMap km{}, vm{};
  if (!cache_map(&km, a.p.kc, a.p, a.p.k_ps, a.p.k_hs, a.p.k_rs, box) ||
      !cache_map(&vm, a.p.vc, a.p, a.p.v_ps, a.p.v_hs, a.p.v_rs, box))
    return cudaSuccess;  // strides that a tensor map cannot hold: the caller takes the other kernel
  *done = true;
  return a.p.D == 64 ? run<64>(a, km, vm, box, nsm, s) : run<128>(a, km, vm, box, nsm, s);
}

}  // namespace gdn
