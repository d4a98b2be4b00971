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
// one warp that issues every MMA, two that feed a ring of key and value tiles by TMA (a box
// per run of rows inside one page; with pages of 16 one warp's issue would be the bound),
// and one that brings the queries (the first item's are the softmax warps'). The tensor
// pipe works on one row tile's products while the other tile's softmax runs:
//   ... PV0(j) QK0(j+1) | PV1(j) QK1(j+1) | PV0(j+1) ...
// P takes the first half of its tile's S columns at D = 128 (MMAs of one shape execute in
// issue order, so QK(j+1) cannot overtake the PV(j) that reads P); at D = 64 it has columns
// of its own.
//
// Two schedules, one body:
//  * few items: one persistent CTA per SM takes an equal run of the call's (item, key tile)
//    units, so neither ragged lengths, nor the causal triangle, nor fewer items than SMs
//    leave SMs idle. Every role walks the run by itself, so that the next item's keys and
//    queries are on their way, and its first product done, while this item's output is
//    written. An item that a CTA holds whole is written at once; at the ends of a CTA's run
//    the parts go to the workspace and a second kernel joins them in the order of the CTAs.
//  * many items (two or more per SM): the grid has a CTA per item, the sequences from the last,
//    each one's items from its longest and the KV heads of a run of rows side by side; the
//    CTAs that run at the same time then read the same keys at the same time, which the L2
//    serves once. A running CTA takes over the next one not yet launched (cluster launch
//    control) and goes on with its item, as above. An item is not cut here: 32 sequences that
//    decode over 16k to 62k keys beside a prompt of 8,192 tokens (48 and 8 heads) take 1,250 us
//    when they stand behind the prompt and 1,464 us in front of it, in calls of their own 774
//    and 565 us.
//
// Measured, heads of 128: a chunk of 2,048 tokens over 63k keys (16 and 4 heads, 128 items)
// 690-700 us, 1.56 PFLOP/s, in bursts and 770-790 us under the power limit; six prompts of up
// to 4,096 tokens (48 and 8 heads, 3,408 items) 604-626 us, 1.2 PFLOP/s, whichever order
// their lengths have (604-610 ascending, descending and mixed), where an item's output, queries and
// first softmax take about a fifth; 16 x 8 draft tokens over up to 16k keys (16 and 2 heads)
// 50 us, of which the stream of keys is 24 us and the start, merge and join the rest.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "paged_attn.cuh"
#include "umma.cuh"

namespace gdn {
namespace {

constexpr int ROWS = 256, HALF = 128, KT = 128;  // query rows of an item, of a tile; keys of a tile
constexpr int THREADS = 384;  // three warpgroups: two of softmax, and one of the warps below
constexpr int MMA_WARP = 8, KEY_WARP = 9, VALUE_WARP = 10, QUERY_WARP = 11;
constexpr int ITEM_READERS = 11;  // warps that read the next item: all but the query warp, which finds it
// Registers a thread, moved from the third warpgroup to the softmax (which holds 128 scores):
// the launch has 168 each, 2 * 216 + 72 = 3 * 168. (Six prompts of up to 4,096 tokens: 610 us; 208 and 88
// 610 us, 224 and 56 662 us.)
constexpr int SOFTMAX_REGS = 216, OTHER_REGS = 72;
constexpr float RESCALE = 8.f;  // growth of the maximum (base 2) that rescales O

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
// Asks for a CTA of the grid that has not been launched; the answer (16 bytes) lands in
// shared memory and completes on the barrier.
__device__ __forceinline__ void ask_next_cta(void* answer, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}
// The CTA taken over, or -1 when all have been launched.
__device__ __forceinline__ int next_cta(const void* answer) {
  uint32_t some, x;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 r;\n .reg .b32 y, z, w;\n ld.shared.b128 r, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, r;\n}\n"
      : "=r"(some), "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  return some ? (int)x : -1;
}

template <int D>
struct TcLay {
  static constexpr int SLOT = KT * D * 2;                // one K or V tile
  static constexpr int SLOTS = D == 128 ? 4 : 8;
  static constexpr int Q = 0;                            // two [128][D] tiles
  static constexpr int RING = 2 * HALF * D * 2;
  static constexpr int OUT = RING + SLOTS * SLOT;        // two fp32 [128][32] stages of a merge
  static constexpr int ML = OUT + HALF * 32 * 4;         // m, l of both row tiles, before the second stage's use
  static constexpr int BAR = OUT + 2 * HALF * 32 * 4;
  // barriers: full[SLOTS], empty[SLOTS], then q, qfree, s, o, p, item, itemfree [2] each,
  // drained, answer
  static constexpr int NBAR = 2 * SLOTS + 16;
  static constexpr int RUN = BAR + NBAR * 8;      // the CTA's run
  static constexpr int ITEM = RUN + 80;           // the next items, two in turn
  static constexpr int ANSWER = ITEM + 2 * 48;
  static constexpr int TSLOT = ANSWER + 16;
  static constexpr int BYTES = TSLOT + 16;
  static_assert(sizeof(Numbering<ROWS, KT, 0>::Run) <= 80 && sizeof(Item) <= 48, "run and items");
  static_assert(BYTES + 1024 <= 227 * 1024, "one CTA per SM");
  // tensor memory columns
  static constexpr int S = 0, O = 256, P = D == 128 ? 0 : 256 + 2 * D;
  static constexpr int P_STEP = D == 128 ? 128 : 64;     // between the two tiles' P
};

// The products of a tile and the arrival on their barrier when they have completed, in one
// block: called by a whole warp and issued by the lane that one elect.sync names. What the
// warp executes between a wait and the first product is on the path softmax, products,
// softmax, so the descriptors' steps are added inside (kept outside, the compiler holds
// every step of every tile in registers).
//
// S = Q K^T, 16 channels a step: both K-major in panels of 64 channels of 16 KB each.
#define GDN_SS_STEP(X) " add.s64 x, %1, " #X ";\n add.s64 y, %2, " #X ";\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n"
template <int D>
__device__ __forceinline__ void issue_scores(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint64_t* bar) {
  if constexpr (D == 64)
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .b64 x, y;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 p, 0, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n setp.eq.b32 p, 0, 0;\n"
        GDN_SS_STEP(2) GDN_SS_STEP(4) GDN_SS_STEP(6)
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(smem_u32(bar))
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .b64 x, y;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 p, 0, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n setp.eq.b32 p, 0, 0;\n"
        GDN_SS_STEP(2) GDN_SS_STEP(4) GDN_SS_STEP(6) GDN_SS_STEP(1024) GDN_SS_STEP(1026) GDN_SS_STEP(1028) GDN_SS_STEP(1030)
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(smem_u32(bar))
        : "memory");
}
#undef GDN_SS_STEP
// O (+)= P V, 16 keys a step. P in tensor memory: 16-bit pairs in 32-bit columns; V MN-major,
// 2048 bytes a step.
#define GDN_TS_STEP(X, Y) " add.u32 x, %1, " #X ";\n add.s64 y, %2, " #Y ";\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, p;\n"
__device__ __forceinline__ void issue_output(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b32 x;\n .reg .b64 y;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n setp.eq.b32 p, 0, 0;\n"
      GDN_TS_STEP(8, 128) GDN_TS_STEP(16, 256) GDN_TS_STEP(24, 384) GDN_TS_STEP(32, 512) GDN_TS_STEP(40, 640)
      GDN_TS_STEP(48, 768) GDN_TS_STEP(56, 896)
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(smem_u32(bar))
      : "memory");
}
#undef GDN_TS_STEP
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

// 32 bytes of a row: one store of whole sectors, or two of 16 bytes where rows are only
// aligned to those.
__device__ __forceinline__ void store32(bf16* dst, const uint32_t (&u)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(u[0]), "r"(u[1]), "r"(u[2]),
                 "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(u[0], u[1], u[2], u[3]);
    *reinterpret_cast<uint4*>(dst + 8) = make_uint4(u[4], u[5], u[6], u[7]);
  }
}

// An item's start and end take a CTA about as long as OVER key tiles.
constexpr int OVER = 3;
typedef Numbering<ROWS, KT, OVER> Num;
constexpr int MIN_UNITS = 3;  // units that make a CTA take part

// What a CTA does of one item: key tiles from t0 on, `need` of them for each row tile (none
// when its run ends before the item's keys, or the rows see none). An item of one row tile
// ("alone") has its rows in both, with the even key tiles for the first and the odd ones for
// the second; the two are merged at the end.
struct Segment {
  int row0, rows, p0, t0, need[2];
  bool alone;
  // the first row of row tile w in the item, and its j-th key tile
  __device__ __forceinline__ int base(int w) const { return alone ? 0 : w * HALF; }
  __device__ __forceinline__ int tile(int w, int j) const { return t0 + (alone ? 2 * j + w : j); }
  __device__ __forceinline__ int tiles() const { return alone ? need[0] + need[1] : max(need[0], need[1]); }
};
__device__ __forceinline__ Segment segment(const Item& it, int G, long long lo, long long hi) {
  Segment g;
  g.row0 = it.i * ROWS;
  g.rows = min(ROWS, it.s.n * G - g.row0);
  g.p0 = it.s.len - it.s.n;
  g.t0 = max((int)(lo > it.start ? lo - it.start : 0) - OVER, 0);
  const int t1 = (int)((hi < it.end ? hi : it.end) - it.start) - OVER;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int last = min(g.rows, (w + 1) * HALF) - 1;
    const int t = last >= w * HALF ? key_blocks<KT>(it.s, G, g.row0 + last) : 0;
    g.need[w] = max(min(t, t1) - g.t0, 0);
  }
  g.alone = g.rows <= HALF;
  if (g.alone) {
    g.need[1] = g.need[0] >> 1;
    g.need[0] -= g.need[1];
  }
  return g;
}

// The queries of row tile w into its shared memory by COUNT threads, `t` the caller's
// number: 16 bytes of every STEP-th row each, all in flight at once (cp.async), rows past the
// end zero. The swizzled places repeat every eight rows, and the global address is stepped
// (G query heads a token). Ends with the data visible to the tensor cores.
template <int D, int COUNT>
__device__ __forceinline__ void load_queries(const AttnArgs& a, const Item& it, const Segment& g, int G, int w, int t, bf16* tile) {
  constexpr int CH = D / 8, STEP = COUNT / CH, TURN = STEP < 8 ? 8 / STEP : 1;
  Tile<bf16, HALF, D> Qs{tile};
  const int row = t / CH, col = t % CH * 8, q = g.row0 + g.base(w) + row, left = g.rows - g.base(w) - row;
  uint32_t place[TURN];
#pragma unroll
  for (int i = 0; i < TURN; ++i) place[i] = smem_u32(Qs.ptr(row + i * STEP, col));
  const long long wrap = a.q_ts - G * a.q_hs, skip = (STEP / G) * a.q_ts + (STEP % G) * a.q_hs;
  int sub = q % G;
  const bf16* src = static_cast<const bf16*>(a.q) + (it.s.first + q / G) * a.q_ts + ((long long)it.h * G + sub) * a.q_hs + col;
#pragma unroll 2
  for (int b = 0; b < HALF / (STEP * TURN); ++b) {
#pragma unroll
    for (int i = 0; i < TURN; ++i) {
      const uint32_t to = place[i] + b * (STEP * TURN * 128);
      if ((b * TURN + i) * STEP < left)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to), "l"(src) : "memory");
      else
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(to), "r"(0) : "memory");
      src += skip;
      sub += STEP % G;
      if (sub >= G) {
        sub -= G;
        src += wrap;
      }
    }
  }
  cp_async_commit();
  cp_async_wait<0>();
  fence_proxy_async();
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    paged_attn_tc_kernel(AttnArgs a, int box_rows, int whole_items, const __grid_constant__ CUtensorMap k_map,
                         const __grid_constant__ CUtensorMap v_map) {
  if (threadIdx.x == 0) {
    prefetch_map(&k_map);
    prefetch_map(&v_map);
  }
  pdl_wait();
  if (!whole_items) pdl_trigger();
  typedef TcLay<D> L;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  const PagedArgs& p = a.p;
  const int G = p.Hq / p.Hk;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint64_t *full = bars, *empty = bars + L::SLOTS, *qbar = bars + 2 * L::SLOTS, *qfree = qbar + 2, *sbar = qfree + 2,
           *obar = sbar + 2, *pbar = obar + 2, *ibar = pbar + 2, *ifree = ibar + 2, *drained = ifree + 2,
           *abar = drained + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + L::TSLOT);
  // one warp finds the CTA's run of units while others set up
  Num::Run* run = reinterpret_cast<Num::Run*>(sm + L::RUN);
  if (warp == 0) {
    Num::Run r;
    const bool some = whole_items ? Num::pick(p, G, lane, blockIdx.x, r)
                                  : Num::plan(p, G, lane, blockIdx.x, gridDim.x, MIN_UNITS, r);
    if (!some) r.lo = r.hi = 0;
    if (lane == 0) *run = r;
  } else if (warp == MMA_WARP) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  } else if (tid == 32) {
    for (int i = 0; i < L::NBAR; ++i) mbar_init(&bars[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&pbar[i], HALF);
      mbar_init(&ifree[i], ITEM_READERS);
    }
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *tslot;
  const long long lo = run->lo;
  long long hi = run->hi;
  PartHead* head = part_heads<ROWS, D>(a.ws, gridDim.x) + blockIdx.x;
  if (lo == hi) {  // no share
    if (tid == 0 && !whole_items) head->more = 0;
    if (warp == MMA_WARP) tmem_dealloc(tm, 512);
    return;
  }
  Item it = run->first;
  // the warp's next item: of the CTA's run, or the one that the query warp has put down
  uint32_t items = 0;
  auto next_item = [&]() {
    if (!whole_items) {
      if (it.end >= hi) return false;
      Num::next_item(p, G, it);
      return true;
    }
    const uint32_t i = items & 1;
    mbar_wait(&ibar[i], items >> 1 & 1, p.err);
    it = *reinterpret_cast<const Item*>(sm + L::ITEM + 48 * i);
    hi = it.end;
    __syncwarp();
    if (lane == 0) mbar_arrive(&ifree[i]);
    ++items;
    return it.b >= 0;
  };

  if (warp < MMA_WARP) {
    // ---------------------------------------------------------------- softmax
    more_registers<SOFTMAX_REGS>();
    const int w = warp >> 2, r = tid & (HALF - 1);  // row tile, row of it
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's quarter of tensor memory
    const uint32_t ts = tm + lanes + L::S + w * 128, tp = tm + lanes + L::P + w * L::P_STEP, to = tm + lanes + L::O + w * D;
    const float c = a.scale * LOG2E;
    {
      const Segment g = segment(it, G, lo, hi);
      if ((w ? g.need[1] : g.need[0]) > 0) {
        load_queries<D, HALF>(a, it, g, G, w, r, reinterpret_cast<bf16*>(sm + L::Q + w * HALF * D * 2));
        asm volatile("bar.sync %0, 128;" ::"r"(2 + w) : "memory");
        if (r == 0) mbar_arrive(&qbar[w]);
      }
    }
    const bool wide = ((reinterpret_cast<uintptr_t>(a.out) | (a.o_ts * 2) | (a.o_hs * 2)) & 31) == 0;
    uint32_t k = 0;  // key tiles of this row tile so far: the parity of its barriers
    while (true) {
      const Segment g = segment(it, G, lo, hi);
      const int need = w ? g.need[1] : g.need[0];
      const int row = g.base(w) + r;  // row of the item
      const int lim = row < g.rows ? g.p0 + (g.row0 + row) / G : -1;
      const int lim_min = g.p0 + (g.row0 + g.base(w)) / G;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < need; ++j, ++k) {
        mbar_wait(&sbar[w], k & 1, p.err);
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32_nowait(ts + 32 * i, s[i]);
        tmem_wait_ld();
        const int key0 = g.tile(w, j) * KT;
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
          mbar_wait(&obar[w], (k - 1) & 1, p.err);  // the last PV has completed
          tc_fence_after();
#pragma unroll 1
          for (int i = 0; i < D / 16; ++i) {
            uint32_t o[16];
            tmem_ld16_nowait(to + 16 * i, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(to + 16 * i, o);
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
            const __nv_bfloat162 b = __floats2bfloat162_rn(x0, x1);
            o[e] = *reinterpret_cast<const uint32_t*>(&b);
          }
          tmem_st16(tp + 16 * i, o);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&pbar[w]);
        float s0, s1;
        unpair(add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      }
      // the tile's output, or its part
      if (need > 0) {
        mbar_wait(&obar[w], (k - 1) & 1, p.err);
        tc_fence_after();
      }
      const bool whole = it.start >= lo && it.end <= hi;
      bool live = row < g.rows, none = need == 0 || l == 0.f;  // (not by the maximum, which passes over NaN)
      if (g.alone) {
        if (g.need[1] > 0) {
          // merge the second row tile into the first, 32 columns at a time through shared memory
          float* ml = reinterpret_cast<float*>(sm + L::ML);
          float* stage = reinterpret_cast<float*>(sm + L::OUT);
          ml[w * HALF + r] = m;
          ml[(2 + w) * HALF + r] = l;
          asm volatile("bar.sync 1, 256;" ::: "memory");
          const float om = ml[(1 - w) * HALF + r], M = fmaxf(m, om);
          const float f = m == -INFINITY ? 0.f : ex2(m - M), of = om == -INFINITY ? 0.f : ex2(om - M);
          l = l * f + ml[(3 - w) * HALF + r] * of;
          m = M;
          none = l == 0.f;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            float* at = stage + (i & 1) * HALF * 32 + r * 32;  // chunks of four columns, swizzled by row
            uint32_t o[32];
            tmem_ld32_nowait(to + 32 * i, o);
            tmem_wait_ld();
            if (w == 1) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(at + (((e >> 2) ^ (r & 7)) << 2)) =
                    make_float4(__uint_as_float(o[e]) * f, __uint_as_float(o[e + 1]) * f, __uint_as_float(o[e + 2]) * f,
                                __uint_as_float(o[e + 3]) * f);
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (w == 0) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 x = *reinterpret_cast<const float4*>(at + (((e >> 2) ^ (r & 7)) << 2));
                o[e] = __float_as_uint(fmaf(__uint_as_float(o[e]), f, x.x));
                o[e + 1] = __float_as_uint(fmaf(__uint_as_float(o[e + 1]), f, x.y));
                o[e + 2] = __float_as_uint(fmaf(__uint_as_float(o[e + 2]), f, x.z));
                o[e + 3] = __float_as_uint(fmaf(__uint_as_float(o[e + 3]), f, x.w));
              }
              tmem_st16(to + 32 * i, *reinterpret_cast<const uint32_t(*)[16]>(&o[0]));
              tmem_st16(to + 32 * i + 16, *reinterpret_cast<const uint32_t(*)[16]>(&o[16]));
            }
          }
          tmem_wait_st();
          asm volatile("bar.sync 1, 256;" ::: "memory");  // the stages are free for the next merge
        }
        live = live && w == 0;  // the first row tile writes
      }
      if (whole) {
        const float inv = none ? 0.f : 1.f / l;
        const int q = g.row0 + row, tok = it.s.first + q / G, head_q = it.h * G + q % G;
        bf16* dst = static_cast<bf16*>(a.out) + (live ? tok * a.o_ts + head_q * a.o_hs : 0);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t o[32];
          if (need > 0) {
            tmem_ld32_nowait(to + 32 * i, o);
            tmem_wait_ld();
          }
          if (live) {
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              uint32_t u[8];
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const float v0 = none ? 0.f : __uint_as_float(o[e + 2 * x]) * inv;
                const float v1 = none ? 0.f : __uint_as_float(o[e + 2 * x + 1]) * inv;
                const __nv_bfloat162 h = __floats2bfloat162_rn(v0, v1);
                u[x] = *reinterpret_cast<const uint32_t*>(&h);
              }
              store32(dst + 32 * i + e, u, wide);
            }
          }
        }
        if (live) {
          if (a.lse) a.lse[(size_t)tok * p.Hq + head_q] = none ? -INFINITY : (m + log2f(l)) * LN2;
        }
      } else {
        // part: four columns of all rows side by side, so that a warp's store is one run
        float* part = Parts<ROWS, D>::slot(a.ws, blockIdx.x, it.start < lo ? 0 : 1);
        const bool mine = !g.alone || w == 0;
        if (mine) {
          part[ROWS * D + row] = none ? -INFINITY : m;
          part[ROWS * D + ROWS + row] = l;
        }
        if (need > 0 && mine) {
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t o[32];
            tmem_ld32_nowait(to + 32 * i, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(part + ((8 * i + e / 4) * ROWS + row) * 4) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
      }
      tc_fence_before();
      if (!next_item()) break;
    }
  } else {
    fewer_registers<OTHER_REGS>();
  }
  if (warp == MMA_WARP) {
    // ---------------------------------------------------------------- products
    constexpr uint32_t id_s = umma_idesc_bf16(HALF, KT), id_o = umma_idesc_bf16(HALF, D, false, true);
    constexpr int PANEL = KT * 128;
    static_assert(PANEL / 16 == 1024, "issue_scores' panels");
    const uint32_t acc = __shfl_sync(0xffffffffu, tm, 0);
    const uint64_t dq = desc_kmajor(sm + L::Q), dring = desc_kmajor(sm + L::RING),
                   dvring = desc_mnmajor(sm + L::RING, PANEL);
    int slot = 0;
    uint32_t phase = 0, np = 0;     // np: bit w is the parity of the next P of row tile w
    uint32_t nq = 0;                // likewise of its next queries
    auto next_slot = [&]() {
      if (++slot == L::SLOTS) {
        slot = 0;
        phase ^= 1;
      }
    };
    while (true) {
      const Segment g = segment(it, G, lo, hi);
      // warp-uniform by construction, and known to be to the compiler
      const int need[2] = {__shfl_sync(0xffffffffu, g.need[0], 0), __shfl_sync(0xffffffffu, g.need[1], 0)};
      const bool alone = __shfl_sync(0xffffffffu, (int)g.alone, 0) != 0;
      const int tiles = __shfl_sync(0xffffffffu, g.tiles(), 0), keys = __shfl_sync(0xffffffffu, it.s.len - g.t0 * KT, 0);
      auto scores = [&](int w, int kslot, bool last) {
        const uint64_t q = dq + (uint64_t)(w * (HALF * D * 2 / 16)), k = dring + (uint64_t)(kslot * (L::SLOT / 16));
        issue_scores<D>(acc + L::S + w * 128, q, k, id_s, &sbar[w]);
        if (last) commit_elected(&qfree[w]);  // the item's queries are done with
      };
      // the first scores of each row tile: of one key tile, or of the first two
      const int ahead = alone ? 2 : 1;
      for (int i = 0; i < ahead && i < tiles; ++i) {
        mbar_wait(&full[slot], phase, p.err);
#pragma unroll
        for (int w = 0; w < 2; ++w)
          if (alone ? w == i : need[w] > 0) {
            mbar_wait(&qbar[w], nq >> w & 1, p.err);
            nq ^= 1u << w;
            tc_fence_after();
            scores(w, slot, need[w] == 1);
          }
        commit_elected(&empty[slot]);
        next_slot();
      }
      for (int i = 0; i < tiles; ++i) {
        const int vslot = slot;
        mbar_wait(&full[vslot], phase, p.err);
        next_slot();
        const int kslot = slot;
        const uint32_t kphase = phase;
        const bool more = i + ahead < tiles;
        if (more) next_slot();
        const int keep = keys - i * KT;
        if (keep < KT) {  // rows past the length hold anything: 0 * NaN is not 0
          Tile<bf16, KT, D> Vs{reinterpret_cast<bf16*>(sm + L::RING + vslot * L::SLOT)};
          for (int q = lane; q < (KT - keep) * (D / 8); q += 32)
            *reinterpret_cast<uint4*>(Vs.ptr(keep + q / (D / 8), q % (D / 8) * 8)) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async();
          __syncwarp();
        }
        bool kready = false;
        const uint64_t v = dvring + (uint64_t)(vslot * (L::SLOT / 16));
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int j = alone ? i >> 1 : i;  // the row tile's own count
          if (alone ? (i & 1) == w : i < need[w]) {
            mbar_wait(&pbar[w], np >> w & 1, p.err);
            tc_fence_after();
            issue_output(acc + L::O + w * D, acc + L::P + w * L::P_STEP, v, id_o, j > 0, &obar[w]);
            np ^= 1u << w;
            if (j + 1 < need[w]) {
              if (!kready) {
                mbar_wait(&full[kslot], kphase, p.err);
                kready = true;
              }
              scores(w, kslot, j + 2 == need[w]);
            }
          }
        }
        commit_elected(&empty[vslot]);
        if (more) commit_elected(&empty[kslot]);
      }
      if (!next_item()) break;
    }
    commit_elected(drained);
    mbar_drain(drained, 0);
    tc_fence_before();
  } else if (warp == KEY_WARP || warp == VALUE_WARP) {
    // ---------------------------------------------------------------- key and value tiles
    // The tiles of an item stand in the ring in the order in which the products take them:
    // `ahead` key tiles, then a value tile and the next key tile in turn.
    const bool value = warp == VALUE_WARP;
    const CUtensorMap* map = value ? &v_map : &k_map;
    const int pieces = KT / box_rows;
    constexpr int PANELS = D / 64;
    uint32_t base = 0;  // tiles of the items before
    while (true) {
      const Segment g = segment(it, G, lo, hi);
      const int n = g.tiles(), ahead = g.alone ? 2 : 1;
      // this lane's piece of a tile: its entry of the page table, read one tile ahead
      const auto look_up = [&](int tile) {
        const int key = (g.t0 + tile) * KT + lane * box_rows;
        return tile < n && lane < pieces && key < it.s.len ? page_entry(p, it.b, key) : 0;
      };
      int coming = look_up(0);
      for (int i = 0; i < n; ++i) {
        const uint32_t at = base + (value ? i + min(n, i + ahead) : i < ahead ? i : 2 * i + 1 - ahead);
        const int slot = at % L::SLOTS;
        const uint32_t use = at / L::SLOTS;
        const int page = checked_page(p, coming), key0 = (g.t0 + i) * KT;
        coming = look_up(i + 1);
        const int have = min(pieces, (it.s.len - key0 + box_rows - 1) / box_rows);  // pieces with cached rows
        const int prow = (key0 + lane * box_rows) % p.page_size;
        if (use > 0) mbar_wait(&empty[slot], (use - 1) & 1, p.err);
        if (lane == 0) mbar_arrive_expect_tx(&full[slot], (uint32_t)(have * box_rows * D * 2));
        __syncwarp();
        if (lane < have) {
          uint8_t* dst = sm + L::RING + slot * L::SLOT + lane * box_rows * 128;
#pragma unroll
          for (int c = 0; c < PANELS; ++c) tma_load_4d(dst + c * KT * 128, map, 64 * c, prow, it.h, page, &full[slot]);
        }
      }
      base += 2 * n;
      if (!next_item()) break;
    }
    // after a failed wait loads may still be on their way: the last one of every slot used
    if (lane == 0 && !value)
      for (uint32_t at = base > L::SLOTS ? base - L::SLOTS : 0; at < base; ++at)
        mbar_drain(&full[at % L::SLOTS], at / L::SLOTS & 1);
    __syncwarp();
  } else if (warp == QUERY_WARP) {
    // ---------------------------------------------------------------- queries, after the first item's, and the join's head
    uint32_t loads[2] = {0, 0};
    for (bool first = true;; first = false) {
      const Segment g = segment(it, G, lo, hi);
#pragma unroll
      for (int w = 0; w < 2; ++w)
        if (g.need[w] > 0) {
          if (!first) {
            if (loads[w] > 0) mbar_wait(&qfree[w], (loads[w] - 1) & 1, p.err);
            load_queries<D, 32>(a, it, g, G, w, lane, reinterpret_cast<bf16*>(sm + L::Q + w * HALF * D * 2));
            __syncwarp();
            if (lane == 0) mbar_arrive(&qbar[w]);
          }
          ++loads[w];
        }
      if (!whole_items) {
        if (next_item()) continue;
        if (lane == 0)
          *head = PartHead{it.start >= lo && it.end > hi ? holder(run->total, run->ncta, it.end - 1) - (int)blockIdx.x : 0,
                           g.row0, g.rows, it.s.first, it.h, {0, 0, 0}};
        break;
      }
      // find the next item while this one is in work, and put it down for the other warps
      if (lane == 0) {
        mbar_arrive_expect_tx(abar, 16);
        ask_next_cta(sm + L::ANSWER, abar);
      }
      __syncwarp();
      Num::Run r;
      r.first = it;
      const bool some = mbar_wait(abar, items & 1, p.err);
      const int cta = some ? next_cta(sm + L::ANSWER) : -1;
      if (cta < 0 || !Num::pick(p, G, lane, cta, r)) r.first.b = -1;
      const uint32_t i = items & 1;
      if (items > 1) mbar_wait(&ifree[i], (items >> 1 & 1) ^ 1, p.err);
      if (lane == 0) {
        *reinterpret_cast<Item*>(sm + L::ITEM + 48 * i) = r.first;
        fence_proxy_async();  // the answer has been read before the next one is written
        mbar_arrive(&ibar[i]);
      }
      __syncwarp();
      ++items;
      it = r.first;
      hi = it.end;
      if (it.b < 0) break;
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == MMA_WARP) tmem_dealloc(tm, 512);
}

// Joins the parts of the item that begins in CTA blockIdx.x and goes on in the next ones,
// in the order of the CTAs: 32 rows per CTA (a row per lane), the columns over the warps.
constexpr int JOIN_WARPS = 8;
template <int D>
__global__ void __launch_bounds__(32 * JOIN_WARPS) paged_attn_tc_join_kernel(AttnArgs a) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x, row = blockIdx.y * 32 + (threadIdx.x & 31), c40 = threadIdx.x >> 5;
  const PartHead h = part_heads<ROWS, D>(a.ws, gridDim.x)[c];
  if (h.more == 0 || row >= h.rows) return;
  constexpr size_t STEP = 2 * Parts<ROWS, D>::SLOT;  // from one CTA's slot to the next CTA's
  constexpr int N = D / 4 / JOIN_WARPS;              // vectors of four columns per thread
  const float *first = Parts<ROWS, D>::slot(a.ws, c, 1), *rest = Parts<ROWS, D>::slot(a.ws, c + 1, 0);
  float M = first[ROWS * D + row];
#pragma unroll 8
  for (int q = 0; q < h.more; ++q) M = fmaxf(M, rest[q * STEP + ROWS * D + row]);
  float4 o[N];
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  const float* part = first;
#pragma unroll 4
  for (int q = 0; q <= h.more; ++q) {
    const float m = part[ROWS * D + row];
    const float lp = part[ROWS * D + ROWS + row], f = m == -INFINITY ? 0.f : ex2(m - M);
    const bool some = lp != 0.f;  // a part without keys has no o; NaN counts, whatever its maximum
    l += lp * f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(part + ((size_t)(c40 + i * JOIN_WARPS) * ROWS + row) * 4);
      if (some) {
        o[i].x += v.x * f; o[i].y += v.y * f; o[i].z += v.z * f; o[i].w += v.w * f;
      }
    }
    part = rest + q * STEP;
  }
  const int G = a.p.Hq / a.p.Hk, q = h.row0 + row, tok = h.first + q / G, head = h.h * G + q % G;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  bf16* dst = static_cast<bf16*>(a.out) + tok * a.o_ts + head * a.o_hs;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float v[4] = {o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv};
    st4(dst + (c40 + i * JOIN_WARPS) * 4, v);
  }
  if (a.lse && c40 == 0) a.lse[(size_t)tok * a.p.Hq + head] = l == 0.f ? -INFINITY : (M + log2f(l)) * LN2;
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

// Whether the call surely has two items or more per SM: the tokens' full items alone. Below
// that the ragged last round can cost more than the parts; above, prompts gain from the shared
// reads of keys, and chunks lose 6 % at most. us by items / by runs, 16 and 4 heads of 128:
//   items                              128      200      304      450       800         1,600
//   2 sequences over 16k keys       217/205  420/307  450/457  676/690  1,352/1,272  2,975/2,947
//   2 prompts                        29/43    45/57    74/78   113/121    260/274      872/909
//   6 prompts, 5 to 25 % of the tokens  -     37/49    47/66    68/94     139/178      412/444
bool whole_items(const AttnArgs& a) {
  const int nsm = device_sm_count() > 0 ? device_sm_count() : 152;
  return (long long)a.p.N * (a.p.Hq / a.p.Hk) / ROWS * a.p.Hk >= 2ll * nsm;
}

template <int D>
cudaError_t run(const AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, int box, cudaStream_t s) {
  const int bytes = TcLay<D>::BYTES + 1024;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_shared(reinterpret_cast<const void*>(paged_attn_tc_kernel<D>), bytes, &allowed);
  if (e != cudaSuccess) return e;
  const bool whole = whole_items(a);
  const unsigned grid = whole ? (unsigned)most_items(a, ROWS) : (unsigned)launch_ctas(a, ROWS, KT, OVER, MIN_UNITS);
  prof_mark(K_ATTN_TC, s, true);
  e = launch_pdl(paged_attn_tc_kernel<D>, dim3(grid), dim3(THREADS), bytes, s, a, box, (int)whole, km, vm);
  prof_mark(K_ATTN_TC, s, false);
  if (e != cudaSuccess || whole) return e;
  prof_mark(K_ATTN_TC_JOIN, s, true);
  e = launch_pdl(paged_attn_tc_join_kernel<D>, dim3(grid, ROWS / 32), dim3(32 * JOIN_WARPS), 0, s, a);
  prof_mark(K_ATTN_TC_JOIN, s, false);
  return e;
}

}  // namespace

// bf16 with more rows than one item of the few-rows kernel has. us of that kernel / of this one,
// two KV heads of 128, by query rows of a KV head:
//   rows                          16       24       32       64        128
//   1 sequence, 2,000 keys     16/27    18/27    19/27    21/29     20/27
//   16 sequences, 2,000 keys   27/31    29/31    29/33    39/33     57/33
//   64 sequences, 2,000 keys   43/55    64/55    66/57   117/57    188/57
//   16 sequences, 30,000 keys 106/113  178/113  176/113  322/113   471/113
// (A second item of 16 rows reads and multiplies all keys again; one short sequence, whose keys
// one item leaves most SMs without, is the exception and stays on the rule.)
bool paged_attn_tc_applies(const AttnArgs& a) {
  const long long G = a.p.Hq / a.p.Hk;
  return a.p.bf16 && (a.max_q < a.p.N ? a.max_q : a.p.N) * G > 16;
}

size_t paged_attn_tc_workspace(const AttnArgs& a) {
  if (whole_items(a)) return 0;
  const int grid = launch_ctas(a, ROWS, KT, OVER, MIN_UNITS);
  return a.p.D == 64 ? Parts<ROWS, 64>::bytes(grid) : Parts<ROWS, 128>::bytes(grid);
}

cudaError_t launch_paged_attn_tc(const AttnArgs& a, cudaStream_t s, bool* done) {
  *done = false;
  int box = KT;  // rows of a box: a run inside one page and inside one tile
  while (a.p.page_size % box != 0) box >>= 1;
  CUtensorMap km{}, vm{};
  if (!cache_map(&km, a.p.kc, a.p, a.p.k_ps, a.p.k_hs, a.p.k_rs, box) ||
      !cache_map(&vm, a.p.vc, a.p, a.p.v_ps, a.p.v_hs, a.p.v_rs, box))
    return cudaSuccess;  // strides that a tensor map cannot hold: the caller takes the other kernel
  *done = true;
  return a.p.D == 64 ? run<64>(a, km, vm, box, s) : run<128>(a, km, vm, box, s);
}

}  // namespace gdn
