// Shared by the paged attention kernels: the new tokens of a sequence, the items a launch
// works on, and the softmax's units.
//
// A query row of KV head h is (token i, head h G + j), numbered i G + j inside the
// sequence: the G query heads that read one KV head sit side by side, so that the keys
// are read once for all of them. An item is a run of ROWS such rows of one (sequence, KV
// head). Row r of an item sees the keys 0 .. limit(r), its token's position (causal), and
// none when that is negative.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace gdn {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct Seq {
  int n, first;  // new tokens, and the first of them
  int len;       // keys in the cache, new ones included
};

// Sequence b, with bounds kept inside the tensors whatever the arrays hold.
__device__ __forceinline__ Seq load_seq(const PagedArgs& p, int b, bool report) {
  Seq s;
  int lo = p.cu[b], hi = p.cu[b + 1];
  lo = lo < 0 ? 0 : (lo > p.N ? p.N : lo);
  hi = hi < lo ? lo : (hi > p.N ? p.N : hi);
  s.first = lo;
  s.n = hi - lo;
  s.len = p.lens[b];
  const long long cap = (long long)p.max_pages * p.page_size;
  if (s.len > cap) {
    if (report && p.err) atomicOr(p.err, ERR_PAGE);
    s.len = (int)cap;
  }
  if (s.len < 0) s.len = 0;
  return s;
}
// The page table's entry for key `key` of sequence b, and the entry clamped into the cache
// (apart, so that the check does not wait for the load where it is issued).
__device__ __forceinline__ int page_entry(const PagedArgs& p, int b, int key) {
  return p.page_table[b * p.pt_stride + key / p.page_size];
}
__device__ __forceinline__ int checked_page(const PagedArgs& p, int page) {
  if (page < 0 || page >= p.num_pages) {
    if (p.err) atomicOr(p.err, ERR_PAGE);
    page = 0;
  }
  return page;
}

// ------------------------------------------------------------------ numbering of the work
// The keys of all items are cut into blocks of UNIT ("units", at least one per item: an
// item without keys still writes its zeros) and numbered through, item after item: the
// items of a KV head, the heads of a sequence, the sequences. Each CTA takes an equal run
// of units, whatever the lengths.
struct Item {
  int b, h, i;           // sequence, KV head, item of the head
  Seq s;
  long long start, end;  // its units, numbered through all items
};

// Blocks of UNIT keys that rows up to `last` of a sequence see.
template <int UNIT>
__device__ __forceinline__ int key_blocks(const Seq& s, int G, int last) {
  const int limit = s.len - s.n + last / G;
  return limit < 0 ? 0 : limit / UNIT + 1;
}

__device__ __forceinline__ long long warp_sum(long long t) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
  return t;
}
__device__ __forceinline__ long long warp_scan(long long t, int lane) {  // inclusive
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, t, off);
    if (lane >= off) t += o;
  }
  return t;
}
// CTA c of n takes the units [cut(c), cut(c + 1)); 32-bit division where it will do.
__device__ __forceinline__ long long cut(long long total, int n, int c) {
  const long long x = total * c;
  return x >> 32 ? x / n : (long long)((uint32_t)x / (uint32_t)n);
}
// The CTA whose run holds unit f.
__device__ __forceinline__ int holder(long long total, int n, long long f) {
  int c = (int)(f * n / total);
  while (c + 1 < n && cut(total, n, c + 1) <= f) ++c;
  while (cut(total, n, c) > f) --c;
  return c;
}

// ROWS query rows per item, UNIT keys per unit; OVER units in front of an item's keys stand
// for the time of its start and end. Called by all lanes of a warp, item_units apart.
template <int ROWS, int UNIT, int OVER>
struct Numbering {
  static __device__ __forceinline__ int item_units(const Seq& s, int G, int item) {
    int last = (item + 1) * ROWS - 1;
    const int rows = s.n * G;
    if (last >= rows) last = rows - 1;
    const int n = key_blocks<UNIT>(s, G, last) + OVER;
    return n < 1 ? 1 : n;
  }
  static __device__ __forceinline__ int seq_items(const Seq& s, int G) { return (s.n * G + ROWS - 1) / ROWS; }

  // Units of one KV head of the sequences b0 + lane, each in its lane: by itself where all
  // have one or two items (single tokens, drafts), else the warp over each one's items.
  static __device__ __forceinline__ long long lane_units(const Seq& s, int G, int lane) {
    const int n = seq_items(s, G);
    long long u = 0;
    if (!__any_sync(0xffffffffu, n > 2)) {
      for (int i = 0; i < n; ++i) u += item_units(s, G, i);
      return u;
    }
    for (unsigned left = __ballot_sync(0xffffffffu, n > 0); left; left &= left - 1) {
      const int l = __ffs(left) - 1;
      const Seq q{__shfl_sync(0xffffffffu, s.n, l), 0, __shfl_sync(0xffffffffu, s.len, l)};
      long long t = 0;
      for (int i = lane, m = seq_items(q, G); i < m; i += 32) t += item_units(q, G, i);
      t = warp_sum(t);
      if (lane == l) u = t;
    }
    return u;
  }

  // The units of 32 sequences b0 + lane over all KV heads, and their running sum.
  struct Chunk {
    Seq s;
    long long u, inc;
  };
  static __device__ __forceinline__ Chunk load_chunk(const PagedArgs& p, int G, int lane, int b0, bool report) {
    Chunk c;
    c.s = b0 + lane < p.B ? load_seq(p, b0 + lane, report) : Seq{0, 0, 0};
    c.u = lane_units(c.s, G, lane);
    c.inc = warp_scan(c.u * p.Hk, lane);
    return c;
  }
  // The item holding unit f < total (one warp, all lanes). c: the first chunk.
  static __device__ __forceinline__ void locate(const PagedArgs& p, int G, int lane, long long f, Chunk c, Item& it) {
    long long base = 0, per = 1;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      if (b0 > 0) c = load_chunk(p, G, lane, b0, false);
      const unsigned hit = __ballot_sync(0xffffffffu, base + c.inc > f);
      if (hit) {
        const int l = __ffs(hit) - 1;
        base += __shfl_sync(0xffffffffu, c.inc - c.u * p.Hk, l);
        per = __shfl_sync(0xffffffffu, c.u, l);
        it.b = b0 + l;
        it.s = Seq{__shfl_sync(0xffffffffu, c.s.n, l), __shfl_sync(0xffffffffu, c.s.first, l),
                   __shfl_sync(0xffffffffu, c.s.len, l)};
        break;
      }
      base += __shfl_sync(0xffffffffu, c.inc, 31);
    }
    it.h = ((f - base) | per) >> 32 ? (int)((f - base) / per) : (int)((uint32_t)(f - base) / (uint32_t)per);
    base += it.h * per;
    const int n = seq_items(it.s, G);
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int u = i0 + lane < n ? item_units(it.s, G, i0 + lane) : 0;
      const long long inc = warp_scan(u, lane);
      const unsigned hit = __ballot_sync(0xffffffffu, base + inc > f);
      if (hit) {
        const int l = __ffs(hit) - 1;
        it.i = i0 + l;
        it.end = base + __shfl_sync(0xffffffffu, inc, l);
        it.start = it.end - __shfl_sync(0xffffffffu, u, l);
        break;
      }
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  // The next item in the numbering (not called past the last).
  static __device__ __forceinline__ void next_item(const PagedArgs& p, int G, Item& it) {
    if (++it.i >= seq_items(it.s, G)) {
      it.i = 0;
      if (++it.h >= p.Hk) {
        it.h = 0;
        do {
          ++it.b;
          it.s = load_seq(p, it.b, false);
        } while (it.s.n == 0 && it.b + 1 < p.B);
      }
    }
    it.start = it.end;
    it.end += item_units(it.s, G, it.i);
  }
  // The run of units of CTA `cta` of `grid`, [lo, hi), out of `total`, and the item its first
  // unit lies in; `ncta` CTAs have one, of `least` units or more. False for the others.
  struct Run {
    long long total, lo, hi;
    int ncta;
    Item first;
  };
  static __device__ __forceinline__ bool plan(const PagedArgs& p, int G, int lane, int cta, int grid, int least, Run& r) {
    const Chunk c = load_chunk(p, G, lane, 0, cta == 0);
    r.total = __shfl_sync(0xffffffffu, c.inc, 31);
    for (int b0 = 32; b0 < p.B; b0 += 32)
      r.total += __shfl_sync(0xffffffffu, load_chunk(p, G, lane, b0, cta == 0).inc, 31);
    r.ncta = active_ctas(r.total, grid, least);
    if (cta >= r.ncta) return false;
    r.lo = cut(r.total, r.ncta, cta);
    r.hi = cut(r.total, r.ncta, cta + 1);
    locate(p, G, lane, r.lo, c, r.first);
    return true;
  }
  // Item `idx` as a run of its own: the KV heads of a run of rows side by side, the items of
  // a sequence from its last, the one with the most keys, and the sequences likewise. False
  // when there are fewer items. Item 0's caller reports the lengths of all sequences.
  static __device__ __forceinline__ bool pick(const PagedArgs& p, int G, int lane, int idx, Run& r) {
    int i = idx / p.Hk;
    Item& it = r.first;
    it.h = idx % p.Hk;
    bool found = false;
    for (int b0 = p.B - 1; b0 >= 0; b0 -= 32) {
      const int b = b0 - lane;
      const Seq s = b >= 0 ? load_seq(p, b, idx == 0) : Seq{0, 0, 0};
      const int n = seq_items(s, G);
      int inc = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += o;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, !found && inc > i);
      if (hit) {
        const int l = __ffs(hit) - 1;
        it.b = b0 - l;
        it.s = Seq{__shfl_sync(0xffffffffu, s.n, l), __shfl_sync(0xffffffffu, s.first, l), __shfl_sync(0xffffffffu, s.len, l)};
        it.i = __shfl_sync(0xffffffffu, inc, l) - 1 - i;
        it.start = r.lo = 0;
        it.end = r.hi = r.total = item_units(it.s, G, it.i);
        r.ncta = 1;
        found = true;
        if (idx != 0) break;
      }
      i -= __shfl_sync(0xffffffffu, inc, 31);
    }
    return found;
  }
  // CTAs that take part: enough units for each to have `least`.
  static __device__ __forceinline__ int active_ctas(long long total, int grid, int least) {
    const long long most = (total + least - 1) / least;
    return most < grid ? (int)most : grid;
  }
};

// The parts of a CTA in the workspace: slot 0 for an item that began in an earlier CTA,
// slot 1 for one that begins here and goes on. o [ROWS][D] (in the kernel's own order)
// relative to m, then m [ROWS] (base 2), l [ROWS].
template <int ROWS, int D>
struct Parts {
  static constexpr size_t SLOT = ROWS * D + 2 * ROWS;  // floats
  static __device__ __forceinline__ float* slot(float* ws, int cta, int second) { return ws + (size_t)(2 * cta + second) * SLOT; }
  static size_t bytes(int ctas) { return (2 * SLOT * sizeof(float) + 32) * (size_t)ctas; }
};
// Most items that a call can have: full ones, and one that is not full per sequence.
inline long long most_items(const AttnArgs& a, int rows) {
  const long long G = a.p.Hq / a.p.Hk, seqs = a.p.B < a.p.N ? a.p.B : a.p.N;
  return ((long long)a.p.N * G / rows + seqs) * a.p.Hk;
}
// The same, by the caller's bound on new tokens too.
inline long long launch_items(const AttnArgs& a, int rows) {
  const long long G = a.p.Hq / a.p.Hk, seqs = a.p.B < a.p.N ? a.p.B : a.p.N, most = most_items(a, rows);
  const long long per_seq = ((long long)(a.max_q < a.p.N ? a.max_q : a.p.N) * G + rows - 1) / rows * seqs * a.p.Hk;
  return per_seq < most ? per_seq : most;
}
// CTAs of a launch: one per SM, or as many as the work can occupy by the caller's bounds on
// new tokens and length (which limit only this). `over`, `least`: as in Numbering and plan.
inline int launch_ctas(const AttnArgs& a, int rows, int unit, int over, int least) {
  const int nsm = device_sm_count() > 0 ? device_sm_count() : 152;
  const long long items = launch_items(a, rows), per_item = ((long long)a.max_kv + unit - 1) / unit + over;
  if (items >= (long long)nsm * least || per_item >= (long long)nsm * least) return nsm;
  const long long want = (items * per_item + least - 1) / least;
  return want < nsm ? (int)want : nsm;
}
// What a join needs of CTA c's slot 1: how many CTAs after it hold the rest (0: no such
// item), the item's first row and rows, the sequence's first token and the KV head. One
// per CTA of the grid, behind the slots.
struct PartHead {
  int more, row0, rows, first, h, pad[3];
};
static_assert(sizeof(PartHead) == 32, "as Parts::bytes counts");
template <int ROWS, int D>
__device__ __forceinline__ PartHead* part_heads(float* ws, int grid) {
  return reinterpret_cast<PartHead*>(Parts<ROWS, D>::slot(ws, grid, 0));
}

}  // namespace gdn
