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

}  // namespace gdn
