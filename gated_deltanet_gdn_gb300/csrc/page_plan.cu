// Plan of a serving step, from the requests' lengths: which requests get their new tokens, the
// pages that are taken from and given back to the free list, and the packed arrays that the
// step's other calls read (offsets, lengths, and each token's request, position and slot).
//
// With page size P, request b of length l and n new tokens (n < 0: gives back its last -n):
//   given back   the pages ceil(max(l + n, 0) / P) .. ceil(l / P) - 1 of each such request, in order,
//                put on top of the free list before anything is taken
//   asked for    ceil((l + n) / P) - ceil(l / P) pages; granted where these and those asked for before it are at most
//                the pages there are, and its tokens and those before it at most max_tokens
//   taken        from the top of the list, in order of request and page
// Requests that are not granted keep their length and have no tokens in the step.
//
// Bound by latency: a few kilobytes of lengths, some prefix sums and one lookup a token. Everything is one launch:
// each CTA forms the prefix sums over all requests for itself in shared memory (two block scans), then takes its share of
// tokens and pages, so that no CTA waits for another. A page from the part of the list that this step gives back is found
// through the sums, not read back from the list, and no array is read where another CTA may write it. Sums are 32 bits and
// saturate, divisions 32 bits unsigned (with 64 bits the 1,024 requests and 131,072 rows of a mixed step took 11.7 us, now 6.5).
#include <climits>

#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;

// Pages given back, pages asked for, tokens asked for; no sum passes INT_MAX.
struct Sums {
  unsigned freed, need, ask;
};
__device__ __forceinline__ unsigned plus(unsigned a, unsigned b) {  // of two up to INT_MAX
  const unsigned s = a + b;
  return s > (unsigned)INT_MAX ? (unsigned)INT_MAX : s;
}
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return Sums{plus(a.freed, b.freed), plus(a.need, b.need), plus(a.ask, b.ask)};
}

__device__ __forceinline__ Sums shfl_up(const Sums& v, int d) {
  return Sums{__shfl_up_sync(~0u, v.freed, d), __shfl_up_sync(~0u, v.need, d), __shfl_up_sync(~0u, v.ask, d)};
}
__device__ __forceinline__ Sums shfl(const Sums& v, int lane) {
  return Sums{__shfl_sync(~0u, v.freed, lane), __shfl_sync(~0u, v.need, lane), __shfl_sync(~0u, v.ask, lane)};
}
// Sum over the warp's lanes up to this one.
__device__ __forceinline__ Sums warp_upto(Sums v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const Sums o = shfl_up(v, d);
    if (lane >= d) v = v + o;
  }
  return v;
}
// Sum over the threads before this one; *total over all. `part` is free again after the next barrier.
__device__ __forceinline__ Sums block_before(const Sums& mine, uint4* part, Sums* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const Sums up = warp_upto(mine, lane);
  if (lane == 31) part[warp] = make_uint4(up.freed, up.need, up.ask, 0u);
  __syncthreads();
  const uint4 v = lane < WARPS ? part[lane] : make_uint4(0u, 0u, 0u, 0u);
  const Sums warps = warp_upto(Sums{v.x, v.y, v.z}, lane), before = shfl(warps, (warp + 31) % 32), ex = shfl_up(up, 1);
  *total = shfl(warps, 31);
  Sums r{0, 0, 0};
  if (warp) r = before;
  if (lane) r = r + ex;
  return r;
}

// First index in [0, n) with upto[index] > v (upto not decreasing); n where there is none.
__device__ __forceinline__ int first_above(const int* upto, int n, int v) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (upto[mid] > v) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

struct Request {
  int len, kept;        // tokens, and those that stay
  int used, keep;       // their pages
  int ask, need;        // new tokens and pages, 0 where they do not fit the table
  bool bad;
};
__device__ __forceinline__ int pages_of(int tokens, int page) { return (int)(((unsigned)tokens + (unsigned)page - 1u) / (unsigned)page); }
__device__ __forceinline__ Request request(int len, int n, int page, int cap) {
  Request r;
  r.bad = len < 0 || len > cap;
  r.len = min(max(len, 0), cap);
  r.kept = n < 0 ? (n < -r.len ? 0 : r.len + n) : r.len;
  r.used = pages_of(r.len, page);
  r.keep = n < 0 ? pages_of(r.kept, page) : r.used;
  r.ask = n > 0 && n <= cap - r.len ? n : 0;
  r.bad |= n > 0 && r.ask == 0;
  r.need = r.ask ? pages_of(r.len + r.ask, page) - r.used : 0;
  return r;
}
// Requests of a thread that stay in registers between the scans; more are read again.
constexpr int HELD = 2;

__global__ void __launch_bounds__(THREADS) page_plan_kernel(PlanArgs a) {
  extern __shared__ int shared[];
  __shared__ uint4 part[2][WARPS];
  pdl_wait();
  pdl_trigger();
  int* upto_freed = shared;             // pages given back by requests 0 .. b
  int* upto_need = shared + a.B;        // pages asked for
  int* upto_tokens = shared + 2 * a.B;  // tokens granted
  int* lens = shared + 3 * a.B;         // tokens before the step
  int* starts = shared + 4 * a.B;       // first page asked for, of all that are
  const long long room = (long long)a.max_pages * a.page_size;
  const int cap = room > INT_MAX ? INT_MAX : (int)room;
  int count = a.free_count[0];
  const int per = (a.B + THREADS - 1) / THREADS, b0 = min((int)threadIdx.x * per, a.B), b1 = min(b0 + per, a.B);
  auto fetch = [&](int b) { return request(a.kv_lens[b], a.new_tokens[b], a.page_size, cap); };
  Request held[HELD];
#pragma unroll
  for (int i = 0; i < HELD; ++i)
    if (b0 + i < b1) held[i] = fetch(b0 + i);
  // body(b, request) of the thread's requests, in order
  auto each = [&](auto body) {
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (b0 + i < b1) body(b0 + i, held[i]);
    for (int b = b0 + HELD; b < b1; ++b) body(b, fetch(b));
  };
  auto sums_of = [](const Request& r) { return Sums{(unsigned)(r.used - r.keep), (unsigned)r.need, (unsigned)r.ask}; };
  bool bad = false;
  Sums mine{0, 0, 0}, all;
  each([&](int, const Request& r) {
    bad |= r.bad;
    mine = mine + sums_of(r);
  });
  const Sums before = block_before(mine, part[0], &all);
  count = count < 0 ? 0 : count > a.num_free ? a.num_free : count;
  const unsigned have = plus(count, all.freed);
  auto granted = [&](const Request& r, const Sums& upto) {
    return (r.need == 0 || upto.need <= have) && upto.ask <= (unsigned)a.max_tokens;
  };
  Sums at = before, got{0, 0, 0}, taken;
  each([&](int b, const Request& r) {
    starts[b] = (int)at.need;
    at = at + sums_of(r);
    upto_freed[b] = (int)at.freed;
    upto_need[b] = (int)at.need;
    lens[b] = r.len;
    if (granted(r, at)) got = got + Sums{0, (unsigned)r.need, (unsigned)r.ask};
  });
  Sums to = block_before(got, part[1], &taken);
  at = before;
  each([&](int b, const Request& r) {
    at = at + sums_of(r);
    const int ask = granted(r, at) ? r.ask : 0;
    if (blockIdx.x == 0) {
      a.cu[b] = (int)to.ask;
      a.lens_out[b] = r.kept + ask;
    }
    to.ask += ask;
    upto_tokens[b] = (int)to.ask;
  });
  const int freed = (int)all.freed, pages = (int)taken.need, tokens = (int)taken.ask;
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) {
      const unsigned left = have - pages;
      a.cu[a.B] = tokens;
      a.count_out[0] = min((int)left, a.num_free);
      bad |= left > (unsigned)a.num_free;
    }
    if (bad && a.err) atomicOr(a.err, ERR_PAGE);
  }
  __syncthreads();

  // the page that is given back as the i-th of all: the last ones of a request's table
  auto given = [&](int i) {
    const int b = first_above(upto_freed, a.B, i);
    if (b >= a.B) return -1;
    return a.page_table[b * a.pt_stride + pages_of(lens[b], a.page_size) - (upto_freed[b] - i)];
  };
  // the p-th page taken
  auto page = [&](int p) {
    const int i = (int)have - 1 - p;
    return i < count ? a.free_pages[i] : given(i - count);
  };
  // rows of tokens, pages taken, pages given back: one item after the other, spread over all threads
  const long long items = (long long)a.max_tokens + pages + freed;
  for (long long it = blockIdx.x * THREADS + threadIdx.x; it < items; it += gridDim.x * THREADS) {
    if (it < a.max_tokens) {
      const int t = (int)it;
      int b = -1, pos = -1;
      long long slot = -1;
      if (t < tokens) {
        b = first_above(upto_tokens, a.B, t);
        const int len = lens[b], used = pages_of(len, a.page_size);
        pos = len + t - (b > 0 ? upto_tokens[b - 1] : 0);
        const int k = (int)((unsigned)pos / (unsigned)a.page_size);
        const int id = k < used ? a.page_table[b * a.pt_stride + k] : page(starts[b] + k - used);
        slot = (long long)id * a.page_size + (pos - k * a.page_size);
      }
      a.requests[t] = b;
      a.positions[t] = pos;
      a.slots[t] = slot;
    } else if (it < (long long)a.max_tokens + pages) {
      const int p = (int)(it - a.max_tokens), b = first_above(upto_need, a.B, p);
      a.page_table[b * a.pt_stride + pages_of(lens[b], a.page_size) + p - starts[b]] = page(p);
    } else {
      const int i = (int)(it - a.max_tokens - pages);
      const long long where = (long long)count + i;
      if (where < a.num_free) a.free_pages[where] = given(i);
    }
  }
}

}  // namespace

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const int bytes = 5 * a.B * (int)sizeof(int);
  if (bytes > 40 * 1024) {
    const cudaError_t e = allow_shared(reinterpret_cast<const void*>(page_plan_kernel), 5 * PLAN_MAX_REQUESTS * (int)sizeof(int), &done);
    if (e != cudaSuccess) return e;
  }
  // an item a thread, as far as one CTA an SM goes: each repeats the sums (131,072 rows: 6.5 us, two an SM 6.8)
  const long long work = (long long)a.max_tokens + a.B, blocks = (work + THREADS - 1) / THREADS;
  prof_mark(K_PAGE_PLAN, s, true);
  const cudaError_t e = launch_pdl(page_plan_kernel, dim3((unsigned)(blocks < 1 ? 1 : blocks > 152 ? 152 : blocks)), dim3(THREADS), bytes, s, a);
  prof_mark(K_PAGE_PLAN, s, false);
  return e;
}

}  // namespace gdn
