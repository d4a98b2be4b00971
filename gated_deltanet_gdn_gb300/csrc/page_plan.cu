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
// each CTA forms the prefix sums over all requests for itself in shared memory (two block scans; 256 requests take
// less than a second launch would), then takes its share of tokens and pages, so that no CTA waits for another. A
// page from the part of the list that this step gives back is found through the sums, not read back from the list,
// and no array is read where another CTA may write it.
#include <climits>

#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;

struct Sums {
  long long freed, need, ask;
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return Sums{a.freed + b.freed, a.need + b.need, a.ask + b.ask};
}
__device__ __forceinline__ Sums shfl_up(const Sums& v, int d) {
  return Sums{__shfl_up_sync(~0u, v.freed, d), __shfl_up_sync(~0u, v.need, d), __shfl_up_sync(~0u, v.ask, d)};
}

// Sum over the threads before this one; *total over all. `part` is free again after the next barrier.
__device__ __forceinline__ Sums block_before(const Sums& mine, Sums* part, Sums* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  Sums up = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const Sums o = shfl_up(up, d);
    if (lane >= d) up = up + o;
  }
  if (lane == 31) part[warp] = up;
  __syncthreads();
  Sums before{0, 0, 0}, all{0, 0, 0};
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    if (i < warp) before = before + part[i];
    all = all + part[i];
  }
  *total = all;
  const Sums ex = shfl_up(up, 1);
  return lane ? before + ex : before;
}
__device__ __forceinline__ int saturate(long long v) { return v > INT_MAX ? INT_MAX : (int)v; }

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
  int len, keep, used;  // tokens, pages that stay, pages it has
  int kept;             // tokens that stay
  int ask, need;        // new tokens and pages, 0 where they do not fit the table
  bool bad;
};
__device__ __forceinline__ int pages_of(long long tokens, int page) { return (int)((tokens + page - 1) / page); }
__device__ __forceinline__ Request request(const PlanArgs& a, int b) {
  Request r;
  const long long cap = (long long)a.max_pages * a.page_size;
  long long len = a.kv_lens[b];
  const long long n = a.new_tokens[b];
  r.bad = len < 0 || len > cap;
  len = len < 0 ? 0 : len > cap ? cap : len;
  r.len = (int)len;
  r.kept = (int)(n < 0 ? (len + n > 0 ? len + n : 0) : len);
  r.used = pages_of(len, a.page_size);
  r.keep = pages_of(r.kept, a.page_size);
  r.ask = n > 0 && len + n <= cap && len + n <= INT_MAX ? (int)n : 0;
  r.bad |= n > 0 && r.ask == 0;
  r.need = r.ask ? pages_of(len + r.ask, a.page_size) - r.used : 0;
  return r;
}

__global__ void __launch_bounds__(THREADS) page_plan_kernel(PlanArgs a) {
  extern __shared__ int shared[];
  __shared__ Sums part[2][WARPS];
  pdl_wait();
  pdl_trigger();
  int* upto_freed = shared;            // pages given back by requests 0 .. b
  int* upto_need = shared + a.B;       // pages asked for
  int* upto_tokens = shared + 2 * a.B; // tokens granted
  int count = a.free_count[0];
  count = count < 0 ? 0 : count > a.num_free ? a.num_free : count;
  const int per = (a.B + THREADS - 1) / THREADS, b0 = min((int)threadIdx.x * per, a.B), b1 = min(b0 + per, a.B);
  bool bad = false;
  Sums mine{0, 0, 0}, all;
  for (int b = b0; b < b1; ++b) {
    const Request r = request(a, b);
    bad |= r.bad;
    mine = mine + Sums{r.used - r.keep, r.need, r.ask};
  }
  const Sums before = block_before(mine, part[0], &all);
  const long long have = count + all.freed;
  Sums at = before, got{0, 0, 0};
  auto granted = [&](const Request& r, const Sums& upto) {
    return (r.need == 0 || upto.need <= have) && upto.ask <= a.max_tokens;
  };
  for (int b = b0; b < b1; ++b) {
    const Request r = request(a, b);
    at = at + Sums{r.used - r.keep, r.need, r.ask};
    upto_freed[b] = saturate(at.freed);
    upto_need[b] = saturate(at.need);
    if (granted(r, at)) got = got + Sums{0, r.need, r.ask};
  }
  Sums taken;
  Sums to = block_before(got, part[1], &taken);
  at = before;
  for (int b = b0; b < b1; ++b) {
    const Request r = request(a, b);
    at = at + Sums{r.used - r.keep, r.need, r.ask};
    const int ask = granted(r, at) ? r.ask : 0;
    if (blockIdx.x == 0) {
      a.cu[b] = (int)to.ask;
      a.lens_out[b] = r.kept + ask;
    }
    to.ask += ask;
    upto_tokens[b] = (int)to.ask;
  }
  const int freed = saturate(all.freed), pages = (int)taken.need, tokens = (int)taken.ask;
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) {
      a.cu[a.B] = tokens;
      const long long left = have - pages;
      a.count_out[0] = (int)(left > a.num_free ? a.num_free : left);
      bad |= left > a.num_free;
    }
    if (bad && a.err) atomicOr(a.err, ERR_PAGE);
  }
  __syncthreads();

  // the page that request b gave back as its i-th, counted over all requests
  auto given = [&](int i) {
    const int b = first_above(upto_freed, a.B, i);
    if (b >= a.B) return -1;
    const Request r = request(a, b);
    return a.page_table[b * a.pt_stride + r.used - (upto_freed[b] - i)];
  };
  // the p-th page taken
  auto page = [&](int p) {
    const long long i = have - 1 - p;
    return i < count ? a.free_pages[i] : given((int)(i - count));
  };
  const int tid = blockIdx.x * THREADS + threadIdx.x, all_threads = gridDim.x * THREADS;
  for (int t = tid; t < a.max_tokens; t += all_threads) {
    int b = -1, pos = -1;
    long long slot = -1;
    if (t < tokens) {
      b = first_above(upto_tokens, a.B, t);
      const Request r = request(a, b);
      const int i = t - (upto_tokens[b] - r.ask), k = (r.len + i) / a.page_size;
      pos = r.len + i;
      const int id = k < r.used ? a.page_table[b * a.pt_stride + k] : page(upto_need[b] - r.need + k - r.used);
      slot = (long long)id * a.page_size + pos % a.page_size;
    }
    a.requests[t] = b;
    a.positions[t] = pos;
    a.slots[t] = slot;
  }
  for (int p = tid; p < pages; p += all_threads) {
    const int b = first_above(upto_need, a.B, p);
    const Request r = request(a, b);
    a.page_table[b * a.pt_stride + r.used + p - (upto_need[b] - r.need)] = page(p);
  }
  for (int i = tid; i < freed; i += all_threads) {
    const long long to_ = (long long)count + i;
    if (to_ < a.num_free) a.free_pages[to_] = given(i);
  }
}

}  // namespace

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const int bytes = 3 * a.B * (int)sizeof(int);
  if (bytes > 40 * 1024) {
    const cudaError_t e = allow_shared(reinterpret_cast<const void*>(page_plan_kernel), 3 * PLAN_MAX_REQUESTS * (int)sizeof(int), &done);
    if (e != cudaSuccess) return e;
  }
  // a token or two a thread, and no more CTAs than SMs: each repeats the sums
  const int work = a.max_tokens > a.B ? a.max_tokens : a.B, blocks = (work + THREADS - 1) / THREADS;
  prof_mark(K_PAGE_PLAN, s, true);
  const cudaError_t e = launch_pdl(page_plan_kernel, dim3(blocks < 1 ? 1 : blocks > 152 ? 152 : blocks), dim3(THREADS), bytes, s, a);
  prof_mark(K_PAGE_PLAN, s, false);
  return e;
}

}  // namespace gdn
