// Appends the new tokens' keys and values to a paged cache, turning the keys (and the
// queries, into q_out) by their position on the way.
//
// A pair (a, b) of a head's first `rot` channels at position p becomes
//   (a cos - b sin, b cos + a sin),  cos, sin = table[p][pair]
// with pairs (i, i + rot/2), or (2i, 2i + 1). Products in fp32, one rounding at the store.
//
// Bound by memory: each value is read once and written once. A thread owns two 16-byte
// vectors of a head row that hold whole pairs ("unit"), the same unit for every head row
// it takes, so a token's cos and sin are read once into registers and serve all of them.
// Rows are taken BATCH at a time, and the first ones' data is on its way before the token's
// sequence, page and table row are looked up, so that the two chains of latency overlap.
// Many small CTAs (one token each in a usual model) keep the memory busy while others look
// up; values that no other thread will read pass the caches by. A prefill of 27,008 tokens
// with 48 + 2 x 8 heads of 128 in bf16 takes 132 us, 6.7 TB/s, the measured copy bandwidth
// (CTAs of 256 threads: 168 us; without the streaming accesses 10 us more).
#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int THREADS = 128;
constexpr int BATCH = 2;  // head rows a thread has in flight

template <class T>
__device__ __forceinline__ void unpack(const uint4& u, float (&x)[16 / sizeof(T)]) {
  const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
  for (int i = 0; i < 16 / (int)sizeof(T); ++i) x[i] = to_f32(e[i]);
}
template <class T>
__device__ __forceinline__ uint4 pack(const float (&x)[16 / sizeof(T)]) {
  uint4 u;
  T* e = reinterpret_cast<T*>(&u);
#pragma unroll
  for (int i = 0; i < 16 / (int)sizeof(T); ++i) e[i] = from_f32<T>(x[i]);
  return u;
}

template <class T, int D>
__global__ void __launch_bounds__(THREADS, 8) kv_append_kernel(AppendArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int V = 16 / (int)sizeof(T), UNITS = D / (2 * V), SLOTS = THREADS / UNITS;
  const PagedArgs& p = a.p;
  const int nq = a.q ? p.Hq : 0, rows = nq + 2 * p.Hk;
  const int per = rows < SLOTS ? SLOTS / rows : 1;  // tokens of a CTA
  const int slot = threadIdx.x / UNITS, u = threadIdx.x % UNITS;
  const int sub = slot / rows < per ? slot / rows : per - 1;
  const long long tok = (long long)blockIdx.x * per + sub;
  int row = per > 1 ? slot - sub * rows : slot;
  if (tok >= p.N || row >= rows) return;
  const int step = per > 1 ? rows : SLOTS;
  const int half = a.rot / (2 * V);  // units of the turned part
  const bool turned = u < half;
  // the unit's two vectors
  const int c0 = a.pairs || !turned ? 2 * u * V : u * V;
  const int c1 = a.pairs || !turned ? c0 + V : c0 + a.rot / 2;

  auto source = [&](int r) -> const T* {
    if (r < nq) return static_cast<const T*>(a.q) + tok * a.q_ts + (long long)r * a.q_hs;
    r -= nq;
    if (r < p.Hk) return static_cast<const T*>(a.k) + tok * a.kn_ts + (long long)r * a.kn_hs;
    return static_cast<const T*>(a.v) + tok * a.vn_ts + (long long)(r - p.Hk) * a.vn_hs;
  };
  uint4 x0[BATCH], x1[BATCH];
  auto load = [&]() {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (row + i * step >= rows) break;
      const T* src = source(row + i * step);
      x0[i] = __ldcs(reinterpret_cast<const uint4*>(src + c0));
      x1[i] = __ldcs(reinterpret_cast<const uint4*>(src + c1));
    }
  };
  load();

  // the token's sequence: the last b with cu[b] <= tok (empty sequences repeat a bound)
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cu[mid] <= tok) lo = mid;
    else hi = mid;
  }
  const int b = lo, first = p.cu[b], end = p.cu[b + 1];
  if (tok < first || tok >= end) return;  // padding outside every sequence
  const long long pos = (long long)p.lens[b] - (end - first) + (tok - first);
  long long page = -1;
  int prow = 0;
  bool turn = false;
  if (pos >= 0) {  // tokens before position 0 are not kept
    bool bad = pos >= (long long)p.max_pages * p.page_size;
    if (!bad) {
      page = p.page_table[b * p.pt_stride + pos / p.page_size];
      prow = (int)(pos % p.page_size);
      if (page < 0 || page >= p.num_pages) {
        bad = true;
        page = -1;
      }
    }
    if (a.rot > 0) {
      turn = pos < a.positions;
      if (!turn) {
        bad = true;
        page = -1;
      }
    }
    if (bad && u == 0 && p.err) atomicOr(p.err, ERR_PAGE);
  }
  float cs[V], sn[V];  // the unit's V pairs
#pragma unroll
  for (int i = 0; i < V; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
  }
  if (turn && turned) {
    const float *c = a.cos + pos * (a.rot / 2) + u * V, *s = a.sin + pos * (a.rot / 2) + u * V;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 fc = *reinterpret_cast<const float4*>(c + i), fs = *reinterpret_cast<const float4*>(s + i);
      cs[i] = fc.x; cs[i + 1] = fc.y; cs[i + 2] = fc.z; cs[i + 3] = fc.w;
      sn[i] = fs.x; sn[i + 1] = fs.y; sn[i + 2] = fs.z; sn[i + 3] = fs.w;
    }
  }
  while (true) {
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      const int r = row + b * step;
      if (r >= rows) break;
      T* dst = nullptr;
      if (r < nq) {
        dst = static_cast<T*>(a.q_out) + tok * a.qo_ts + (long long)r * a.qo_hs;
      } else if (page >= 0) {
        const int h = r - nq;
        dst = h < p.Hk ? static_cast<T*>(p.kc) + page * p.k_ps + h * p.k_hs + prow * p.k_rs
                       : static_cast<T*>(p.vc) + page * p.v_ps + (h - p.Hk) * p.v_hs + prow * p.v_rs;
      }
      if (!dst) continue;
      if (turn && turned && r < nq + p.Hk) {
        float f0[V], f1[V];
        unpack<T>(x0[b], f0);
        unpack<T>(x1[b], f1);
        if (a.pairs) {  // neighbours: pair i of the unit is channels 2i, 2i + 1 of its 2 V channels
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            const float e0 = f0[i], o0 = f0[i + 1], e1 = f1[i], o1 = f1[i + 1];
            const float ca = cs[i / 2], sa = sn[i / 2], cb = cs[V / 2 + i / 2], sb = sn[V / 2 + i / 2];
            f0[i] = e0 * ca - o0 * sa;
            f0[i + 1] = o0 * ca + e0 * sa;
            f1[i] = e1 * cb - o1 * sb;
            f1[i + 1] = o1 * cb + e1 * sb;
          }
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float e = f0[i], o = f1[i];
            f0[i] = e * cs[i] - o * sn[i];
            f1[i] = o * cs[i] + e * sn[i];
          }
        }
        x0[b] = pack<T>(f0);
        x1[b] = pack<T>(f1);
      }
      __stcs(reinterpret_cast<uint4*>(dst + c0), x0[b]);
      __stcs(reinterpret_cast<uint4*>(dst + c1), x1[b]);
    }
    row += BATCH * step;
    if (per > 1 || row >= rows) break;
    load();
  }
}

template <class T, int D>
cudaError_t run(const AppendArgs& a, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T), SLOTS = THREADS / (D / (2 * V));
  const int rows = (a.q ? a.p.Hq : 0) + 2 * a.p.Hk, per = rows < SLOTS ? SLOTS / rows : 1;
  prof_mark(K_KV_APPEND, s, true);
  const cudaError_t e = launch_pdl(kv_append_kernel<T, D>, dim3((unsigned)(((long long)a.p.N + per - 1) / per)),
                                   dim3(THREADS), 0, s, a);
  prof_mark(K_KV_APPEND, s, false);
  return e;
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t s) {
  if (a.p.bf16) return a.p.D == 64 ? run<bf16, 64>(a, s) : run<bf16, 128>(a, s);
  return a.p.D == 64 ? run<float, 64>(a, s) : run<float, 128>(a, s);
}

}  // namespace gdn
