// Short causal convolution of every channel along the tokens, forward and backward:
//   pre_t = bias + sum_j w_j x_{t - K + 1 + j},  y_t = pre_t, or pre_t sigmoid(pre_t)
// with the state (the K - 1 inputs before the call's first) in front of a sequence.
//
// Bound by memory: forward reads x and writes y, backward reads x and dy and writes dx.
// A thread owns a vector of channels and a run of tokens, keeps the window of the last K
// inputs in registers and has a batch of BATCH tokens' loads in flight; neighbouring
// threads own neighbouring vectors, so rows are read whole. A run reads the K - 1 inputs
// before it again (from L2). The sequence's first run alone reads the state and alone writes the next one, so
// that both may be the same memory however long the sequence is.
//
// Backward, with dpre = dy act'(pre): dx_t = sum_j w_j dpre_{t + K - 1 - j} looks K - 1 tokens ahead, so a run forms
// pre and dpre for its own tokens and K - 1 more, and its weight gradient dw_j = sum_t dpre_t x_{t - K + 1 + j} for
// its own. A thread takes several runs, so that the partial weight gradients, added in a fixed
// order by a second kernel, stay a small share of the traffic.
#include "packed.cuh"
#include "pairs.cuh"

namespace gdn {
namespace {

constexpr int THREADS = 128;
constexpr int BATCH = 8;       // tokens whose loads are in flight
constexpr int BWD_BATCH = 4;

template <class T, int V>
__device__ __forceinline__ void load_v(const T* p, float (&x)[V]) {
  if constexpr (V == 1) {
    x[0] = to_f32(*p);
  } else {
    alignas(16) T e[V];
    if constexpr (sizeof(T) * V == 16) *reinterpret_cast<uint4*>(e) = *reinterpret_cast<const uint4*>(p);
    else *reinterpret_cast<uint2*>(e) = *reinterpret_cast<const uint2*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = to_f32(e[i]);
  }
}
template <class T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&x)[V]) {
  if constexpr (V == 1) {
    *p = from_f32<T>(x[0]);
  } else {
    alignas(16) T e[V];
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = from_f32<T>(x[i]);
    if constexpr (sizeof(T) * V == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(e);
    else *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(e);
  }
}
// The vector as loaded, to be converted where it is used.
template <class T, int V>
struct Raw {
  static constexpr int W = (int)sizeof(T) * V >= 4 ? (int)sizeof(T) * V / 4 : 1;
  uint32_t w[W];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (sizeof(T) * V == 16) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
    else if constexpr (sizeof(T) * V == 8) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
    else if constexpr (sizeof(T) == 4) w[0] = __float_as_uint(*p);
    else w[0] = (uint32_t)__bfloat16_as_ushort(*p) << 16;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void floats(float (&x)[V]) const {
    if constexpr (V == 1) {
      x[0] = __uint_as_float(w[0]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
};

// Weights [C][K] of channels c .. c + V - 1, and the bias.
template <class T, int V, int K>
__device__ __forceinline__ void load_weights(const ConvArgs& a, int c, float (&w)[K][V], float (&bias)[V]) {
  const T* wp = static_cast<const T*>(a.w) + (long long)c * K;
  if constexpr (V == 1) {
#pragma unroll
    for (int j = 0; j < K; ++j) w[j][0] = to_f32(wp[j]);
  } else {
    float flat[V * K];
#pragma unroll
    for (int i = 0; i < V * K; i += V) {
      float part[V];
      load_v<T, V>(wp + i, part);
#pragma unroll
      for (int e = 0; e < V; ++e) flat[i + e] = part[e];
    }
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) w[j][e] = flat[e * K + j];
  }
#pragma unroll
  for (int e = 0; e < V; ++e) bias[e] = 0.f;
  if (a.bias) load_v<T, V>(static_cast<const T*>(a.bias) + c, bias);
}

// The K - 1 inputs before token t of the sequence: its own rows, or the state's (zeros without one).
template <class T, int V, int K>
__device__ __forceinline__ void load_past(const ConvArgs& a, const Chunk& k, int t, const T* state, int c, float (&past)[K - 1][V]) {
  const T* x = static_cast<const T*>(a.x);
#pragma unroll
  for (int i = 0; i < K - 1; ++i) {
    const int at = t - (K - 1) + i;
    if (at >= 0) {
      load_v<T, V>(x + (k.first + (long long)at) * a.x_ts + c, past[i]);
    } else if (state) {
      load_v<T, V>(state + (long long)(at + K - 1) * a.C + c, past[i]);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) past[i][e] = 0.f;
    }
  }
}

template <class T, int V, int K, bool SILU>
__global__ void __launch_bounds__(THREADS) causal_conv_fwd_kernel(ConvArgs a) {
  pdl_wait();
  pdl_trigger();
  const int vecs = a.C / V;
  const long long item = (long long)blockIdx.x * THREADS + threadIdx.x;
  const long long number = item / vecs;
  const int c = (int)(item - number * vecs) * V;
  if (number >= packed_numbers(a.q, a.run)) return;
  Chunk k;
  if (!packed_chunk(a.q, number, a.run, &k)) return;
  T* y = static_cast<T*>(a.y);
  const int t0 = k.j * a.run, t1 = min(k.len, t0 + a.run);
  if (k.b == a.q.B) {
    float none[V] = {};
    if (a.q.zero_tail)
      for (int t = t0; t < t1; ++t) store_v<T, V>(y + (k.first + (long long)t) * a.y_ts + c, none);
    return;
  }
  const T* state = nullptr;
  T* next = nullptr;
  if (k.j == 0) {  // runs are longer than a state
    const int slot = packed_slot(a.q, k.b);
    const long long at = (long long)slot * (K - 1) * a.C;
    if (slot >= 0 && a.state0 && packed_goes_on(a.q, k.b, k.len)) state = static_cast<const T*>(a.state0) + at;
    if (slot >= 0 && a.state_final) next = static_cast<T*>(a.state_final) + at;
  }
  float w[K][V], bias[V], win[K][V];  // win[K - 1]: the current input
  float old[K - 1][V];
  load_past<T, V, K>(a, k, t0, state, c, old);
#pragma unroll
  for (int i = 0; i < K - 1; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) win[i][e] = old[i][e];
  load_weights<T, V, K>(a, c, w, bias);
  const T* x = static_cast<const T*>(a.x) + (long long)k.first * a.x_ts + c;
  y += (long long)k.first * a.y_ts + c;
  for (int t = t0; t < t1; t += BATCH) {
    Raw<T, V> raw[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (t + i < t1) raw[i].load(x + (long long)(t + i) * a.x_ts);
      else raw[i].zero();
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      raw[i].floats(win[K - 1]);
      float out[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float pre = bias[e];
#pragma unroll
        for (int j = 0; j < K; ++j) pre = fmaf(w[j][e], win[j][e], pre);
        out[e] = SILU ? pre * sigmoid(pre) : pre;
      }
      if (t + i < t1) store_v<T, V>(y + (long long)(t + i) * a.y_ts, out);
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) win[j][e] = win[j + 1][e];
    }
  }
  if (next) {  // the last K - 1 of the state's inputs and the sequence's
    float last[K - 1][V];
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      const int at = k.len - (K - 1) + i;
      if (at >= 0) {
        load_v<T, V>(x + (long long)at * a.x_ts, last[i]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          last[i][e] = 0.f;
#pragma unroll
          for (int o = 0; o < K - 1; ++o) last[i][e] = o == at + K - 1 ? old[o][e] : last[i][e];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < K - 1; ++i) store_v<T, V>(next + (long long)i * a.C + c, last[i]);
  }
}

// Gradients. Token indexes run from -(K - 1), the state's inputs, to len - 1.
template <class T, int V, int K, bool SILU>
__global__ void __launch_bounds__(THREADS) causal_conv_bwd_kernel(ConvArgs a, int parts, long long numbers) {
  pdl_wait();
  pdl_trigger();
  const int vecs = a.C / V;
  const long long item = (long long)blockIdx.x * THREADS + threadIdx.x;
  const int part = (int)(item / vecs);
  const int c = (int)(item - (long long)part * vecs) * V;
  if (part >= parts) return;
  float w[K][V], bias[V], dw[K][V] = {}, db[V] = {};
  load_weights<T, V, K>(a, c, w, bias);
  for (long long number = part; number < numbers; number += parts) {
    Chunk k;
    if (!packed_chunk(a.q, number, a.run, &k)) continue;
    T* dx = static_cast<T*>(a.dx) + (long long)k.first * a.C + c;
    const int t0 = k.j * a.run, t1 = min(k.len, t0 + a.run);
    if (k.b == a.q.B) {
      float none[V] = {};
      for (int t = t0; t < t1; ++t) store_v<T, V>(dx + (long long)t * a.C, none);
      continue;
    }
    const long long held = (long long)k.b * (K - 1) * a.C + c;
    const T* state = a.state0 ? static_cast<const T*>(a.state0) + held - c : nullptr;
    const T* dstate = a.dstate ? static_cast<const T*>(a.dstate) + held : nullptr;
    float win[K][V], dpre[K][V];  // inputs t - K + 1 .. t and their outputs' gradients
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) dpre[j][e] = 0.f;
    {
      float old[K - 1][V];
      load_past<T, V, K>(a, k, t0, state, c, old);
#pragma unroll
      for (int i = 0; i < K - 1; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) win[i][e] = old[i][e];
    }
    const T* x = static_cast<const T*>(a.x) + (long long)k.first * a.x_ts + c;
    const T* dy = static_cast<const T*>(a.dy) + (long long)k.first * a.dy_ts + c;
    // the gradient of input t, once dpre of t .. t + K - 1 is in dpre[0 .. K - 1]
    auto emit = [&](int t) {
      float g[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        g[e] = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) g[e] = fmaf(w[j][e], dpre[K - 1 - j][e], g[e]);
      }
      // the last K - 1 inputs are the next state
      if (dstate && t >= k.len - (K - 1)) {
        float more[V];
        load_v<T, V>(dstate + (long long)(t - (k.len - (K - 1))) * a.C, more);
#pragma unroll
        for (int e = 0; e < V; ++e) g[e] += more[e];
      }
      if (t >= 0) store_v<T, V>(dx + (long long)t * a.C, g);
      else if (a.dstate0) store_v<T, V>(static_cast<T*>(a.dstate0) + held + (long long)(t + K - 1) * a.C, g);
    };
    // inputs whose gradients are this run's: its own tokens, and the state's for the first run
    const int from = k.j == 0 ? -(K - 1) : t0, stop = t1 + K - 1;
    for (int t = t0; t < stop; t += BWD_BATCH) {
      Raw<T, V> rx[BWD_BATCH], rd[BWD_BATCH];
#pragma unroll
      for (int i = 0; i < BWD_BATCH; ++i) {
        if (t + i < min(stop, k.len)) {
          rx[i].load(x + (long long)(t + i) * a.x_ts);
          rd[i].load(dy + (long long)(t + i) * a.dy_ts);
        } else {
          rx[i].zero();
          rd[i].zero();
        }
      }
#pragma unroll
      for (int i = 0; i < BWD_BATCH; ++i) {
        const int at = t + i;
        rx[i].floats(win[K - 1]);
        float g[V];
        rd[i].floats(g);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if (SILU) {
            float pre = bias[e];
#pragma unroll
            for (int j = 0; j < K; ++j) pre = fmaf(w[j][e], win[j][e], pre);
            const float s = sigmoid(pre);
            g[e] = at < k.len ? g[e] * fmaf(pre * s, 1.f - s, s) : 0.f;
          }
          dpre[K - 1][e] = g[e];
        }
        if (at < t1) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            db[e] += dpre[K - 1][e];
#pragma unroll
            for (int j = 0; j < K; ++j) dw[j][e] = fmaf(dpre[K - 1][e], win[j][e], dw[j][e]);
          }
        }
        if (at - (K - 1) >= from && at - (K - 1) < t1) emit(at - (K - 1));
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            win[j][e] = win[j + 1][e];
            dpre[j][e] = dpre[j + 1][e];
          }
      }
    }
  }
  float* to = a.partial + (long long)part * (K + 1) * a.C + c;
#pragma unroll
  for (int j = 0; j < K + 1; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) to[(long long)j * a.C + e] = j < K ? dw[j < K ? j : 0][e] : db[e];
}

// Adds the partial weight gradients: 8 warps take every eighth part of 32 channels, then add up in order.
template <class T>
__global__ void __launch_bounds__(256) causal_conv_wgrad_kernel(ConvArgs a, int parts) {
  __shared__ float sum[8][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, j = blockIdx.y;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < a.C) {
    const float* p = a.partial + (long long)j * a.C + c;
    const long long step = (long long)(a.taps + 1) * a.C;
#pragma unroll 4
    for (int i = warp; i < parts; i += 8) s += p[i * step];
  }
  sum[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= a.C) return;
  for (int i = 1; i < 8; ++i) s += sum[i][lane];
  if (j < a.taps) static_cast<T*>(a.dw)[(long long)c * a.taps + j] = from_f32<T>(s);
  else if (a.dbias) static_cast<T*>(a.dbias)[c] = from_f32<T>(s);
}

// Tokens of a run: short ones for more threads when tokens are few, long ones for fewer repeated
// inputs, at least a thread in 16 warps an SM.
int run_of(const ConvArgs& a, int vecs, int least) {
  const long long threads = (long long)152 * 16 * 32;
  int run = 64;
  while (run > least && (long long)a.q.N / run * vecs < threads) run /= 2;
  return run;
}
template <class T>
constexpr int fwd_vec() {
  return 16 / (int)sizeof(T);
}
// Parts of the weight gradients: threads for 8 warps an SM, and no more than there are runs.
long long parts_of(const ConvArgs& a, int vecs) {
  const long long numbers = packed_numbers(a.q, a.run), most = ((long long)152 * 16 * 32 + vecs - 1) / vecs;
  return numbers < most ? numbers : most;
}

template <class T, int V, int K, bool SILU>
cudaError_t fwd(ConvArgs a, cudaStream_t s) {
  const int vecs = a.C / V;
  a.run = a.max_q <= BATCH ? BATCH : run_of(a, vecs, 2 * BATCH);
  const long long blocks = (packed_numbers(a.q, a.run) * vecs + THREADS - 1) / THREADS;
  if (blocks > 0x7fffffff) return cudaErrorNotSupported;
  prof_mark(K_CONV_FWD, s, true);
  const cudaError_t e = launch_pdl(causal_conv_fwd_kernel<T, V, K, SILU>, dim3((unsigned)blocks), dim3(THREADS), 0, s, a);
  prof_mark(K_CONV_FWD, s, false);
  return e;
}
template <class T, int V, int K, bool SILU>
cudaError_t bwd(ConvArgs a, cudaStream_t s) {
  const int vecs = a.C / V;
  a.run = run_of(a, vecs, 16);
  const int parts = (int)parts_of(a, vecs);
  const long long blocks = ((long long)parts * vecs + THREADS - 1) / THREADS;
  prof_mark(K_CONV_BWD, s, true);
  cudaError_t e = launch_pdl(causal_conv_bwd_kernel<T, V, K, SILU>, dim3((unsigned)blocks), dim3(THREADS), 0, s, a, parts,
                             packed_numbers(a.q, a.run));
  prof_mark(K_CONV_BWD, s, false);
  if (e != cudaSuccess) return e;
  prof_mark(K_CONV_WGRAD, s, true);
  e = launch_pdl(causal_conv_wgrad_kernel<T>, dim3((a.C + 31) / 32, K + 1), dim3(256), 0, s, a, parts);
  prof_mark(K_CONV_WGRAD, s, false);
  return e;
}

template <class T, int V, bool BWD>
cudaError_t pick(const ConvArgs& a, cudaStream_t s) {
  auto go = [&](auto k, auto act) {
    if constexpr (BWD) return bwd<T, V, decltype(k)::value, decltype(act)::value>(a, s);
    else return fwd<T, V, decltype(k)::value, decltype(act)::value>(a, s);
  };
  auto with = [&](auto act) {
    if (a.taps == 2) return go(std::integral_constant<int, 2>(), act);
    if (a.taps == 3) return go(std::integral_constant<int, 3>(), act);
    return go(std::integral_constant<int, 4>(), act);
  };
  return a.silu ? with(BoolTag<true>()) : with(BoolTag<false>());
}

}  // namespace

cudaError_t launch_causal_conv(const ConvArgs& a, bool wide, cudaStream_t s) {
  if (a.bf16) return wide ? pick<bf16, fwd_vec<bf16>(), false>(a, s) : pick<bf16, 1, false>(a, s);
  return wide ? pick<float, fwd_vec<float>(), false>(a, s) : pick<float, 1, false>(a, s);
}
cudaError_t launch_causal_conv_bwd(const ConvArgs& a, bool wide, cudaStream_t s) {
  if (a.bf16) return wide ? pick<bf16, 4, true>(a, s) : pick<bf16, 1, true>(a, s);
  return wide ? pick<float, 4, true>(a, s) : pick<float, 1, true>(a, s);
}
size_t causal_conv_workspace(const ConvArgs& a0) {
  ConvArgs a = a0;
  size_t most = 0;
  for (int V : {1, 4}) {  // whichever width the call's pointers and strides allow
    if (a.C % V) continue;
    a.run = run_of(a, a.C / V, 16);
    const size_t n = (size_t)parts_of(a, a.C / V) * (a.taps + 1) * a.C * sizeof(float);
    most = n > most ? n : most;
  }
  return most;
}

}  // namespace gdn
