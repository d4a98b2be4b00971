// Short causal convolution of every channel along the tokens, forward and backward:
//   pre_t = bias + sum_j w_j x_{t - K + 1 + j},  y_t = pre_t, or pre_t sigmoid(pre_t)
// with the state (the K - 1 inputs before the call's first) in front of a sequence.
//
// Bound by memory: forward reads x and writes y, backward reads x and dy and writes dx.
// A thread owns a vector of channels and a run of tokens, keeps the window of the last K
// inputs in registers and has the next BATCH tokens' loads in flight while it works on these; neighbouring
// threads own neighbouring vectors, so rows are read whole. A run reads the K - 1 inputs
// before it again (from L2). The sequence's first run alone reads the state and alone writes the next one, so
// that both may be the same memory however long the sequence is.
//
// Backward, with dpre = dy act'(pre): dx_t = sum_j w_j dpre_{t + K - 1 - j} looks K - 1 tokens ahead, so a run forms
// pre and dpre for its own tokens and K - 1 more, and its weight gradient dw_j = sum_t dpre_t x_{t - K + 1 + j} for
// its own. Runs are as long as a few threads per lane of the GPU allow, so that the partial weight gradients, added in a
// fixed order by a second kernel, stay a small share of the traffic.
//
// Values go two by two through the fp32 instructions (fma.rn.f32x2): with one by one, the arithmetic of 2304 channels x
// 32,768 tokens took as long as their bytes (75 us forward, 200 us backward).
#include "packed.cuh"
#include "pairs.cuh"

namespace gdn {
namespace {

constexpr int THREADS = 128;

// V channels of a token as they lie in memory, and as pairs (V = 1: one pair, its second half unused).
template <class T, int V>
struct Raw {
  static constexpr int W = (int)sizeof(T) * V >= 4 ? (int)sizeof(T) * V / 4 : 1, NP = V > 1 ? V / 2 : 1;
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
  __device__ __forceinline__ void pairs(f32x2 (&x)[NP]) const {
    if constexpr (V == 1) {
      x[0] = pack2(__uint_as_float(w[0]), 0.f);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < NP; ++i) x[i] = pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i) x[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
  }
};
template <class T, int V>
__device__ __forceinline__ void load_v(const T* p, f32x2 (&x)[Raw<T, V>::NP]) {
  Raw<T, V> r;
  r.load(p);
  r.pairs(x);
}
template <class T, int V>
__device__ __forceinline__ void store_v(T* p, const f32x2 (&x)[Raw<T, V>::NP]) {
  if constexpr (V == 1) {
    *p = from_f32<T>(split2(x[0]).x);
  } else {
    alignas(16) T e[V];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 f = split2(x[i]);
      store2(e + 2 * i, f.x, f.y);
    }
    if constexpr (sizeof(T) * V == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(e);
    else *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(e);
  }
}

// Weights [C][K] of channels c .. c + V - 1, and the bias.
template <class T, int V, int K, int NP>
__device__ __forceinline__ void load_weights(const ConvArgs& a, int c, f32x2 (&w)[K][NP], f32x2 (&bias)[NP]) {
  const T* wp = static_cast<const T*>(a.w) + (long long)c * K;
  float flat[2 * NP * K];
  if constexpr (V == 1) {
#pragma unroll
    for (int j = 0; j < 2 * K; ++j) flat[j] = j < K ? to_f32(wp[j]) : 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < V * K; i += V) {
      f32x2 part[NP];
      load_v<T, V>(wp + i, part);
#pragma unroll
      for (int e = 0; e < NP; ++e) {
        const float2 f = split2(part[e]);
        flat[i + 2 * e] = f.x;
        flat[i + 2 * e + 1] = f.y;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < K; ++j)
#pragma unroll
    for (int e = 0; e < NP; ++e) w[j][e] = pack2(flat[2 * e * K + j], flat[(2 * e + 1) * K + j]);
#pragma unroll
  for (int e = 0; e < NP; ++e) bias[e] = both(0.f);
  if (a.bias) load_v<T, V>(static_cast<const T*>(a.bias) + c, bias);
}

// The input i - (K - 1) before token t of the sequence: its own row, or the state's (zeros without one).
template <class T, int V, int K>
__device__ __forceinline__ void load_past(const ConvArgs& a, const Chunk& k, int at, const T* state, int c,
                                          f32x2 (&past)[Raw<T, V>::NP]) {
  Raw<T, V> r;
  r.zero();
  if (at >= 0) r.load(static_cast<const T*>(a.x) + (k.first + (long long)at) * a.x_ts + c);
  else if (state) r.load(state + (long long)(at + K - 1) * a.C + c);
  r.pairs(past);
}

// Zeros in the padding's rows of y or dx.
template <class T, int V>
__device__ __forceinline__ void zero_padding(const ConvArgs& a, unsigned from, void* p, long long ts) {
  packed_padding<THREADS>(a.q, from, a.C / V, [&](long long r, int v) {
    f32x2 none[Raw<T, V>::NP];
#pragma unroll
    for (int e = 0; e < Raw<T, V>::NP; ++e) none[e] = both(0.f);
    store_v<T, V>(static_cast<T*>(p) + r * ts + v * V, none);
  });
}

template <class T, int V, int K, bool SILU, int BATCH>
__global__ void __launch_bounds__(THREADS) causal_conv_fwd_kernel(ConvArgs a, unsigned ctas) {
  constexpr int NP = Raw<T, V>::NP;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x >= ctas) {
    zero_padding<T, V>(a, ctas, a.y, a.y_ts);
    return;
  }
  const int vecs = a.C / V;
  const long long item = (long long)blockIdx.x * THREADS + threadIdx.x;
  const long long number = item / vecs;
  const int c = (int)(item - number * vecs) * V;
  if (number >= packed_numbers(a.q, a.run)) return;
  f32x2 w[K][NP], bias[NP], win[K][NP];  // win[K - 1]: the current input
  if constexpr (BATCH == 1) load_weights<T, V, K>(a, c, w, bias);  // on their way during the look-up
  Chunk k;
  if (!packed_chunk(a.q, number, a.run, &k)) return;
  const int t0 = k.j * a.run, t1 = min(k.len, t0 + a.run);
  T* y = static_cast<T*>(a.y) + (k.first + (long long)t0) * a.y_ts + c;
  const T* x = static_cast<const T*>(a.x) + (k.first + (long long)t0) * a.x_ts + c;
  Raw<T, V> raw[BATCH];
  auto fetch = [&](int t) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (t + i < t1) raw[i].load(x + i * a.x_ts);
    x += BATCH * a.x_ts;
  };
  fetch(t0);
  const T* state = nullptr;
  T* next = nullptr;
  if (k.j == 0) {  // runs are longer than a state
    const int slot = packed_slot(a.q, k.b);
    const long long at = (long long)slot * (K - 1) * a.C;
    if (slot >= 0 && a.state0 && packed_goes_on(a.q, k.b, k.len)) state = static_cast<const T*>(a.state0) + at;
    if (slot >= 0 && a.state_final) next = static_cast<T*>(a.state_final) + at;
  }
#pragma unroll
  for (int i = 0; i < K - 1; ++i) load_past<T, V, K>(a, k, t0 - (K - 1) + i, state, c, win[i]);
  if constexpr (BATCH != 1) load_weights<T, V, K>(a, c, w, bias);
  // The last K - 1 of the state's inputs and the sequence's: all that this thread reads of the state is
  // read by now, whatever it writes.
  if (next) {
    f32x2 last[K - 1][NP];
#pragma unroll
    for (int i = 0; i < K - 1; ++i) load_past<T, V, K>(a, k, k.len - (K - 1) + i, state, c, last[i]);
#pragma unroll
    for (int i = 0; i < K - 1; ++i) store_v<T, V>(next + (long long)i * a.C + c, last[i]);
  }
  for (int t = t0; t < t1; t += BATCH) {
    Raw<T, V> now[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) now[i] = raw[i];
    fetch(t + BATCH);
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      now[i].pairs(win[K - 1]);
      f32x2 out[NP];
#pragma unroll
      for (int e = 0; e < NP; ++e) {
        f32x2 pre = bias[e];
#pragma unroll
        for (int j = 0; j < K; ++j) pre = fma2(w[j][e], win[j][e], pre);
        out[e] = SILU ? mul2(pre, sigmoid2(pre)) : pre;
      }
      if (t + i < t1) store_v<T, V>(y, out);
      y += a.y_ts;
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
#pragma unroll
        for (int e = 0; e < NP; ++e) win[j][e] = win[j + 1][e];
    }
  }
}

// Gradients. Token indexes run from -(K - 1), the state's inputs, to len - 1.
template <class T, int V, int K, bool SILU>
__global__ void __launch_bounds__(THREADS, 4) causal_conv_bwd_kernel(ConvArgs a, int parts, long long numbers, unsigned ctas) {
  constexpr int NP = Raw<T, V>::NP, BATCH = 4;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x >= ctas) {
    zero_padding<T, V>(a, ctas, a.dx, a.C);
    return;
  }
  const int vecs = a.C / V;
  const long long item = (long long)blockIdx.x * THREADS + threadIdx.x;
  const int part = (int)(item / vecs);
  const int c = (int)(item - (long long)part * vecs) * V;
  if (part >= parts) return;
  f32x2 w[K][NP], bias[NP], dw[K][NP], db[NP];
#pragma unroll
  for (int e = 0; e < NP; ++e) {
    db[e] = both(0.f);
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j][e] = both(0.f);
  }
  load_weights<T, V, K>(a, c, w, bias);
  for (long long number = part; number < numbers; number += parts) {
    Chunk k;
    if (!packed_chunk(a.q, number, a.run, &k)) continue;
    const int t0 = k.j * a.run, t1 = min(k.len, t0 + a.run);
    T* dx = static_cast<T*>(a.dx) + (k.first + (long long)t0) * a.C + c;  // of token t0, moving on with the tokens
    const long long held = (long long)k.b * (K - 1) * a.C + c;
    const T* state = a.state0 ? static_cast<const T*>(a.state0) + held - c : nullptr;
    const T* dstate = a.dstate ? static_cast<const T*>(a.dstate) + held : nullptr;
    // inputs whose gradients are this run's: its own tokens, and the state's for the first run
    const int from = k.j == 0 ? -(K - 1) : t0, stop = t1 + K - 1, real = min(stop, k.len);
    const T* x = static_cast<const T*>(a.x) + (k.first + (long long)t0) * a.x_ts + c;
    const T* dy = static_cast<const T*>(a.dy) + (k.first + (long long)t0) * a.dy_ts + c;
    Raw<T, V> rx[BATCH], rd[BATCH];
    auto fetch = [&](int t) {
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        rx[i].zero();
        rd[i].zero();
        if (t + i < real) {
          rx[i].load(x + i * a.x_ts);
          rd[i].load(dy + i * a.dy_ts);
        }
      }
      x += BATCH * a.x_ts;
      dy += BATCH * a.dy_ts;
    };
    fetch(t0);
    f32x2 win[K][NP], dpre[K][NP];  // inputs t - K + 1 .. t and their outputs' gradients
#pragma unroll
    for (int i = 0; i < K - 1; ++i) load_past<T, V, K>(a, k, t0 - (K - 1) + i, state, c, win[i]);
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int e = 0; e < NP; ++e) dpre[j][e] = both(0.f);
    dx -= (K - 1) * (long long)a.C;  // the gradient that is complete at token t is of token t - (K - 1)
    for (int t = t0; t < stop; t += BATCH) {
      Raw<T, V> nx[BATCH], nd[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        nx[i] = rx[i];
        nd[i] = rd[i];
      }
      fetch(t + BATCH);
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int at = t + i, done = at - (K - 1);
        nx[i].pairs(win[K - 1]);
        nd[i].pairs(dpre[K - 1]);
        if constexpr (SILU) {
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            f32x2 pre = bias[e];
#pragma unroll
            for (int j = 0; j < K; ++j) pre = fma2(w[j][e], win[j][e], pre);
            const f32x2 s = sigmoid2(pre);  // silu' = s + pre s (1 - s)
            dpre[K - 1][e] = mul2(dpre[K - 1][e], fma2(mul2(pre, s), fma2(s, both(-1.f), both(1.f)), s));
            if (at >= k.len) dpre[K - 1][e] = both(0.f);
          }
        }
        if (at < t1) {
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            db[e] = add2(db[e], dpre[K - 1][e]);
#pragma unroll
            for (int j = 0; j < K; ++j) dw[j][e] = fma2(dpre[K - 1][e], win[j][e], dw[j][e]);
          }
        }
        if (done >= from && done < t1) {
          f32x2 g[NP];
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            g[e] = mul2(w[0][e], dpre[K - 1][e]);
#pragma unroll
            for (int j = 1; j < K; ++j) g[e] = fma2(w[j][e], dpre[K - 1 - j][e], g[e]);
          }
          // the last K - 1 inputs are the next state
          if (dstate && done >= k.len - (K - 1)) {
            f32x2 more[NP];
            load_v<T, V>(dstate + (long long)(done - (k.len - (K - 1))) * a.C, more);
#pragma unroll
            for (int e = 0; e < NP; ++e) g[e] = add2(g[e], more[e]);
          }
          if (done >= 0) store_v<T, V>(dx, g);
          else if (a.dstate0) store_v<T, V>(static_cast<T*>(a.dstate0) + held + (long long)(done + K - 1) * a.C, g);
        }
        dx += a.C;
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
#pragma unroll
          for (int e = 0; e < NP; ++e) {
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
    for (int e = 0; e < NP; ++e) {
      const float2 f = split2(j < K ? dw[j < K ? j : 0][e] : db[e]);
      to[(long long)j * a.C + 2 * e] = f.x;
      if (V > 1) to[(long long)j * a.C + 2 * e + 1] = f.y;
    }
}

// Adds the partial weight gradients of 32 channels: a CTA's warps take the parts in turn, then add up in order. About 16
// parts a warp: with 8 warps always, the 1216 parts of 512 fp32 channels took 17 us in place of 10, with 32 always the 102 parts
// of 6144 channels 14 in place of 9.
template <class T>
__global__ void __launch_bounds__(1024) causal_conv_wgrad_kernel(ConvArgs a, int parts) {
  __shared__ float sum[32][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32, j = blockIdx.y;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < a.C) {
    const float* p = a.partial + (long long)j * a.C + c;
    const long long step = (long long)(a.taps + 1) * a.C;
#pragma unroll 8
    for (int i = warp; i < parts; i += warps) s += p[i * step];
  }
  sum[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= a.C) return;
  for (int i = 1; i < warps; ++i) s += sum[i][lane];
  if (j < a.taps) static_cast<T*>(a.dw)[(long long)c * a.taps + j] = from_f32<T>(s);
  else if (a.dbias) static_cast<T*>(a.dbias)[c] = from_f32<T>(s);
}

// Tokens of a forward run: short ones for more threads when tokens are few, long ones for fewer repeated
// inputs, at least a thread in 16 warps an SM.
int run_of(const ConvArgs& a, int vecs) {
  const long long threads = (long long)152 * 16 * 32;
  int run = 128;
  while (run > 16 && (long long)a.q.N / run * vecs < threads) run /= 2;
  return run;
}
// Backward: as many parts of the weight gradients as give 32 warps an SM, a run or two for each part (at least 16 tokens: a
// run reads and forms 3 tokens more).
constexpr int BWD_WARPS = 32;
void bwd_plan(ConvArgs* a, int vecs, int* parts, long long* numbers) {
  const long long most = ((long long)152 * BWD_WARPS * 32 + vecs - 1) / vecs;
  if (a->q.cu) {
    const long long left = most > a->q.B + 1 ? most - a->q.B - 1 : 1;
    a->run = (int)((a->q.N + left - 1) / left);
  } else {
    const long long per = a->q.B > 0 && most > a->q.B ? most / a->q.B : 1;
    a->run = (int)((a->q.T + per - 1) / per);
  }
  if (a->run < 16) a->run = 16;
  *numbers = packed_numbers(a->q, a->run);
  *parts = (int)(*numbers < most ? *numbers : most);
}
// A sequence's new tokens up to which a run is a sequence, with 16-byte vectors and one token's loads at a time (32 tokens of
// 18,432 channels 4.0 us); longer runs take vectors of four channels and sixteen tokens' loads, of float32 eight (32,768 tokens of 2,304
// channels 53 us, with 16-byte vectors and eight tokens 58 us).
constexpr int FEW = 8;

template <class T, int V, int K, bool SILU, int BATCH>
cudaError_t fwd(ConvArgs a, cudaStream_t s) {
  const int vecs = a.C / V;
  a.run = a.max_q <= FEW ? PACKED_WHOLE : run_of(a, vecs);
  const long long blocks = (packed_numbers(a.q, a.run) * vecs + THREADS - 1) / THREADS;
  const unsigned pad = packed_pad_ctas(a.q, a.q.zero_tail, vecs, THREADS);
  if (blocks + pad > 0x7fffffff) return cudaErrorNotSupported;
  prof_mark(K_CONV_FWD, s, true);
  const cudaError_t e = launch_pdl(causal_conv_fwd_kernel<T, V, K, SILU, BATCH>, dim3((unsigned)blocks + pad), dim3(THREADS), 0, s, a,
                                   (unsigned)blocks);
  prof_mark(K_CONV_FWD, s, false);
  return e;
}
template <class T, int V, int K, bool SILU>
cudaError_t bwd(ConvArgs a, cudaStream_t s) {
  const int vecs = a.C / V;
  int parts;
  long long numbers;
  bwd_plan(&a, vecs, &parts, &numbers);
  const long long blocks = ((long long)parts * vecs + THREADS - 1) / THREADS;
  const unsigned pad = packed_pad_ctas(a.q, true, vecs, THREADS);
  prof_mark(K_CONV_BWD, s, true);
  cudaError_t e = launch_pdl(causal_conv_bwd_kernel<T, V, K, SILU>, dim3((unsigned)blocks + pad), dim3(THREADS), 0, s, a, parts, numbers,
                             (unsigned)blocks);
  prof_mark(K_CONV_BWD, s, false);
  if (e != cudaSuccess) return e;
  prof_mark(K_CONV_WGRAD, s, true);
  const int warps = parts < 128 ? 8 : parts < 512 ? parts / 16 : 32;
  e = launch_pdl(causal_conv_wgrad_kernel<T>, dim3((a.C + 31) / 32, K + 1), dim3(32 * warps), 0, s, a, parts);
  prof_mark(K_CONV_WGRAD, s, false);
  return e;
}

// BATCH: tokens of a forward batch, 0 for the backward.
template <class T, int V, int BATCH>
cudaError_t pick(const ConvArgs& a, cudaStream_t s) {
  auto go = [&](auto k, auto act) {
    if constexpr (BATCH == 0) return bwd<T, V, decltype(k)::value, decltype(act)::value>(a, s);
    else return fwd<T, V, decltype(k)::value, decltype(act)::value, BATCH>(a, s);
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
  if (a.max_q <= FEW) {
    if (a.bf16) return wide ? pick<bf16, 8, 1>(a, s) : pick<bf16, 1, 1>(a, s);
    return wide ? pick<float, 4, 1>(a, s) : pick<float, 1, 1>(a, s);
  }
  if (a.bf16) return wide ? pick<bf16, 4, 16>(a, s) : pick<bf16, 1, 16>(a, s);
  return wide ? pick<float, 4, 8>(a, s) : pick<float, 1, 16>(a, s);
}
cudaError_t launch_causal_conv_bwd(const ConvArgs& a, bool wide, cudaStream_t s) {
  if (a.bf16) return wide ? pick<bf16, 4, 0>(a, s) : pick<bf16, 1, 0>(a, s);
  return wide ? pick<float, 4, 0>(a, s) : pick<float, 1, 0>(a, s);
}
size_t causal_conv_workspace(const ConvArgs& a0) {
  ConvArgs a = a0;
  size_t most = 0;
  for (int V : {1, 4}) {  // whichever width the call's pointers and strides allow
    if (a.C % V) continue;
    int parts;
    long long numbers;
    bwd_plan(&a, a.C / V, &parts, &numbers);
    const size_t n = (size_t)parts * (a.taps + 1) * a.C * sizeof(float);
    most = n > most ? n : most;
  }
  return most;
}

}  // namespace gdn
