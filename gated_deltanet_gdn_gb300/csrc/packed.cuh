// Packed sequences: B sequences' tokens in the rows of [N, ...] tensors, sequence b in rows
// cu[b] .. cu[b+1] - 1 (or b T .. b T + T - 1 without cu), and the rows of a pool that hold
// their states.
//
// Kernels cut every sequence into chunks of L tokens of its own, and the chunks of all
// sequences are numbered without a prefix sum: sequence b's chunk j has number
// floor(cu[b] / L) + b + j. Its first number never reaches the one before's last, since
// floor(e / L) + 1 >= floor(s / L) + ceil((e - s) / L); so floor(N / L) + B + 1 numbers hold
// every chunk. Some numbers stay unused, those below floor(cu[0] / L) and from the last sequence's end on among them.
// (Without cu a sequence's chunks are numbered one after the other, none unused.)
#pragma once

#include "kernels.h"

namespace gdn {

constexpr int PACKED_WHOLE = 0x40000000;  // chunk length where sequences are not cut

// Chunks of a sequence of T tokens; one, without tokens, where T is 0.
__host__ __device__ __forceinline__ int packed_per(int T, int L) { return T > L ? (T - 1) / L + 1 : 1; }

struct Chunk {
  int b;       // sequence
  int first;   // row of the sequence's first token
  int len;     // its tokens
  int j;       // chunk of the sequence
};

// Bounds of sequence b, within [0, N] whatever the array holds.
__device__ __forceinline__ int packed_start(const PackedArgs& q, int b) {
  if (!q.cu) return b * q.T;
  const int s = q.cu[b];
  return s < 0 ? 0 : s > q.N ? q.N : s;
}
__device__ __forceinline__ void packed_bounds(const PackedArgs& q, int b, int* first, int* len) {
  *first = packed_start(q, b);
  if (b == q.B) {
    *len = q.N - *first;
  } else if (!q.cu) {
    *len = q.T;
  } else {
    const int n = packed_start(q, b + 1) - *first;
    *len = n < 0 ? 0 : n;
  }
}
// Number of sequence b's first chunk.
__device__ __forceinline__ long long packed_number(const PackedArgs& q, int b, int first, int L) {
  return q.cu ? (long long)(first / L) + b : (long long)b * packed_per(q.T, L);
}
// The chunk with this number; false for an unused one. A sequence without tokens has one empty
// chunk, in which its state is handed on.
__device__ __forceinline__ bool packed_chunk(const PackedArgs& q, long long number, int L, Chunk* c) {
  if (!q.cu) {
    const int per = packed_per(q.T, L);
    c->b = (int)(number / per);
    c->j = (int)(number % per);
    c->first = c->b * q.T;
    c->len = q.T;
    return c->b < q.B;
  }
  int lo = 0, hi = q.B + 1;  // the last b with number(b) <= number; number(0) is 0
  if (L > q.N) {  // a chunk for every sequence: nothing to search
    lo = (int)number;
    hi = 0;
  }
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (packed_start(q, mid) / L + mid <= number) lo = mid;
    else hi = mid;
  }
  c->b = lo;
  packed_bounds(q, lo, &c->first, &c->len);
  c->j = (int)(number - (c->first / L + lo));
  if (c->j < 0 || lo == q.B) return false;  // below the first sequence's first number, or behind the last one's
  return (long long)c->j * L < c->len || c->j == 0;
}
// The rows before the first sequence and behind the last belong to none. Where they are to become zeros, a grid has CTAs for
// them behind its own: one for every PAD_VECS vectors a thread that there can be, up to sixteen warps an SM. (By the CTAs of
// the sequences themselves, after their work: other registers and spills in most of the kernels. As chunks like a sequence's,
// which were rows one after the other for a single token's step: 1 token in 8,192 rows x 6,144 channels took 256 us,
// now 16; 4 in its own row.)
constexpr int PAD_VECS = 8;
inline unsigned packed_pad_ctas(const PackedArgs& q, bool wanted, int vecs, int threads) {
  if (!q.cu || !wanted) return 0;
  const long long n = ((long long)q.N * vecs + PAD_VECS * threads - 1) / (PAD_VECS * threads), most = 152 * 512 / threads;
  return (unsigned)(n < most ? n : most);
}
// body(row, vector) of these rows, each of so many vectors; from: the first of the CTAs.
template <int THREADS, class F>
__device__ __forceinline__ void packed_padding(const PackedArgs& q, unsigned from, int vecs, F body) {
  const int front = packed_start(q, 0), end = packed_start(q, q.B);
  const int wide = vecs < THREADS ? vecs : THREADS, each = THREADS / wide, mine = threadIdx.x / wide, v0 = threadIdx.x % wide;
  if (mine >= each) return;
  const long long rows = (long long)front + q.N - end, step = (long long)(gridDim.x - from) * each;
#pragma unroll 1
  for (long long r = (long long)(blockIdx.x - from) * each + mine; r < rows; r += step)
#pragma unroll 1
    for (int v = v0; v < vecs; v += wide) body(r < front ? r : end + r - front, v);
}
// Row of the pool with sequence b's state, -1 for none.
__device__ __forceinline__ int packed_slot(const PackedArgs& q, int b) {
  if (!q.slots) return b;
  const int s = q.slots[b];
  if (s >= q.pool) {
    if (q.err) atomicOr(q.err, ERR_SLOT);
    return -1;
  }
  return s < 0 ? -1 : s;
}
// Whether sequence b of len new tokens goes on from a state (else it starts from zeros).
__device__ __forceinline__ bool packed_goes_on(const PackedArgs& q, int b, int len) {
  return !q.lens || q.lens[b] > len;
}
__host__ __device__ __forceinline__ long long packed_numbers(const PackedArgs& q, int L) {
  return q.cu ? (long long)(q.N / L) + q.B + 1 : (long long)q.B * packed_per(q.T, L);
}

}  // namespace gdn
