// linattn.h -- what the kernels of the head-decay linear attention share: arguments, segments of a
// sequence, powers of a decay.  Internal, not exported.
#pragma once

#include "common.cuh"

namespace rwkv7 {
namespace lin {

// One pass of the recurrence over [B, T, H, 64] (or packed ragged) operands, for every (b, h):
//   forward  S <- w S + v k^T;  out = S q          reverse (tokens from the last)  S <- S + v k^T;  out = S q;  S <- w S
// Rows of S are the channels of v, columns those of k.
template <typename TIn> struct Pass {
  const TIn *q, *k, *v;
  TIn *out;
  const float *s_in;     // [B, H, 64, 64] or nullptr (zero)
  float *s_out;          // [B, H, 64, 64] or nullptr
  int s_in_t, s_out_t;   // the state is stored transposed there
  float *ws;             // nseg > 1: [B, H, nseg, 64, 64], slot z is the state that segment z begins with
                         // (joined), or what the segment before it adds to the state
  int reverse;
  int terms;             // on the tensor cores, bf16 terms of v that the state is summed from: 2, or 3 where it is an output
};
// Passes over operands of one shape that run side by side (the backward has three).
template <typename TIn> struct Passes {
  Pass<TIn> p[3];
  int n;
  int state_only;  // no outputs: what each segment adds to the state, for the segment after it (q, out unused)
};

struct Shape {
  const float *w;  // [H]
  const int32_t *cu_seqlens;  // nullptr: fixed length T
  int T;
  long long total_T;
  int H;
  int nseg;     // segments per sequence (1: the whole sequence)
  int joined;   // nseg > 1: the slots of ws hold the states that segments begin with, not yet what they add
  int seg_len;  // tokens per segment (on the tensor cores whole chunks); the last segment runs to the sequence's end
};

// Tokens lo .. lo + len - 1 of the packed operands; `first` / `last`: this segment begins / ends the
// sequence, which has n segments, the last one of last_len tokens.  len = -1: nothing to do.
struct Segment {
  long long lo;
  int len;
  bool first, last;
  int n, last_len;
};
__device__ __forceinline__ Segment segment(const Shape &P, int b, int z) {
  const SeqBounds sb = seq_bounds(P.cu_seqlens, b, P.T, P.total_T);
  Segment s{0, -1, z == 0, false, 0, 0};
  if (sb.len < 0) return s;
  const long long off = static_cast<long long>(z) * P.seg_len;
  const int segs = sb.len <= P.seg_len ? 1 : (sb.len - 1) / P.seg_len + 1;
  s.n = segs < P.nseg ? segs : P.nseg;
  s.last_len = sb.len - (s.n - 1) * P.seg_len;  // below 2^31: the segments before are within the sequence
  if (z > 0 && off >= sb.len) return s;
  const long long left = sb.len - off;
  s.lo = sb.start + off;
  s.last = z == P.nseg - 1 || left <= P.seg_len;
  s.len = static_cast<int>(s.last ? left : P.seg_len);
  return s;
}

// w^n in float64 by squaring (w^0 = 1 for every w, zero included); one rounding per product, so far
// below float32's step for every n here.
__device__ __forceinline__ double powi(double w, long long n) {
  double r = 1.0, p = w;
  for (; n > 0; n >>= 1) {
    if (n & 1) r *= p;
    p *= p;
  }
  return r;
}

// w^n in two float32 terms.  A state that is scaled by the same power again and again would be off by its
// rounding as often, all in one direction (float32 B4 T8192 H64, 1024 steps of w^4: 1e-5, and 1e-6 with the second
// term).
struct Power {
  float hi, lo;
};
__device__ __forceinline__ Power power(double w, long long n) {
  const double p = powi(w, n);
  const float hi = static_cast<float>(p);
  return {hi, static_cast<float>(p - static_cast<double>(hi))};
}

// element (row, col) of a state as it is stored
__device__ __forceinline__ int state_at(int transposed, int row, int col) {
  return transposed ? col * kN + row : row * kN + col;
}

// Launches a kernel that waits (pdl_wait) before it touches memory: its CTAs may be placed while the grid
// before it on the stream drains.
template <typename... KArgs, typename... Args>
cudaError_t launch_waiting(void (*kernel)(KArgs...), dim3 grid, unsigned block, size_t smem, cudaStream_t stream,
                           const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// The batch row of a CTA: rows of a ragged batch are taken from the longest to the shortest (up to kMaxSorted
// rows; equal ones in order), so that none is left to the end: 16 rows of up to 2500 tokens, H32, 95 us against
// 112 in their own order.  `lens`: kMaxSorted + 1 ints of shared memory.  Called by a whole CTA.
constexpr int kMaxSorted = 256;
__device__ __forceinline__ int sorted_row(const Shape &P, int b, int B, int *lens) {
  if (P.cu_seqlens == nullptr || B > kMaxSorted) return b;
  for (int i = threadIdx.x; i < B; i += blockDim.x) lens[i] = seq_bounds(P.cu_seqlens, i, P.T, P.total_T).len;
  __syncthreads();
  for (int i = threadIdx.x; i < B; i += blockDim.x) {
    int before = 0;
    const int len = lens[i];
#pragma unroll 8
    for (int j = 0; j < B; ++j) before += lens[j] > len || (lens[j] == len && j < i);
    if (before == b) lens[kMaxSorted] = i;
  }
  __syncthreads();
  return lens[kMaxSorted];
}

}  // namespace lin

// Launchers of the passes; TIn: float or uint16_t (bfloat16 bits).
template <typename TIn>
cudaError_t launch_linattn_scan(const lin::Passes<TIn> &passes, const lin::Shape &shape, int B, cudaStream_t stream);
// Passes with state_only leave what each segment adds to the state in the slot of the segment
// after it.  This turns the slots into the states that the segments begin with; the segments read
// only those, so s_in may be s_out.
template <typename TIn>
cudaError_t launch_linattn_join(const lin::Passes<TIn> &passes, const lin::Shape &shape, int B, cudaStream_t stream);
// The same on the tensor cores (linattn_chunk.cu); total_T > 0.  err_word: where its bounded waits report.
cudaError_t launch_linattn_chunk(const lin::Passes<uint16_t> &passes, const lin::Shape &shape, int B, int *err_word,
                                 cudaStream_t stream);
template <typename TIn>
cudaError_t launch_linattn_decode(const TIn *r, const TIn *k, const TIn *v, const float *w, float *s, TIn *y, int B,
                                  int H, cudaStream_t stream);

}  // namespace rwkv7
