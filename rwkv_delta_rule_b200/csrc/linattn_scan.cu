// linattn_scan.cu -- linear attention with one decay per head, token by token with the float32 state
// in registers:  S <- w S + v k^T,  y = S q,  and the same walked from the last token for gradients.
//
// One CTA of 128 threads holds a (b, h) pair's 64 x 64 state: thread (rs, q) has rows 4 rs .. 4 rs + 3
// and columns 4 q .. 4 q + 3, 32 + 4 q .. 32 + 4 q + 3, in pairs (packed operations are the scalar ones, two at a
// time).  The chain through the state is one multiply-add per token, so the walk is bound by its 48 packed
// operations, 5 shared-memory loads and the row sums per thread and token.  These sums meet in a 4-shuffle
// reduce-scatter over the 8 lanes of a row group.  Operands are staged by cp.async in double-buffered tiles.
// Measured on B200: float32 B1 T1000 H12 28 us (states, join and outputs in three launches, 42
// segments of 24 tokens); B8 T4096 H12 418, B4 T8192 H64 1999.  B8 T4096 H12 took 558 with tiles twice as long and 4
// CTAs per SM, 603 with scalar operations.
#include "linattn.h"
#include "packed.cuh"

namespace rwkv7 {
namespace lin {

constexpr int kThreads = 128;
template <typename TIn> struct Tile {
  static constexpr int kTok = sizeof(TIn) == 2 ? 16 : 8;     // tokens per tile
  static constexpr int kEPC = 16 / static_cast<int>(sizeof(TIn));
  static constexpr int kElems = kTok * 3 * kN;                // q, k, v
  static constexpr size_t kSmem = 2 * kElems * sizeof(TIn) + kTok * kN * sizeof(float);
};

template <int n> struct Count {
  static constexpr int value = n;
};

template <typename TIn> __device__ __forceinline__ void load_pairs(const TIn *p, f32x2 *x) {
  float f[4];
  Elem<TIn>::load4(p, f);
  x[0] = make2(f[0], f[1]);
  x[1] = make2(f[2], f[3]);
}

template <typename TIn, bool kOut>
__device__ __forceinline__ void stage(const Pass<TIn> &A, TIn *buf, long long tok0, int ntok, int H, int h) {
  using C = Tile<TIn>;
  constexpr int kPer = kN / C::kEPC;  // 16-byte pieces of a vector
  for (int c = threadIdx.x; c < ntok * 3 * kPer; c += kThreads) {
    const int tt = c / (3 * kPer), rem = c - tt * (3 * kPer), vid = rem / kPer, part = rem - vid * kPer;
    if (!kOut && vid == 0) continue;
    const TIn *src = vid == 0 ? A.q : vid == 1 ? A.k : A.v;
    cp_async16(buf + (tt * 3 + vid) * kN + part * C::kEPC, src + ((tok0 + tt) * H + h) * kN + part * C::kEPC);
  }
}

// Reversed walks are bf16 (gradients), passes for the states alone float32: bf16 sequences that come here are too short
// to be split.
template <typename TIn, bool kRev, bool kOut>
__device__ __forceinline__ void scan_segment(const Pass<TIn> &A, const Shape &P, int b, int z, uint8_t *smem_raw) {
  static_assert(sizeof(TIn) == 2 ? kOut : !kRev, "no call asks for it");
  using C = Tile<TIn>;
  TIn *bufs = reinterpret_cast<TIn *>(smem_raw);
  float *ys = reinterpret_cast<float *>(smem_raw + 2 * C::kElems * sizeof(TIn));
  const int h = blockIdx.x;
  const Segment sg = segment(P, b, z);
  if (sg.len < 0) return;
  if (!kOut && sg.last) return;
  const long long pair = static_cast<long long>(b) * P.H + h;
  const int tid = threadIdx.x, q = tid & 7, row0 = 4 * (tid >> 3);
  const float w = P.w[h];
  const f32x2 w2 = make2(w, w);
  // states alone: powers, for 4 tokens at once, and what the rounding of w^4 takes from the state with each four, as a
  // part of it
  float wp[5] = {1.f, w, 0.f, 0.f, 0.f}, lost = 0.f;
  if (!kOut) {
    const double wd = w;
    wp[2] = static_cast<float>(wd * wd);
    wp[3] = static_cast<float>(wd * wd * wd);
    const Power p4 = power(wd, 4);
    wp[4] = p4.hi;
    lost = p4.hi > 1e-30f ? p4.lo / p4.hi : 0.f;
  }

  f32x2 s[4][4];  // columns in pairs
  const float *from = !kOut ? nullptr : P.nseg > 1 ? A.ws + (pair * P.nseg + z) * (kN * kN) : A.s_in + pair * (kN * kN);
  const int from_t = P.nseg == 1 && A.s_in_t;
  if (P.nseg == 1 && A.s_in == nullptr) from = nullptr;
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int col = (e >> 1) * 32 + 4 * q + 2 * (e & 1);
      s[m][e] = from == nullptr ? make2(0.f, 0.f)
                                : make2(from[state_at(from_t, row0 + m, col)], from[state_at(from_t, row0 + m, col + 1)]);
    }

  const int ntiles = (sg.len + C::kTok - 1) / C::kTok;
  auto tile_tok = [&](int i) { return (kRev ? ntiles - 1 - i : i) * C::kTok; };
  if (ntiles > 0) {
    const int t0 = tile_tok(0);
    stage<TIn, kOut>(A, bufs, sg.lo + t0, min(C::kTok, sg.len - t0), P.H, h);
    cp_async_commit();
  }
  for (int i = 0; i < ntiles; ++i) {
    const int t0 = tile_tok(i), ntok = min(C::kTok, sg.len - t0);
    if (i + 1 < ntiles) {
      const int t1 = tile_tok(i + 1);
      stage<TIn, kOut>(A, bufs + ((i + 1) & 1) * C::kElems, sg.lo + t1, min(C::kTok, sg.len - t1), P.H, h);
      cp_async_commit();
      cp_async_wait<1>();
    } else {
      cp_async_wait<0>();
    }
    __syncthreads();
    const TIn *buf = bufs + (i & 1) * C::kElems;
    // kG tokens at a time: their operands are loaded before, and their row sums meet after the walk through
    // the state, so that neither's latency is paid per token
    auto group = [&](int u0, auto count) {
      constexpr int kG = decltype(count)::value;
      f32x2 kk[kG][4], vv[kG][4], qq[kOut ? kG : 1][4];
#pragma unroll
      for (int j = 0; j < kG; ++j) {
        const TIn *tk = buf + (kRev ? ntok - 1 - u0 - j : u0 + j) * 3 * kN;
        load_pairs(tk + kN + 4 * q, kk[j]);
        load_pairs(tk + kN + 32 + 4 * q, kk[j] + 2);
        float v[4];
        Elem<TIn>::load4(tk + 2 * kN + row0, v);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          // states alone: all that decays by the group's end is scaled here
          if (!kOut) v[m] *= wp[kG - 1 - j];
          vv[j][m] = make2(v[m], v[m]);
        }
        if (kOut) {
          load_pairs(tk + 4 * q, qq[j]);
          load_pairs(tk + 32 + 4 * q, qq[j] + 2);
        }
      }
      if constexpr (!kOut) {
        const f32x2 f = make2(wp[kG], wp[kG]);
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[m][e] = mul2(s[m][e], f);
#pragma unroll
            for (int j = 0; j < kG; ++j) s[m][e] = fma2(vv[j][m], kk[j][e], s[m][e]);
          }
      } else {
        float p[kG][4];
#pragma unroll
        for (int j = 0; j < kG; ++j) {
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              s[m][e] = kRev ? fma2(vv[j][m], kk[j][e], s[m][e]) : fma2(s[m][e], w2, mul2(vv[j][m], kk[j][e]));
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            f32x2 t = mul2(s[m][0], qq[j][0]);
#pragma unroll
            for (int e = 1; e < 4; ++e) t = fma2(s[m][e], qq[j][e], t);
            float x, y;
            split2(t, x, y);
            p[j][m] = x + y;
          }
          if (kRev) {
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[m][e] = mul2(s[m][e], w2);
          }
        }
        const bool h4 = (q & 4) != 0, h2 = (q & 2) != 0;
        float y[kG];
#pragma unroll
        for (int j = 0; j < kG; ++j) {
          const float a0 = (h4 ? p[j][2] : p[j][0]) + __shfl_xor_sync(0xffffffffu, h4 ? p[j][0] : p[j][2], 4);
          const float a1 = (h4 ? p[j][3] : p[j][1]) + __shfl_xor_sync(0xffffffffu, h4 ? p[j][1] : p[j][3], 4);
          y[j] = (h2 ? a1 : a0) + __shfl_xor_sync(0xffffffffu, h2 ? a0 : a1, 2);
        }
#pragma unroll
        for (int j = 0; j < kG; ++j) {
          y[j] += __shfl_xor_sync(0xffffffffu, y[j], 1);
          if ((q & 1) == 0)
            ys[(kRev ? ntok - 1 - u0 - j : u0 + j) * kN + row0 + (h4 ? 2 : 0) + (h2 ? 1 : 0)] = y[j];
        }
      }
    };
    int u = 0;
    for (; u + 4 <= ntok; u += 4) group(u, Count<4>());
    if (!kOut) {
      // (its own tokens get up to a rounding too much of it, once)
      const float l = lost * static_cast<float>(u >> 2);
      const f32x2 l2 = make2(l, l);
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[m][e] = fma2(s[m][e], l2, s[m][e]);
    }
    for (; u < ntok; ++u) group(u, Count<1>());
    __syncthreads();
    if (kOut) {
      for (int e = 4 * tid; e < ntok * kN; e += 4 * kThreads) {
        const float4 f = *reinterpret_cast<const float4 *>(ys + e);
        TIn *out = A.out + ((sg.lo + t0 + (e >> 6)) * P.H + h) * kN + (e & 63);
        if constexpr (sizeof(TIn) == 4)
          *reinterpret_cast<float4 *>(out) = f;
        else
          *reinterpret_cast<uint2 *>(out) = make_uint2(pack2(make2(f.x, f.y)), pack2(make2(f.z, f.w)));
      }
      // the next tile writes ys only behind the barrier after its loads
    }
  }

  const bool ends = kRev ? sg.first : sg.last;
  float *to = !kOut ? A.ws + (pair * P.nseg + z + 1) * (kN * kN) : A.s_out + pair * (kN * kN);
  if (!kOut || (ends && A.s_out != nullptr)) {
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int col = (e >> 1) * 32 + 4 * q + 2 * (e & 1), t = kOut && A.s_out_t;
        split2(s[m][e], to[state_at(t, row0 + m, col)], to[state_at(t, row0 + m, col + 1)]);
      }
  }
}

// blockIdx = (head, batch row, pass and segment); the passes for the states alone leave out the segment
// that none continues from.
template <typename TIn, bool kOut>
__global__ void __launch_bounds__(kThreads, 7) linattn_scan_kernel(const __grid_constant__ Passes<TIn> A, const Shape P) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ int lens[kMaxSorted + 1];
  pdl_wait();
  pdl_trigger();
  const int b = sorted_row(P, blockIdx.y, gridDim.y, lens);
  if constexpr (sizeof(TIn) == 4) {
    scan_segment<TIn, false, kOut>(A.p[0], P, b, blockIdx.z, smem_raw);
  } else {
    const int role = blockIdx.z / P.nseg, z = blockIdx.z - role * P.nseg;
    if (A.p[role].reverse)
      scan_segment<TIn, true, kOut>(A.p[role], P, b, z, smem_raw);
    else
      scan_segment<TIn, false, kOut>(A.p[role], P, b, z, smem_raw);
  }
}

// One thread per 4 columns of a state row, along the segments.
template <typename TIn> __global__ void __launch_bounds__(256) linattn_join_kernel(const __grid_constant__ Passes<TIn> passes,
                                                                                    const Shape P) {
  const int h = blockIdx.x, b = blockIdx.y;
  const Pass<TIn> &A = passes.p[blockIdx.z >> 2];
  pdl_wait();
  pdl_trigger();
  const SeqBounds sb = seq_bounds(P.cu_seqlens, b, P.T, P.total_T);
  if (sb.len < 0) return;
  const Segment sg = segment(P, b, 0);
  const int n = sg.n;
  const long long pair = static_cast<long long>(b) * P.H + h;
  const int e4 = (blockIdx.z & 3) * 256 + threadIdx.x, row = e4 >> 4, col = 4 * (e4 & 15);
  const double w = P.w[h];
  const Power wl = power(w, P.seg_len);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (A.s_in != nullptr) {
    const float *f = A.s_in + pair * (kN * kN);
    s = make_float4(f[state_at(A.s_in_t, row, col)], f[state_at(A.s_in_t, row, col + 1)],
                    f[state_at(A.s_in_t, row, col + 2)], f[state_at(A.s_in_t, row, col + 3)]);
  }
  float *ws = A.ws + pair * P.nseg * (kN * kN) + row * kN + col;
  auto slot = [&](int i) {
    return reinterpret_cast<float4 *>(ws + static_cast<long long>(A.reverse ? n - 1 - i : i) * (kN * kN));
  };
  *slot(0) = s;
  // the slots in order, 8 loads at a time
  for (int i0 = 1; i0 < n; i0 += 8) {
    float4 u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i0 + j < n) u[j] = *slot(i0 + j);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i0 + j < n) {
        // the decay over the segment before; the sequence's last one may be of another length
        const Power f = A.reverse && i0 + j == 1 ? power(w, sg.last_len) : wl;
        s = make_float4(fmaf(s.x, f.hi, fmaf(s.x, f.lo, u[j].x)), fmaf(s.y, f.hi, fmaf(s.y, f.lo, u[j].y)),
                        fmaf(s.z, f.hi, fmaf(s.z, f.lo, u[j].z)), fmaf(s.w, f.hi, fmaf(s.w, f.lo, u[j].w)));
        *slot(i0 + j) = s;
      }
  }
}

}  // namespace lin

template <typename TIn>
cudaError_t launch_linattn_scan(const lin::Passes<TIn> &A, const lin::Shape &P, int B, cudaStream_t stream) {
  using namespace lin;
  const int nz = A.state_only ? P.nseg - 1 : P.nseg;
  if (nz <= 0) return cudaSuccess;
  const dim3 grid(P.H, B, nz * A.n);
  if constexpr (sizeof(TIn) == 4) {
    if (A.state_only)
      return launch_waiting(linattn_scan_kernel<TIn, false>, grid, kThreads, Tile<TIn>::kSmem, stream, A, P);
  }
  return launch_waiting(linattn_scan_kernel<TIn, true>, grid, kThreads, Tile<TIn>::kSmem, stream, A, P);
}

template <typename TIn>
cudaError_t launch_linattn_join(const lin::Passes<TIn> &A, const lin::Shape &P, int B, cudaStream_t stream) {
  return lin::launch_waiting(lin::linattn_join_kernel<TIn>, dim3(P.H, B, 4 * A.n), 256, 0, stream, A, P);
}

template cudaError_t launch_linattn_scan<float>(const lin::Passes<float> &, const lin::Shape &, int, cudaStream_t);
template cudaError_t launch_linattn_scan<uint16_t>(const lin::Passes<uint16_t> &, const lin::Shape &, int, cudaStream_t);
template cudaError_t launch_linattn_join<float>(const lin::Passes<float> &, const lin::Shape &, int, cudaStream_t);
template cudaError_t launch_linattn_join<uint16_t>(const lin::Passes<uint16_t> &, const lin::Shape &, int, cudaStream_t);

}  // namespace rwkv7
