// layer_norm.cu -- layer norm over groups of D channels, forward and backward, with the reduction of
// the weight's and bias's gradients over the rows.
//
//   mean, var (divisor D) over x[m, g, :],  rstd = 1 / sqrt(var + eps),  xh = (x - mean) rstd
//   y  = xh w + b
//   g  = dy w,   dx = rstd (g - mean_D(g) - xh mean_D(g xh)),   dw = sum_m dy xh,   db = sum_m dy
//
// G = 1 is the norm of a token (ln1 / ln2 of a block), D = 64 with G = heads the ln_x of the time mix.
//
// Everything is bound by HBM: two tensors forward, three backward, so each element is loaded once, in
// 16-byte pieces where the rows allow it, and kept in registers between the sums and the result (the
// variance is that of the centred values, which costs no second load).  A "unit" is a set of lanes
// that owns one (m, g) vector: 1 to 32 lanes of a warp while it fits there (4 pieces a lane), else a
// whole CTA.  A unit keeps its group g and steps over the rows m, so it also keeps its columns' sums
// for dw and db in registers; CTAs then leave one partial sum each, and a second launch adds those up
// in a fixed order.  Vectors too long for a CTA's registers are walked in loops instead.
#include "layer_norm.h"

#include "common.cuh"

namespace rwkv7 {
namespace ln {

constexpr int kSMs = 148;

// V consecutive elements of T as they lie in memory, and as floats
template <typename T, int V> struct Piece;
template <> struct Piece<float, 4> {
  float4 u;
  __device__ __forceinline__ void load(const float *p) { u = *reinterpret_cast<const float4 *>(p); }
  __device__ __forceinline__ void zero() { u = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&o)[4]) const { o[0] = u.x; o[1] = u.y; o[2] = u.z; o[3] = u.w; }
  static __device__ __forceinline__ void store(float *p, const float (&o)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(o[0], o[1], o[2], o[3]);
  }
};
template <> struct Piece<float, 1> {
  float u;
  __device__ __forceinline__ void load(const float *p) { u = *p; }
  __device__ __forceinline__ void zero() { u = 0.f; }
  __device__ __forceinline__ void get(float (&o)[1]) const { o[0] = u; }
  static __device__ __forceinline__ void store(float *p, const float (&o)[1]) { *p = o[0]; }
};
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return static_cast<uint32_t>(float_to_bf16_bits(lo)) | (static_cast<uint32_t>(float_to_bf16_bits(hi)) << 16);
}
template <> struct Piece<uint16_t, 8> {
  uint4 u;
  __device__ __forceinline__ void load(const uint16_t *p) { u = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&o)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __uint_as_float(w[i] << 16);
      o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(uint16_t *p, const float (&o)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack2(o[0], o[1]), pack2(o[2], o[3]), pack2(o[4], o[5]), pack2(o[6], o[7]));
  }
};
template <> struct Piece<uint16_t, 2> {
  uint32_t u;
  __device__ __forceinline__ void load(const uint16_t *p) { u = *reinterpret_cast<const uint32_t *>(p); }
  __device__ __forceinline__ void zero() { u = 0u; }
  __device__ __forceinline__ void get(float (&o)[2]) const {
    o[0] = __uint_as_float(u << 16);
    o[1] = __uint_as_float(u & 0xffff0000u);
  }
  static __device__ __forceinline__ void store(uint16_t *p, const float (&o)[2]) {
    *reinterpret_cast<uint32_t *>(p) = pack2(o[0], o[1]);
  }
};
template <> struct Piece<uint16_t, 1> {
  uint16_t u;
  __device__ __forceinline__ void load(const uint16_t *p) { u = *p; }
  __device__ __forceinline__ void zero() { u = 0; }
  __device__ __forceinline__ void get(float (&o)[1]) const { o[0] = bf16_bits_to_float(u); }
  static __device__ __forceinline__ void store(uint16_t *p, const float (&o)[1]) { *p = float_to_bf16_bits(o[0]); }
};

template <typename T> struct Args {
  const T *x, *dy;
  const float *w, *b;
  float eps;
  T *out;  // y, or dx
  float *mean, *rstd;
  float *partial;  // [CTA rows][2][G, D], or nullptr
  int M, G, D;
  // lanes per unit (block units: the CTA); groups a CTA covers, units per group in it, CTAs that cover all groups
  int lanes, gper, slots, gblocks;
};

// V float32 parameters from w + c (ones or zeros where there is none); w is only 4-byte aligned for odd D
template <int V> __device__ __forceinline__ void params(const float *w, long long c, float missing, float (&o)[V]) {
  if (w == nullptr) {
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = missing;
  } else if constexpr (V % 4 == 0) {
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      const float4 u = *reinterpret_cast<const float4 *>(w + c + e);
      o[e] = u.x; o[e + 1] = u.y; o[e + 2] = u.z; o[e + 3] = u.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = w[c + e];
  }
}

// Sums over a unit's lanes.  Block units: the warps' sums meet in red (2 x 32 floats per call site
// parity), with one barrier per call; a call's slots are rewritten two calls later at the earliest.
template <bool kBlock> __device__ __forceinline__ float2 unit_sum(float2 v, int lanes, float2 *red, int &turn) {
  const int top = kBlock ? 16 : lanes >> 1;
  for (int off = top; off >= 1; off >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, off);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, off);
  }
  if (kBlock) {
    float2 *slot = red + 32 * turn;
    turn ^= 1;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
    __syncthreads();
    float2 t = (threadIdx.x & 31) < warps ? slot[threadIdx.x & 31] : make_float2(0.f, 0.f);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
      t.x += __shfl_xor_sync(0xffffffffu, t.x, off);
      t.y += __shfl_xor_sync(0xffffffffu, t.y, off);
    }
    v = t;
  }
  return v;
}

// Where a thread stands: its unit's group, the row it begins with, the step between its rows.
struct Place {
  int lane, unit, g;
  long long m, step;
  bool active;
};
template <bool kBlock, typename T> __device__ __forceinline__ Place place(const Args<T> &A) {
  Place p;
  p.lane = kBlock ? threadIdx.x : threadIdx.x & (A.lanes - 1);
  p.unit = kBlock ? 0 : threadIdx.x / A.lanes;
  const int gb = blockIdx.x % A.gblocks, mb = blockIdx.x / A.gblocks, mblocks = gridDim.x / A.gblocks;
  p.g = gb * A.gper + p.unit % A.gper;
  const int slot = p.unit / A.gper;
  p.m = static_cast<long long>(mb) * A.slots + slot;
  p.step = static_cast<long long>(mblocks) * A.slots;
  p.active = slot < A.slots && p.g < A.G;
  return p;
}

template <typename T, int V, int NV, bool kBlock>
__global__ void __launch_bounds__(kBlock ? 1024 : 256) layer_norm_kernel(const Args<T> A) {
  __shared__ float2 red[64];
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const Place p = place<kBlock>(A);
  const float inv = 1.f / static_cast<float>(A.D);
  // every lane of a warp takes the same number of turns (the sums are over whole warps)
  const long long rows = (A.M + p.step - 1) / p.step;
  for (long long i = 0; i < rows; ++i) {
    const long long m = p.m + i * p.step;
    const bool on = p.active && m < A.M;
    const long long base = (m * A.G + p.g) * A.D;
    Piece<T, V> u[NV];
    float x[NV][V];
    float s = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c = (n * A.lanes + p.lane) * V;
      if (on && c < A.D) u[n].load(A.x + base + c); else u[n].zero();
    }
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      u[n].get(x[n]);
#pragma unroll
      for (int e = 0; e < V; ++e) s += x[n][e];
    }
    const float mean = unit_sum<kBlock>(make_float2(s, 0.f), A.lanes, red, turn).x * inv;
    float q = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c = (n * A.lanes + p.lane) * V;
      if (c < A.D) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          x[n][e] -= mean;
          q = fmaf(x[n][e], x[n][e], q);
        }
      }
    }
    const float var = unit_sum<kBlock>(make_float2(q, 0.f), A.lanes, red, turn).x * inv;
    const float rstd = 1.f / sqrtf(var + A.eps);
    if (!on) continue;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c = (n * A.lanes + p.lane) * V;
      if (c < A.D) {
        float w[V], b[V];
        const long long pc = static_cast<long long>(p.g) * A.D + c;
        params<V>(A.w, pc, 1.f, w);
        params<V>(A.b, pc, 0.f, b);
#pragma unroll
        for (int e = 0; e < V; ++e) x[n][e] = fmaf(x[n][e] * rstd, w[e], b[e]);
        Piece<T, V>::store(A.out + base + c, x[n]);
      }
    }
    if (p.lane == 0) {
      if (A.mean != nullptr) A.mean[m * A.G + p.g] = mean;
      if (A.rstd != nullptr) A.rstd[m * A.G + p.g] = rstd;
    }
  }
}

// threads of a CTA unit in the backward: 3 float32 values per element are kept
constexpr int backward_threads(int v, int nv) { return v * nv > 8 ? 512 : 1024; }

template <typename T, int V, int NV, bool kBlock>
__global__ void __launch_bounds__(kBlock ? backward_threads(V, NV) : 256) layer_norm_backward_kernel(const Args<T> A) {
  __shared__ float2 red[64];
  extern __shared__ float sums[];  // units of a warp only: [2][slots][gper * lanes * NV * V]
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const Place p = place<kBlock>(A);
  const float inv = 1.f / static_cast<float>(A.D);
  float w[NV][V], aw[NV][V], ab[NV][V];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int c = (n * A.lanes + p.lane) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) w[n][e] = aw[n][e] = ab[n][e] = 0.f;
    if (p.active && c < A.D) params<V>(A.w, static_cast<long long>(p.g) * A.D + c, 1.f, w[n]);
  }
  const long long rows = (A.M + p.step - 1) / p.step;
  for (long long i = 0; i < rows; ++i) {
    const long long m = p.m + i * p.step;
    const bool on = p.active && m < A.M;
    const long long base = (m * A.G + p.g) * A.D;
    Piece<T, V> ux[NV], ud[NV];
    const float mean = on ? A.mean[m * A.G + p.g] : 0.f, rstd = on ? A.rstd[m * A.G + p.g] : 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c = (n * A.lanes + p.lane) * V;
      if (on && c < A.D) {
        ux[n].load(A.x + base + c);
        ud[n].load(A.dy + base + c);
      } else {
        ux[n].zero();
        ud[n].zero();
      }
    }
    float2 s = make_float2(0.f, 0.f);  // sums of g and g xh
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      float x[V], d[V];
      ux[n].get(x);
      ud[n].get(d);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float xh = (x[e] - mean) * rstd, g = d[e] * w[n][e];
        s.x += g;
        s.y = fmaf(g, xh, s.y);
        aw[n][e] = fmaf(d[e], xh, aw[n][e]);
        ab[n][e] += d[e];
      }
    }
    s = unit_sum<kBlock>(s, A.lanes, red, turn);
    if (!on) continue;
    const float mg = s.x * inv, mgx = s.y * inv;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c = (n * A.lanes + p.lane) * V;
      if (c < A.D) {
        float x[V], d[V];
        ux[n].get(x);
        ud[n].get(d);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float xh = (x[e] - mean) * rstd;
          d[e] = rstd * (fmaf(d[e], w[n][e], -mg) - xh * mgx);
        }
        Piece<T, V>::store(A.out + base + c, d);
      }
    }
  }
  if (A.partial == nullptr) return;
  // this CTA's sums: over its units of each group, in order
  const long long GD = static_cast<long long>(A.G) * A.D;
  float *out = A.partial + (blockIdx.x / A.gblocks) * 2 * GD;
  if (kBlock || A.slots == 1) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c = (n * A.lanes + p.lane) * V;
      if (p.active && c < A.D) {
        const long long pc = static_cast<long long>(p.g) * A.D + c;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          out[pc + e] = aw[n][e];
          out[GD + pc + e] = ab[n][e];
        }
      }
    }
    return;
  }
  const int width = A.gper * A.lanes * NV * V, slot = p.unit / A.gper, col0 = (p.unit % A.gper) * A.lanes * NV * V;
  if (slot < A.slots) {
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int col = col0 + (n * A.lanes + p.lane) * V + e;
        sums[slot * width + col] = aw[n][e];
        sums[(A.slots + slot) * width + col] = ab[n][e];
      }
  }
  __syncthreads();
  const int gb = blockIdx.x % A.gblocks, per = A.lanes * NV * V;
  for (int i = threadIdx.x; i < 2 * width; i += blockDim.x) {
    const int which = i / width, col = i - which * width, g = gb * A.gper + col / per, c = col % per;
    if (g >= A.G || c >= A.D) continue;
    float t = 0.f;
    for (int s = 0; s < A.slots; ++s) t += sums[(which * A.slots + s) * width + col];
    out[which * GD + static_cast<long long>(g) * A.D + c] = t;
  }
}

// Vectors that no CTA holds in registers: one CTA per (m, g), read again for each sum.
template <typename T> __global__ void __launch_bounds__(1024) layer_norm_long_kernel(const Args<T> A) {
  __shared__ float2 red[64];
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const long long m = blockIdx.x / A.G, base = blockIdx.x * static_cast<long long>(A.D);
  const long long gc = static_cast<long long>(blockIdx.x - m * A.G) * A.D;
  float s = 0.f;
  for (int c = threadIdx.x; c < A.D; c += blockDim.x) s += Elem<T>::load(A.x + base + c);
  const float mean = unit_sum<true>(make_float2(s, 0.f), 32, red, turn).x / static_cast<float>(A.D);
  float q = 0.f;
  for (int c = threadIdx.x; c < A.D; c += blockDim.x) {
    const float d = Elem<T>::load(A.x + base + c) - mean;
    q = fmaf(d, d, q);
  }
  const float var = unit_sum<true>(make_float2(q, 0.f), 32, red, turn).x / static_cast<float>(A.D);
  const float rstd = 1.f / sqrtf(var + A.eps);
  for (int c = threadIdx.x; c < A.D; c += blockDim.x) {
    const float xh = (Elem<T>::load(A.x + base + c) - mean) * rstd;
    Elem<T>::store(A.out + base + c, fmaf(xh, A.w ? A.w[gc + c] : 1.f, A.b ? A.b[gc + c] : 0.f));
  }
  if (threadIdx.x == 0) {
    if (A.mean != nullptr) A.mean[blockIdx.x] = mean;
    if (A.rstd != nullptr) A.rstd[blockIdx.x] = rstd;
  }
}

template <typename T> __global__ void __launch_bounds__(1024) layer_norm_backward_long_kernel(const Args<T> A) {
  __shared__ float2 red[64];
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const long long m = blockIdx.x / A.G, base = blockIdx.x * static_cast<long long>(A.D);
  const long long gc = static_cast<long long>(blockIdx.x - m * A.G) * A.D;
  const float mean = A.mean[blockIdx.x], rstd = A.rstd[blockIdx.x];
  float2 s = make_float2(0.f, 0.f);
  for (int c = threadIdx.x; c < A.D; c += blockDim.x) {
    const float xh = (Elem<T>::load(A.x + base + c) - mean) * rstd;
    const float g = Elem<T>::load(A.dy + base + c) * (A.w ? A.w[gc + c] : 1.f);
    s.x += g;
    s.y = fmaf(g, xh, s.y);
  }
  s = unit_sum<true>(s, 32, red, turn);
  const float mg = s.x / static_cast<float>(A.D), mgx = s.y / static_cast<float>(A.D);
  for (int c = threadIdx.x; c < A.D; c += blockDim.x) {
    const float xh = (Elem<T>::load(A.x + base + c) - mean) * rstd;
    const float g = Elem<T>::load(A.dy + base + c) * (A.w ? A.w[gc + c] : 1.f);
    Elem<T>::store(A.out + base + c, rstd * (g - mg - xh * mgx));
  }
}

// The column sums of long vectors: one thread per column, rows mb, mb + mblocks, ...; blockIdx = (mb, column tile).
template <typename T> __global__ void __launch_bounds__(256) layer_norm_columns_kernel(const Args<T> A) {
  pdl_wait();
  pdl_trigger();
  const long long GD = static_cast<long long>(A.G) * A.D, c = static_cast<long long>(blockIdx.y) * 256 + threadIdx.x;
  if (c >= GD) return;
  const int g = static_cast<int>(c / A.D);
  float aw = 0.f, ab = 0.f;
  for (long long m = blockIdx.x; m < A.M; m += gridDim.x) {
    const float d = Elem<T>::load(A.dy + m * GD + c);
    aw = fmaf(d, (Elem<T>::load(A.x + m * GD + c) - A.mean[m * A.G + g]) * A.rstd[m * A.G + g], aw);
    ab += d;
  }
  A.partial[blockIdx.x * 2 * GD + c] = aw;
  A.partial[(blockIdx.x * 2 + 1) * GD + c] = ab;
}

// dw and db from the partial sums [n][2][GD]: 32 columns and 32 slices of n per CTA.
__global__ void __launch_bounds__(1024) layer_norm_reduce_kernel(const float *partial, int n, long long GD, float *dw,
                                                                float *db) {
  __shared__ float part[32][33];
  pdl_wait();
  pdl_trigger();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const long long c = static_cast<long long>(blockIdx.x) * 32 + tx;
  float t = 0.f;
  if (c < 2 * GD)
    for (int i = ty; i < n; i += 32) t += partial[i * 2 * GD + c];
  part[ty][tx] = t;
  __syncthreads();
  t = part[tx][ty];
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
  const long long o = static_cast<long long>(blockIdx.x) * 32 + ty;
  if (tx == 0 && o < 2 * GD) (o < GD ? dw[o] : db[o - GD]) = t;
}

// How the vectors are laid over lanes and CTAs.
struct Plan {
  int v;         // elements per piece
  int nv;        // pieces per lane
  bool block;    // units are CTAs
  bool loop;     // vectors too long for registers
  int lanes, threads, gper, slots, gblocks, mblocks;
};

int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

Plan make_plan(size_t elem, int M, int G, int D, bool backward) {
  Plan P{};
  const int full = static_cast<int>(16 / elem);
  P.v = D % full == 0 ? full : (elem == 2 && D % 2 == 0) ? 2 : 1;
  const int pieces = ceil_div(D, P.v);
  if (pieces <= 128) {
    P.lanes = 1;
    while (P.lanes < pieces && P.lanes < 32) P.lanes *= 2;
    P.nv = ceil_div(pieces, P.lanes);
    P.threads = 256;
    const int units = P.threads / P.lanes;
    P.gper = G < units ? G : units;
    P.slots = units / P.gper;
  } else {
    P.block = true;
    P.gper = P.slots = 1;
    // the backward keeps three more values per element, so half as many elements per thread
    const int most = backward ? 16 / P.v : 32 / P.v;
    const int cap = most < 8 ? most : 8;
    for (P.nv = cap >= 2 && pieces >= 256 ? 2 : 1; P.nv < cap && ceil_div(pieces, P.nv) > 512; P.nv *= 2) {}
    P.threads = (ceil_div(pieces, P.nv) + 31) / 32 * 32;
    P.lanes = P.threads;
    if (P.threads > (backward ? backward_threads(P.v, P.nv) : 1024)) P.loop = true;
  }
  P.gblocks = ceil_div(G, P.gper);
  const int rowblocks = ceil_div(M, P.slots);  // CTAs that would take one row per unit
  const int resident = P.loop ? 2 : backward ? 2048 / P.threads / 2 : 2048 / P.threads;
  const int want = ceil_div(static_cast<long long>(kSMs) * (resident > 0 ? resident : 1), P.gblocks);
  P.mblocks = rowblocks < want ? rowblocks : want;
  return P;
}

cudaLaunchConfig_t config(dim3 grid, int threads, size_t smem, cudaStream_t stream, cudaLaunchAttribute *attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <typename K, typename... A>
cudaError_t launch(K kern, dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config(grid, threads, smem, stream, &attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int V, int NV, bool kBlock>
cudaError_t launch_planned(const Plan &P, const Args<T> &A, bool backward, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(P.gblocks * P.mblocks));
  if (!backward) return launch(layer_norm_kernel<T, V, NV, kBlock>, grid, P.threads, 0, stream, A);
  if constexpr (kBlock && V * NV > 16) return cudaErrorInvalidValue;  // no plan asks for it
  size_t smem = 0;
  if (!kBlock && P.slots > 1) smem = sizeof(float) * 2 * P.slots * P.gper * P.lanes * P.nv * P.v;
  auto kern = layer_norm_backward_kernel<T, V, (kBlock && V * NV > 16 ? 1 : NV), kBlock>;
  if (smem > 48 * 1024 - 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch(kern, grid, P.threads, smem, stream, A);
}

template <typename T, int V> cudaError_t launch_v(const Plan &P, const Args<T> &A, bool backward, cudaStream_t stream) {
  if (!P.block) {
    switch (P.nv) {
      case 1: return launch_planned<T, V, 1, false>(P, A, backward, stream);
      case 2: return launch_planned<T, V, 2, false>(P, A, backward, stream);
      case 3: return launch_planned<T, V, 3, false>(P, A, backward, stream);
      case 4: return launch_planned<T, V, 4, false>(P, A, backward, stream);
    }
  } else {
    switch (P.nv) {
      case 1: return launch_planned<T, V, 1, true>(P, A, backward, stream);
      case 2: return launch_planned<T, V, 2, true>(P, A, backward, stream);
      case 4: return launch_planned<T, V, 4, true>(P, A, backward, stream);
      case 8: if constexpr (V < 8) return launch_planned<T, V, 8, true>(P, A, backward, stream);
    }
  }
  return cudaErrorInvalidValue;
}

template <typename T> cudaError_t launch_any(const Plan &P, const Args<T> &A, bool backward, cudaStream_t stream) {
  constexpr int full = static_cast<int>(16 / sizeof(T));
  if (P.v == full) return launch_v<T, full>(P, A, backward, stream);
  if constexpr (sizeof(T) == 2) {
    if (P.v == 2) return launch_v<T, 2>(P, A, backward, stream);
  }
  return launch_v<T, 1>(P, A, backward, stream);
}

}  // namespace ln

template <typename TIn>
cudaError_t launch_layer_norm(const TIn *x, const float *w, const float *b, float eps, TIn *y, float *mean, float *rstd,
                              int M, int G, int D, cudaStream_t stream) {
  using namespace ln;
  if (M == 0) return cudaSuccess;
  const Plan P = make_plan(sizeof(TIn), M, G, D, false);
  const Args<TIn> A{x, nullptr, w, b, eps, y, mean, rstd, nullptr, M, G, D, P.lanes, P.gper, P.slots, P.gblocks};
  if (P.loop) return launch(layer_norm_long_kernel<TIn>, dim3(static_cast<unsigned>(M) * G), 1024, 0, stream, A);
  return launch_any(P, A, false, stream);
}

long long layer_norm_partial_bytes(size_t elem, int M, int G, int D) {
  const ln::Plan P = ln::make_plan(elem, M, G, D, true);
  return static_cast<long long>(P.mblocks) * 2 * G * D * static_cast<long long>(sizeof(float));
}

template <typename TIn>
cudaError_t launch_layer_norm_backward(const TIn *dy, const TIn *x, const float *w, const float *mean,
                                       const float *rstd, TIn *dx, float *dw, float *db, float *partial, int M, int G,
                                       int D, cudaStream_t stream) {
  using namespace ln;
  const Plan P = make_plan(sizeof(TIn), M, G, D, true);
  const long long GD = static_cast<long long>(G) * D;
  if (M > 0) {
    const Args<TIn> A{x, dy, w, nullptr, 0.f, dx, const_cast<float *>(mean), const_cast<float *>(rstd),
                      dw != nullptr ? partial : nullptr, M, G, D, P.lanes, P.gper, P.slots, P.gblocks};
    cudaError_t e;
    if (P.loop) {
      e = launch(layer_norm_backward_long_kernel<TIn>, dim3(static_cast<unsigned>(M) * G), 1024, 0, stream, A);
      if (e == cudaSuccess && dw != nullptr)
        e = launch(layer_norm_columns_kernel<TIn>, dim3(P.mblocks, ceil_div(GD, 256)), 256, 0, stream, A);
    } else {
      e = launch_any(P, A, true, stream);
    }
    if (e != cudaSuccess) return e;
  }
  if (dw == nullptr) return cudaSuccess;
  return launch(layer_norm_reduce_kernel, dim3(ceil_div(2 * GD, 32)), 1024, 0, stream,
                static_cast<const float *>(partial), M > 0 ? P.mblocks : 0, GD, dw, db);
}

template cudaError_t launch_layer_norm<float>(const float *, const float *, const float *, float, float *, float *,
                                              float *, int, int, int, cudaStream_t);
template cudaError_t launch_layer_norm<uint16_t>(const uint16_t *, const float *, const float *, float, uint16_t *,
                                                 float *, float *, int, int, int, cudaStream_t);
template cudaError_t launch_layer_norm_backward<float>(const float *, const float *, const float *, const float *,
                                                       const float *, float *, float *, float *, float *, int, int, int,
                                                       cudaStream_t);
template cudaError_t launch_layer_norm_backward<uint16_t>(const uint16_t *, const uint16_t *, const float *,
                                                          const float *, const float *, uint16_t *, float *, float *,
                                                          float *, int, int, int, cudaStream_t);

}  // namespace rwkv7
