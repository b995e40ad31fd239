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
// that owns one (m, g) vector: 1 to 32 lanes of a warp while it fits there (2 pieces a lane), else a
// whole CTA.  A unit keeps its group g and steps over the rows m, so it also keeps its columns' sums
// for dw and db in registers; CTAs then leave one partial sum each, and a second launch adds those up
// in a fixed order.  Vectors too long for a CTA's registers are walked in loops instead.
//
// Measured on B200 (us, share of measured HBM): forward 65536 x 4096 bf16 197 to 201, 82 %; gradients
// 16384 x 64 x 64 82, 76 %; 32768 x 768 37, 61 % (31 for the rows, 6 for the sum of the partials and the
// launch between).  Steps that carried, for the forward: rows fetched ahead and weights in registers 288 to
// 227, pointers instead of index arithmetic per row 227 to 201 (it was bound by its instructions).
#include "layer_norm.h"

#include "common.cuh"
#include "packed.cuh"

namespace rwkv7 {
namespace ln {

constexpr int kSMs = 148;

// Loads of what is read once: past L1, which keeps the weights.
__device__ __forceinline__ uint4 ld_once(const void *p) {
  uint4 u;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(p));
  return u;
}

// V consecutive elements of T as they lie in memory.  get / put: element e of the piece is half (o + e) % 2
// of pair (o + e) / 2, o being where the piece begins in a lane's elements (its multiple of V).
template <typename T, int V> struct Piece;
template <> struct Piece<float, 4> {
  uint4 u;
  __device__ __forceinline__ void load(const float *p) { u = ld_once(p); }
  __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(f32x2 *x, int o) const {
    x[o / 2] = make2(__uint_as_float(u.x), __uint_as_float(u.y));
    x[o / 2 + 1] = make2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ void put(float *p, const f32x2 *x, int o) {
    float4 f;
    split2(x[o / 2], f.x, f.y);
    split2(x[o / 2 + 1], f.z, f.w);
    *reinterpret_cast<float4 *>(p) = f;
  }
};
template <> struct Piece<uint16_t, 8> {
  uint4 u;
  __device__ __forceinline__ void load(const uint16_t *p) { u = ld_once(p); }
  __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(f32x2 *x, int o) const {
    x[o / 2] = unpack2(u.x);
    x[o / 2 + 1] = unpack2(u.y);
    x[o / 2 + 2] = unpack2(u.z);
    x[o / 2 + 3] = unpack2(u.w);
  }
  static __device__ __forceinline__ void put(uint16_t *p, const f32x2 *x, int o) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack2(x[o / 2]), pack2(x[o / 2 + 1]), pack2(x[o / 2 + 2]), pack2(x[o / 2 + 3]));
  }
};
template <> struct Piece<uint16_t, 2> {
  uint32_t u;
  __device__ __forceinline__ void load(const uint16_t *p) { u = *reinterpret_cast<const uint32_t *>(p); }
  __device__ __forceinline__ void zero() { u = 0u; }
  __device__ __forceinline__ void get(f32x2 *x, int o) const { x[o / 2] = unpack2(u); }
  static __device__ __forceinline__ void put(uint16_t *p, const f32x2 *x, int o) {
    *reinterpret_cast<uint32_t *>(p) = pack2(x[o / 2]);
  }
};
template <typename T> struct Piece<T, 1> {
  T u;
  __device__ __forceinline__ void load(const T *p) { u = *p; }
  __device__ __forceinline__ void zero() { u = 0; }
  __device__ __forceinline__ void get(f32x2 *x, int o) const {
    float a, b;
    split2(x[o / 2], a, b);
    const float f = Elem<T>::load(&u);
    x[o / 2] = o % 2 ? make2(a, f) : make2(f, 0.f);
  }
  static __device__ __forceinline__ void put(T *p, const f32x2 *x, int o) {
    float a, b;
    split2(x[o / 2], a, b);
    Elem<T>::store(p, o % 2 ? b : a);
  }
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

// V float32 parameters from w + c, placed as a piece's elements (ones or zeros where there is no w, which
// is only 4-byte aligned for odd D)
template <int V> __device__ __forceinline__ void params(const float *w, long long c, float missing, f32x2 *x, int o) {
  if constexpr (V == 1) {
    float a, b;
    split2(x[o / 2], a, b);
    const float f = w == nullptr ? missing : w[c];
    x[o / 2] = o % 2 ? make2(a, f) : make2(f, 0.f);
  } else if (w == nullptr) {
#pragma unroll
    for (int e = 0; e < V; e += 2) x[(o + e) / 2] = make2(missing, missing);
  } else if constexpr (V % 4 == 0) {
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      const float4 u = *reinterpret_cast<const float4 *>(w + c + e);
      x[(o + e) / 2] = make2(u.x, u.y);
      x[(o + e) / 2 + 1] = make2(u.z, u.w);
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      const float2 u = *reinterpret_cast<const float2 *>(w + c + e);
      x[(o + e) / 2] = make2(u.x, u.y);
    }
  }
}

__device__ __forceinline__ float lane_sum(float v, int lanes) {
  for (int off = lanes >> 1; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ float2 lane_sum(float2 v, int lanes) {
  for (int off = lanes >> 1; off >= 1; off >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, off);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, off);
  }
  return v;
}
// Sums over a unit's lanes.  Block units: the warps' sums meet in red (two sets of 32), with one barrier per
// call; a set is rewritten two calls later at the earliest.  `warps`: of the CTA, rounded up to a power of 2.
template <bool kBlock, typename F> __device__ __forceinline__ F unit_sum(F v, int lanes, int warps, F *red, int &turn) {
  if (!kBlock) return lane_sum(v, lanes);
  v = lane_sum(v, 32);
  F *slot = red + 32 * turn;
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  const int l = threadIdx.x & (warps - 1);
  F t{};
  if (l < static_cast<int>(blockDim.x >> 5)) t = slot[l];
  return lane_sum(t, warps);
}
__device__ __forceinline__ int warps_pow2() {
  const int w = blockDim.x >> 5;
  return w <= 1 ? 1 : 1 << (32 - __clz(w - 1));
}

// Where a thread stands: its unit's group g, and `count` rows from m0 on, `step` apart.  Every unit of a CTA goes
// through `turns` rows (the sums are over whole warps), the last of them perhaps empty.
struct Place {
  int lane, unit, g, m0, step, count, turns;
};
template <bool kBlock, typename T> __device__ __forceinline__ Place place(const Args<T> &A) {
  Place p;
  p.lane = kBlock ? threadIdx.x : threadIdx.x & (A.lanes - 1);
  p.unit = kBlock ? 0 : threadIdx.x / A.lanes;
  const int gb = blockIdx.x % A.gblocks, mb = blockIdx.x / A.gblocks, mblocks = gridDim.x / A.gblocks;
  p.g = gb * A.gper + p.unit % A.gper;
  const int slot = p.unit / A.gper;
  p.m0 = mb * A.slots + slot;  // below 2^31: mblocks * slots is at most M + slots
  p.step = mblocks * A.slots;
  p.turns = (A.M - 1) / p.step + 1;
  p.count = slot < A.slots && p.g < A.G && p.m0 < A.M ? (A.M - 1 - p.m0) / p.step + 1 : 0;
  return p;
}
// The lane's first element in the vector of a unit's first row, and the elements from one of its rows to the next.
template <typename T> __device__ __forceinline__ long long first_at(const Args<T> &A, const Place &p, int V) {
  return (static_cast<long long>(p.m0) * A.G + p.g) * A.D + p.lane * V;
}
template <typename T> __device__ __forceinline__ long long row_step(const Args<T> &A, const Place &p) {
  return static_cast<long long>(p.step) * A.G * A.D;
}

// A lane's pieces of the vector at `row`, zeros past its end (`left` elements are left from the lane's first)
// and where there is no row.
template <typename T, int V, int NV>
__device__ __forceinline__ void fetch(const T *row, bool on, int stride, int left, Piece<T, V> (&u)[NV]) {
#pragma unroll
  for (int n = 0; n < NV; ++n)
    if (on && n * stride < left) u[n].load(row + n * stride); else u[n].zero();
}

// Registers a thread may take with E elements.  Forward: two float32 parameters (beyond 16 elements they
// are read again from L1) and the value per element, and one or two rows fetched ahead: with rows of
// 8 KB, 48 KB are in flight per SM.  Backward: the weight, two sums, and the row under way and the next of
// two tensors (24 elements per lane spilled: 32768 x 768 took 73 us with one warp per row, 39 with three).
// At these limits several kernels with 8 and 16 elements spill, 4 to 76 bytes a thread.
constexpr int forward_regs(int E) { return E <= 8 ? 64 : E <= 16 ? 80 : 128; }
constexpr int backward_regs(int E) { return E <= 8 ? 80 : 128; }
constexpr int kMaxThreads = 512;

template <typename T, int V, int NV, bool kBlock>
__global__ void __launch_bounds__(kBlock ? kMaxThreads : 256) __maxnreg__(forward_regs(V *NV))
    layer_norm_kernel(const Args<T> A) {
  constexpr int kPairs = (V * NV + 1) / 2, kAhead = V * NV * sizeof(T) <= 32 ? 2 : 1;
  constexpr bool kKeepW = V * NV <= 16;
  __shared__ float red[64];
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const Place p = place<kBlock>(A);
  const int warps = warps_pow2(), stride = A.lanes * V, left = A.D - p.lane * V;
  const float inv = 1.f / static_cast<float>(A.D);
  const long long gc = static_cast<long long>(p.g) * A.D + p.lane * V, jump = row_step(A, p);
  f32x2 w[kPairs] = {}, b[kPairs] = {};
#pragma unroll
  for (int n = 0; n < NV; ++n)
    if (kKeepW && p.count > 0 && n * stride < left) {
      params<V>(A.w, gc + n * stride, 1.f, w, n * V);
      params<V>(A.b, gc + n * stride, 0.f, b, n * V);
    }
  const T *in = A.x + first_at(A, p, V);
  T *out = A.out + first_at(A, p, V);
  long long stat = static_cast<long long>(p.m0) * A.G + p.g;
  Piece<T, V> next[kAhead][NV];
#pragma unroll
  for (int k = 0; k < kAhead; ++k, in += jump) fetch(in, k < p.count, stride, left, next[k]);
  for (int i = 0; i < p.turns; ++i) {
    f32x2 x[kPairs] = {}, s2 = make2(0.f, 0.f);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      next[0][n].get(x, n * V);
#pragma unroll
      for (int k = 0; k + 1 < kAhead; ++k) next[k][n] = next[k + 1][n];
    }
    fetch(in, p.count - i > kAhead, stride, left, next[kAhead - 1]);
    in += jump;
#pragma unroll
    for (int e = 0; e < kPairs; ++e) s2 = add2(s2, x[e]);
    float s, t;
    split2(s2, s, t);
    const float mean = unit_sum<kBlock>(s + t, A.lanes, warps, red, turn) * inv;
    // centred values; what lies past the vector's end counts as zero
    const f32x2 mm = make2(-mean, -mean);
    f32x2 q2 = make2(0.f, 0.f);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      if constexpr (V == 1) {
        float a, z;
        split2(x[n / 2], a, z);
        const float d = n * stride < left ? (n % 2 ? z : a) - mean : 0.f;
        x[n / 2] = n % 2 ? make2(a, d) : make2(d, z);
        q2 = fma2(make2(d, 0.f), make2(d, 0.f), q2);
      } else if (n * stride < left) {
#pragma unroll
        for (int e = n * V / 2; e < (n + 1) * V / 2; ++e) {
          x[e] = add2(x[e], mm);
          q2 = fma2(x[e], x[e], q2);
        }
      }
    }
    split2(q2, s, t);
    const float var = unit_sum<kBlock>(s + t, A.lanes, warps, red, turn) * inv;
    const float rstd = rsqrtf(var + A.eps);  // within 2 steps of float32
    if (i < p.count) {
      const f32x2 rr = make2(rstd, rstd);
      if constexpr (kKeepW) {
#pragma unroll
        for (int e = 0; e < kPairs; ++e) x[e] = fma2(mul2(x[e], rr), w[e], b[e]);
      }
#pragma unroll
      for (int n = 0; n < NV; ++n)
        if (n * stride < left) {
          if constexpr (!kKeepW) {
            f32x2 wp[V / 2], bp[V / 2];
            params<V>(A.w, gc + n * stride, 1.f, wp, 0);
            params<V>(A.b, gc + n * stride, 0.f, bp, 0);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) x[n * V / 2 + e] = fma2(mul2(x[n * V / 2 + e], rr), wp[e], bp[e]);
          }
          Piece<T, V>::put(out + n * stride, x, n * V);
        }
      if (p.lane == 0) {
        if (A.mean != nullptr) A.mean[stat] = mean;
        if (A.rstd != nullptr) A.rstd[stat] = rstd;
      }
    }
    out += jump;
    stat += static_cast<long long>(p.step) * A.G;
  }
}

template <typename T, int V, int NV, bool kBlock>
__global__ void __launch_bounds__(kBlock ? kMaxThreads : 256) __maxnreg__(backward_regs(V *NV))
    layer_norm_backward_kernel(const Args<T> A) {
  constexpr int kPairs = (V * NV + 1) / 2;
  __shared__ float2 red[64];
  extern __shared__ float sums[];  // units of a warp only: [2][slots][gper * lanes * NV * V]
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const Place p = place<kBlock>(A);
  const int warps = warps_pow2(), stride = A.lanes * V, left = A.D - p.lane * V;
  const float inv = 1.f / static_cast<float>(A.D);
  const long long gc = static_cast<long long>(p.g) * A.D + p.lane * V, jump = row_step(A, p);
  f32x2 w[kPairs] = {}, aw[kPairs] = {}, ab[kPairs] = {};
#pragma unroll
  for (int n = 0; n < NV; ++n)
    if (p.count > 0 && n * stride < left) params<V>(A.w, gc + n * stride, 1.f, w, n * V);
  const T *inx = A.x + first_at(A, p, V), *ind = A.dy + first_at(A, p, V);
  T *out = A.out + first_at(A, p, V);
  long long stat = static_cast<long long>(p.m0) * A.G + p.g;
  Piece<T, V> nx[NV], nd[NV];
  float nmean = 0.f, nrstd = 0.f;
  auto fetch_all = [&](bool on) {
    fetch(inx, on, stride, left, nx);
    fetch(ind, on, stride, left, nd);
    if (on) {
      nmean = A.mean[stat];
      nrstd = A.rstd[stat];
    }
    inx += jump;
    ind += jump;
    stat += static_cast<long long>(p.step) * A.G;
  };
  fetch_all(p.count > 0);
  for (int i = 0; i < p.turns; ++i) {
    Piece<T, V> ux[NV], ud[NV];
    const float rstd = nrstd;
    const f32x2 rr = make2(rstd, rstd), mm = make2(-nmean, -nmean);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      ux[n] = nx[n];
      ud[n] = nd[n];
    }
    fetch_all(i + 1 < p.count);
    f32x2 sg = make2(0.f, 0.f), sx = make2(0.f, 0.f);  // sums of g and g xh
    // (past the vector's end dy is zero, and so is what it adds)
    {
      f32x2 x[kPairs] = {}, d[kPairs] = {};
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        ux[n].get(x, n * V);
        ud[n].get(d, n * V);
      }
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        const f32x2 xh = mul2(add2(x[e], mm), rr), g = mul2(d[e], w[e]);
        sg = add2(sg, g);
        sx = fma2(g, xh, sx);
        aw[e] = fma2(d[e], xh, aw[e]);
        ab[e] = add2(ab[e], d[e]);
      }
    }
    float a, b, c0, d0;
    split2(sg, a, b);
    split2(sx, c0, d0);
    const float2 s = unit_sum<kBlock>(make_float2(a + b, c0 + d0), A.lanes, warps, red, turn);
    if (i < p.count) {
      // dx = rstd (g - mg - xh mgx)
      const float mg = -s.x * inv * rstd, mgx = -s.y * inv * rstd;
      const f32x2 mg2 = make2(mg, mg), mgx2 = make2(mgx, mgx);
      f32x2 x[kPairs] = {}, d[kPairs] = {};
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        ux[n].get(x, n * V);
        ud[n].get(d, n * V);
      }
#pragma unroll
      for (int e = 0; e < kPairs; ++e)
        d[e] = fma2(mul2(d[e], w[e]), rr, fma2(mul2(add2(x[e], mm), rr), mgx2, mg2));
#pragma unroll
      for (int n = 0; n < NV; ++n)
        if (n * stride < left) Piece<T, V>::put(out + n * stride, d, n * V);
    }
    out += jump;
  }
  if (A.partial == nullptr) return;
  // this CTA's sums: over its units of each group, in order
  const long long GD = static_cast<long long>(A.G) * A.D;
  float *part = A.partial + (blockIdx.x / A.gblocks) * 2 * GD;
  // units that the groups leave over (G = 12 groups on 16 units) stand in a slot past the last: their p.g is that of a
  // unit with rows, and they store nothing
  const int slot = p.unit / A.gper;
  if (kBlock || A.slots == 1) {
    constexpr int kF = V % 4 == 0 ? 4 : 1;
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if (slot < A.slots && p.g < A.G && n * stride < left) {
#pragma unroll
        for (int e = 0; e < V; e += kF) {
          Piece<float, kF>::put(part + gc + n * stride + e, aw, n * V + e);
          Piece<float, kF>::put(part + GD + gc + n * stride + e, ab, n * V + e);
        }
      }
    return;
  }
  const int width = A.gper * A.lanes * NV * V, col0 = (p.unit % A.gper) * A.lanes * NV * V;
  if (slot < A.slots) {
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int col = col0 + (n * A.lanes + p.lane) * V + e;
        Piece<float, 1>::put(sums + slot * width + col, aw, n * V + e);
        Piece<float, 1>::put(sums + (A.slots + slot) * width + col, ab, n * V + e);
      }
  }
  __syncthreads();
  const int gb = blockIdx.x % A.gblocks, per = A.lanes * NV * V;
  for (int i = threadIdx.x; i < 2 * width; i += blockDim.x) {
    const int which = i / width, col = i - which * width, g = gb * A.gper + col / per, c = col % per;
    if (g >= A.G || c >= A.D) continue;
    float t = 0.f;
    for (int s = 0; s < A.slots; ++s) t += sums[(which * A.slots + s) * width + col];
    part[which * GD + static_cast<long long>(g) * A.D + c] = t;
  }
}

// Vectors that no CTA holds in registers: one CTA per (m, g), read again for each sum.
template <typename T> __global__ void __launch_bounds__(1024) layer_norm_long_kernel(const Args<T> A) {
  __shared__ float red[64];
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const long long m = blockIdx.x / A.G, base = blockIdx.x * static_cast<long long>(A.D);
  const long long gc = static_cast<long long>(blockIdx.x - m * A.G) * A.D;
  float s = 0.f;
  for (int c = threadIdx.x; c < A.D; c += blockDim.x) s += Elem<T>::load(A.x + base + c);
  const float mean = unit_sum<true>(s, 32, 32, red, turn) / static_cast<float>(A.D);
  float q = 0.f;
  for (int c = threadIdx.x; c < A.D; c += blockDim.x) {
    const float d = Elem<T>::load(A.x + base + c) - mean;
    q = fmaf(d, d, q);
  }
  const float var = unit_sum<true>(q, 32, 32, red, turn) / static_cast<float>(A.D);
  const float rstd = rsqrtf(var + A.eps);
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
  s = unit_sum<true>(s, 32, 32, red, turn);
  const float mg = s.x / static_cast<float>(A.D), mgx = s.y / static_cast<float>(A.D);
  for (int c = threadIdx.x; c < A.D; c += blockDim.x) {
    const float xh = (Elem<T>::load(A.x + base + c) - mean) * rstd;
    const float g = Elem<T>::load(A.dy + base + c) * (A.w ? A.w[gc + c] : 1.f);
    Elem<T>::store(A.out + base + c, rstd * (g - mg - xh * mgx));
  }
}

// The column sums of long vectors: one thread per column, rows mb, mb + mblocks, ...; blockIdx = (column tile, mb):
// there may be 65536 tiles, one more than a grid has in y.
template <typename T> __global__ void __launch_bounds__(256) layer_norm_columns_kernel(const Args<T> A) {
  pdl_wait();
  pdl_trigger();
  const long long GD = static_cast<long long>(A.G) * A.D, c = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= GD) return;
  const int g = static_cast<int>(c / A.D);
  float aw = 0.f, ab = 0.f;
  for (long long m = blockIdx.y; m < A.M; m += gridDim.y) {
    const float d = Elem<T>::load(A.dy + m * GD + c);
    aw = fmaf(d, (Elem<T>::load(A.x + m * GD + c) - A.mean[m * A.G + g]) * A.rstd[m * A.G + g], aw);
    ab += d;
  }
  A.partial[blockIdx.y * 2 * GD + c] = aw;
  A.partial[(blockIdx.y * 2 + 1) * GD + c] = ab;
}

// dw and db from the partial sums [n][2][GD]: 8 columns and 128 slices of n per CTA.
__global__ void __launch_bounds__(256) layer_norm_reduce_kernel(const float *partial, int n, long long GD, float *dw,
                                                               float *db) {
  __shared__ float4 part[2][8];
  pdl_wait();
  pdl_trigger();
  const int tx = threadIdx.x & 1, ty = threadIdx.x >> 1;
  const long long cols = 2 * GD, c = static_cast<long long>(blockIdx.x) * 8 + 4 * tx;
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  if ((cols & 3) == 0 && c < cols) {
#pragma unroll 8
    for (int i = ty; i < n; i += 128) {
      const float4 u = *reinterpret_cast<const float4 *>(partial + i * cols + c);
      t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
    }
  } else {
    for (int i = ty; i < n; i += 128) {
      const float *p = partial + i * cols + c;
      if (c < cols) t.x += p[0];
      if (c + 1 < cols) t.y += p[1];
      if (c + 2 < cols) t.z += p[2];
      if (c + 3 < cols) t.w += p[3];
    }
  }
#pragma unroll
  for (int off = 16; off >= 2; off >>= 1) {
    t.x += __shfl_xor_sync(0xffffffffu, t.x, off);
    t.y += __shfl_xor_sync(0xffffffffu, t.y, off);
    t.z += __shfl_xor_sync(0xffffffffu, t.z, off);
    t.w += __shfl_xor_sync(0xffffffffu, t.w, off);
  }
  if ((threadIdx.x & 31) < 2) part[tx][threadIdx.x >> 5] = t;
  __syncthreads();
  if (threadIdx.x >= 8) return;
  const float *q = reinterpret_cast<const float *>(part[threadIdx.x >> 2]) + (threadIdx.x & 3);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += q[4 * i];
  const long long o = static_cast<long long>(blockIdx.x) * 8 + threadIdx.x;
  if (o < cols) (o < GD ? dw[o] : db[o - GD]) = s;
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
  if (pieces <= 64) {
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
    const int most = (backward ? 16 : static_cast<int>(64 / elem)) / P.v, cap = most < 8 ? most : 8;  // pieces per lane
    for (P.nv = 1; P.nv < cap && ceil_div(pieces, P.nv) > 256; P.nv *= 2) {}
    P.threads = (ceil_div(pieces, P.nv) + 31) / 32 * 32;
    P.lanes = P.threads;
    P.loop = P.threads > kMaxThreads;
  }
  P.gblocks = ceil_div(G, P.gper);
  if (P.loop) {
    // the backward's column sums: tiles of 256 columns, and row blocks for 8 rounds of 8 CTAs per SM, so that the last
    // round counts little.  Each row block is a partial sum: 296 of them whatever the width would be 40 GB for 300
    // rows of 2^24.  Measured (us; 296 row blocks / 1, 4, 8 rounds), bf16: 4096 x 16384 357 / 400, 331, 339;
    // 8192 x 12288 518 / 613, 524, 516; 300 x 16384 61 / 35, 42, 46.
    const int want = ceil_div(8LL * 8 * kSMs, ceil_div(static_cast<long long>(G) * D, 256));
    P.mblocks = M < want ? M : want;
    return P;
  }
  const int rowblocks = ceil_div(M, P.slots);  // CTAs that would take one row per unit
  const int regs = backward ? backward_regs(P.v * P.nv) : forward_regs(P.v * P.nv);
  const int resident = 65536 / regs / P.threads;
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
  if constexpr (V * NV > 16) return cudaErrorInvalidValue;  // no plan asks for it
  size_t smem = 0;
  // at most 256 lanes of 16 elements, 32 KB: below what a launch has without asking
  if (!kBlock && P.slots > 1) smem = sizeof(float) * 2 * P.slots * P.gper * P.lanes * P.nv * P.v;
  auto kern = layer_norm_backward_kernel<T, V, (V * NV > 16 ? 1 : NV), kBlock>;
  return launch(kern, grid, P.threads, smem, stream, A);
}

template <typename T, int V> cudaError_t launch_v(const Plan &P, const Args<T> &A, bool backward, cudaStream_t stream) {
  if (!P.block) {
    switch (P.nv) {
      case 1: return launch_planned<T, V, 1, false>(P, A, backward, stream);
      case 2: return launch_planned<T, V, 2, false>(P, A, backward, stream);
    }
  } else {
    switch (P.nv) {
      case 1: return launch_planned<T, V, 1, true>(P, A, backward, stream);
      case 2: return launch_planned<T, V, 2, true>(P, A, backward, stream);
      case 4: return launch_planned<T, V, 4, true>(P, A, backward, stream);
      case 8: if constexpr (V < 4) return launch_planned<T, V, 8, true>(P, A, backward, stream);
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
        e = launch(layer_norm_columns_kernel<TIn>, dim3(ceil_div(GD, 256), P.mblocks), 256, 0, stream, A);
    } else {
      e = launch_any(P, A, true, stream);
    }
    if (e != cudaSuccess) return e;
  }
  if (dw == nullptr) return cudaSuccess;
  return launch(layer_norm_reduce_kernel, dim3(ceil_div(2 * GD, 8)), 256, 0, stream,
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
