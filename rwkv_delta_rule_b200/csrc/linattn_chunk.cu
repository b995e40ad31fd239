// linattn_chunk.cu -- linear attention with one decay per head, 128 tokens at a time on the tcgen05
// tensor cores, forward and (for gradients) walked from the last token.
//
// For a chunk of L <= 128 tokens (rows t, s from 0) that begins with state S0, the recurrence
// S <- w S + v k^T, out = S q is
//     P_ts  = (q_t . k_s) w^(t-s)  for s <= t, else 0
//     out_t = w^(t+1) S0 q_t + sum_s P_ts v_s
//     S_L   = w^L S0 + sum_s (w^(L-1-s) v_s) k_s^T
// and reversed (S <- S + v k^T, out = S q, S <- w S, tokens from the last)
//     P_ts  = (q_t . k_s) w^(s-t)  for s >= t;   out_t = w^(L-1-t) S0 q_t + ...;
//     S_0   = w^L S0 + sum_s (w^(s+1) v_s) k_s^T.
// Only powers of the head's decay appear, w^0 .. w^128 and, where segments are joined, those of their lengths; all
// <= 1, so every w in [0, 1] is exact.  Those that scale the state are applied in two float32 terms.
//
// One CTA of eight warps walks the chunks of one (b, h) (or of one segment of it), two CTAs per SM: 106 KB of
// shared memory and 256 TMEM columns each, and what one waits for overlaps the other's work.  Warp w has
// token rows (TMEM lanes) 32 (w % 4) .. + 31 and half w / 4 of their columns; the warp with nothing to do
// in P issues the TMA loads and the MMAs.  Per chunk, float32 accumulation:
//     MMA1  [128 x 192] = Q [K; S0]^T                K-major tiles, as TMA and the warps left them
//     MMA2  [128 x 64]  = P V                        P from TMEM in bf16, V as TMA left it (MN-major)
//     MMA3  [64 x 64]   = V1 K + V2 K (+ V3 K)       V1 + V2 (+ V3) = w^(L-1-s) v_s, MN-major
// MMA3 and the new state run beside P and MMA2, and the tiles of the next chunk arrive meanwhile.
// The state stays in float32 registers across chunks (16 elements per thread).  Roundings to bf16:
//   P: one per product, as large as the rounding of out itself, and averaged over the tokens;
//   S0 in MMA1: once, 2^-8 at most like P; it reaches out only (out's error against float64 is 0.0023 of
//   its norm, 0.0017 of which is out's own rounding).  A second term cost the shared memory and the TMEM
//   columns that let MMA3 run beside P (B4 T16384 H64: 685 us with it, 625 without);
//   w^(L-1-s) v_s in MMA3: three terms, 2^-24 at most, because these sums are the state: with two terms
//   they would be 2.7e-6 off on average, the three leave 4e-7 (float32 sums of products alone: 2e-7).
//   Where the state is no output (dr and dk) two, 2^-16 at most: the outputs are bf16, and S0's 2^-8 is
//   larger (backward B8 T1024 H12 39 us with three there, 34 with two; B2 T4001 H64 220 and 190).  dv's pass
//   has three whether or not its state, ds_in, is asked for, so that dv does not depend on that.
// k, q and v enter their products as they are, exactly.
//
// NaN and infinity: zero times them is NaN, so a bad k or v would also spoil the rows of its chunk before it (reversed:
// behind it).  Such a chunk shows in MMA3's result, whose row (v) or column (k) is not finite then, and its out is
// formed again by redo_out.  Looking for it there takes 8 operations per thread and chunk and costs nothing that
// can be measured; selects in P and a sum over the pieces of v instead cost 3 to 5 % of a prefill.
//
// Code size counts: both directions of the backward run on an SM at once.  With the polling of a wait unrolled
// by the compiler and a descriptor formed per MMA, 10 KB more in all, B2 T4001 H64 takes 221 us and 196 as it is.
//
// Measured on B200: B4 T16384 H64 (2.15 GB) 431 us, 476 to 540 us back to back, where the card's power
// limit takes the clock from 1.97 to 1.55 GHz; 296 chains (2 per SM) of 8192 tokens 5.4 TB/s, 83 % of
// measured HBM.  A chunk takes 2.5 us alone on an SM and 3.6 us with another CTA: no unit is full (issue
// slots 33 %, tensor pipe 40 %, shared memory about half), the chain from barrier to barrier is what is
// left.  Steps that carried: MMAs under elect.sync (7 cycles to issue against 90), M = 64 for MMA3 (35 cycles
// an MMA against 50), no spills (L1 is 4 KB here), powers in registers, tiles that change places.  Tried and
// not kept, no faster: a ninth warp for the issuing, 16 warps per CTA, a second term of S0.
#include <cuda.h>

#include "linattn.h"
#include "packed.cuh"
#include "tc_ptx.cuh"

namespace rwkv7 {
namespace lin {

constexpr int kChunk = 128;
constexpr int kThreads = 256;
constexpr uint32_t kMaxPolls = 1u << 22;
constexpr uint32_t kTile = kChunk * kN * 2;  // one bf16 128 x 64 tile, 128-byte swizzled rows

// TMEM columns.  MMA1 fills 0 .. 191 (q k, then q S0); P (bf16 pairs) replaces the first 64 of the
// products as they are read, MMA2's result the second 64.  MMA3's 64 rows lie 16 to each warp's 32 lanes.
constexpr uint32_t TM_P = 0, TM_Y = 64, TM_YS = 128, TM_X = 192, kTmemCols = 256;

// shared memory, from a 1024-aligned base.  V1's tile is where the rows of out are put together for
// their TMA store.
constexpr uint32_t OFF_Q = 0, OFF_K = kTile;
constexpr uint32_t OFF_S = 2 * kTile;  // [64 value channels][64 key channels]; MMA1's rows behind K
constexpr uint32_t OFF_V = OFF_S + kN * kN * 2, OFF_V1 = OFF_V + kTile, OFF_V2 = OFF_V1 + kTile, OFF_V3 = OFF_V2 + kTile;
constexpr uint32_t OFF_PW = OFF_V3 + kTile;  // float [132]: w^n for n <= 128
constexpr uint32_t OFF_PL = OFF_PW + 528;    // float [132]: what the rounding of w^n to float32 leaves
constexpr uint32_t OFF_BAR = OFF_PL + 528;   // mbarriers, TMEM address, flags
constexpr uint32_t OFF_EDGE = OFF_BAR + 128;  // unsigned [64]: see redo_out
constexpr uint32_t kSmemBytes = OFF_EDGE + 256 + 1024;
// Tiles landed (Q and K; V); all warps ready for MMA1, MMA3, MMA2; each of those done; V1's tile free again; a product
// of redo_out done (two phases per call).
enum { B_QK, B_V, B_READY, B_SPLIT, B_P, B_M1, B_M3, B_M2, B_OUT, B_REDO, kBars };
constexpr uint32_t OFF_SLOT = OFF_BAR + 8 * kBars;  // words: TMEM address, bad, stop, redo
static_assert(OFF_SLOT % 8 == 0 && 8 * kBars + 16 <= 128, "stop and redo are read together");

struct Maps {
  CUtensorMap q, k, v, out;  // [tokens, H, 64] bf16, box {64, 1, 128}
};

// the values cut to their upper 16 bits, which are bf16: what is cut off is left exactly by sub2
__device__ __forceinline__ f32x2 cut2(f32x2 x) { return x & 0xffff0000ffff0000ull; }
__device__ __forceinline__ uint32_t high_halves(f32x2 x) {
  return __byte_perm(static_cast<uint32_t>(x), static_cast<uint32_t>(x >> 32), 0x7632);
}
// shared memory by 32-bit address
__device__ __forceinline__ void sts128(uint32_t p, const uint32_t (&u)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3])
               : "memory");
}
__device__ __forceinline__ void sts32(uint32_t p, uint32_t u) {
  asm volatile("st.shared.b32 [%0], %1;\n" ::"r"(p), "r"(u) : "memory");
}
__device__ __forceinline__ void lds128(uint32_t p, uint32_t (&u)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "r"(p)
               : "memory");
}
__device__ __forceinline__ float lds32(uint32_t p) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(v) : "r"(p) : "memory");
  return v;
}
// 16 lanes x 32 columns of 32-bit, spread over the warp: pair 2 n + u of a thread is lane t / 4 + 8 u,
// columns 8 n + 2 (t % 4), + 1.  Load followed by the wait.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, f32x2 (&v)[8]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = make2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
}
// true in one lane of the (converged) warp.  MMAs are issued under this predicate, in a branch that is
// uniform for the warp: then an MMA takes 7 cycles to issue, under lane == 0 it takes 90 (measured
// with 32 MMAs of 128 x 64 x 16, which take 50 each to run).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory"); }
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, uint32_t src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];\n" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// P in bf16 from 32 columns of products q k: a block on the diagonal, w^(t-s), zero past it: 1 on it, then a factor w
// per column ...
template <bool kRev> __device__ __forceinline__ void diagonal_p(float (&v)[32], float (&pk)[16], int lane, float w1) {
  float f = 0.f;
#pragma unroll
  for (int x = 0; x < 32; ++x) {
    const int e = kRev ? x : 31 - x;
    f = e == lane ? 1.f : f * w1;
    v[e] *= f;
  }
#pragma unroll
  for (int x = 0; x < 16; ++x) pk[x] = __uint_as_float(pack2(make2(v[2 * x], v[2 * x + 1])));
}
// ... and one off it, w^(t-s) = w^(t - 32 g - 31) w^(31 - x), reversed w^(s-t) = w^(32 g - t) w^x; a is the first factor
template <bool kRev>
__device__ __forceinline__ void full_p(const float (&v)[32], float (&pk)[16], float a, float w1, f32x2 w2) {
  f32x2 f = kRev ? make2(a, a * w1) : make2(a * w1, a);
#pragma unroll
  for (int x = 0; x < 16; ++x) {
    const int e = kRev ? x : 15 - x;
    pk[e] = __uint_as_float(pack2(mul2(make2(v[2 * e], v[2 * e + 1]), f)));
    f = mul2(f, w2);
  }
}

// The rows of out again, for a chunk with a k or v that is not finite: P with nothing past its diagonal, a bad v as zero
// in P V and then NaN from its own row on (reversed: up to it).  All other results keep their bits.  Called by the whole
// CTA behind the chunk's last barrier, when the tiles of V1 to V3 and the first 128 TMEM columns are free and q S0 still
// is in TMEM; q, k, v, out: the chunk's first row of this head.  edge[channel] = number << 8 | kChunk - n says that
// from the n-th row on (reversed: counted from the last) the channel is NaN in the CTA's chunk `number`, counted from
// 1; later chunks' words are larger, so none has to be cleared.  Not inlined: the loop's code has to stay small.
template <bool kRev>
__device__ __noinline__ void redo_out(uint32_t sm, uint32_t tmem, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                                      uint16_t *out, int H, int L, int number) {
  constexpr int kLead = kRev ? 3 : 4;
  uint8_t *smem = static_cast<uint8_t *>(__cvta_shared_to_generic(sm));
  unsigned *edge = reinterpret_cast<unsigned *>(smem + OFF_EDGE);
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + OFF_BAR) + B_REDO;
  volatile int *bad = reinterpret_cast<volatile int *>(smem + OFF_SLOT + 4);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, rb = warp & 3, half = warp >> 2;
  const int row = 32 * rb + lane, nth = kRev ? kChunk - 1 - row : row;
  const bool elected = elect_one();
  const uint32_t at = sm + row * 128u + (((4 * half) ^ (row & 7)) << 4), tml = tmem + (static_cast<uint32_t>(rb) << 21);
  const long long mine = row * (static_cast<long long>(H) * kN) + 32 * half;
#pragma unroll 1
  for (int x = 0; x < 4; ++x) {
    uint4 u[3] = {};
    if (row < L) {
      u[0] = *reinterpret_cast<const uint4 *>(q + mine + 8 * x);
      u[1] = *reinterpret_cast<const uint4 *>(k + mine + 8 * x);
      u[2] = *reinterpret_cast<const uint4 *>(v + mine + 8 * x);
    }
    uint32_t w[4] = {u[2].x, u[2].y, u[2].z, u[2].w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t ones = e & 1 ? 0x7f800000u : 0x7f80u;
      if ((w[e >> 1] & ones) == ones) {
        w[e >> 1] &= e & 1 ? 0xffffu : 0xffff0000u;
        atomicMax(edge + 32 * half + 8 * x + e, static_cast<unsigned>(number) << 8 | static_cast<unsigned>(kChunk - nth));
      }
    }
    const uint32_t wq[4] = {u[0].x, u[0].y, u[0].z, u[0].w}, wk[4] = {u[1].x, u[1].y, u[1].z, u[1].w};
    sts128((at ^ (16 * x)) + OFF_V1, wq);
    sts128((at ^ (16 * x)) + OFF_V2, wk);
    sts128((at ^ (16 * x)) + OFF_V3, w);
  }
  // a product issued by the leading warp, which all wait for
  auto product = [&](int phase, auto issue) {
    tc::fence_proxy_async_smem();
    tc::tc_fence_before();
    named_sync(1, kThreads);
    tc::tc_fence_after();
    if (warp == kLead && elected) {
      issue();
      tc::mma_commit(bar);
      if (!tc::mbar_wait_bounded(bar, phase, kMaxPolls)) *bad = 1;
    }
    __syncwarp();
    if (!tc::mbar_wait_bounded(bar, phase, kMaxPolls)) *bad = 1;
    tc::tc_fence_after();
  };
  product(0, [&]() {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
      tc::mma_ss(0, tmem + TM_P, tc::smem_desc(sm + OFF_V1 + ks * 32, 16, 1024),
                 tc::smem_desc(sm + OFF_V2 + ks * 32, 16, 1024), tc::instr_desc(tc::kFmtBF16, 128, 128, false, false), ks > 0);
  });
  const float w1 = lds32(sm + OFF_PW + 4);
#pragma unroll 1
  for (int n = 0; n < 2; ++n) {
    const int g = half + 2 * n;
    float p[32], pk[16] = {};
    tc::tmem_ld32(tml + TM_P + 32 * g, p);
    if (g == rb) {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (kRev ? e < lane : e > lane) p[e] = 0.f;
      diagonal_p<kRev>(p, pk, lane, w1);
    } else if (kRev ? g > rb : g < rb) {
      full_p<kRev>(p, pk, lds32(sm + OFF_PW + 4 * (kRev ? 32 * g - row : row - 32 * g - 31)), w1, make2(w1 * w1, w1 * w1));
    }
    tc::tmem_st16(tml + TM_P + 32 * half + 16 * n, pk);
  }
  tc::tmem_st_wait();
  product(1, [&]() {
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
      tc::mma_ts_bf16(tmem + TM_Y, tmem + TM_P + 32 * ((ks >> 1) & 1) + 16 * (ks >> 2) + 8 * (ks & 1),
                      tc::smem_desc(sm + OFF_V3 + ks * 2048, kTile, 1024),
                      tc::instr_desc(tc::kFmtBF16, 128, 64, false, true), ks > 0);
  });
  const float f1 = lds32(sm + OFF_PW + 4 * (kRev ? max(L - 1 - row, 0) : row + 1));
  float y[32], p[32];
  tc::tmem_ld32(tml + TM_YS + 32 * half, y);
  tc::tmem_ld32(tml + TM_Y + 32 * half, p);
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const unsigned c = edge[32 * half + 8 * x + e];
      if (c >> 8 == static_cast<unsigned>(number) && nth >= kChunk - static_cast<int>(c & 255u))
        p[8 * x + e] = __int_as_float(0x7fffffff);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      u[e] = pack2(fma2(make2(y[8 * x + 2 * e], y[8 * x + 2 * e + 1]), make2(f1, f1),
                        make2(p[8 * x + 2 * e], p[8 * x + 2 * e + 1])));
    sts128((at ^ (16 * x)) + OFF_V1, u);
    if (L < kChunk && row < L) *reinterpret_cast<uint4 *>(out + mine + 8 * x) = make_uint4(u[0], u[1], u[2], u[3]);
  }
  tc::fence_proxy_async_smem();
  tc::tc_fence_before();
  named_sync(1, kThreads);
}

// One segment of one pass.
template <bool kRev, bool kOut>
__device__ __forceinline__ void walk(const Maps &maps, const Pass<uint16_t> &A, const Shape &P, int b, int z,
                                     uint8_t *smem_raw, int *err_word) {
  const uint32_t sm = (smem_u32(smem_raw) + 1023u) & ~1023u;  // shared-memory addresses from here on
  uint8_t *smem = smem_raw + (sm - smem_u32(smem_raw));
  const int h = blockIdx.x;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const bool elected = elect_one();
  const Segment sg = segment(P, b, z);
  if (sg.len < 0) return;
  if (!kOut && (kRev ? sg.first : sg.last)) return;
  const long long pair = static_cast<long long>(b) * P.H + h;

  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + OFF_BAR);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + OFF_SLOT);
  volatile int *bad = reinterpret_cast<volatile int *>(smem + OFF_SLOT + 4);  // a wait ran out
  volatile int *stop = bad + 1;  // tid 0's copy of it, which all warps act on together
  volatile int *redo = bad + 2;  // the last chunk, counted from 1, with a k or v that is not finite

  const int nchunks = (sg.len + kChunk - 1) / kChunk;
  auto chunk_at = [&](int i) { return kRev ? nchunks - 1 - i : i; };
  // one tile of chunk `it`, and that of the chunk after it on its way to L2
  auto load = [&](const CUtensorMap *map, uint32_t to, int bar, int it) {
    const int tok = static_cast<int>(sg.lo) + chunk_at(it) * kChunk;
    tc::mbar_arrive_expect_tx(bars + bar, kTile);
    tc::tma_load_3d(smem + to, map, bars + bar, 0, h, tok);
    if (it + 1 < nchunks) tc::tma_prefetch_l2_3d(map, 0, h, tok + (kRev ? -kChunk : kChunk));
  };
  // issues loads and MMAs; of the two warps of its rows the one without products of its own in P
  constexpr int kLead = kRev ? 3 : 4;
  constexpr int kStore = kRev ? 4 : 3;  // issues the TMA stores of out
  if (warp == kLead) {
    if (elected) {
      for (int i = 0; i < kBars; ++i)
        tc::mbar_init(bars + i, i == B_READY || i == B_SPLIT ? 8 : i == B_P ? 7 : i == B_QK && kOut ? 2 : 1);
      tc::fence_mbar_init();
      *bad = 0;
      *stop = 0;
      *redo = 0;
      if (nchunks > 0) {
        load(&maps.k, OFF_K, B_QK, 0);
        load(&maps.v, OFF_V, B_V, 0);
        if (kOut) load(&maps.q, OFF_Q, B_QK, 0);
      }
    }
    __syncwarp();
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  {
    float *pw = reinterpret_cast<float *>(smem + OFF_PW), *pl = reinterpret_cast<float *>(smem + OFF_PL);
    for (int n = tid; n <= kChunk; n += kThreads) {
      const double p = powi(static_cast<double>(P.w[h]), n);
      const float f = static_cast<float>(p);
      pw[n] = f;
      pl[n] = static_cast<float>(p - static_cast<double>(f));
    }
  }

  const int rb = warp & 3, half = warp >> 2;  // row block and column half of this warp
  const int row = 32 * rb + lane;
  if (kOut && tid < kN) *reinterpret_cast<unsigned *>(smem + OFF_EDGE + 4 * tid) = 0u;
  // chunk x of this thread's half row of a swizzled tile is at tile + (at ^ 16 x)
  const uint32_t at = sm + row * 128u + (((4 * half) ^ (row & 7)) << 4);
  // this thread's part of the state, as MMA3's result is read: pair 2 n + u is row (value channel)
  // i0 + 8 u, columns j0 + 8 n, + 1
  const int i0 = 16 * rb + (lane >> 2), j0 = 32 * half + 2 * (lane & 3);
  const uint32_t at_s = sm + OFF_S + i0 * 128u + 4 * (lane & 3) + (((4 * half) ^ (lane >> 2)) << 4);
  // of w^(L-1-s) v_s in MMA3, the second of two rounded (a choice of two constants: taken as a number, the backward of
  // B2 T4001 H64 took 227 us, 193 so)
  const int terms = kOut && A.terms == 2 ? 2 : 3;
  f32x2 S[8];
  auto put_state = [&]() {  // S in bf16, rows of MMA1's B operand
#pragma unroll
    for (int e = 0; e < 8; ++e) sts32((at_s ^ (16 * (e >> 1))) + 1024 * (e & 1), pack2(S[e]));
  };
  {
    // from where the segments' states are joined already, its slot; else the initial state, and what the
    // segments on the way here add to it
    const bool joined = P.nseg > 1 && P.joined;
    const float *from = !kOut ? nullptr : joined ? A.ws + (pair * P.nseg + z) * (kN * kN) : A.s_in;
    if (kOut && !joined && from != nullptr) from += pair * (kN * kN);
    const int t = !joined && A.s_in_t;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      S[e] = from == nullptr ? make2(0.f, 0.f)
                             : make2(from[state_at(t, i0 + 8 * (e & 1), j0 + 8 * (e >> 1))],
                                     from[state_at(t, i0 + 8 * (e & 1), j0 + 8 * (e >> 1) + 1)]);
    if (kOut && !joined && P.nseg > 1) {
      const double wd = P.w[h];
      const Power wl = power(wd, P.seg_len);
      const int steps = kRev ? sg.n - 1 - z : z;
      for (int s = 1; s <= steps; ++s) {
        const float *u = A.ws + (pair * P.nseg + (kRev ? sg.n - 1 - s : s)) * (kN * kN);
        const Power f = kRev && s == 1 ? power(wd, sg.last_len) : wl;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 x = *reinterpret_cast<const float2 *>(u + (i0 + 8 * (e & 1)) * kN + j0 + 8 * (e >> 1));
          S[e] = fma2(S[e], make2(f.hi, f.hi), fma2(S[e], make2(f.lo, f.lo), make2(x.x, x.y)));
        }
      }
    }
    if (kOut) put_state();
  }
  tc::fence_proxy_async_smem();
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Bounded wait for phase n of a barrier.  After a wait has run out anywhere in the CTA, all others
  // return at once: the warps finish their chunk (on whatever is there, within bounds), so that every
  // named barrier is reached by all, and stop together at its end.
  auto wait = [&](int k, int n) -> bool {
#pragma unroll 1
    for (uint32_t p = 0; p < kMaxPolls; ++p) {
      if (tc::mbar_try_wait(bars + k, n & 1)) return true;
      if ((p & 63u) == 63u && *bad) return false;
    }
    *bad = 1;
    return false;
  };

  const float w1 = lds32(sm + OFF_PW + 4);
  const f32x2 w2 = make2(w1 * w1, w1 * w1);
  // phases under way, for the leading lane to wait out if it has to give up
  int begun[kBars] = {};
  if (nchunks > 0) begun[B_QK] = begun[B_V] = 1;
  const uint32_t tml = tmem + (static_cast<uint32_t>(rb) << 21);  // this warp's lanes
  for (int it = 0; it < nchunks; ++it) {
    const int c = chunk_at(it), L = min(kChunk, sg.len - c * kChunk);
    // rows past the end hold other sequences' tokens: K and V count as zero there (Q's rows give
    // outputs that are not stored)
    const uint32_t zero[4] = {0u, 0u, 0u, 0u};
    // The next V arrives in Q's tile once MMA1 is through with it, the next Q in V's behind MMA2, so the two
    // change places from chunk to chunk.  Without outputs Q's tile is K's second one.
    const uint32_t tile_k = !kOut && (it & 1) ? OFF_Q : OFF_K;
    const uint32_t tile_q = it & 1 ? OFF_V : OFF_Q, tile_v = kOut && (it & 1) ? OFF_Q : OFF_V;
    if (L < kChunk) {
      wait(B_QK, it);
      if (row >= L) {
#pragma unroll
        for (int x = 0; x < 4; ++x) sts128((at ^ (16 * x)) + tile_k, zero);
      }
      tc::fence_proxy_async_smem();
    }
    if (kOut) {
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bars + B_READY);
      if (warp == kLead) {
        if (wait(B_QK, it) && wait(B_READY, it) && elected) {
          tc::tc_fence_after();
          constexpr uint32_t d1 = tc::instr_desc(tc::kFmtBF16, 128, 192, false, false);
          // (offsets within a tile are added to a descriptor's address field, 16 bytes a step: shared memory ends below
          // 2^18, so that nothing carries out of it)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc::mma_ss(0, tmem + TM_P, tc::smem_desc(sm + tile_q, 16, 1024) + ks * 2,
                       tc::smem_desc(sm + OFF_K, 16, 1024) + ks * 2, d1, ks > 0);
          tc::mma_commit(bars + B_M1);
          ++begun[B_M1];
        }
        __syncwarp();
      }
    }

    // V1, V2 (and V3): this thread's half of its token row, scaled and cut into 8-bit pieces
    wait(B_V, it);
    if (row >= L) {
#pragma unroll
      for (int x = 0; x < 4; ++x) sts128((at ^ (16 * x)) + tile_v, zero);
    }
    {
      const float f1 = lds32(sm + OFF_PW + 4 * (kRev ? row + 1 : max(L - 1 - row, 0)));
      const f32x2 f = make2(f1, f1);
      if (kOut && it > 0) {  // V1's tile has been stored from
        if (warp == kStore && elected) {
          bulk_wait_read();
          tc::mbar_arrive(bars + B_OUT);
        }
        wait(B_OUT, it - 1);
      }
      uint32_t in[4];
      lds128(at + tile_v, in);
#pragma unroll 1
      for (int x = 0; x < 64; x += 16) {
        uint32_t p1[4], p2[4], p3[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f32x2 v = mul2(unpack2(in[e]), f);
          p1[e] = high_halves(v);
          const f32x2 r = sub2(v, cut2(v));
          p2[e] = terms == 2 ? pack2(r) : high_halves(r);
          p3[e] = high_halves(sub2(r, cut2(r)));
        }
        if (x < 48) lds128((at ^ (x + 16)) + tile_v, in);
        sts128((at ^ x) + OFF_V1, p1);
        sts128((at ^ x) + OFF_V2, p2);
        if (terms == 3) sts128((at ^ x) + OFF_V3, p3);
      }
    }
    tc::fence_proxy_async_smem();
    tc::tc_fence_before();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bars + B_SPLIT);
    if (warp == kLead) {
      if ((kOut || wait(B_QK, it)) && wait(B_SPLIT, it) && elected) {
        tc::tc_fence_after();
        if (!kOut && it + 1 < nchunks && !*bad) {
          // every warp is through with V and with its waits for these tiles, and MMA3 of the chunk before with
          // the other K
          load(&maps.k, OFF_Q + OFF_K - tile_k, B_QK, it + 1);
          load(&maps.v, OFF_V, B_V, it + 1);
          ++begun[B_QK];
          ++begun[B_V];
        }
        constexpr uint32_t d3 = tc::instr_desc(tc::kFmtBF16, 64, 64, true, true);
        for (int t = 0; t < terms; ++t)
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            tc::mma_ss(0, tmem + TM_X, tc::smem_desc(sm + OFF_V1 + t * kTile, kTile, 1024) + ks * 128,
                       tc::smem_desc(sm + tile_k, kTile, 1024) + ks * 128, d3, t + ks > 0);
        tc::mma_commit(bars + B_M3);
        ++begun[B_M3];
      }
      __syncwarp();
    }

    if (kOut) {
      wait(B_M1, it);
      tc::tc_fence_after();
      if (warp == kLead && elected && it + 1 < nchunks && !*bad) {
        load(&maps.v, tile_q, B_V, it + 1);
        ++begun[B_V];
      }
      // P by column groups of 32: half and half + 2 for a warp, all four for the partner of kLead.  P goes over
      // products that this warp has read: group g to columns 32 (g % 2) + 16 (g / 2) .. + 15.
      // (The powers come from repeated products: tables in shared memory had to wait for MMA3, which takes
      // nearly all of its bandwidth meanwhile.)
      if (warp != kLead) {
#pragma unroll 1
        for (int n = 0; n < 2; ++n) {
          const int g = half + 2 * n;
          const uint32_t to = tml + TM_P + 32 * half + 16 * n;
          float pk[16];
          if (g == rb) {
            float v[32];
            tc::tmem_ld32(tml + TM_P + 32 * g, v);
            diagonal_p<kRev>(v, pk, lane, w1);
          } else if (kRev ? g > rb : g < rb) {
            float v[32];
            tc::tmem_ld32(tml + TM_P + 32 * g, v);
            full_p<kRev>(v, pk, lds32(sm + OFF_PW + 4 * (kRev ? 32 * g - row : row - 32 * g - 31)), w1, w2);
          } else {
#pragma unroll
            for (int x = 0; x < 16; ++x) pk[x] = 0.f;
          }
          tc::tmem_st16(to, pk);
          if (rb == (kLead & 3)) {
#pragma unroll
            for (int x = 0; x < 16; ++x) pk[x] = 0.f;
            tc::tmem_st16(tml + TM_P + 32 * (half ^ 1) + 16 * n, pk);
          }
        }
        tc::tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bars + B_P);
      }
      if (warp == kLead) {
        if (wait(B_P, it) && elected) {
          tc::tc_fence_after();
          constexpr uint32_t d2 = tc::instr_desc(tc::kFmtBF16, 128, 64, false, true);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            tc::mma_ts_bf16(tmem + TM_Y, tmem + TM_P + 32 * ((ks >> 1) & 1) + 16 * (ks >> 2) + 8 * (ks & 1),
                            tc::smem_desc(sm + tile_v, kTile, 1024) + ks * 128, d2,
                            ks > 0);
          tc::mma_commit(bars + B_M2);
          ++begun[B_M2];
        }
        __syncwarp();
      }
    }

    // the state behind this chunk
    wait(B_M3, it);
    tc::tc_fence_after();
    if (kOut && warp == kLead && elected && it + 1 < nchunks && !*bad) {
      load(&maps.k, OFF_K, B_QK, it + 1);
      ++begun[B_QK];
    }
    {
      f32x2 x[8];
      tmem_ld_16x32(tml + TM_X + 32 * half, x);
      const float f1 = lds32(sm + OFF_PW + 4 * L), f2 = lds32(sm + OFF_PL + 4 * L);
      const f32x2 f = make2(f1, f1), fl = make2(f2, f2);
#pragma unroll
      for (int e = 0; e < 8; ++e) S[e] = fma2(S[e], f, fma2(S[e], fl, x[e]));
      if (kOut) {
        // a bad v spoils its whole row of x, a bad k its column: this thread's columns in one row, its other row in one
        float a, b2, c2, d2;
        split2(add2(add2(x[0], x[2]), add2(x[4], x[6])), a, b2);
        split2(x[1], c2, d2);
        if (!(fabsf(a + b2 + c2) <= 3e38f)) *redo = it + 1;
      }
    }
    if (kOut) {
      put_state();
      // out: the state's part and that of the chunk's own tokens
      const float f1 = lds32(sm + OFF_PW + 4 * (kRev ? max(L - 1 - row, 0) : row + 1));
      const f32x2 f = make2(f1, f1);
      float y[32], v[32];
      tc::tmem_ld32(tml + TM_YS + 32 * half, y);
      wait(B_M2, it);
      tc::tc_fence_after();
      if (warp == kLead && elected && it + 1 < nchunks && !*bad) load(&maps.q, tile_v, B_QK, it + 1);
      tc::tmem_ld32(tml + TM_Y + 32 * half, v);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          u[e] = pack2(fma2(make2(y[8 * x + 2 * e], y[8 * x + 2 * e + 1]), f, make2(v[8 * x + 2 * e], v[8 * x + 2 * e + 1])));
        sts128((at ^ (16 * x)) + OFF_V1, u);
      }
      tc::fence_proxy_async_smem();  // the rows of out, and the state
      if (L < kChunk) {
        // not the whole tile: the warp's 32 half rows, 4 lanes to each
        __syncwarp();
        const int r0 = 32 * rb + (lane >> 2), ch = 4 * half + (lane & 3);
        uint16_t *out = A.out + ((sg.lo + c * kChunk + r0) * P.H + h) * kN + 8 * ch;
        const uint32_t from = sm + OFF_V1 + r0 * 128 + ((ch ^ (r0 & 7)) << 4);
        for (int n = 0; r0 + 8 * n < L && n < 4; ++n) {
          uint32_t u[4];
          lds128(from + 1024 * n, u);
          *reinterpret_cast<uint4 *>(out + static_cast<long long>(8 * n) * P.H * kN) = make_uint4(u[0], u[1], u[2], u[3]);
        }
      }
    }
    tc::tc_fence_before();
    if (tid == 0) *stop = *bad;
    named_sync(1, kThreads);
    int stopped, again;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];\n" : "=r"(stopped), "=r"(again) : "r"(sm + OFF_SLOT + 8) : "memory");
    if (stopped) break;
    if (kOut && again == it + 1) {
      const long long first = ((sg.lo + c * kChunk) * P.H + h) * kN;
      redo_out<kRev>(sm, tmem, A.q + first, A.k + first, A.v + first, A.out + first, P.H, L, it + 1);
    }
    if (kOut && L == kChunk && warp == kStore && elected) {
      tma_store_3d(&maps.out, sm + OFF_V1, 0, h, static_cast<int>(sg.lo) + c * kChunk);
      tc::bulk_commit_group();
    }
  }
  if (kOut && warp == kStore && elected) tc::bulk_wait_all();
  if (warp == kLead && elected && *bad) {
    // give up: whatever is still in flight lands first
    report_device_error(err_word, kDevErrTimeout);
    for (int k : {B_QK, B_V, B_M1, B_M3, B_M2})
      if (begun[k] > 0) tc::mbar_wait_bounded(bars + k, (begun[k] - 1) & 1, kMaxPolls);
  }
  const bool ends = kRev ? sg.first : sg.last;
  float *to = !kOut ? A.ws + (pair * P.nseg + (kRev ? z - 1 : z + 1)) * (kN * kN)
              : ends && A.s_out != nullptr ? A.s_out + pair * (kN * kN) : nullptr;
  if (to != nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float x, y;
      split2(S[e], x, y);
      to[state_at(kOut && A.s_out_t, i0 + 8 * (e & 1), j0 + 8 * (e >> 1))] = x;
      to[state_at(kOut && A.s_out_t, i0 + 8 * (e & 1), j0 + 8 * (e >> 1) + 1)] = y;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == kLead) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

struct AllMaps {
  Maps m[3];
};

// blockIdx = (head, batch row, pass and segment); the passes for the states alone leave out the segment
// that none continues from.
template <bool kOut>
__global__ void __launch_bounds__(kThreads, 2) linattn_chunk_kernel(const __grid_constant__ AllMaps maps,
                                                                    const __grid_constant__ Passes<uint16_t> A,
                                                                    const Shape P, int *err_word) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ int lens[kMaxSorted + 1];
  pdl_wait();
  pdl_trigger();
  const int b = sorted_row(P, blockIdx.y, gridDim.y, lens);
  const int nz = kOut ? P.nseg : P.nseg - 1, role = blockIdx.z / nz, z = blockIdx.z - role * nz;
  if (A.p[role].reverse)
    walk<true, kOut>(maps.m[role], A.p[role], P, b, kOut ? z : z + 1, smem_raw, err_word);
  else
    walk<false, kOut>(maps.m[role], A.p[role], P, b, z, smem_raw, err_word);
}

using PFN_encodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                     const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                                     CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                     CUtensorMapFloatOOBfill);

static PFN_encodeTiled encoder() {
  static const PFN_encodeTiled fn = []() -> PFN_encodeTiled {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_encodeTiled>(p);
    return nullptr;
  }();
  return fn;
}

static bool make_map(CUtensorMap *map, const void *base, long long tokens, int H) {
  const PFN_encodeTiled enc = encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kN), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kN) * 2, static_cast<cuuint64_t>(H) * kN * 2};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(kN), 1, static_cast<cuuint32_t>(kChunk)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace lin

cudaError_t launch_linattn_chunk(const lin::Passes<uint16_t> &A, const lin::Shape &P, int B, int *err_word,
                                 cudaStream_t stream) {
  using namespace lin;
  const int nz = A.state_only ? P.nseg - 1 : P.nseg;
  if (nz <= 0) return cudaSuccess;
  AllMaps maps;
  for (int i = 0; i < A.n; ++i) {
    const Pass<uint16_t> &p = A.p[i];
    Maps &m = maps.m[i];
    // a call for the states alone loads no q and stores no out: any valid map does
    if (!make_map(&m.k, p.k, P.total_T, P.H) || !make_map(&m.v, p.v, P.total_T, P.H) ||
        !make_map(&m.q, A.state_only ? p.k : p.q, P.total_T, P.H) ||
        !make_map(&m.out, A.state_only ? p.k : p.out, P.total_T, P.H))
      return cudaErrorInvalidValue;
  }
  auto run = [&](auto kern) -> cudaError_t {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
    if (e != cudaSuccess) return e;
    return launch_waiting(kern, dim3(P.H, B, nz * A.n), kThreads, kSmemBytes, stream, maps, A, P, err_word);
  };
  return A.state_only ? run(linattn_chunk_kernel<false>) : run(linattn_chunk_kernel<true>);
}

}  // namespace rwkv7
