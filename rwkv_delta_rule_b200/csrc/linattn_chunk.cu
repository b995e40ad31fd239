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
// Only powers w^0 .. w^128 of the head's decay appear, all <= 1, so every w in [0, 1] is exact.
//
// One CTA of 128 threads walks the chunks of one (b, h) (or of one segment of it); thread t owns token
// row t and TMEM lane t.  Per chunk, on the tensor cores with float32 accumulation:
//     MMA1  [128 x 128] = Q K^T                      Q, K as TMA left them (K-major)
//     MMA2  [128 x 64]  = Q S0^T                     S0 in two bf16 terms
//     MMA3  [128 x 64]  = P V                        P from TMEM in bf16, V as TMA left it (MN-major)
//     MMA4  [128 x 64]  = [V'; V''] K (+ V''' twice)   V' = w^(L-1-s) v_s, see below
// The state stays in float32 registers across chunks (32 elements per thread).  Roundings to bf16:
//   P: one per product, as large as the rounding of out itself, and averaged over the tokens;
//   S0 in MMA2: hi + lo, 2^-17 of each element; it reaches out only;
//   w^(L-1-s) v_s in MMA4: hi + mid + lo (2^-25), because these sums are the state: two terms were
//   2.7e-6 off on average, three are within float32's own rounding.  hi and mid are the two halves of
//   MMA4's 128 rows; half of lo is added to both by a second pass, and the halves are added in float32.
// k, q and v enter their products as they are, exactly.
#include <cuda.h>

#include "linattn.h"
#include "tc_ptx.cuh"

namespace rwkv7 {
namespace lin {

constexpr int kChunk = 128;
constexpr int kThreads = 128;
constexpr uint32_t kMaxPolls = 1u << 22;
constexpr uint32_t kTile = kChunk * kN * 2;  // one bf16 128 x 64 tile, 128-byte swizzled rows

// TMEM columns: MMA1's result; P (bf16 pairs) replaces its first half as it is read, MMA3's result its second
constexpr uint32_t TM_P = 0, TM_Y1 = 64, TM_Y2 = 128, TM_X = 192, kTmemCols = 256;

// shared memory, from a 1024-aligned base.  Q's tile takes V''' once MMA1 and MMA2 are through with it;
// V' is where the threads swap halves of MMA4's result afterwards, V'' where out waits for its TMA store.
constexpr uint32_t OFF_Q = 0, OFF_K = kTile, OFF_V = 2 * kTile, OFF_V1 = 3 * kTile, OFF_V2 = 4 * kTile;
constexpr uint32_t OFF_S = 5 * kTile;                // hi, then lo: [64 value channels][64 key channels]
constexpr uint32_t kStateTile = kN * kN * 2;
constexpr uint32_t OFF_PW = OFF_S + 2 * kStateTile;  // float2 [129]: w^n as a float32 and what that leaves
constexpr uint32_t OFF_BAR = OFF_PW + 1040;          // three mbarriers, TMEM address, abort flag
constexpr uint32_t kSmemBytes = OFF_BAR + 64 + 1024;

struct Maps {
  CUtensorMap q, k, v, out;  // [tokens, H, 64] bf16, box {64, 1, 128}
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float lo_of(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float hi_of(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory"); }
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *smem_src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];\n" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(smem_src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

template <bool kRev, bool kOut>
__global__ void __launch_bounds__(kThreads, 2) linattn_chunk_kernel(const __grid_constant__ Maps maps,
                                                                    const Pass<uint16_t> A, const Shape P,
                                                                    int *err_word) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int h = blockIdx.x, b = blockIdx.y, z = blockIdx.z + (!kOut && kRev ? 1 : 0);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  const Segment sg = segment(P, b, z);
  if (sg.len < 0) return;
  if (!kOut && (kRev ? sg.first : sg.last)) return;
  const long long pair = static_cast<long long>(b) * P.H + h;

  float2 *pw = reinterpret_cast<float2 *>(smem + OFF_PW);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + OFF_BAR);  // tiles landed, MMA1 + MMA2 done, MMA3 + MMA4 done
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + OFF_BAR + 32);
  volatile int *bad = reinterpret_cast<volatile int *>(smem + OFF_BAR + 40);

  const int nchunks = (sg.len + kChunk - 1) / kChunk;
  auto chunk_at = [&](int i) { return kRev ? nchunks - 1 - i : i; };
  auto load_tiles = [&](int c) {
    const int tok = static_cast<int>(sg.lo) + c * kChunk;
    tc::mbar_arrive_expect_tx(bars, (kOut ? 3 : 2) * kTile);
    tc::tma_load_3d(smem + OFF_K, &maps.k, bars, 0, h, tok);
    if (kOut) tc::tma_load_3d(smem + OFF_Q, &maps.q, bars, 0, h, tok);
    tc::tma_load_3d(smem + OFF_V, &maps.v, bars, 0, h, tok);
  };
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) tc::mbar_init(bars + i, 1);
    tc::fence_mbar_init();
    *bad = 0;
    if (nchunks > 0) load_tiles(chunk_at(0));
  }
  if (warp == 0) {
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  for (int n = tid; n <= kChunk; n += kThreads) {
    const double p = powi(static_cast<double>(P.w[h]), n);
    const float f = static_cast<float>(p);
    pw[n] = make_float2(f, static_cast<float>(p - static_cast<double>(f)));
  }

  // this thread's part of the state: row i (value channel), columns 32 half .. + 31
  const int i = tid & 63, half = tid >> 6;
  float S[32];
  {
    const float *from = !kOut ? nullptr : P.nseg > 1 ? A.ws + (pair * P.nseg + z) * (kN * kN) : A.s_in;
    if (kOut && P.nseg == 1 && from != nullptr) from += pair * (kN * kN);
    const int t = P.nseg == 1 && A.s_in_t;
#pragma unroll
    for (int e = 0; e < 32; ++e) S[e] = from == nullptr ? 0.f : from[state_at(t, i, 32 * half + e)];
  }
  auto put_state = [&]() {  // S as two bf16 terms, the B operand of MMA2
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = S[8 * c + 2 * e], y = S[8 * c + 2 * e + 1];
        hi[e] = pack2(x, y);
        lo[e] = pack2(x - lo_of(hi[e]), y - hi_of(hi[e]));
      }
      uint8_t *p = smem + OFF_S + tc::sw128(i, 4 * half + c);
      *reinterpret_cast<uint4 *>(p) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4 *>(p + kStateTile) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  };
  if (kOut) put_state();
  tc::fence_proxy_async_smem();
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tml = tmem + (static_cast<uint32_t>(warp) << 21);  // this warp's lanes
  const uint32_t sQ = smem_u32(smem + OFF_Q), sK = smem_u32(smem + OFF_K), sV = smem_u32(smem + OFF_V);
  const uint32_t sV1 = smem_u32(smem + OFF_V1), sS = smem_u32(smem + OFF_S);
  int waited[3] = {0, 0, 0}, begun[3] = {nchunks > 0 ? 1 : 0, 0, 0};  // phases of the barriers (begun: thread 0's view)
  auto wait = [&](int k) {
    if (!tc::mbar_wait_bounded(bars + k, waited[k] & 1, kMaxPolls)) {
      *bad = 1;
      return;
    }
    ++waited[k];
  };

  for (int it = 0; it < nchunks; ++it) {
    const int c = chunk_at(it), L = min(kChunk, sg.len - c * kChunk);
    wait(0);
    if (L < kChunk) {
      // rows past the end hold other sequences' tokens: K and V count as zero there (Q's rows give
      // outputs that are not stored)
      if (tid >= L) {
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          *reinterpret_cast<uint4 *>(smem + OFF_K + tid * 128 + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4 *>(smem + OFF_V + tid * 128 + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      tc::fence_proxy_async_smem();
      __syncthreads();
    }
    if (kOut) {
      if (tid == 0 && !*bad) {
        tc::tc_fence_after();
        constexpr uint32_t d1 = tc::instr_desc(tc::kFmtBF16, 128, 128, false, false);
        constexpr uint32_t d2 = tc::instr_desc(tc::kFmtBF16, 128, 64, false, false);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          tc::mma_ss(0, tmem + TM_P, tc::smem_desc(sQ + ks * 32, 16, 1024), tc::smem_desc(sK + ks * 32, 16, 1024), d1,
                     ks > 0);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          tc::mma_ss(0, tmem + TM_Y2, tc::smem_desc(sQ + (ks & 3) * 32, 16, 1024),
                     tc::smem_desc(sS + (ks >> 2) * kStateTile + (ks & 3) * 32, 16, 1024), d2, ks > 0);
        tc::mma_commit(bars + 1);
        begun[1]++;
      }
      // the last chunk's outputs have left V''
      if (tid == 0) bulk_wait_read();
      __syncthreads();
      if (*bad) break;
    }

    // V', V'' and V''': token row tid scaled and split
    uint32_t third[32];
    {
      const float f = pw[kRev ? min(tid + 1, kChunk) : max(L - 1 - tid, 0)].x;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const uint32_t at = tc::sw128(tid, x);
        const uint4 u = *reinterpret_cast<const uint4 *>(smem + OFF_V + at);
        const uint32_t in[4] = {u.x, u.y, u.z, u.w};
        uint32_t p1[4], p2[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float a = lo_of(in[e]) * f, bb = hi_of(in[e]) * f;
          p1[e] = pack2(a, bb);
          a -= lo_of(p1[e]);
          bb -= hi_of(p1[e]);
          p2[e] = pack2(a, bb);
          third[4 * x + e] = pack2(0.5f * (a - lo_of(p2[e])), 0.5f * (bb - hi_of(p2[e])));
        }
        *reinterpret_cast<uint4 *>(smem + OFF_V1 + at) = make_uint4(p1[0], p1[1], p1[2], p1[3]);
        *reinterpret_cast<uint4 *>(smem + OFF_V2 + at) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
      }
    }
    if (kOut) {
      wait(1);
      tc::tc_fence_after();
    }
#pragma unroll
    for (int x = 0; x < 8; ++x)
      *reinterpret_cast<uint4 *>(smem + OFF_Q + tc::sw128(tid, x)) =
          make_uint4(third[4 * x], third[4 * x + 1], third[4 * x + 2], third[4 * x + 3]);
    if (kOut) {
      // P, 32 columns at a time: P's columns are behind those still to be read
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float pk[16];
        if (g == warp || (kRev ? g > warp : g < warp)) {
          float v[32];
          tc::tmem_ld32(tml + TM_P + 32 * g, v);
          if (g == warp) {
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const int d = kRev ? x - lane : lane - x;
              v[x] = d >= 0 ? v[x] * pw[d].x : 0.f;
            }
          } else {
            // w^(t-s) = w^(t - 32 g - 31) w^(31 - x), reversed w^(s-t) = w^(32 g - t) w^x
            const float a = pw[kRev ? 32 * g - tid : tid - 32 * g - 31].x;
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] = v[x] * a * pw[kRev ? x : 31 - x].x;
          }
#pragma unroll
          for (int x = 0; x < 16; ++x) pk[x] = __uint_as_float(pack2(v[2 * x], v[2 * x + 1]));
        } else {
#pragma unroll
          for (int x = 0; x < 16; ++x) pk[x] = 0.f;
        }
        tc::tmem_st16(tml + TM_P + 16 * g, pk);
      }
      tc::tmem_st_wait();
      tc::tc_fence_before();
    }
    tc::fence_proxy_async_smem();
    __syncthreads();
    if (*bad) break;
    if (tid == 0) {
      tc::tc_fence_after();
      constexpr uint32_t d3 = tc::instr_desc(tc::kFmtBF16, 128, 64, false, true);
      constexpr uint32_t d4 = tc::instr_desc(tc::kFmtBF16, 128, 64, true, true);
      if (kOut) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          tc::mma_ts_bf16(tmem + TM_Y1, tmem + TM_P + 8 * ks, tc::smem_desc(sV + ks * 2048, kTile, 1024), d3, ks > 0);
      }
#pragma unroll
      for (int ks = 0; ks < 16; ++ks)  // V' over V''; then V''' over itself (block stride 0)
        tc::mma_ss(0, tmem + TM_X, tc::smem_desc((ks < 8 ? sV1 : sQ) + (ks & 7) * 2048, ks < 8 ? kTile : 0, 1024),
                   tc::smem_desc(sK + (ks & 7) * 2048, kTile, 1024), d4, ks > 0);
      tc::mma_commit(bars + 2);
      begun[2]++;
    }
    float y[64];
    if (kOut) {
      // meanwhile the state's part of the outputs
      const float f = pw[kRev ? max(L - 1 - tid, 0) : tid + 1].x;
      float v[32];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        tc::tmem_ld32(tml + TM_Y2 + 32 * g, v);
#pragma unroll
        for (int x = 0; x < 32; ++x) y[32 * g + x] = v[x] * f;
      }
    }
    wait(2);
    tc::tc_fence_after();
    if (tid == 0 && it + 1 < nchunks && !*bad) {
      load_tiles(chunk_at(it + 1));
      begun[0]++;
    }
    {
      // the two halves of MMA4: this thread keeps its 32 columns and swaps the others with tid ^ 64
      float mine[32], other[32];
      tc::tmem_ld32(tml + TM_X + 32 * half, mine);
      tc::tmem_ld32(tml + TM_X + 32 * (half ^ 1), other);
#pragma unroll
      for (int x = 0; x < 8; ++x)
        *reinterpret_cast<float4 *>(smem + OFF_V1 + tc::sw128(tid, x)) =
            make_float4(other[4 * x], other[4 * x + 1], other[4 * x + 2], other[4 * x + 3]);
      if (kOut) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float v[32];
          tc::tmem_ld32(tml + TM_Y1 + 32 * g, v);
#pragma unroll
          for (int x = 0; x < 32; ++x) y[32 * g + x] += v[x];
        }
        uint16_t *row = A.out + ((sg.lo + c * kChunk + tid) * P.H + h) * kN;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const uint4 u = make_uint4(pack2(y[8 * x], y[8 * x + 1]), pack2(y[8 * x + 2], y[8 * x + 3]),
                                     pack2(y[8 * x + 4], y[8 * x + 5]), pack2(y[8 * x + 6], y[8 * x + 7]));
          if (L == kChunk)
            *reinterpret_cast<uint4 *>(smem + OFF_V2 + tc::sw128(tid, x)) = u;
          else if (tid < L)
            reinterpret_cast<uint4 *>(row)[x] = u;
        }
      }
      tc::fence_proxy_async_smem();
      __syncthreads();
      if (kOut && tid == 0 && L == kChunk) {
        tma_store_3d(&maps.out, smem + OFF_V2, 0, h, static_cast<int>(sg.lo) + c * kChunk);
        tc::bulk_commit_group();
      }
      const float2 f = pw[L];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const float4 u = *reinterpret_cast<const float4 *>(smem + OFF_V1 + tc::sw128(tid ^ 64, x));
        const float o[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) S[4 * x + e] = fmaf(S[4 * x + e], f.x, fmaf(S[4 * x + e], f.y, mine[4 * x + e] + o[e]));
      }
      if (kOut) put_state();
      tc::fence_proxy_async_smem();
      tc::tc_fence_before();
      __syncthreads();
      if (*bad) break;
    }
  }

  if (*bad && tid == 0) {
    // give up: whatever is still in flight lands first
    report_device_error(err_word, kDevErrTimeout);
    for (int k = 0; k < 3; ++k)
      while (waited[k] < begun[k] && tc::mbar_wait_bounded(bars + k, waited[k] & 1, kMaxPolls)) ++waited[k];
  }
  if (tid == 0) tc::bulk_wait_all();
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc(tmem, kTmemCols);

  const bool ends = kRev ? sg.first : sg.last;
  float *to = !kOut ? A.ws + (pair * P.nseg + (kRev ? z - 1 : z + 1)) * (kN * kN)
              : ends && A.s_out != nullptr ? A.s_out + pair * (kN * kN) : nullptr;
  if (to != nullptr) {
#pragma unroll
    for (int e = 0; e < 32; ++e) to[state_at(kOut && A.s_out_t, i, 32 * half + e)] = S[e];
  }
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

cudaError_t launch_linattn_chunk(const lin::Pass<uint16_t> &A, const lin::Shape &P, int B, int *err_word,
                                 cudaStream_t stream) {
  using namespace lin;
  const int nz = A.state_only ? P.nseg - 1 : P.nseg;
  if (nz <= 0) return cudaSuccess;
  Maps maps;
  // a call without outputs loads no q and stores nothing: any valid map does
  if (!make_map(&maps.k, A.k, P.total_T, P.H) || !make_map(&maps.v, A.v, P.total_T, P.H) ||
      !make_map(&maps.q, A.state_only ? A.k : A.q, P.total_T, P.H) ||
      !make_map(&maps.out, A.state_only ? static_cast<const void *>(A.k) : A.out, P.total_T, P.H))
    return cudaErrorInvalidValue;
  auto run = [&](auto kern) -> cudaError_t {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
    if (e != cudaSuccess) return e;
    kern<<<dim3(P.H, B, nz), kThreads, kSmemBytes, stream>>>(maps, A, P, err_word);
    return cudaGetLastError();
  };
  if (A.state_only) return A.reverse ? run(linattn_chunk_kernel<true, false>) : run(linattn_chunk_kernel<false, false>);
  return A.reverse ? run(linattn_chunk_kernel<true, true>) : run(linattn_chunk_kernel<false, true>);
}

}  // namespace rwkv7
