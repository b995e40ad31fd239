// linattn_decode.cu -- one token of the head-decay linear attention for every (b, h), state in place:
//   S <- w S + v k^T,  y = S r.
// Bound by HBM: each pair reads and writes its 16 KiB state once.  One CTA of 256 threads per pair;
// thread t holds columns 4 (t % 16) .. + 3 of rows t / 16 + 16 m, so the four 16-byte state loads are
// in flight together and the row sums of y take four shuffles inside 16 lanes.
#include "linattn.h"

namespace rwkv7 {
namespace lin {

template <typename TIn>
__global__ void __launch_bounds__(256) linattn_decode_kernel(const TIn *r, const TIn *k, const TIn *v, const float *w,
                                                             float *s, TIn *y, int H) {
  const long long pair = blockIdx.x;
  const int tid = threadIdx.x, c4 = 4 * (tid & 15), rg = tid >> 4;
  // the previous grid on the stream may still run: nothing is read before it has finished, and the
  // next one is let in only then, so that no more than two grids are ever in flight here
  pdl_wait();
  pdl_trigger();
  float *S = s + pair * (kN * kN) + rg * kN + c4;
  float4 st[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) st[m] = *reinterpret_cast<const float4 *>(S + 16 * m * kN);
  float kk[4], rr[4], vv[4], p[4];
  Elem<TIn>::load4(k + pair * kN + c4, kk);
  Elem<TIn>::load4(r + pair * kN + c4, rr);
#pragma unroll
  for (int m = 0; m < 4; ++m) vv[m] = Elem<TIn>::load(v + pair * kN + rg + 16 * m);
  const float wh = w[static_cast<int>(pair % H)];
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    float4 x = st[m];
    x.x = fmaf(x.x, wh, vv[m] * kk[0]);
    x.y = fmaf(x.y, wh, vv[m] * kk[1]);
    x.z = fmaf(x.z, wh, vv[m] * kk[2]);
    x.w = fmaf(x.w, wh, vv[m] * kk[3]);
    *reinterpret_cast<float4 *>(S + 16 * m * kN) = x;
    p[m] = fmaf(x.x, rr[0], x.y * rr[1]) + fmaf(x.z, rr[2], x.w * rr[3]);
  }
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1)
#pragma unroll
    for (int m = 0; m < 4; ++m) p[m] += __shfl_xor_sync(0xffffffffu, p[m], off);
  if ((tid & 15) == 0) {
#pragma unroll
    for (int m = 0; m < 4; ++m) Elem<TIn>::store(y + pair * kN + rg + 16 * m, p[m]);
  }
}

}  // namespace lin

template <typename TIn>
cudaError_t launch_linattn_decode(const TIn *r, const TIn *k, const TIn *v, const float *w, float *s, TIn *y, int B,
                                  int H, cudaStream_t stream) {
  const long long pairs = static_cast<long long>(B) * H;
  if (pairs > 0x7fffffffLL) return cudaErrorInvalidValue;
  return lin::launch_waiting(lin::linattn_decode_kernel<TIn>, dim3(static_cast<unsigned>(pairs)), 256, 0, stream, r, k,
                             v, w, s, y, H);
}

template cudaError_t launch_linattn_decode<float>(const float *, const float *, const float *, const float *, float *,
                                                  float *, int, int, cudaStream_t);
template cudaError_t launch_linattn_decode<uint16_t>(const uint16_t *, const uint16_t *, const uint16_t *,
                                                     const float *, float *, uint16_t *, int, int, cudaStream_t);

}  // namespace rwkv7
