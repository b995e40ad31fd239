// linattn_api.cu -- the extern "C" entry points of the head-decay linear attention and of the layer
// norm (include/rwkv7.h): host-side checks, the split of a sequence into segments, launches.
#include "../../include/rwkv7.h"
#include "common.cuh"
#include "launch.h"
#include "layer_norm.h"
#include "linattn.h"

namespace rwkv7 {
namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <typename... P> bool all_aligned(const P *...ps) { return (aligned16(ps) && ...); }
template <typename... P> bool none_null(const P *...ps) { return ((ps != nullptr) && ...); }
rwkv7_status from_cuda(cudaError_t e) { return e == cudaSuccess ? RWKV7_OK : RWKV7_ERR_CUDA; }

constexpr long long kStateBytes = kN * kN * sizeof(float);

// bf16 passes run on the tensor cores from this length on.  Measured on B200 (token by token / tensor cores,
// us): B1 H12 T16 4.8 / 6.1, T32 9.1 / 6.1; B8 H12 T32 9.3 / 6.4; B64 H32 T32 48 / 52, T40 59 / 52; B256 H16
// T32 93 / 102, T40 114 / 102.
constexpr long long kChunkMinT = 32;
template <typename TIn> bool use_chunk(long long max_T) { return sizeof(TIn) == 2 && max_T >= kChunkMinT; }

// Segments a sequence of at most T tokens is split into, for `chains` sequences that run side by side: as
// many as fill the CTAs that the device runs at once (2 per SM on the tensor cores, 7 of the token-by-token
// kernel; float32 B4 T1000 H12 87 us with 4, 62 with 7), of whole chunks, or of 24 tokens, 48 tokens staying
// whole (float32 B1 H12: T1000 45 us in segments of 96 tokens, 33 of 32; T64 13.3 whole, 12.5 in three;
// bf16 T32 9.1 whole, 9.7 in two).  Lengths are multiples of 8 tokens, of 128 on the tensor cores.
int segments(long long chains, long long T, bool chunk) {
  const long long want = (chunk ? 296 : 1036) / chains, most = chunk ? T / 128 : T <= 48 ? 1 : (T + 23) / 24;
  const long long n = want < most ? want : most;
  return n < 1 ? 1 : static_cast<int>(n);
}
// Workspace of one pass: a state per segment and pair where there is more than one segment.
long long pass_bytes(long long pairs, int nseg) { return nseg > 1 ? pairs * nseg * kStateBytes : 0; }

long long workspace(int B, int max_T, int H, int passes) {
  if (B <= 0 || H <= 0 || max_T <= 0) return 0;
  const long long pairs = static_cast<long long>(B) * H;
  const int a = segments(passes * pairs, max_T, false), b = segments(passes * pairs, max_T, true);
  return passes * pass_bytes(pairs, a > b ? a : b);
}

// Splits for the workspace given: fewer segments where it holds no more.
lin::Shape shape(const float *w, const int32_t *cu, int B, int T, long long total_T, long long max_T, int H,
                 long long bytes, int passes, bool chunk) {
  const long long pairs = static_cast<long long>(B) * H;
  int n = segments(passes * pairs, max_T, chunk);
  const long long room = bytes / (passes * pairs * kStateBytes);
  if (n > room) n = room < 2 ? 1 : static_cast<int>(room);
  const long long u = chunk ? 128 : 8, len = ((max_T + n - 1) / n + u - 1) / u * u;
  if (n > 1) n = static_cast<int>((max_T + len - 1) / len);
  return lin::Shape{w, cu, T, total_T, H, n, 1, n > 1 ? static_cast<int>(len) : 0x7fffff80};
}

template <typename TIn> cudaError_t one_sweep(const lin::Passes<TIn> &p, const lin::Shape &s, int B, bool chunk,
                                              cudaStream_t stream) {
  if constexpr (sizeof(TIn) == 2) {
    if (chunk) return launch_linattn_chunk(p, s, B, device_error_word(), stream);
  }
  return launch_linattn_scan(p, s, B, stream);
}

// Up to this many segments the tensor-core pass joins their states itself, in place of a launch between
// (B8 T4096 H12, 3 segments: 66.5 us against 75.7); each CTA then reads the 16 KB of every segment before its
// own.
constexpr int kOwnJoin = 8;

template <typename TIn> cudaError_t run_passes(const lin::Passes<TIn> &p, lin::Shape s, int B, bool chunk,
                                               cudaStream_t stream) {
  if (s.nseg > 1) {
    lin::Passes<TIn> states = p;
    states.state_only = 1;
    const cudaError_t e = one_sweep(states, s, B, chunk, stream);
    if (e != cudaSuccess) return e;
    // a state written in place must have been read by every segment before any of them ends
    bool in_place = false;
    for (int i = 0; i < p.n; ++i)
      for (int j = 0; j < p.n; ++j) in_place = in_place || (p.p[i].s_in != nullptr && p.p[i].s_in == p.p[j].s_out);
    s.joined = !chunk || s.nseg > kOwnJoin || in_place;
    if (s.joined) {
      const cudaError_t f = launch_linattn_join(states, s, B, stream);
      if (f != cudaSuccess) return f;
    }
  }
  return one_sweep(p, s, B, chunk, stream);
}

template <typename TIn>
rwkv7_status check(int B, long long tokens, int H, int N, const TIn *r, const TIn *k, const TIn *v, const float *w,
                   const float *s_in, const TIn *y, const float *s_out, const void *ws, long long ws_bytes) {
  if (N != kN) return RWKV7_ERR_UNSUPPORTED;
  if (B <= 0 || H <= 0 || tokens < 0 || B > 65535 || H > 65535 || ws_bytes < 0) return RWKV7_ERR_INVALID;
  if (w == nullptr || s_out == nullptr || (ws == nullptr && ws_bytes > 0)) return RWKV7_ERR_INVALID;
  if (tokens > 0 && !none_null(r, k, v, y)) return RWKV7_ERR_INVALID;
  if (tokens > 0x7fffffffLL) return RWKV7_ERR_INVALID;
  if (!all_aligned(r, k, v, y) || !all_aligned(w, s_in, s_out) || !aligned16(ws)) return RWKV7_ERR_ALIGN;
  return RWKV7_OK;
}

template <typename TIn>
rwkv7_status prefill(int B, int T, long long total_T, long long max_T, int H, int N, const int32_t *cu, const TIn *r,
                     const TIn *k, const TIn *v, const float *w, const float *s_in, TIn *y, float *s_out, void *ws,
                     long long ws_bytes, rwkv7_stream_t stream) {
  const rwkv7_status st = check(B, total_T, H, N, r, k, v, w, s_in, y, s_out, ws, ws_bytes);
  if (st != RWKV7_OK) return st;
  if (total_T == 0) max_T = 0;
  const bool chunk = use_chunk<TIn>(max_T);
  const lin::Shape s = shape(w, cu, B, T, total_T, max_T, H, ws_bytes, 1, chunk);
  const lin::Passes<TIn> p{{{r, k, v, y, s_in, s_out, 0, 0, static_cast<float *>(ws), 0, 3}}, 1, 0};
  return from_cuda(run_passes(p, s, B, chunk, reinterpret_cast<cudaStream_t>(stream)));
}

template <typename TIn>
rwkv7_status decode(int B, int H, int N, const TIn *r, const TIn *k, const TIn *v, const float *w, float *s, TIn *y,
                    rwkv7_stream_t stream) {
  if (N != kN) return RWKV7_ERR_UNSUPPORTED;
  if (B <= 0 || H <= 0 || !none_null(r, k, v, y) || !none_null(w, s)) return RWKV7_ERR_INVALID;
  if (!all_aligned(r, k, v, y) || !all_aligned(w, s)) return RWKV7_ERR_ALIGN;
  return from_cuda(launch_linattn_decode(r, k, v, w, s, y, B, H, reinterpret_cast<cudaStream_t>(stream)));
}

bool norm_sizes(int M, int G, int D) {
  return M >= 0 && G > 0 && D > 0 && static_cast<long long>(M) * G <= 0x7fffffffLL &&
         static_cast<long long>(G) * D <= (1LL << 24);
}

template <typename TIn>
rwkv7_status norm(int M, int G, int D, float eps, const TIn *x, const float *w, const float *b, TIn *y, float *mean,
                  float *rstd, rwkv7_stream_t stream) {
  if (!norm_sizes(M, G, D) || !(eps >= 0.f)) return RWKV7_ERR_INVALID;
  if (M > 0 && !none_null(x, y)) return RWKV7_ERR_INVALID;
  if (!all_aligned(x, y) || !all_aligned(w, b, mean, rstd)) return RWKV7_ERR_ALIGN;
  return from_cuda(launch_layer_norm(x, w, b, eps, y, mean, rstd, M, G, D, reinterpret_cast<cudaStream_t>(stream)));
}

template <typename TIn>
rwkv7_status norm_backward(int M, int G, int D, const TIn *dy, const TIn *x, const float *w, const float *mean,
                           const float *rstd, TIn *dx, float *dw, float *db, void *ws, long long ws_bytes,
                           rwkv7_stream_t stream) {
  if (!norm_sizes(M, G, D)) return RWKV7_ERR_INVALID;
  if (M > 0 && (!none_null(dy, x, dx) || !none_null(mean, rstd))) return RWKV7_ERR_INVALID;
  if ((dw == nullptr) != (db == nullptr)) return RWKV7_ERR_INVALID;
  const long long need = dw != nullptr ? layer_norm_partial_bytes(sizeof(TIn), M, G, D) : 0;
  if (ws_bytes < need || (need > 0 && ws == nullptr)) return RWKV7_ERR_INVALID;
  if (!all_aligned(dy, x, dx) || !all_aligned(w, mean, rstd, dw, db) || !aligned16(ws)) return RWKV7_ERR_ALIGN;
  return from_cuda(launch_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, static_cast<float *>(ws), M, G, D,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace rwkv7

using namespace rwkv7;

extern "C" {

long long rwkv7_linattn_workspace(int B, int max_T, int H) { return workspace(B, max_T, H, 1); }

long long rwkv7_linattn_backward_workspace(int B, int T, int H) { return workspace(B, T, H, 3); }

rwkv7_status rwkv7_linattn_prefill(int B, int T, int H, int N, const float *r, const float *k, const float *v,
                                   const float *w, const float *s_in, float *y, float *s_out, void *workspace,
                                   long long workspace_bytes, rwkv7_stream_t stream) {
  if (T < 0) return RWKV7_ERR_INVALID;
  return prefill(B, T, static_cast<long long>(B) * T, T, H, N, nullptr, r, k, v, w, s_in, y, s_out, workspace,
                 workspace_bytes, stream);
}

rwkv7_status rwkv7_linattn_prefill_bf16(int B, int T, int H, int N, const uint16_t *r, const uint16_t *k,
                                        const uint16_t *v, const float *w, const float *s_in, uint16_t *y,
                                        float *s_out, void *workspace, long long workspace_bytes,
                                        rwkv7_stream_t stream) {
  if (T < 0) return RWKV7_ERR_INVALID;
  return prefill(B, T, static_cast<long long>(B) * T, T, H, N, nullptr, r, k, v, w, s_in, y, s_out, workspace,
                 workspace_bytes, stream);
}

rwkv7_status rwkv7_linattn_prefill_varlen_bf16(int B, int total_T, int max_T, int H, int N, const int32_t *cu_seqlens,
                                               const uint16_t *r, const uint16_t *k, const uint16_t *v, const float *w,
                                               const float *s_in, uint16_t *y, float *s_out, void *workspace,
                                               long long workspace_bytes, rwkv7_stream_t stream) {
  if (max_T < 0 || cu_seqlens == nullptr) return RWKV7_ERR_INVALID;
  if (!aligned16(cu_seqlens)) return RWKV7_ERR_ALIGN;
  return prefill(B, 0, total_T, max_T, H, N, cu_seqlens, r, k, v, w, s_in, y, s_out, workspace, workspace_bytes,
                 stream);
}

rwkv7_status rwkv7_linattn_decode(int B, int H, int N, const float *r, const float *k, const float *v, const float *w,
                                  float *s_inout, float *y, rwkv7_stream_t stream) {
  return decode(B, H, N, r, k, v, w, s_inout, y, stream);
}

rwkv7_status rwkv7_linattn_decode_bf16(int B, int H, int N, const uint16_t *r, const uint16_t *k, const uint16_t *v,
                                       const float *w, float *s_inout, uint16_t *y, rwkv7_stream_t stream) {
  return decode(B, H, N, r, k, v, w, s_inout, y, stream);
}

rwkv7_status rwkv7_linattn_backward_bf16(int B, int T, int H, int N, const uint16_t *r, const uint16_t *k,
                                         const uint16_t *v, const float *w, const float *s_in, const uint16_t *dy,
                                         const float *ds_out, uint16_t *dr, uint16_t *dk, uint16_t *dv, float *ds_in,
                                         void *workspace, long long workspace_bytes, rwkv7_stream_t stream) {
  if (N != kN) return RWKV7_ERR_UNSUPPORTED;
  if (T < 0) return RWKV7_ERR_INVALID;
  const long long tokens = static_cast<long long>(B) * T;
  const float *any = ds_in != nullptr ? ds_in : w;  // ds_in may be left out
  const rwkv7_status st = check(B, tokens, H, N, r, k, v, w, s_in, dr, any, workspace, workspace_bytes);
  if (st != RWKV7_OK) return st;
  if (tokens > 0 && !none_null(dy, dk, dv)) return RWKV7_ERR_INVALID;
  if (!all_aligned(dy, dk, dv) || !aligned16(ds_out)) return RWKV7_ERR_ALIGN;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (ds_in == nullptr || ds_in == ds_out) return RWKV7_OK;
    const size_t bytes = static_cast<size_t>(B) * H * kStateBytes;
    return from_cuda(ds_out ? cudaMemcpyAsync(ds_in, ds_out, bytes, cudaMemcpyDeviceToDevice, cs)
                            : cudaMemsetAsync(ds_in, 0, bytes, cs));
  }
  const bool chunk = use_chunk<uint16_t>(T);
  const lin::Shape s = shape(w, nullptr, B, T, tokens, T, H, workspace_bytes, 3, chunk);
  float *ws = static_cast<float *>(workspace);
  const long long part = s.nseg > 1 ? static_cast<long long>(B) * H * s.nseg * kN * kN : 0;
  const lin::Passes<uint16_t> p{{{dy, v, k, dr, s_in, nullptr, 1, 0, ws, 0, 2},
                                 {v, dy, r, dk, ds_out, nullptr, 1, 0, ws + part, 1, 2},
                                 {k, r, dy, dv, ds_out, ds_in, 0, 0, ws + 2 * part, 1, 3}},
                                3, 0};
  if (ds_in != nullptr && (ds_in == ds_out || ds_in == s_in) && s.nseg == 1) {
    // in place, and no workspace that holds the state meanwhile: the pass that writes it goes last
    lin::Passes<uint16_t> first = p, last = p;
    first.n = 2;
    last.n = 1;
    last.p[0] = p.p[2];
    const cudaError_t e = run_passes(first, s, B, chunk, cs);
    return from_cuda(e != cudaSuccess ? e : run_passes(last, s, B, chunk, cs));
  }
  return from_cuda(run_passes(p, s, B, chunk, cs));
}

long long rwkv7_layer_norm_workspace(int bf16, int M, int G, int D) {
  if (!norm_sizes(M, G, D) || M == 0) return 0;
  return layer_norm_partial_bytes(bf16 ? 2 : 4, M, G, D);
}

rwkv7_status rwkv7_layer_norm(int M, int G, int D, float eps, const float *x, const float *weight, const float *bias,
                              float *y, float *mean, float *rstd, rwkv7_stream_t stream) {
  return norm(M, G, D, eps, x, weight, bias, y, mean, rstd, stream);
}

rwkv7_status rwkv7_layer_norm_bf16(int M, int G, int D, float eps, const uint16_t *x, const float *weight,
                                   const float *bias, uint16_t *y, float *mean, float *rstd, rwkv7_stream_t stream) {
  return norm(M, G, D, eps, x, weight, bias, y, mean, rstd, stream);
}

rwkv7_status rwkv7_layer_norm_backward(int M, int G, int D, const float *dy, const float *x, const float *weight,
                                       const float *mean, const float *rstd, float *dx, float *dweight, float *dbias,
                                       void *workspace, long long workspace_bytes, rwkv7_stream_t stream) {
  return norm_backward(M, G, D, dy, x, weight, mean, rstd, dx, dweight, dbias, workspace, workspace_bytes, stream);
}

rwkv7_status rwkv7_layer_norm_backward_bf16(int M, int G, int D, const uint16_t *dy, const uint16_t *x,
                                            const float *weight, const float *mean, const float *rstd, uint16_t *dx,
                                            float *dweight, float *dbias, void *workspace, long long workspace_bytes,
                                            rwkv7_stream_t stream) {
  return norm_backward(M, G, D, dy, x, weight, mean, rstd, dx, dweight, dbias, workspace, workspace_bytes, stream);
}

}  // extern "C"
