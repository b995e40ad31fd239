// layer_norm.h -- launchers of the layer norm over groups (internal, not exported).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rwkv7 {

// x, y [M, G, D] of TIn (float or bfloat16 bits); w, b float32 [G, D] or nullptr (ones / zeros); mean,
// rstd float32 [M, G] or nullptr.
template <typename TIn>
cudaError_t launch_layer_norm(const TIn *x, const float *w, const float *b, float eps, TIn *y, float *mean, float *rstd,
                              int M, int G, int D, cudaStream_t stream);

// Bytes of the partial sums that the backward's two launches pass on (0: it needs none).
long long layer_norm_partial_bytes(size_t elem, int M, int G, int D);
// dw, db float32 [G, D], both or neither.
template <typename TIn>
cudaError_t launch_layer_norm_backward(const TIn *dy, const TIn *x, const float *w, const float *mean,
                                       const float *rstd, TIn *dx, float *dw, float *db, float *partial, int M, int G,
                                       int D, cudaStream_t stream);

}  // namespace rwkv7
