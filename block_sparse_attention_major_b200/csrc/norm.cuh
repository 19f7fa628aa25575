// What the C ABI calls of the layer norm (norm.cu).
#pragma once

#include "common.cuh"

namespace bsa {
size_t norm_workspace(const bsa_norm_shape& f);
cudaError_t launch_norm_fwd(const bsa_norm_shape& f, const void* x, const void* w, const void* b, void* y,
                            float* mean, float* rstd, cudaStream_t s);
cudaError_t launch_norm_bwd(const bsa_norm_shape& f, const void* x, const void* dy, const float* mean,
                            const float* rstd, const void* w, void* dx, float* dw, float* db, void* ws,
                            cudaStream_t s);
}  // namespace bsa
