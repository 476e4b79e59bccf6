// norm.cuh -- argument block and launch entry points of the normalisation
// over rows (internal to the library; the public ABI is include/ssm.h).
//
//   layer: xhat = (x - mean(x)) rstd, rstd = (mean((x - mean)^2) + eps)^-1/2
//   RMS:   xhat = x rstd,             rstd = (mean(x^2) + eps)^-1/2
//   out = (xhat weight + bias) silu(z)
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace ssm {

struct NormArgs {
    const void *x, *z, *dout;          // (rows, dim); z null: no gate
    const float *weight, *bias;        // (dim) or null (one, zero)
    const float *mean_in, *rstd_in;    // backward: (rows); mean_in null: RMS
    void *out, *dx, *dz;
    float *mean, *rstd;                // forward: (rows) or null
    float *dweight, *dbias;            // (dim) or null
    float *partial;                    // backward workspace: partial column sums, set by the launcher
    int64_t rows;
    int dim;
    float eps;
    int center;                        // 1: layer norm, 0: RMS norm
};

cudaError_t launch_norm_fwd(const NormArgs &a, bool bf16, int sms, cudaStream_t st);
// Stream-ordered workspace for the column sums (freed with cudaFreeAsync).
typedef cudaError_t (*NormAlloc)(size_t bytes, cudaStream_t st, float **p);
cudaError_t launch_norm_bwd(const NormArgs &a, bool bf16, int sms, NormAlloc alloc, cudaStream_t st);

}  // namespace ssm
