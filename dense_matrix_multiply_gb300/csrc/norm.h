// Root-mean-square norm with the residual's addition: launchers (rms_norm.cu).
#pragma once

#include "internal.h"

namespace gemm_gb300 {

// H = X + R rounded to the element type (R null: H is X, none is stored), and of it
// Y = w H rstd, rstd = 1 / sqrt(mean(H^2) + eps), or Y's E4M3 codes Q and scales.
// All row-major [M, K] without gaps; w [K] (null: ones) of the element type.
struct NormProblem {
    const void *X, *R, *w;
    void *H;      // null: not stored; may be X or R
    void *Y;      // 16 bits, or null
    void *Q;      // E4M3, where Y is null
    float *scale; // with Q: a row's largest |Y| / 448
    float *rstd;  // null: not stored
    float eps;
    int M, K;
    Elt elt;
};
// dX = rstd w dY - H rstd^3 mean(w dY H) + dH (null: 0), dw = sum over rows of
// dY H rstd; a null one is left out.  dX may be dH.
struct NormBackward {
    const void *H, *w;
    const float *rstd;
    const void *dY, *dH;
    void *dX;
    float *dw;
    int M, K;
    Elt elt;
};
cudaError_t launch_rms_norm(const NormProblem &p, cudaStream_t s);
cudaError_t launch_rms_norm_backward(const NormBackward &p, int num_sms, int *status, cudaStream_t s);

}  // namespace gemm_gb300
