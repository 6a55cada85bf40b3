// Orthogonalised update of a weight matrix: launcher (orthogonalize.cu).
#pragma once

#include "internal.h"

namespace gemm_gb300 {

// O [M, N] = the matrix that `steps` times X <- a X + (b A + c A^2) X, A = X X^T (from the
// right, with X^T X, where M > N), makes of G / |G|_F.  Row-major 16-bit; O may be G.
struct OrthProblem {
    const void *G;
    long long ldg;
    void *O;
    long long ldo;
    int M, N, steps;
    float a, b, c;
    Elt elt;
};
cudaError_t launch_orthogonalize(const OrthProblem &p, int num_sms, int *status, cudaStream_t s);

}  // namespace gemm_gb300
