// Softmax cross entropy of a linear head: launchers (cross_entropy.cu).
#pragma once

#include "internal.h"

namespace gemm_gb300 {

// Logits Z = X W^T of X [M, K] and W [N, K] (16 bits, row-major without gaps), never
// stored whole; of row i lse_i = log sum_j exp Z_ij and loss_i = lse_i - Z_i,t_i, or 0
// where the target t_i is no column.
struct HeadProblem {
    const void *X, *W;
    const long long *target;
    float *loss, *lse;  // lse null: not stored
    int M, N, K;
    Elt elt;
};
// dZ_ij = (exp(Z_ij - lse_i) - [j = t_i]) dloss_i (0 in rows without a target),
// dX = dZ W, dW = dZ^T X; a null one is left out.
struct HeadBackward {
    const void *X, *W;
    const long long *target;
    const float *lse, *dloss;
    void *dX, *dW;
    int M, N, K;
    Elt elt;
};
// K >= 1, M >= 1, N >= 1.
cudaError_t launch_cross_entropy(const HeadProblem &p, int *status, cudaStream_t s);
cudaError_t launch_cross_entropy_backward(const HeadBackward &p, int *status, cudaStream_t s);
// Logits of empty sums (K = 0), or none (N = 0).
cudaError_t launch_cross_entropy_flat(const HeadProblem &p, cudaStream_t s);

}  // namespace gemm_gb300
