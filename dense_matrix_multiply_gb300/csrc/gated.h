// Gated feed-forward block: launchers (gated.cu, gated_skinny.cu, gated_pad.cu) and
// the activations they share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace gemm_gb300 {

// Z [M,N] = act(X Wg) * (X Wu); X [M,K], Wg and Wu [K,N], row-major, 16-bit.
// G and U [M,N] FP32: both stored, or both null.
struct GatedProblem {
    const void *X, *Wg, *Wu;
    void *Z;
    float *G, *U;
    int M, N, K;
    Elt elt;
    bool gelu;      // GELU (tanh form), else SiLU
    long long ldx;  // elements from one row of X to the next
};
// The gradients of X, Wg and Wu from dZ and the saved G and U; a null one is
// left out.
struct GatedBackward {
    const void *X, *Wg, *Wu, *dZ;
    const float *G, *U;
    void *dX, *dWg, *dWu;
    int M, N, K;
    Elt elt;
    bool gelu;
};
// Any N, K >= 1 and alignment of elements (gated_pad.cu); the launchers below need
// N and K to be multiples of 8 and every base on 16 bytes.
cudaError_t launch_gated_forward(const GatedProblem &p, int num_sms, int *status, cudaStream_t s);
cudaError_t launch_gated_gradients(const GatedBackward &p, int num_sms, int *status, cudaStream_t s);

cudaError_t launch_gated(const GatedProblem &p, int *status, cudaStream_t s);            // any M
constexpr int kGatedSkinnyMaxM = 64;
cudaError_t launch_gated_skinny(const GatedProblem &p, int num_sms, int *status, cudaStream_t s);
// dX from dG and dU [2][M][N], rows gated_ldg(N) elements apart.
constexpr long long gated_ldg(int N) { return ((long long)N + 63) / 64 * 64; }
// beside: the launch before is dW's, which writes nothing that dX reads.
cudaError_t launch_gated_skinny_dx(const GatedBackward &p, const void *dGU, bool beside, int num_sms, int *status,
                                   cudaStream_t s);
cudaError_t launch_gated_backward(const GatedBackward &p, int num_sms, int *status, cudaStream_t s);

#ifdef __CUDACC__
// Both activations are g s(z), s the logistic function: SiLU with z = g, the tanh
// form of GELU with z = 2 sqrt(2/pi) (g + 0.044715 g^3), since (1 + tanh y) / 2 =
// s(2 y) -- which also keeps the relative accuracy of the negative tail, where 1 +
// tanh cancels.  s from t = e^-|z|, at most 1: 1 / (1 + t), or t / (1 + t) for negative
// z, whose divisor stays within the fast division's range (1 / (1 + e^-z) would be 0
// from z = -87.3 down, where g s is still a normal number of bf16).  The fast
// exponential's relative error grows with its argument, 2 + 1.2 |z| units of 2^-23: under
// 2^-20 for |z| < 5 and 2^-16 at the end of the range, far below the 2^-9 or 2^-12 of
// the rounding that follows; the division adds 2 units.
template <bool GELU>
__device__ __forceinline__ float gate_sigmoid(float g) {
    constexpr float c2 = 1.5957691216057308f, c3 = 0.044715f;  // 2 sqrt(2 / pi)
    const float z = GELU ? c2 * g * fmaf(c3 * g, g, 1.0f) : g;
    const float t = __expf(-fabsf(z));
    return __fdividef(z < 0.0f ? t : 1.0f, 1.0f + t);
}
template <bool GELU>
__device__ __forceinline__ float gate_act(float g) { return g * gate_sigmoid<GELU>(g); }
// act and its derivative s + g s (1 - s) z'; where g s (1 - s) is 0 the last term
// is, however large z'.
template <bool GELU>
__device__ __forceinline__ void gate_act_grad(float g, float &a, float &da) {
    constexpr float c2 = 1.5957691216057308f, c33 = 3.0f * 0.044715f;
    const float s = gate_sigmoid<GELU>(g);
    a = g * s;
    float t = a * (1.0f - s);
    if (GELU) t = t == 0.0f ? 0.0f : t * (c2 * fmaf(c33 * g, g, 1.0f));
    da = s + t;
}
#endif

}  // namespace gemm_gb300
