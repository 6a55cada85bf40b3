"""The activations' negative tail, down to the least number that bf16 holds: Z, dU
and dG against 64-bit values where the gate's exponential leaves FP32's normal
range.

Inputs make the products exact: X holds one 1 a row, so G and U are weights and
the weight gradients are dG and dU (rounded to bf16).  What is left is the
activation's error, relative in |z| <= 100: ten FP32 roundings of z and of the
exponent's multiplication, 10 x 2^-24 x 100 < 2^-13, of which the exponential itself and
the division are a few 2^-23; the result's rounding to bf16 (2^-8), for dG and dU
again when the product is rounded (nothing is lost there); and, near the least
number, half of its distance 2^-133 and a few FP32 subnormal steps (2^-149 x 100)."""

import numpy as np
import pytest
import torch

import gated_ref

import dense_matrix_multiply_gb300 as g

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
REL, ABS = 2.0 ** -8 + 2.0 ** -13, 2.0 ** -133


@pytest.fixture(scope="module", autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return lib


def gates(act):
    """bf16 gate values of the tail, 264 of them; z of the logistic down to -98."""
    if act == "silu":
        v = -np.arange(20.0, 98.5, 0.5)
    else:
        v = -np.arange(4.0, 10.05, 0.0625)
    v = torch.from_numpy(np.resize(v, 264)).to(BF16)
    return v


def exact(act, v):
    """act and act' in 64 bits, without the cancellation of 1 + tanh."""
    z = v if act == "silu" else 2 * gated_ref.C * (v + 0.044715 * v ** 3)
    s = np.exp(z) / (1 + np.exp(z))
    dz = 1.0 if act == "silu" else 2 * gated_ref.C * (1 + 3 * 0.044715 * v * v)
    return v * s, s + v * s * (1 - s) * dz, s + np.abs(v * s * (1 - s) * dz)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M", [3, 64, 300])
def test_forward(act, M):
    v = gates(act)
    N, K = v.numel(), 16
    X = torch.zeros(M, K, dtype=BF16, device="cuda")
    X[torch.arange(M), torch.arange(M) % K] = 1
    Wg = v.cuda().expand(K, N).contiguous()
    Wu = torch.ones(K, N, dtype=BF16, device="cuda")
    Z = torch.empty(M, N, dtype=BF16, device="cuda")
    g.gemm_gated("bf16", act, X, Wg, Wu, Z, None, None, M, N, K)
    g.gemm_synchronize()
    want, _, _ = exact(act, v.double().numpy())
    assert (np.abs(Z.double().cpu().numpy() - want) <= REL * np.abs(want) + ABS).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients(act):
    v = gates(act)
    M, N, K = 1, v.numel(), 8
    X = torch.zeros(M, K, dtype=BF16, device="cuda")
    X[0, 0] = 1
    G = v.float().cuda().view(M, N)
    U = torch.full((M, N), 3.0, device="cuda")
    dZ = torch.full((M, N), 2.0, dtype=BF16, device="cuda")
    dWg, dWu = (torch.empty(K, N, dtype=BF16, device="cuda") for _ in range(2))
    g.gemm_gated_backward("bf16", act, X, None, None, G, U, dZ, None, dWg, dWu, M, N, K)
    g.gemm_synchronize()
    a, da, size = exact(act, v.double().numpy())
    assert (np.abs(dWu[0].double().cpu().numpy() - 2 * a) <= REL * np.abs(2 * a) + ABS).all()
    # act' is a difference: its rounding errors are of the size of its terms
    bound = 6 * (2.0 ** -8 * np.abs(da) + 2.0 ** -13 * size) + ABS
    assert (np.abs(dWg[0].double().cpu().numpy() - 6 * da) <= bound).all()
