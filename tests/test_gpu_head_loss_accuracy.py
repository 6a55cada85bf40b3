"""The head's loss and lse where the logits are exact in FP32: what is left is the softmax's
own error, which neither the logits' size nor the number of partial sums adds to."""

import numpy as np
import pytest
import torch

import dense_matrix_multiply_gb300 as g

pytestmark = pytest.mark.gpu
U = 2.0 ** -24  # an FP32 rounding


@pytest.fixture(scope="module", autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return lib


def head(z, targets, K=8):
    """loss, lse of one row of logits z (bf16 numbers) for each target, and X, W."""
    M, N = len(targets), len(z)
    X, W = torch.zeros(M, K, dtype=torch.bfloat16), torch.zeros(N, K, dtype=torch.bfloat16)
    X[:, 0] = 1
    W[:, 0] = torch.from_numpy(z.astype(np.float32))
    assert (W[:, 0].double().numpy() == z).all()
    X, W, t = X.cuda(), W.cuda(), torch.from_numpy(np.asarray(targets)).cuda()
    loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    g.gemm_cross_entropy("bf16", X, W, t, loss, lse, M, N, K)
    g.gemm_synchronize()
    return loss, lse, X, W, t


def check(z, targets):
    """2^x is 2 units of 2^-23 off; its exponent, a difference from the largest logit's rounded
    product with log2 e, by half a unit of values up to 128 (2^-18 of e^z's where that is
    e^-88 or less: nothing) and log2 e itself by 2^-26 of itself, both in proportion to the
    distance d: (d 2^-24 + d 2^-26) e^-d is below 2^-25; joins' exponents the same.  Then a sum
    of at most 4 + 8 + 4 + N / 4096 + 64 additions in a row, the logarithm, the maximum's own
    correction and the last additions.  lse has the last one's rounding at its own size."""
    loss, lse, *_ = head(z, targets)
    m = z.max()
    tail = np.log(np.exp(z - m).sum())
    e = 4 * U + 4 * U + (4 + 8 + 4 + len(z) / 4096 + 64) * U + 4 * U * abs(tail)
    off = np.abs(lse.double().cpu().numpy() - (m + tail)).max()
    assert off <= e + 2 * U * abs(m + tail), ("lse", off / (e + 2 * U * abs(m + tail)))
    want = m - z[np.asarray(targets)] + tail
    off = np.abs(loss.double().cpu().numpy() - want)
    tol = e + 2 * U * np.abs(want)
    assert (off <= tol).all(), ("loss", float((off / tol).max()))


@pytest.mark.parametrize("M", [1, 3, 130])
@pytest.mark.parametrize("N", [1000, 50257, 2000000])
@pytest.mark.parametrize("m", [0.0, 5.0, 20.5, 100.0, -100.0, 1000.0, 29952.0, -2.0 ** 60, 2.0 ** 100])
def test_equal_logits(M, N, m):
    """Every partial sum has the same largest logit: lse = m + log N, loss = log N."""
    check(np.full(N, m), [i * 7 % N for i in range(M)])


@pytest.mark.parametrize("M", [1, 130])
@pytest.mark.parametrize("m", [16.0, 120.0, 1000.0, 2000.0])
def test_a_probable_target(M, m):
    """The target's logit stands 8 or 16 above the rest: a small loss, and one that is the
    rest's distance, with lse much larger than both."""
    z = np.full(32000, m - 8)
    z[17::1000] = m - 16
    z[4321] = m
    check(z, [(4321, 17, 5)[i % 3] for i in range(M)])


@pytest.mark.parametrize("N", [300, 40000])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_logits_next_to_fp32s_largest(N, sign):
    """Products of logits with log2 e past FP32's range: lse is the largest logit (log N is
    nothing to it), loss the distance, and the softmax all on the largest."""
    big = float(torch.tensor(3e38, dtype=torch.bfloat16))
    low = float(torch.tensor(2.5e38, dtype=torch.bfloat16))
    z = np.full(N, sign * (low if sign > 0 else big))
    z[N // 3] = sign * (big if sign > 0 else low)
    M = 2
    loss, lse, X, W, t = head(z, [N // 3, 0])
    assert (lse.double().cpu().numpy() == z[N // 3]).all()
    want = np.array([0.0, z[N // 3] - z[0]])
    assert (np.abs(loss.double().cpu().numpy() - want) <= 2 * U * want).all(), loss
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    g.gemm_cross_entropy_backward("bf16", X, W, t, lse, torch.tensor([1.0, 0.5], device="cuda"), dX, dW, M, N, 8)
    g.gemm_synchronize()
    # dZ: row 0 all zeros; row 1 +0.5 at the largest, -0.5 at its target
    dw = torch.zeros(N, 8)
    dw[N // 3, 0], dw[0, 0] = 0.5, -0.5
    assert torch.equal(dW.float().cpu(), dw)
    assert not dX[0].any() and abs(float(dX[1, 0]) / (0.5 * want[1]) - 1) <= 2.0 ** -8 + 4 * U


@pytest.mark.parametrize("m", [12.0, 29952.0, 2.0 ** 20, -2.0 ** 27])
def test_the_softmax_is_of_the_lse_given(m):
    """p = e^(z - lse) with lse as it is, however large: dW of one row is dZ, rounded to bf16
    twice; p's exponent by a rounding of at most 8 and 2^x by two units of 2^-23."""
    N = 700
    z = np.full(N, m)
    _, lse, X, W, t = head(z, [5])
    lse.add_(3.0)
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    g.gemm_cross_entropy_backward("bf16", X, W, t, lse, torch.ones(1, device="cuda"), dX, dW, 1, N, 8)
    g.gemm_synchronize()
    want = np.exp(z - float(lse[0]))
    want[5] -= 1
    got = dW[:, 0].double().cpu().numpy()
    tol = np.abs(want) * (2 * 2.0 ** -8 + 2.0 ** -16) + (8 + 8) * U * np.exp(m - float(lse[0]))
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())
