"""The norm at the ends of bf16's range, against 64-bit values within norm_ref's
tolerances."""

import numpy as np
import pytest
import torch

import norm_ref as ref

import dense_matrix_multiply_gb300 as g

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return lib


def f64(t, *shape):
    return t.double().cpu().numpy().reshape(shape)


def close(got, want, tol, name):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (name, int(bad.sum()), float((np.abs(got - want) / tol).max()))


def run_e4m3(X, w, eps):
    M, K = X.shape
    x, Q, scale = X.cuda().reshape(-1), torch.empty(M * K, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(M, device="cuda")
    g.gemm_rms_norm_e4m3("bf16", x, None, None if w is None else w.cuda(), eps, None, Q, scale, M, K)
    g.gemm_synchronize()
    return f64(Q.float(), M, K), f64(scale, M)


# 1 / sqrt of a mean of squares up to 2^256 is an FP32 subnormal: half a step of those
LEAST = 2.0 ** -150


@pytest.mark.parametrize("K", [2048, 4096, 4099, 8192, 16000, 16371, 40000])
def test_rows_of_the_largest_numbers(K):
    """All elements next to the largest, whose squares' sum overflows even when they are
    taken down by 2^70: 16-bit and E4M3 results, rstd, and the gradients that read it."""
    rng = np.random.default_rng(K)
    top = float(torch.finfo(torch.bfloat16).max)
    x = np.where(rng.random((3, K)) < 0.5, 1.0, -1.0) * np.array([1.0, 0.9, 1.0])[:, None] * top
    x[2, ::3] *= 1e-30
    X = torch.from_numpy(x.astype(np.float32)).bfloat16()
    w = torch.from_numpy((1 + 0.3 * rng.standard_normal(K)).astype(np.float32)).bfloat16()
    dY = torch.from_numpy(rng.standard_normal((3, K)).astype(np.float32)).bfloat16()
    xc, wc = X.cuda().reshape(-1), w.cuda()
    Y, dX = torch.empty_like(xc), torch.empty_like(xc)
    rstd, dw = torch.empty(3, device="cuda"), torch.empty(K, device="cuda")
    g.gemm_rms_norm("bf16", xc, None, wc, EPS, None, Y, rstd, 3, K)
    g.gemm_rms_norm_backward("bf16", xc, wc, rstd, dY.cuda().reshape(-1), None, dX, dw, 3, K)
    Q, scale = run_e4m3(X, w, EPS)
    h, wd, d = X.double().numpy(), w.double().numpy(), dY.double().numpy()
    r, y = ref.forward(h, wd, EPS)
    er, ey = ref.forward_error(K)
    close(f64(rstd, 3), r, r * er + LEAST, "rstd")
    close(f64(Y, 3, K), y, ref.round_tolerance(y, ey, "bf16"), "Y")
    s = np.abs(y).max(1) / 448
    close(scale, s, s * (ey + 2 * ref.U), "scale")
    v = y / s[:, None]
    close(Q, v, ref.e4m3_tolerance(v, ey), "Q")
    want_x, want_w = ref.backward(h, wd, d, 0.0, EPS)
    tol_x, tol_w = ref.backward_tolerance(h, wd, d, np.zeros((3, K)), EPS, "bf16")
    # rstd half a step of subnormals off: as much more of dw's terms, which it multiplies
    close(f64(dw, K), want_w, tol_w + np.abs(d * h).sum(0) * LEAST, "dw")
    close(f64(dX, 3, K), want_x, tol_x, "dX")


def check_e4m3(x, w, eps):
    """Codes within half a step of Y / scale, no NaN; FP32 operations as elsewhere, one product
    more, and scales down to FP32's subnormals."""
    X = torch.from_numpy(x.astype(np.float32)).bfloat16()
    wt = None if w is None else torch.from_numpy(w.astype(np.float32)).bfloat16()
    Q, scale = run_e4m3(X, wt, eps)
    _, y = ref.forward(X.double().numpy(), 1.0 if w is None else wt.double().numpy(), eps)
    _, ey = ref.forward_error(x.shape[1])
    s = np.abs(y).max(1) / 448
    s[s < 2.0 ** -150 / 448] = 0  # Y is 0 in FP32
    close(scale, s, s * (ey + 4 * ref.U) + LEAST, "scale")
    v = np.where(s[:, None] > 0, y / np.where(s > 0, s, 1)[:, None], 0)
    close(Q, v, ref.e4m3_tolerance(v, ey + ref.U), "Q")


LENGTHS = [(7, 64), (7, 512), (6, 1027), (5, 2040), (5, 2047), (3, 4096), (3, 8200), (6, 20000)]
NEARLY_ZERO = np.array([1e-40, 9.2e-41, 0.0, 1e-39, 3.0, 1e-38, 2e-37])


@pytest.mark.parametrize("eps", [EPS, 1.0, 2.0 ** 29])
@pytest.mark.parametrize("M,K", LENGTHS)
def test_codes_of_rows_that_are_nearly_zero(M, K, eps):
    """bf16's least numbers, with zeros between them, beside rows of zeros and ordinary ones."""
    rng = np.random.default_rng(K)
    x = (1 + rng.random((M, K))) * NEARLY_ZERO[:M, None] * rng.choice([1.0, -1.0, 0.0], (M, K))
    check_e4m3(x, None, eps)
    check_e4m3(x, 1 + 0.3 * rng.standard_normal(K), eps)
    # gains that take Y to FP32's subnormals, below them, or back among the normal numbers
    for gain in (1e-5, 1e-12, 1e25):
        check_e4m3(x, gain * (1 + rng.random(K)), eps)


@pytest.mark.parametrize("M,K", LENGTHS)
def test_codes_of_gains_that_take_h_out_of_fp32(M, K):
    """w H above FP32's largest number, or below its least, where Y = w H rstd is neither."""
    rng = np.random.default_rng(K)
    x = rng.standard_normal((M, K)) * np.array([1e10, 1.0, 1e30, 0.0, 1e18, 1e-3, 1e9])[:M, None]
    check_e4m3(x, 1e30 * (1 + 0.3 * rng.standard_normal(K)), EPS)
    check_e4m3(x * 1e-8, 1e-30 * (1 + 0.3 * rng.standard_normal(K)), 1.2e-38)
    w = 10.0 ** rng.uniform(-37, 37, K)
    check_e4m3(x, w, EPS)
