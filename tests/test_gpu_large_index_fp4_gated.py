"""4-bit and gated operators on matrices whose element offsets pass 2^31: rows at
both ends of the range against 64-bit values."""

import numpy as np
import pytest
import torch

import fp4_ref as ref
import gated_ref

import dense_matrix_multiply_gb300 as g

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield lib
    torch.cuda.empty_cache()


def ends(M, n=3):
    return list(range(n)) + [M // 2, 2 ** 31 // 8200, 2 ** 31 // 8200 + 1] + list(range(M - n, M))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_quantize_and_read_back(fmt):
    M, K = 70001, 32768
    assert M * K > 2 ** 31
    a = torch.randn(M, K, dtype=BF16, device="cuda")
    gs = 0.002 if fmt == "nv" else None
    t = None if gs is None else torch.tensor([gs], device="cuda")
    Q = torch.empty(g.gemm_fp4_code_bytes(M, K), dtype=torch.uint8, device="cuda")
    S = torch.empty(g.gemm_fp4_scale_bytes(fmt, M, K), dtype=torch.uint8, device="cuda")
    g.gemm_fp4_quantize("bf16", fmt, a, K, t, Q, S, M, K)
    out = torch.empty_like(a)
    g.gemm_fp4_dequantize("bf16", fmt, Q, S, t, out, K, M, K)
    g.gemm_synchronize()
    rows = [0, 1, 65535, 65536, M - 2, M - 1]
    code, byte = ref.quantize(fmt, a[rows].float().cpu().numpy(), gs)
    v = ref.values(fmt, code, byte).astype(np.float32) * np.float32(1 if gs is None else gs)
    assert torch.equal(out[rows].cpu(), torch.from_numpy(v).to(BF16))


def test_product():
    M, N, K, fmt = 262200, 8200, 64, "nv"
    assert M * N > 2 ** 31
    gs = torch.tensor([0.002], device="cuda")
    sides = []
    for rows in (M, N):
        x = torch.randn(rows, K, dtype=BF16, device="cuda")
        Q = torch.empty(g.gemm_fp4_code_bytes(rows, K), dtype=torch.uint8, device="cuda")
        S = torch.empty(g.gemm_fp4_scale_bytes(fmt, rows, K), dtype=torch.uint8, device="cuda")
        g.gemm_fp4_quantize("bf16", fmt, x, K, gs, Q, S, rows, K)
        sides += [x, Q, S]
    a, Qa, Sa, b, Qb, Sb = sides
    C = torch.empty(M, N, dtype=BF16, device="cuda")
    g.gemm_fp4("bf16", fmt, Qa, Sa, gs, Qb, Sb, gs, C, N, M, N, K)
    g.gemm_synchronize()
    rows, s = ends(M), float(gs.item())
    va = ref.values(fmt, *ref.quantize(fmt, a[rows].float().cpu().numpy(), s), s)
    vb = ref.values(fmt, *ref.quantize(fmt, b.float().cpu().numpy(), s), s)
    want = va @ vb.T
    err = np.abs(C[rows].double().cpu().numpy() - want)
    assert (err <= ref.tolerance(va, vb, want, "bf16", K)).all()


def test_gated():
    M, N, K = 262200, 8200, 8
    X, Wg, Wu = (torch.randn(*s, device="cuda").to(BF16) for s in ((M, K), (K, N), (K, N)))
    Z, dZ = torch.empty(M, N, dtype=BF16, device="cuda"), torch.empty(M, N, dtype=BF16, device="cuda").normal_()
    G, U = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    dX, dWg, dWu = torch.empty_like(X), torch.empty_like(Wg), torch.empty_like(Wu)
    g.gemm_gated("bf16", "silu", X, Wg, Wu, Z, G, U, M, N, K)
    g.gemm_gated_backward("bf16", "silu", X, Wg, Wu, G, U, dZ, dX, dWg, dWu, M, N, K)
    g.gemm_synchronize()
    rows = ends(M)
    x, wg, wu, d = (t.double().cpu().numpy() for t in (X[rows], Wg, Wu, dZ[rows]))
    for got, want, tol in zip((Z, G, U), gated_ref.forward("silu", x, wg, wu),
                              gated_ref.forward_tolerance("silu", x, wg, wu, "bf16")):
        assert (np.abs(got[rows].double().cpu().numpy() - want) <= tol).all()
    want, tol = gated_ref.backward("silu", x, wg, wu, d)[0], gated_ref.backward_tolerance("silu", x, wg, wu, d, "bf16")[0]
    assert (np.abs(dX[rows].double().cpu().numpy() - want) <= tol).all()
    # dW sums over every row: against 64-bit sums on the GPU, row piece by row
    # piece.  Its M terms' roundings to bf16 are independent: 8 deviations of
    # 2^-8 / sqrt(3) each; FP32 sums of M terms, 2^-24 of the running sum a term, are
    # under that; one rounding at the end.
    for got, which in ((dWg, 0), (dWu, 1)):
        total, square = (torch.zeros(K, N, dtype=torch.float64, device="cuda") for _ in range(2))
        for r in range(0, M, 8192):
            xx, gg, uu, dd = (t[r:r + 8192].double() for t in (X, G, U, dZ))
            s = torch.sigmoid(gg)
            e = dd * (uu * s * (1 + gg * (1 - s)) if which == 0 else gg * s)
            total += xx.T @ e
            square += xx.square().T @ e.square()
        bound = 8 * 2.0 ** -8 / 3 ** 0.5 * square.sqrt() + 2.0 ** -8 * total.abs()
        assert ((got.double() - total).abs() <= bound).all()
