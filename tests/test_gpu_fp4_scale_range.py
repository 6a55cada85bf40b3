"""NV products whose two tensor scales' product is not an FP32 number of full
precision, though the result is one: small operands (ga gb below 2^-126) and large
ones (ga gb above 2^128)."""

import numpy as np
import pytest
import torch

import fp4_ref as ref

import dense_matrix_multiply_gb300 as g

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return lib


def scale(v):
    return torch.tensor([v], dtype=torch.float32, device="cuda")


def side(rows, K, size, seed):
    a = torch.from_numpy(np.random.default_rng(seed).standard_normal((rows, K)).astype(np.float32)) * size
    return a.bfloat16()


def quantize(a, gs):
    M, K = a.shape
    Q = torch.empty(g.gemm_fp4_code_bytes(M, K), dtype=torch.uint8, device="cuda")
    S = torch.empty(g.gemm_fp4_scale_bytes("nv", M, K), dtype=torch.uint8, device="cuda")
    g.gemm_fp4_quantize("bf16", "nv", a.cuda(), K, scale(gs), Q, S, M, K)
    return Q, S


# (size of a, ga), (size of b, gb): ga gb some 2^-148, 2^-150 and 2^-152 (0 in FP32), 2^132
# and 2^130 (infinite); 2^-146 and 2^134 with one scale far from 1 and one nearer to it
CASES = [((2.0 ** -64, 1.3 * 2.0 ** -74), (2.0 ** -64, 1.7 * 2.0 ** -74)),
         ((2.0 ** -60, 2.0 ** -70), (2.0 ** -66, 2.0 ** -80)), ((2.0 ** -62, 2.0 ** -76), (2.0 ** -62, 2.0 ** -76)),
         ((2.0 ** 58, 2.0 ** 66), (2.0 ** 58, 2.0 ** 66)), ((2.0 ** 96, 2.0 ** 100), (2.0 ** 22, 2.0 ** 30)),
         ((2.0 ** -110, 1.7 * 2.0 ** -120), (2.0 ** -17, 1.3 * 2.0 ** -26)),
         ((2.0 ** 98, 2.0 ** 106), (2.0 ** 21, 2.0 ** 28))]


@pytest.mark.parametrize("M", [1, 16, 130])
@pytest.mark.parametrize("a_case,b_case", CASES)
def test_product_and_linear(M, a_case, b_case):
    N, K = 136, 2048
    a, b = side(M, K, a_case[0], M), side(N, K, b_case[0], M + 1)
    if M > 1:
        a[M // 2] = 0      # a row of exact zeros stays 0
    (ga, gb) = a_case[1], b_case[1]
    va, vb = (ref.values("nv", *ref.quantize("nv", x.float().numpy(), s), s) for x, s in ((a, ga), (b, gb)))
    want = va @ vb.T
    assert np.abs(want).max() < 2.0 ** 127 and np.abs(want).max() > 2.0 ** -126
    # two roundings of the scales more than tolerance() counts, 2^-24 each: well under its
    # 16 x 2^-23 of the magnitudes added
    tol = ref.tolerance(va, vb, want, "bf16", K)
    Qa, Sa = quantize(a, ga)
    Qb, Sb = quantize(b, gb)
    C, D = (torch.full((M, N), 77.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g.gemm_fp4("bf16", "nv", Qa, Sa, scale(ga), Qb, Sb, scale(gb), C, N, M, N, K)
    g.gemm_fp4_linear("bf16", "nv", a.cuda(), K, scale(ga), Qb, Sb, scale(gb), D, N, M, N, K)
    g.gemm_synchronize()
    for out in (C, D):
        assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
