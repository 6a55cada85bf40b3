"""NV with a tensor scale of 0, the scale (amax / 2688) of a tensor of zeros: a
block of zeros has scale byte 0 whatever the tensor's scale, everything reads
back as 0, and products with it are 0, as with a tensor whose scale was taken from
zeros but which has values."""

import numpy as np
import pytest
import torch

import fp4_ref as ref

import dense_matrix_multiply_gb300 as g

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return lib


def scale(v):
    return torch.tensor([v], dtype=torch.float32, device="cuda")


def quantize(a, gs):
    M, K = a.shape
    name = "bf16" if a.dtype == torch.bfloat16 else "f16"
    Q = torch.full((g.gemm_fp4_code_bytes(M, K),), 0x5A, dtype=torch.uint8, device="cuda")
    S = torch.full((g.gemm_fp4_scale_bytes("nv", M, K),), 0x5A, dtype=torch.uint8, device="cuda")
    g.gemm_fp4_quantize(name, "nv", a.cuda(), K, gs, Q, S, M, K)
    return Q, S


def values(kind, M, K, dtype, seed):
    """zeros; values; or rows of zeros among rows of values, and blocks of zeros in these"""
    a = torch.randn(M, K, generator=torch.Generator().manual_seed(seed))
    if kind == "zeros":
        a.zero_()
    elif kind == "some":
        a[::2] = 0
        a[:, 16:32] = 0
    return a.to(DT[dtype])


# K of whole groups of 256 (no padded blocks) and not; rows on 16, 8 and 2 bytes
@pytest.mark.parametrize("K", [256, 1024, 16, 300, 1, 513])
@pytest.mark.parametrize("kind", ["zeros", "some", "values"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_and_read_back(K, kind, dtype):
    M = 130
    a = values(kind, M, K, dtype, K)
    Q, S = quantize(a, scale(0.0))
    out = torch.full((M, K), 77.0, dtype=DT[dtype], device="cuda")
    g.gemm_fp4_dequantize(dtype, "nv", Q, S, scale(0.0), out, K, M, K)
    g.gemm_synchronize()
    assert (out == 0).all()
    # a block with values saturates (448: byte 126), one of zeros has byte 0, padding too
    x = np.zeros((M, -(-K // 16) * 16), dtype=np.float32)
    x[:, :K] = a.float().numpy()
    byte = np.where(np.abs(x.reshape(M, -1, 16)).max(-1) > 0, 126, 0)
    assert np.array_equal(S.cpu().numpy(), ref.tile_scales("nv", byte, K))


@pytest.mark.parametrize("gs", [0.0, 2.0 ** -149, 1e-30, 1.0, 1e30])
def test_zeros_under_any_scale(gs):
    M, K = 3, 300
    Q, S = quantize(torch.zeros(M, K, dtype=torch.bfloat16), scale(gs))
    g.gemm_synchronize()
    assert not Q.any() and not S.any()


# both product kernels, the quantiser inside one of them (M <= 8), and before it
@pytest.mark.parametrize("M", [1, 8, 16, 64, 65, 300])
@pytest.mark.parametrize("K", [512, 300, 33])
@pytest.mark.parametrize("kind", ["zeros", "some", "values"])
def test_products(M, K, kind):
    N = 136
    w = torch.randn(N, K, generator=torch.Generator().manual_seed(K)).bfloat16()
    gw = scale(float(w.float().abs().max()) / 2688)
    Qw, Sw = quantize(w, gw)
    a = values(kind, M, K, "bf16", M + K)
    zero = scale(0.0)
    Qa, Sa = quantize(a, zero)
    C = torch.full((M, N), 77.0, dtype=torch.bfloat16, device="cuda")
    D = C.clone()
    g.gemm_fp4("bf16", "nv", Qa, Sa, zero, Qw, Sw, gw, C, N, M, N, K)
    g.gemm_fp4_linear("bf16", "nv", a.cuda(), K, zero, Qw, Sw, gw, D, N, M, N, K)
    g.gemm_synchronize()
    assert (C == 0).all() and (D == 0).all()
    # weights of zeros
    Qz, Sz = quantize(torch.zeros(N, K, dtype=torch.bfloat16), zero)
    x = torch.randn(M, K, device="cuda").bfloat16()
    C.fill_(77.0)
    g.gemm_fp4_linear("bf16", "nv", x, K, scale(0.002), Qz, Sz, zero, C, N, M, N, K)
    g.gemm_synchronize()
    assert (C == 0).all()
