"""Refusals of the norm's entry points, on the host (no GPU)."""

import pytest
import torch

import dense_matrix_multiply_gb300 as g


@pytest.fixture(scope="module", autouse=True)
def built(lib):
    return lib.load()


h = lambda n: torch.zeros(n, dtype=torch.bfloat16)
u8 = lambda n: torch.zeros(n, dtype=torch.uint8)
f32 = lambda n: torch.zeros(n, dtype=torch.float32)
M, K = 3, 16


def refused(fn, *args, match, error=ValueError):
    before = g.gemm_kernel_launches()
    with pytest.raises(error, match=match):
        fn(*args)
    assert g.gemm_kernel_launches() == before


def call(fn, good, **k):
    return (fn, "bf16", *({**good, **k}.values()), M, K)


def test_tensors():
    fwd = dict(X=h(M * K), R=h(M * K), w=h(K), eps=1e-6, H=h(M * K), Y=h(M * K), rstd=f32(M))
    q = dict(X=h(M * K), R=h(M * K), w=h(K), eps=1e-6, H=h(M * K), Q=u8(M * K), scale=f32(M))
    bwd = dict(H=h(M * K), w=h(K), rstd=f32(M), dY=h(M * K), dH=h(M * K), dX=h(M * K), dw=f32(K))
    for fn, good in ((g.gemm_rms_norm, fwd), (g.gemm_rms_norm_e4m3, q), (g.gemm_rms_norm_backward, bwd)):
        refused(*call(fn, good), match="CUDA device")
        for name, t in good.items():
            if name == "eps":
                continue
            refused(*call(fn, good, **{name: t[:-1].clone()}), match=f"{name} holds")
            wrong = u8(t.numel()) if t.dtype != torch.uint8 else h(t.numel())
            refused(*call(fn, good, **{name: wrong}), match="-byte elements")
            refused(*call(fn, good, **{name: torch.zeros(t.numel(), 2, dtype=t.dtype)[:, 0]}), match="contiguous")
        refused(fn, "f32", *good.values(), M, K, match="dtype")


A = 1 << 20  # addresses that are checked and never read


@pytest.mark.parametrize("eps", [0.0, -1.0, float("nan"), float("inf"), 1e-40, 2e9])
def test_eps(eps):
    refused(g.gemm_rms_norm, "bf16", A, 0, 0, eps, 0, 2 * A, 0, M, K, match="INVALID_VALUE.*eps", error=g.GemmError)


def test_addresses():
    n, e4 = g.gemm_rms_norm, g.gemm_rms_norm_e4m3
    bad = lambda fn, *a, match: refused(fn, "bf16", *a, M, K, match=match, error=g.GemmError)
    bad(n, 0, 0, 0, 1e-6, 0, A, 0, match="INVALID")                    # no X
    bad(n, A, 0, 0, 1e-6, 0, 0, 0, match="INVALID")                    # no Y
    bad(n, A, 0, 0, 1e-6, 2 * A, 3 * A, 0, match="INVALID")            # H without R
    bad(n, A + 1, 0, 0, 1e-6, 0, 2 * A, 0, match="INVALID")            # off the element
    bad(n, A, 0, 0, 1e-6, 0, 2 * A, 3 * A + 2, match="INVALID")        # rstd off 4 bytes
    bad(n, A, 0, 0, 1e-6, 0, A, 0, match="ALIAS")                      # Y in place
    bad(n, A, 2 * A, 0, 1e-6, A + 2, 3 * A, 0, match="ALIAS")          # H over part of X
    bad(n, A, 2 * A, 0, 1e-6, 2 * A, 2 * A, 0, match="ALIAS")          # Y over H
    bad(n, A, 2 * A, A + 8, 1e-6, A, 3 * A, 0, match="ALIAS")          # H over the gains
    bad(e4, A, 0, 0, 1e-6, 0, 0, 2 * A, match="INVALID")               # no Q
    bad(e4, A, 0, 0, 1e-6, 0, 2 * A, 0, match="INVALID")               # no scale
    bad(e4, A, 0, 0, 1e-6, 0, A + M * K, 3 * A, match="ALIAS")         # Q over X
    b = g.gemm_rms_norm_backward
    bad(b, A, 0, 0, 2 * A, 0, 3 * A, 0, match="INVALID")               # no rstd
    bad(b, A, 0, 4 * A, 0, 0, 3 * A, 0, match="INVALID")               # no dY
    bad(b, A, 0, 4 * A, 2 * A, 0, 2 * A, 0, match="ALIAS")             # dX over dY
    bad(b, A, 0, 4 * A, 2 * A, 3 * A, 3 * A + 2, 0, match="ALIAS")     # dX over part of dH
    bad(b, A, 0, 4 * A, 2 * A, 3 * A, 0, 3 * A, match="ALIAS")         # dw over dH
    bad(b, A, 0, 4 * A, 2 * A, 0, 3 * A, 3 * A, match="ALIAS")         # dw over dX
    refused(n, "bf16", A, 0, 0, 1e-6, 0, 2 * A, 0, -1, K, match="INVALID", error=g.GemmError)


def test_nothing_to_do():
    before = g.gemm_kernel_launches()
    g.gemm_rms_norm("bf16", 0, 0, 0, 1e-6, 0, 0, 0, 0, K)
    g.gemm_rms_norm("bf16", 0, 0, 0, 1e-6, 0, 0, 0, M, 0)
    g.gemm_rms_norm_e4m3("f16", 0, 0, 0, 1e-6, 0, 0, 0, 0, K)
    g.gemm_rms_norm_backward("f16", 0, 0, 0, 0, 0, 0, 0, M, K)
    assert g.gemm_last_kernel() == "noop" and g.gemm_kernel_launches() == before
