"""Refusals of the head's entry points, on the host (no GPU)."""

import pytest
import torch

import dense_matrix_multiply_gb300 as g


@pytest.fixture(scope="module", autouse=True)
def built(lib):
    return lib.load()


h = lambda n: torch.zeros(n, dtype=torch.bfloat16)
f32 = lambda n: torch.zeros(n, dtype=torch.float32)
i64 = lambda n: torch.zeros(n, dtype=torch.int64)
M, N, K = 3, 5, 16
A = 1 << 20  # addresses that are checked and never read


def refused(fn, *args, match, error=ValueError):
    before = g.gemm_kernel_launches()
    with pytest.raises(error, match=match):
        fn(*args)
    assert g.gemm_kernel_launches() == before


def test_tensors():
    fwd = dict(X=h(M * K), W=h(N * K), targets=i64(M), loss=f32(M), lse=f32(M))
    bwd = dict(X=h(M * K), W=h(N * K), targets=i64(M), lse=f32(M), dloss=f32(M), dX=h(M * K), dW=h(N * K))
    for fn, good in ((g.gemm_cross_entropy, fwd), (g.gemm_cross_entropy_backward, bwd)):
        call = lambda **k: (fn, "bf16", *({**good, **k}.values()), M, N, K)
        refused(*call(), match="CUDA device")
        for name, t in good.items():
            refused(*call(**{name: t[:-1].clone()}), match=f"{name} holds")
            refused(*call(**{name: torch.zeros(t.numel(), dtype=torch.uint8)}), match="-byte elements")
            refused(*call(**{name: torch.zeros(t.numel(), 2, dtype=t.dtype)[:, 0]}), match="contiguous")
        refused(*call(targets=torch.zeros(M, dtype=torch.int32)), match="8-byte elements")
        refused(fn, "f32", *good.values(), M, N, K, match="dtype")


def test_addresses():
    fwd, bwd = g.gemm_cross_entropy, g.gemm_cross_entropy_backward
    bad = lambda fn, *a, match, dims=(M, N, K): refused(fn, "bf16", *a, *dims, match=match, error=g.GemmError)
    bad(fwd, 0, A, 2 * A, 3 * A, 0, match="INVALID")              # no X
    bad(fwd, A, 0, 2 * A, 3 * A, 0, match="INVALID")              # no W
    bad(fwd, A, A, 0, 3 * A, 0, match="INVALID")                  # no targets
    bad(fwd, A, A, 2 * A, 0, 3 * A, match="INVALID")              # no loss
    bad(fwd, A + 1, A, 2 * A, 3 * A, 0, match="INVALID")          # off the element
    bad(fwd, A, A, 2 * A + 4, 3 * A, 0, match="INVALID.*targets need 8")
    bad(fwd, A, A, 2 * A, 3 * A, 3 * A + 8, match="ALIAS")        # lse over loss
    bad(fwd, A, 2 * A, 3 * A, A, 0, match="ALIAS")                # loss over X
    bad(fwd, A, A, 2 * A, 3 * A, 0, match="INVALID", dims=(M, -1, K))
    bad(bwd, A, 2 * A, 3 * A, 0, 4 * A, 5 * A, 0, match="INVALID")          # no lse
    bad(bwd, A, 2 * A, 3 * A, 4 * A, 0, 5 * A, 0, match="INVALID")          # no dloss
    bad(bwd, A, 2 * A, 3 * A, 4 * A, 5 * A, A, 0, match="ALIAS")            # dX over X
    bad(bwd, A, 2 * A, 3 * A, 4 * A, 5 * A, 0, 2 * A + 2, match="ALIAS")    # dW over W
    bad(bwd, A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, 6 * A, match="ALIAS")    # dX over dW


def test_nothing_to_do():
    before = g.gemm_kernel_launches()
    g.gemm_cross_entropy("bf16", 0, 0, 0, 0, 0, 0, N, K)
    g.gemm_cross_entropy_backward("bf16", 0, 0, 0, 0, 0, 0, 0, M, N, K)
    g.gemm_cross_entropy_backward("bf16", 0, 0, 0, 0, 0, A, A, M, N, 0)
    assert g.gemm_last_kernel() == "noop" and g.gemm_kernel_launches() == before
