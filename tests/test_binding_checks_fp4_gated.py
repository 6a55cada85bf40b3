"""The binding's host-side checks of the 4-bit and gated entry points (no GPU):
short, mistyped or non-contiguous tensors and tensors off the GPU are refused
before an address reaches the library."""

import pytest
import torch

import dense_matrix_multiply_gb300 as g


@pytest.fixture(scope="module", autouse=True)
def built(lib):
    return lib.load()


def refused(fn, *args, match):
    before = g.gemm_kernel_launches()
    with pytest.raises(ValueError, match=match):
        fn(*args)
    assert g.gemm_kernel_launches() == before


h = lambda n: torch.zeros(n, dtype=torch.bfloat16)
u8 = lambda n: torch.zeros(n, dtype=torch.uint8)
f32 = lambda n: torch.zeros(n, dtype=torch.float32)


@pytest.mark.parametrize("fmt,blocks", [("mx", 1024), ("nv", 2048)])
def test_fp4(fmt, blocks):
    M, N, K, ld = 3, 5, 40, 44
    A, Qm, Qn, S = h(2 * ld + K), u8(M * 32), u8(N * 32), u8(blocks)
    gs = f32(1) if fmt == "nv" else None
    q, d = g.gemm_fp4_quantize, g.gemm_fp4_dequantize
    for fn, order in ((q, lambda a, qq, s, t: (a, ld, t, qq, s)), (d, lambda a, qq, s, t: (qq, s, t, a, ld))):
        args = lambda a=A, qq=Qm, s=S, t=gs: ("bf16", fmt, *order(a, qq, s, t), M, K)
        refused(fn, *args(), match="CUDA device")
        refused(fn, *args(a=A[:-1].clone()), match=f"A holds {2 * ld + K - 1} elements")
        refused(fn, *args(qq=Qm[:-1]), match="Q holds 95 elements")
        refused(fn, *args(s=S[:-1]), match="S holds")
        refused(fn, *args(a=f32(2 * ld + K)), match="2-byte elements")
        refused(fn, *args(qq=h(M * 32)), match="1-byte elements")
        refused(fn, *args(t=h(1)), match="4-byte elements")
    C = h(M * N)
    args = lambda **k: ("bf16", fmt, *({**dict(Qa=Qm, Sa=S, ga=gs, Qb=Qn, Sb=S, gb=gs, C=C), **k}.values()), N, M, N, K)
    refused(g.gemm_fp4, *args(), match="CUDA device")
    refused(g.gemm_fp4, *args(Qb=Qn[1:]), match="Qb holds 159 elements, the call needs 160")
    refused(g.gemm_fp4, *args(Sa=S[1:]), match="Sa holds")
    refused(g.gemm_fp4, *args(C=C[:-1].clone()), match="C holds 14")
    lin = lambda **k: ("bf16", fmt, *({**dict(X=A, ldx=ld, gx=gs, Q=Qn, S=S, gw=gs, C=C), **k}.values()), N, M, N, K)
    refused(g.gemm_fp4_linear, *lin(), match="CUDA device")
    refused(g.gemm_fp4_linear, *lin(X=A[:-1].clone()), match="X holds")
    refused(g.gemm_fp4_linear, *lin(Q=Qn[:-1]), match="Qw holds")
    # nothing is read or written: only the device is checked
    refused(g.gemm_fp4_linear, *(lin()[:-3]), 0, N, K, match="CUDA device")


def test_gated():
    M, N, K = 3, 8, 16
    good = dict(X=h(M * K), Wg=h(K * N), Wu=h(K * N), Z=h(M * N), G=f32(M * N), U=f32(M * N))
    fwd = lambda **k: ("bf16", "silu", *({**good, **k}.values()), M, N, K)
    refused(g.gemm_gated, *fwd(), match="CUDA device")
    refused(g.gemm_gated, *fwd(Wu=h(K * N - 1)), match="W_u holds 127 elements, the call needs 128")
    refused(g.gemm_gated, *fwd(G=h(M * N)), match="4-byte elements")
    refused(g.gemm_gated, *fwd(X=h(M * K).view(K, M).t()), match="contiguous")
    good2 = dict(X=h(M * K), Wg=h(K * N), Wu=h(K * N), G=f32(M * N), U=f32(M * N), dZ=h(M * N), dX=h(M * K), dWg=h(K * N),
                 dWu=h(K * N))
    bwd = lambda **k: ("bf16", "gelu", *({**good2, **k}.values()), M, N, K)
    refused(g.gemm_gated_backward, *bwd(), match="CUDA device")
    refused(g.gemm_gated_backward, *bwd(dX=None, dWg=None, dWu=h(1)), match="dW_u holds 1")
    refused(g.gemm_gated_backward, *bwd(dZ=f32(M * N)), match="2-byte elements")
