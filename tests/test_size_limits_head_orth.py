"""Sizes whose last tile would end past 2^31 are refused, on the host (no GPU): there the
kernels' 32-bit columns would turn negative."""

import pytest

import dense_matrix_multiply_gb300 as g

TOP = (1 << 31) - 256  # the largest that is taken
A = 1 << 50  # addresses that are checked and never read, far apart


@pytest.fixture(scope="module", autouse=True)
def built(lib):
    return lib.load()


def refused(fn, *args):
    before = g.gemm_kernel_launches()
    with pytest.raises(g.GemmError, match="INVALID_VALUE.*at most 2\\^31 - 256"):
        fn(*args)
    assert g.gemm_kernel_launches() == before


@pytest.mark.parametrize("dims", [(1, TOP + 1, 8), (1, (1 << 31) - 1, 8), (1, 1, TOP + 1), (TOP + 1, 1, 8)])
def test_head(dims):
    if dims[0] == 1:  # the loss takes any rows: they go in pieces
        refused(g.gemm_cross_entropy, "bf16", A, 2 * A, 3 * A, 4 * A, 5 * A, *dims)
    refused(g.gemm_cross_entropy_backward, "bf16", A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, 7 * A, *dims)


@pytest.mark.parametrize("M,N", [(1, TOP + 1), (TOP + 1, 1), (1, (1 << 31) - 1)])
def test_update(M, N):
    refused(g.gemm_orthogonalize, "bf16", A, N, 2 * A, N, 5, M, N)


def test_nothing_to_do_takes_any():
    g.gemm_cross_entropy("bf16", 0, 0, 0, 0, 0, 0, (1 << 31) - 1, 8)
    g.gemm_cross_entropy_backward("bf16", 0, 0, 0, 0, 0, 0, 0, 8, (1 << 31) - 1, 8)
    g.gemm_orthogonalize("bf16", 0, (1 << 31) - 1, 0, (1 << 31) - 1, 5, 0, (1 << 31) - 1)
    assert g.gemm_last_kernel() == "noop"
