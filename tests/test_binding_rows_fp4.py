"""The 4-bit entry points' matrices with a leading dimension (A, X, C and the
read-back's output; no GPU): a tensor whose elements do not lie where the leading
dimension says is refused, a transposed view above all; flat buffers and slices of
wider rows pass on to the check of the device, the last one."""

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


M, N, K = 40, 24, 56
h = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
u8 = lambda n: torch.zeros(n, dtype=torch.uint8)
Q = lambda rows, k: u8(g.gemm_fp4_code_bytes(rows, k))
S = lambda rows, k: u8(g.gemm_fp4_scale_bytes("mx", rows, k))


def calls(rows, cols):
    """Each call with a [rows, cols] matrix t of leading dimension ld in one of its places."""
    def linear_x(t, ld):
        return g.gemm_fp4_linear, "bf16", "mx", t, ld, None, Q(N, cols), S(N, cols), None, h(rows, N), N, rows, N, cols

    def linear_c(t, ld):
        return g.gemm_fp4_linear, "bf16", "mx", h(rows, K), K, None, Q(cols, K), S(cols, K), None, t, ld, rows, cols, K

    def product_c(t, ld):
        return (g.gemm_fp4, "bf16", "mx", Q(rows, K), S(rows, K), None, Q(cols, K), S(cols, K), None, t, ld, rows, cols,
                K)

    def quantize(t, ld):
        return g.gemm_fp4_quantize, "bf16", "mx", t, ld, None, Q(rows, cols), S(rows, cols), rows, cols

    def read_back(t, ld):
        return g.gemm_fp4_dequantize, "bf16", "mx", Q(rows, cols), S(rows, cols), None, t, ld, rows, cols

    return linear_x, linear_c, product_c, quantize, read_back


OFF = "elements apart"
BAD = {
    "transposed": (lambda r, c: h(c, r).t(), lambda r, c: c),
    "transposed, its own stride": (lambda r, c: h(3 * c, r).t()[:, :c], lambda r, c: max(r, c)),
    "not transposed at all": (lambda r, c: h(c, r), lambda r, c: c),
    "every second column": (lambda r, c: h(r, 2 * c)[:, ::2], lambda r, c: 2 * c),
    "every second row": (lambda r, c: h(2 * r, c)[::2], lambda r, c: c),
    "a slice with its own width": (lambda r, c: h(r, c + 8)[:, :c], lambda r, c: c),
    "contiguous with another width": (lambda r, c: h(2 * r, c), lambda r, c: c + 8),
    "every second value": (lambda r, c: h(2 * r * c)[::2], lambda r, c: c),
    "a row repeated": (lambda r, c: h(2 * r * c)[:c].expand(r, c), lambda r, c: c),
    "three dimensions, uneven": (lambda r, c: h(2, r, c)[:, :r // 2], lambda r, c: c),
}
GOOD = {
    "flat": (lambda r, c: h(r * c), lambda r, c: c),
    "flat, wider rows": (lambda r, c: h(r * (c + 8)), lambda r, c: c + 8),
    "two dimensions": (lambda r, c: h(r, c), lambda r, c: c),
    "a slice": (lambda r, c: h(r, c + 8)[:, :c], lambda r, c: c + 8),
    "a slice off the front": (lambda r, c: h(r, c + 8)[:, 8:], lambda r, c: c + 8),
    "every second row": (lambda r, c: h(2 * r, c)[::2], lambda r, c: 2 * c),
    "more rows": (lambda r, c: h(r + 3, c + 4), lambda r, c: c + 4),
    "three dimensions": (lambda r, c: h(2, r // 2, c), lambda r, c: c),
    "three dimensions, a slice": (lambda r, c: h(2, r // 2, c + 8)[..., :c], lambda r, c: c + 8),
    "a transposed transposed": (lambda r, c: h(r, c).t().contiguous().t().contiguous(), lambda r, c: c),
}


@pytest.mark.parametrize("case", BAD)
def test_other_strides_are_refused(case):
    tensor, ld = BAD[case]
    for call in calls(M, N):
        fn, *args = call(tensor(M, N), ld(M, N))
        refused(fn, *args, match=OFF)


@pytest.mark.parametrize("case", GOOD)
def test_rows_of_the_leading_dimension_pass(case):
    tensor, ld = GOOD[case]
    for call in calls(M, N):
        fn, *args = call(tensor(M, N), ld(M, N))
        refused(fn, *args, match="CUDA device")


def test_one_row_or_one_column():
    """One row: the leading dimension says nothing.  One column: the rows' distance is all."""
    for call in calls(1, N):
        for t in (h(1, N), h(5, 2 * N), h(5, 2 * N)[2:3, :N]):
            fn, *args = call(t, N)
            refused(fn, *args, match="CUDA device")
        fn, *args = call(h(1, 2 * N)[:, ::2], N)
        refused(fn, *args, match=OFF)
    for call in calls(M, 1):
        fn, *args = call(h(M, 8)[:, 3:4], 8)
        refused(fn, *args, match="CUDA device")
        fn, *args = call(h(M, 8)[:, 3:4], 1)
        refused(fn, *args, match=OFF)


def test_nothing_to_read():
    """Empty calls look at the device alone, as before."""
    refused(g.gemm_fp4_linear, "bf16", "mx", h(K, M).t(), K, None, Q(N, K), S(N, K), None, h(N, M).t(), N, 0, N, K,
            match="CUDA device")
