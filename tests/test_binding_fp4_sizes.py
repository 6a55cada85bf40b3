"""gemm_fp4_code_bytes and gemm_fp4_scale_bytes (no GPU): an unknown format is a
ValueError, as in the calls that take one; sizes as the header's layout has them."""

import pytest

import dense_matrix_multiply_gb300 as g


@pytest.fixture(scope="module", autouse=True)
def built(lib):
    return lib.load()


@pytest.mark.parametrize("fmt", ["fp4", "NV", "", None, 0])
def test_unknown_format(fmt):
    with pytest.raises(ValueError, match=r"format 'mx' \| 'nv'"):
        g.gemm_fp4_scale_bytes(fmt, 4, 64)


@pytest.mark.parametrize("rows,K", [(0, 0), (0, 5), (1, 1), (128, 256), (129, 257), (3, 0)])
def test_sizes(rows, K):
    assert g.gemm_fp4_code_bytes(rows, K) == rows * (-(-K // 32) * 16)
    for fmt, per in (("mx", 1024), ("nv", 2048)):
        assert g.gemm_fp4_scale_bytes(fmt, rows, K) == -(-rows // 128) * -(-K // 256) * per


def test_negative_sizes():
    assert g.gemm_fp4_code_bytes(-1, 5) == -1 and g.gemm_fp4_scale_bytes("nv", 5, -1) == -1
