"""Pins of the CPU reference of the 4-bit formats, and the entry points' host-side
refusals and sizes.  No GPU."""

import ctypes

import numpy as np
import pytest

import fp4_ref as ref

import dense_matrix_multiply_gb300 as g


@pytest.fixture(scope="module")
def built():
    g.ensure_built()
    return g.load()


def test_ties_go_to_the_even_code():
    # one block whose largest magnitude is 4: MX step 1
    x = np.zeros((1, 32), dtype=np.float32)
    x[0, :9] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -0.75, 0.2500001]
    code, byte = ref.quantize("mx", x)
    assert byte[0, 0] == 127
    assert code[0, :9].tolist() == [6, 0, 2, 2, 4, 4, 6, 10, 1]


def test_mx_scale_is_the_power_of_two_two_below_amax():
    for amax, byte in ((4.0, 127), (7.9, 127), (8.0, 128), (3.99, 126), (1.0, 125), (2.0 ** -126, 0), (0.0, 0),
                       (2.0 ** -125, 0), (2.0 ** -124, 1), (np.float32(3.3e38), 252)):
        x = np.full((1, 32), amax, dtype=np.float32)
        assert ref.quantize("mx", x)[1][0, 0] == byte, amax
    assert ref.values("mx", *ref.quantize("mx", np.full((1, 32), 7.9, dtype=np.float32)))[0, 0] == 6.0


def test_nv_scale_and_step():
    x = np.full((1, 16), 6.0, dtype=np.float32)
    code, byte = ref.quantize("nv", x, 1.0)
    assert ref.e4m3_value(byte[0, 0]) == 1.0 and code[0, 0] == 7
    code, byte = ref.quantize("nv", x * 1000, 1.0)  # 1000 saturates at 448
    assert ref.e4m3_value(byte[0, 0]) == 448.0 and code[0, 0] == 7
    code, byte = ref.quantize("nv", x * np.float32(1e-6), 1.0)  # the scale underflows
    assert byte[0, 0] == 0 and code[0, 0] == 0


def test_scale_offsets_cover_the_buffer_once():
    for fmt in ("mx", "nv"):
        byte = (1 + np.arange(256 * 24) % 200).reshape(256, 24).astype(np.uint8)
        K = 24 * ref.BLOCK[fmt]
        t = ref.tile_scales(fmt, byte, K)
        assert np.count_nonzero(t) == byte.size
        assert t[(1 * (-(-K // 256) * (64 // ref.BLOCK[fmt])) + 2) * 512 + 5 * 16 + 1 * 4 + 3] == byte[128 + 37, 11]


def test_sizes(built):
    assert g.gemm_fp4_code_bytes(3, 33) == 3 * 32 and g.gemm_fp4_code_bytes(5, 0) == 0
    assert g.gemm_fp4_scale_bytes("mx", 1, 1) == 1024 and g.gemm_fp4_scale_bytes("nv", 129, 257) == 2 * 2 * 2048
    assert g.gemm_fp4_scale_bytes("mx", 0, 256) == 0 and g.gemm_fp4_code_bytes(-1, 4) == -1
    # one row of a matrix with 2^31 - 1 rows: no overflow of 32 bits
    assert g.gemm_fp4_scale_bytes("nv", 2 ** 31 - 1, 4096) == 2 ** 24 * 64 * 512
    assert built.gemm_fp4_scale_bytes(2, 4, 4) == -1


def test_host_side_errors(built):
    buf = ctypes.create_string_buffer(1 << 17)
    p = (ctypes.addressof(buf) + 15) // 16 * 16
    A, Q, S, G, C = p, p + 16384, p + 32768, p + 49152, p + 65536
    q = built.gemm_fp4_quantize
    assert q(0, 0, A, 64, None, Q, S, 4, 64) == 1 and q(2, 2, A, 64, None, Q, S, 4, 64) == 1   # enums
    assert q(2, 0, A, 64, None, Q, S, -1, 64) == 1 and q(2, 0, A, 63, None, Q, S, 4, 64) == 1  # sizes
    assert q(2, 0, None, 64, None, Q, S, 4, 64) == 1 and q(2, 0, A, 64, None, Q, None, 4, 64) == 1
    assert q(2, 0, A, 64, G, Q, S, 4, 64) == 1                   # MX has no tensor scale
    assert b"tensor scale" in built.gemm_last_error()
    assert q(2, 1, A, 64, G, Q + 8, S, 4, 64) == 1               # alignment
    assert q(2, 1, A, 64, G, A + 16, S, 4, 64) == 2 and q(2, 1, A, 64, S + 16, Q, S, 4, 64) == 2
    assert q(2, 1, A, 64, G, Q, S, 0, 64) == 0 and q(2, 1, A, 64, G, Q, S, 4, 0) == 0
    assert q(2, 1, A + 1, 64, G, Q, S, 4, 64) == 1 and q(2, 1, A, 64, G + 2, Q, S, 4, 64) == 1
    assert b"on 4" in built.gemm_last_error()
    d = built.gemm_fp4_dequantize
    assert d(2, 1, Q, S, G, None, 64, 4, 64) == 1 and d(2, 1, Q, S, G, Q, 64, 4, 64) == 2
    assert d(2, 1, Q, S, A + 4, A, 64, 4, 64) == 2               # the scale inside the output
    f = built.gemm_fp4
    assert f(2, 1, Q, S, G, Q, S, G, C + 1, 4, 4, 4, 64) == 1 and f(2, 1, Q, S, G, Q, S, G + 1, C, 4, 4, 4, 64) == 1
    assert f(2, 1, Q, S, G, Q, S, G, C, 3, 4, 4, 64) == 1        # ldc
    assert f(2, 1, Q, S, G, Q, S, G, None, 4, 4, 4, 64) == 1 and f(2, 1, Q, None, G, Q, S, G, C, 4, 4, 4, 64) == 1
    assert f(2, 1, Q, S, G, Q, S, G, S, 4, 4, 4, 64) == 2 and f(2, 1, Q, S, C, Q, S, G, C, 4, 4, 4, 64) == 2
    assert f(2, 0, Q, S, G, Q, S, None, C, 4, 4, 4, 64) == 1
    assert f(2, 1, Q, S, G, Q, S, G, C, 4, 0, 4, 64) == 0
    li = built.gemm_fp4_linear
    assert li(2, 1, A + 1, 64, G, Q, S, G, C, 4, 4, 4, 64) == 1 and li(2, 1, A, 64, G + 2, Q, S, G, C, 4, 4, 4, 64) == 1
    assert li(2, 1, A, 63, G, Q, S, G, C, 4, 4, 4, 64) == 1 and li(2, 1, None, 64, G, Q, S, G, C, 4, 4, 4, 64) == 1
    assert li(2, 1, A, 64, G, Q, S, G, A + 8, 4, 4, 4, 64) == 2
    with pytest.raises(ValueError):
        g.gemm_fp4_quantize("f32", "mx", 0, 4, None, 0, 0, 1, 4)
    with pytest.raises(ValueError):
        g.gemm_fp4("bf16", "fp4", 0, 0, None, 0, 0, None, 0, 4, 1, 4, 4)
