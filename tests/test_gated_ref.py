"""The gated block's 64-bit reference against differences, and the entry points'
host-side refusals.  No GPU."""

import ctypes

import numpy as np
import pytest

import gated_ref as ref

import dense_matrix_multiply_gb300 as g


@pytest.fixture(scope="module")
def built():
    g.ensure_built()
    return g.load()


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_derivatives_against_differences(name):
    x = np.linspace(-8, 8, 4001)
    h = 1e-5
    a, da, d2 = ref.act(name, x)
    assert np.allclose((ref.act(name, x + h)[0] - ref.act(name, x - h)[0]) / (2 * h), da, atol=1e-8)
    assert np.abs(da).max() < 1.13
    assert np.abs((ref.act(name, x + h)[1] - ref.act(name, x - h)[1]) / (2 * h)).max() <= d2
    rng = np.random.default_rng(1)
    X, Wg, Wu, dZ = (rng.standard_normal(s) for s in ((5, 7), (7, 6), (7, 6), (5, 6)))
    grads = ref.backward(name, X, Wg, Wu, dZ)
    ops = [X, Wg, Wu]
    for i in range(3):
        V = rng.standard_normal(ops[i].shape)
        up, dn = [o.copy() for o in ops], [o.copy() for o in ops]
        up[i] += h * V
        dn[i] -= h * V
        diff = ((ref.forward(name, *up)[0] - ref.forward(name, *dn)[0]) * dZ).sum() / (2 * h)
        assert diff == pytest.approx((grads[i] * V).sum(), rel=1e-7)


def test_activations_at_known_points():
    assert ref.act("silu", np.array([0.0]))[0][0] == 0 and ref.act("silu", np.array([0.0]))[1][0] == 0.5
    assert ref.act("gelu", np.array([0.0]))[1][0] == 0.5
    assert ref.act("silu", np.array([1.0]))[0][0] == pytest.approx(0.7310585786300049)
    assert ref.act("gelu", np.array([1.0]))[0][0] == pytest.approx(0.8411919906082768)


def test_host_side_errors(built):
    buf = ctypes.create_string_buffer(1 << 17)
    p = (ctypes.addressof(buf) + 15) // 16 * 16
    X, Wg, Wu, Z, G, U, dZ, dX, dWg, dWu = (p + 8192 * i for i in range(10))
    f = built.gemm_gated
    ok = dict(d=2, a=0, X=X, Wg=Wg, Wu=Wu, Z=Z, G=None, U=None, M=4, N=16, K=8)
    call = lambda **k: f(*{**ok, **k}.values())
    assert call(d=0) == 1 and call(a=2) == 1 and call(M=-1) == 1 and call(N=-8) == 1 and call(K=-4) == 1
    assert call(G=G + 2, U=U) == 1 and b"on 4" in built.gemm_last_error()
    assert call(X=X + 1) == 1 and call(Z=None) == 1 and call(Wu=None) == 1
    assert call(G=G) == 1                        # G without U
    assert call(Z=X + 16) == 2 and call(G=G, U=G + 64) == 2 and call(G=Z + 16, U=U) == 2
    assert call(M=0) == 0 and built.gemm_last_kernel() == b"noop"
    b = built.gemm_gated_backward
    okb = dict(d=2, a=1, X=X, Wg=Wg, Wu=Wu, G=G, U=U, dZ=dZ, dX=dX, dWg=dWg, dWu=dWu, M=4, N=16, K=8)
    callb = lambda **k: b(*{**okb, **k}.values())
    assert callb(d=0) == 1 and callb(a=-1) == 1 and callb(K=-8) == 1 and callb(dX=dX + 1) == 1 and callb(U=U + 2) == 1
    assert callb(G=None) == 1 and callb(dZ=None) == 1 and callb(Wg=None) == 1 and callb(X=None) == 1
    assert callb(dX=X) == 2 and callb(dWu=dWg + 16) == 2 and callb(dWg=G) == 2
    assert callb(dX=None, dWg=None, dWu=None) == 0 and callb(K=0) == 0
    with pytest.raises(ValueError):
        g.gemm_gated("f32", "silu", 0, 0, 0, 0, None, None, 1, 8, 8)
    with pytest.raises(ValueError):
        g.gemm_gated_backward("bf16", "relu", 0, 0, 0, 0, 0, 0, 0, 0, 0, 1, 8, 8)
