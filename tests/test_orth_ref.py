"""The 64-bit update: singular values follow the scalar polynomial, vectors stay."""

import numpy as np
import pytest

import orth_ref as ref


@pytest.mark.parametrize("shape", [(6, 20), (20, 6), (9, 9), (1, 5)])
def test_singular_values_follow_the_polynomial(shape):
    G = np.random.default_rng(0).standard_normal(shape)
    a, b, c = ref.QUINTIC
    U, s, V = np.linalg.svd(G, full_matrices=False)
    x = s / np.sqrt((s * s).sum())
    for _ in range(5):
        x = a * x + b * x ** 3 + c * x ** 5
    assert np.allclose(ref.orthogonalize(G, 5), (U * x) @ V, atol=1e-10)
    assert x.min() > 0.3 and x.max() < 1.3


def test_tolerances_are_met_by_an_emulation_and_not_by_a_wrong_step():
    """The kernel's roundings in numpy on 64-bit products; a coefficient off by 5 % fails."""
    G = np.random.default_rng(1).standard_normal((40, 100)).astype(np.float16).astype(np.float64)
    half = lambda x: x.astype(np.float16).astype(np.float64)
    for q in (ref.QUINTIC, (3.4445, -4.7750 * 1.05, 2.0315)):
        X = G / np.sqrt((G * G).sum())
        hi, lo = X, 0 * X
        for step in range(5):
            A = half(hi @ hi.T)
            B = half(q[1] * A + q[2] * (A @ A))
            X = q[0] * (hi + lo) + B @ hi
            if step == 0:
                got = half(X)
                good = (np.abs(got - ref.orthogonalize(G, 1)) <= ref.one_step_tolerance(G, "f16")).all()
                assert good == (q == ref.QUINTIC)
            hi = half(X)
            lo = X - hi
        off = np.linalg.norm(half(X) - ref.orthogonalize(G, 5))
        assert (off <= ref.frobenius_tolerance(G, 5, "f16")) == (q == ref.QUINTIC)
