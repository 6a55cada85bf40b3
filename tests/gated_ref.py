"""Gated feed-forward block in 64 bits, from its definition, and how far a kernel
with FP32 sums and 16-bit results may be from it."""

from __future__ import annotations

import numpy as np

C = np.sqrt(2 / np.pi)
ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}     # half an ulp, relative
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25}
FAST = 2.0 ** -16   # exponential and division: a few ulps of FP32, and |z| 2^-23 of the exponent, |z| < 100


def act(name, g):
    """act(g), act'(g) and a bound of |act''|."""
    if name == "silu":
        s = 1 / (1 + np.exp(-g))
        return g * s, s * (1 + g * (1 - s)), 0.5
    t = np.tanh(C * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * C * (1 + 3 * 0.044715 * g * g), 1.2


def forward(name, X, Wg, Wu):
    G, U = X @ Wg, X @ Wu
    return act(name, G)[0] * U, G, U


def backward(name, X, Wg, Wu, dZ):
    G, U = X @ Wg, X @ Wu
    a, da, _ = act(name, G)
    dU, dG = dZ * a, dZ * U * da
    return dG @ Wg.T + dU @ Wu.T, X.T @ dG, X.T @ dU


def sum_error(A, B):
    """FP32 sums of A B in blocks of 16, each step off by 2^-23 of the magnitudes so far."""
    return (A.shape[1] / 16 + 16) * 2.0 ** -23 * (np.abs(A) @ np.abs(B))


def forward_tolerance(name, X, Wg, Wu, dtype):
    """Of Z, G and U.  |act'| <= 1.13."""
    Z, G, U = forward(name, X, Wg, Wu)
    eG, eU = sum_error(X, Wg), sum_error(X, Wu)
    a = np.abs(act(name, G)[0])
    e = 1.13 * eG * (np.abs(U) + eU) + a * eU + FAST * a * np.abs(U)
    return e + ROUND[dtype] * (np.abs(Z) + e) + TINY[dtype], eG, eU


def backward_tolerance(name, X, Wg, Wu, dZ, dtype):
    """Of dX, dWg and dWu: the error of dG and dU before their rounding summed in
    full, their roundings (independent, uniform within half an ulp: deviation
    ROUND / sqrt(3) each) at eight deviations, the sums' and the result's own."""
    G, U = X @ Wg, X @ Wu
    eG, eU = sum_error(X, Wg), sum_error(X, Wu)
    a, da, d2 = act(name, G)
    dU, dG = dZ * a, dZ * U * da
    z = np.abs(dZ)
    fU = z * (1.13 * eG + FAST * np.abs(a)) + TINY[dtype]
    fG = z * ((np.abs(U) + eU) * (d2 * eG + FAST * (np.abs(da) + np.abs(G))) + eU * np.abs(da)) + TINY[dtype]

    def out(parts):
        want = sum(p @ q for p, _, q in parts)
        e = sum(f @ np.abs(q) + sum_error(p, q) for p, f, q in parts)
        r2 = sum((p * p) @ (q * q) for p, _, q in parts)
        e = e + 8 * ROUND[dtype] / np.sqrt(3) * np.sqrt(r2)
        return e + ROUND[dtype] * (np.abs(want) + e) + TINY[dtype]

    dX = out([(dG, fG, Wg.T), (dU, fU, Wu.T)])
    dWg = out([(dG.T, fG.T, X)]).T
    dWu = out([(dU.T, fU.T, X)]).T
    return dX, dWg, dWu
