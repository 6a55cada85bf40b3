"""Softmax cross entropy of a linear head and its gradients in 64 bits, from the
definitions, and how far a kernel with FP32 sums and 16-bit results may be from them."""

from __future__ import annotations

import numpy as np

ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}     # a 16-bit rounding, relative: torch.finfo(t).eps / 2
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}    # half the least subnormal
U = 2.0 ** -24                                     # an FP32 rounding


def counts(t, N):
    return (t >= 0) & (t < N)


def forward(X, W, t):
    Z = X @ W.T
    m = Z.max(1)
    lse = m + np.log(np.exp(Z - m[:, None]).sum(1))
    c = counts(t, W.shape[0])
    return np.where(c, lse - Z[np.arange(len(t)), np.where(c, t, 0)], 0.0), lse, Z


def backward(X, W, t, dloss):
    _, lse, Z = forward(X, W, t)
    c = counts(t, W.shape[0])
    dZ = np.exp(Z - lse[:, None])
    dZ[np.nonzero(c)[0], t[c]] -= 1
    dZ *= np.where(c, dloss, 0)[:, None]
    return dZ @ W, np.where(c[:, None], X, 0).T.dot(dZ).T, dZ


def sum_error(A, B):
    """FP32 sums of A B in blocks of 16, each step off by 2^-23 of the magnitudes so far."""
    return (A.shape[1] / 16 + 16) * 2.0 ** -23 * (np.abs(A) @ np.abs(B))


def logit_error(X, W):
    return sum_error(X, W.T)


def forward_tolerance(X, W, t):
    """Of loss and lse.  exp is 1-Lipschitz in its exponent's logarithm: lse moves by at most
    the largest logit error.  Exponents are products with log2 e rounded once each (|z|
    log2 e 2^-24, twice: the term and the maximum) and taken down the tiles' and the joining
    kernel's maxima (one rounding of |m| each, at most N / 4096 + 32 of a warp's and 32 of
    warps, but a maximum that stays costs nothing: two count); 2^x is two units of 2^-23 off,
    a sum of at most 8 + 4 + N / 4096 + 64 additions in a row; the logarithm and the last
    two additions."""
    loss, lse, Z = forward(X, W, t)
    N = W.shape[0]
    top = np.abs(Z).max(1)
    e = logit_error(X, W).max(1) + 4 * 1.4427 * top * U + (4 + 4 + 8 + 4 + N / 4096 + 64) * U + 2 * np.abs(lse) * U + 4 * U
    c = counts(t, N)
    zt = np.abs(Z[np.arange(len(t)), np.where(c, t, 0)])
    return np.where(c, e + logit_error(X, W)[np.arange(len(t)), np.where(c, t, 0)] + (np.abs(loss) + zt) * U, 0), e


def backward_tolerance(X, W, t, dloss, dtype):
    """dZ before its rounding: the exponent's error (a logit's, lse's, two roundings) times
    p, 2^x's own, a subtraction and a product; its roundings to 16 bits (independent, uniform
    within half a step: deviation ROUND / sqrt(3) each) at eight deviations, and in half at
    most 2^-25 of subnormals after scaling by at least 2^14 / max |dloss|; the sums' errors;
    the result's rounding."""
    dX, dW, dZ = backward(X, W, t, dloss)
    _, lse, Z = forward(X, W, t)
    _, el = forward_tolerance(X, W, t)
    c = counts(t, W.shape[0])
    d = np.abs(np.where(c, dloss, 0))[:, None]
    p = np.exp(Z - lse[:, None])
    f = d * (p * (logit_error(X, W) + el[:, None] + 2 * 1.4427 * (np.abs(Z) + np.abs(lse)[:, None]) * U + 6 * U) + 2 * U * np.abs(dZ) / np.maximum(d, 1e-300))
    f += 2.0 ** -25 * d.max() * 2.0 ** -14 if dtype == "f16" else TINY["bf16"]
    Xc = np.where(c[:, None], X, 0)

    def out(A, fA, B, want):
        e = fA @ np.abs(B) + sum_error(A, B) + 8 * ROUND[dtype] / np.sqrt(3) * np.sqrt((A * A) @ (B * B))
        return e + ROUND[dtype] * (np.abs(want) + e) + TINY[dtype]

    return out(dZ, f, W, dX), out(dZ.T, f.T, Xc, dW)
