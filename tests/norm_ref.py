"""Root-mean-square norm and its gradients in 64 bits, from the definitions, and how far
a kernel with FP32 sums and 16-bit (or E4M3) results may be from them."""

from __future__ import annotations

import numpy as np

ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}     # a 16-bit rounding, relative: torch.finfo(t).eps / 2
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}    # half the least subnormal
U = 2.0 ** -24                                     # an FP32 rounding


def sum_roundings(K):
    """Roundings that a term of a row's sum goes through: 32 of its thread (or K / 512 of a
    thread of a long row), five shuffles, sixteen warps."""
    return 32 + K / 512 + 5 + 16


def forward(H, w, eps):
    """rstd [M] and Y [M,K]."""
    r = 1 / np.sqrt((H * H).mean(1) + eps)
    return r, H * w * r[:, None]


def forward_error(K):
    """Relative, of rstd: the squares and their sum (all positive), halved by the root; a
    division by K, eps added, the root and the reciprocal.  Of Y: two products more."""
    r = (0.5 * (1 + sum_roundings(K)) + 4) * U
    return r, r + 3 * U


def round_tolerance(Y, rel, dtype):
    return np.abs(Y) * (rel + ROUND[dtype] * (1 + rel)) + TINY[dtype]


def e4m3_tolerance(V, rel):
    """Of codes of the values V = Y / scale, |V| <= 448: half a step, and the FP32
    operations before it (Y and amax each `rel` off, two divisions and a product)."""
    return np.maximum(np.abs(V) * 2.0 ** -4, 2.0 ** -10) + np.abs(V) * (2 * rel + 4 * U)


def backward(H, w, dY, dH, eps):
    r, _ = forward(H, w, eps)
    X = H * r[:, None]
    g = dY * w
    dX = r[:, None] * (g - X * (g * X).mean(1, keepdims=True)) + dH
    return dX, (dY * X).sum(0)


def backward_tolerance(H, w, dY, dH, eps, dtype):
    """dX: |rstd g|, three roundings and rstd's error; |rstd X| mean|g X|, the sum's
    roundings and rstd's error four times; the addition of dH; one rounding to dtype.  dw: X
    twice off, the sums over a CTA's rows (at most M / 152 + 1), over partials (608 / 8 a warp)
    and over eight warps."""
    (M, K), (er, _) = H.shape, forward_error(H.shape[1])
    r, _ = forward(H, w, eps)
    X = H * r[:, None]
    g = dY * w
    dX, _ = backward(H, w, dY, dH, eps)
    e = np.abs(r[:, None] * g) * (er + 4 * U)
    e += np.abs(r[:, None] * X) * np.abs(g * X).mean(1, keepdims=True) * (4 * er + (sum_roundings(K) + 8) * U)
    e += (np.abs(dX) + np.abs(dH)) * 2 * U
    return e + ROUND[dtype] * (np.abs(dX) + e) + TINY[dtype], np.abs(dY * X).sum(0) * (er + (M / 152 + 90) * U)
