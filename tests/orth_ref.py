"""The orthogonalised update in 64 bits, from its definition, and how far a kernel with
half-precision operands (X in two halves) and FP32 sums may be from it."""

from __future__ import annotations

import numpy as np

ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}     # a 16-bit rounding, relative: torch.finfo(t).eps / 2
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}    # half the least subnormal
H, HT = 2.0 ** -11, 2.0 ** -25                     # of half
QUINTIC = (3.4445, -4.7750, 2.0315)


def steps_of(G, steps, coefficients=QUINTIC):
    """X before every step, wide (rows at most columns), and after the last."""
    a, b, c = coefficients
    X = G if G.shape[0] <= G.shape[1] else G.T
    norm = np.sqrt((X * X).sum())
    X = X / norm if norm > 0 else X
    out = [X]
    for _ in range(steps):
        A = X @ X.T
        X = a * X + (b * A + c * (A @ A)) @ X
        out.append(X)
    return out


def orthogonalize(G, steps, coefficients=QUINTIC):
    X = steps_of(G, steps, coefficients)[-1]
    return X if G.shape[0] <= G.shape[1] else X.T


def sum_error(K, magnitudes):
    """FP32 sums of K products in blocks of 16, each step off by 2^-23 of the magnitudes so far."""
    return (K / 16 + 16) * 2.0 ** -23 * magnitudes


def one_step_tolerance(G, dtype, coefficients=QUINTIC):
    """Element by element, of one step: A rounded to half (and its sum, and |G|'s factor
    twice), B from it, rounded to half, its sum; B X, its sum and the FP32 operations
    behind it; the result's rounding.  X itself goes in exact, but for elements that fall
    among half's subnormals after |G| is scaled to 2^14: 2^-25 each."""
    a, b, c = map(abs, coefficients)
    wide = G if G.shape[0] <= G.shape[1] else G.T
    norm = np.sqrt((wide * wide).sum())
    X, m, n = wide / norm, *wide.shape
    x0 = 2.0 ** -25 / 2.0 ** 14
    A, aX = X @ X.T, np.abs(X)
    aa = aX @ aX.T
    eA = sum_error(n, aa) + 4 * 2.0 ** -24 * np.abs(A) + 2 * x0 * aX.sum(1).max()
    eA = eA + H * (np.abs(A) + eA) + HT
    B = coefficients[1] * A + coefficients[2] * (A @ A)
    abs_a = np.abs(A) + eA
    eB = b * eA + c * (eA @ abs_a + abs_a @ eA + sum_error(m, abs_a @ abs_a)) + 3 * 2.0 ** -24 * (b * abs_a + c * abs_a @ abs_a)
    eB = eB + H * (np.abs(B) + eB) + HT
    want = coefficients[0] * X + B @ X
    e = eB @ aX + sum_error(m, (np.abs(B) + eB) @ aX) + (a + np.abs(B).sum(1).max()) * x0
    e = e + 4 * 2.0 ** -24 * (a * aX + np.abs(want) + e)
    e = e + ROUND[dtype] * (np.abs(want) + e) + TINY[dtype]
    return e if G.shape[0] <= G.shape[1] else e.T


def frobenius_tolerance(G, steps, dtype, coefficients=QUINTIC):
    """Of the difference's Frobenius norm after any number of steps.  A step's map has
    derivative at most L = max |p'|, |p / x| over the singular values met (its divided
    differences); what a step adds is carried on by the L of the steps after it.  Added:
    A's rounding dA (deviation H / sqrt 3 of each element, independent, |dA| at most that
    times |A|_F with room for chance: twice) through b dA X + c (dA A + A dA) X; B's, the
    same way, times |X|_2; hi alone in B X: H |X|_F |B|_2; lo's rounding, 2^-22 |X|_F; and
    FP32 sums, 2^-20 of the three products' norms.  The result's rounding in the end."""
    a, b, c = coefficients
    X = steps_of(G, steps, coefficients)
    s = [np.linalg.svd(x, compute_uv=False) for x in X]
    total = 0.0
    for x, sv in zip(X[:-1], s[:-1]):
        top, fro = sv[0], np.sqrt((sv * sv).sum())
        grid = np.linspace(0, top * 1.02, 2001)
        d = np.abs(a + 3 * b * grid ** 2 + 5 * c * grid ** 4).max()
        q = np.abs(a + b * grid ** 2 + c * grid ** 4).max()
        Af = np.sqrt((sv ** 4).sum())
        Bv = b * sv ** 2 + c * sv ** 4
        Bf, B2 = np.sqrt((Bv * Bv).sum()), np.abs(Bv).max()
        r = 2 * H / np.sqrt(3)
        m = len(sv)
        added = (r * Af + m * HT) * (abs(b) + 2 * abs(c) * top ** 2) * top + (r * Bf + m * HT) * top
        added += H / np.sqrt(3) * fro * B2 + 2.0 ** -22 * abs(a) * fro + 2.0 ** -20 * (Af * top * (abs(b) + 2 * abs(c) * top * top) + Bf * top + abs(a) * fro)
        total = total * max(d, q) + added
    fro = np.sqrt((s[-1] ** 2).sum())
    return total + ROUND[dtype] / np.sqrt(3) * fro * 1.1 + TINY[dtype] * np.sqrt(X[-1].size)
