"""4-bit block-scaled formats on the CPU, from their definition (include/gemm.h):
quantisation with every FP32 step in FP32, values and products in 64 bits."""

from __future__ import annotations

import numpy as np

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
BLOCK = {"mx": 32, "nv": 16}


def e4m3_value(b):
    """Values of E4M3FN bytes (127 and 255 are NaN)."""
    b = np.asarray(b, dtype=np.int64)
    e, f = (b >> 3) & 15, b & 7
    v = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    return np.where((b & 127) == 127, np.nan, np.where(b & 128, -v, v))


def nearest(v, table):
    """Index of the nearest entry of an increasing table (last index: saturation),
    ties to the even index, in 64 bits."""
    v = np.asarray(v, dtype=np.float64)
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = v - table[lo], table[hi] - v
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


E4M3 = e4m3_value(np.arange(127))


def quantize(fmt, a, g=None):
    """a: float32 [M,K] holding 16-bit values.  Codes [M,K] (0 .. 15) and scale
    bytes [M, ceil(K/B)]."""
    B, (M, K) = BLOCK[fmt], a.shape
    g = np.float32(1.0 if g is None else g)
    nb = -(-K // B)
    x = np.zeros((M, nb * B), dtype=np.float32)
    x[:, :K] = a
    x = x.reshape(M, nb, B)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], np.float32(0), x)
    amax = np.abs(x).max(-1)
    if fmt == "mx":
        with np.errstate(divide="ignore"):
            e = np.where(amax > 0, np.clip(np.frexp(amax.astype(np.float64))[1] - 3, -127, 125), -127)
        byte = e + 127
        q = x.astype(np.float64) / np.exp2(e.astype(np.float64))[..., None]
    else:
        byte = nearest(np.minimum((amax / (np.float32(6) * g)).astype(np.float64), 448.0), E4M3)
        step = (E4M3[byte].astype(np.float32) * g)[..., None]
        with np.errstate(divide="ignore", invalid="ignore"):
            q = np.where(step > 0, x / step, np.float32(0)).astype(np.float64)
    code = nearest(np.abs(q), LEVELS) + 8 * (np.signbit(q) & (np.abs(q) > 0.25))
    byte = np.where(bad, 255 if fmt == "mx" else 127, byte)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(M, -1)[:, :K].astype(np.uint8), byte.astype(np.uint8)


def values(fmt, code, byte, g=None):
    """64-bit values of codes [M,K] and scale bytes."""
    B, K = BLOCK[fmt], code.shape[1]
    v = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)
    if fmt == "mx":
        s = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
    else:
        s = e4m3_value(byte) * np.float64(1.0 if g is None else np.float32(g))
    return v * np.repeat(s, B, axis=1)[:, :K]


def pack(code):
    """Two codes to a byte, the even k low, rows padded to 32 codes."""
    M, K = code.shape
    p = np.zeros((M, -(-K // 32) * 32), dtype=np.uint8)
    p[:, :K] = code
    return p[:, 0::2] | (p[:, 1::2] << 4)


def tile_scales(fmt, byte, K):
    """Scale bytes in the stored order, padding 0."""
    M, nb = byte.shape
    atoms = -(-K // 256) * (64 // BLOCK[fmt])
    out = np.zeros(-(-M // 128) * atoms * 512, dtype=np.uint8)
    r, j = np.arange(M)[:, None], np.arange(nb)[None, :]
    out[((r // 128) * atoms + j // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + j % 4] = byte
    return out


def tolerance(a, b, C, dtype, K):
    """Bound of |C_gpu - C| for a product of 64-bit values a [M,K], b [N,K]: half
    an ulp of the output type on C (and on the error below it), and FP32 sums of
    exact products in blocks of 16 or more k, each step off by at most 2^-23 of
    the magnitudes added so far."""
    S = np.abs(a) @ np.abs(b).T
    acc = S * (K / 16 + 16) * 2.0 ** -23
    u, tiny = (2.0 ** -8, 2.0 ** -133) if dtype == "bf16" else (2.0 ** -11, 2.0 ** -25)
    return acc + u * (np.abs(C) + acc) + tiny
