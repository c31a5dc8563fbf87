"""Plain float64 forms of the 8-bit operators (test infrastructure only).

Codes are the e4m3 values themselves (float64); ``e4m3_bytes`` maps them to
their encoding.  Token scales are [ceil(d / 128), M], weight scales
[ceil(N / 128), ceil(K / 128)].
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
MAX_CODE = 448.0
FLOOR = 1e-12


def e4m3_table() -> np.ndarray:
    """Value of each of the 256 e4m3 encodings: sign, 4 exponent bits (bias 7),
    3 fraction bits, no infinities, NaN at 0x7F and 0xFF."""
    out = np.empty(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        v = (1 + f / 8) * 2.0 ** (e - 7) if e else f / 8 * 2.0 ** -6
        out[b] = np.nan if (e, f) == (15, 7) else v
    out[128:] *= -1
    return out


def round_e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value by search in the table, ties to the even fraction, saturating."""
    pos = e4m3_table()[:127]
    a = np.abs(np.asarray(v, np.float64))
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    mid = (pos[lo] + pos[hi]) / 2
    up = (a > mid) | ((a == mid) & (hi % 2 == 0))
    r = np.where(up, pos[hi], pos[lo])
    return np.where(np.isnan(a), np.nan, np.copysign(r, v))


def e4m3_bytes(v: np.ndarray) -> np.ndarray:
    """Encoding of exact e4m3 values (zeros keep their sign)."""
    pos = e4m3_table()[:127]
    b = np.searchsorted(pos, np.abs(v)).astype(np.uint8)
    assert np.array_equal(pos[b], np.abs(v))
    return b | (np.signbit(v).astype(np.uint8) << 7)


def _quant(v, rows):
    M, d = v.shape
    codes = np.empty_like(v)
    nr, nb = -(-M // rows), -(-d // BLOCK)
    scale = np.empty((nr, nb))
    for r in range(nr):
        for b in range(nb):
            at = np.s_[r * rows:(r + 1) * rows, b * BLOCK:(b + 1) * BLOCK]
            m = np.abs(v[at]).max()
            if not np.isfinite(m):
                codes[at], scale[r, b] = np.nan, np.nan
                continue
            m = max(m, FLOOR)
            codes[at], scale[r, b] = round_e4m3(v[at] * MAX_CODE / m), m / MAX_CODE
    return codes, scale


def quant_tokens(v):
    codes, scale = _quant(np.asarray(v, np.float64), 1)
    return codes, scale.T.copy()


def quant_block(v):
    return _quant(np.asarray(v, np.float64), BLOCK)


def norm_quant(h, weight, eps):
    """h: the stored sum of x and residual -> codes and scales of its RMSNorm times weight."""
    h = np.asarray(h, np.float64)
    rms = np.sqrt((h * h).mean(axis=1) + eps)
    codes, scale = quant_tokens(h if weight is None else h * np.asarray(weight, np.float64))
    return codes, scale / rms


def token_values(codes, scale):
    return codes * np.repeat(np.asarray(scale, np.float64).T, BLOCK, axis=1)[:, :codes.shape[1]]


def block_values(codes, scale):
    s = np.repeat(np.repeat(np.asarray(scale, np.float64), BLOCK, axis=0), BLOCK, axis=1)
    return codes * s[:codes.shape[0], :codes.shape[1]]


def product(a, a_scale, w, w_scale):
    """(P, sum of the magnitudes of P's terms): the second bounds the rounding of any fp32 summation."""
    A, W = token_values(a, a_scale), block_values(w, w_scale)
    return A @ W.T, np.abs(A) @ np.abs(W).T


def silu(g):
    return g / (1.0 + np.exp(-g))


def gated(a, a_scale, wg, wg_scale, wu, wu_scale):
    """(z, bound on the error of an fp32 z for products with relative error e: e * second + third)."""
    g, ga = product(a, a_scale, wg, wg_scale)
    u, ua = product(a, a_scale, wu, wu_scale)
    z = silu(g) * u
    # |silu'| < 1.1; the fp32 exp, division and two products add a few roundings of z
    return z, 1.1 * ga * np.abs(u) + np.abs(silu(g)) * ua, np.abs(z) * 2.0 ** -20
