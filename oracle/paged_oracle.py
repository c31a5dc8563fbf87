"""Rotary positions and the paged 4-bit cache in float64 numpy: what the kernels are compared with.

A batch is (table [B, pages], lengths [B], cu [B + 1] or None, page size); a cache (k_q, k_s, v_q, v_s) with codes
[pages, Hkv, page size, d / 2] and scales [pages, Hkv, page size].
"""
from __future__ import annotations

import numpy as np


def hadamard(d: int) -> np.ndarray:
    h = np.ones((1, 1))
    while h.shape[0] < d:
        h = np.kron(np.array([[1.0, 1.0], [1.0, -1.0]]), h)
    return h / np.sqrt(d)


def rope(x, positions, inv_freq, interleaved=False, scale=1.0):
    """x [N, H, d]; pairs of the first 2 len(inv_freq) elements turned."""
    y = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    a = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)
    c, s = scale * np.cos(a)[:, None, :], scale * np.sin(a)[:, None, :]
    lo = np.arange(half) * 2 if interleaved else np.arange(half)
    hi = lo + 1 if interleaved else lo + half
    u, w = y[..., lo].copy(), y[..., hi].copy()
    y[..., lo], y[..., hi] = u * c - w * s, w * c + u * s
    return y


def places(lengths, cu, n):
    """[(sequence or -1, position)] of n tokens."""
    out = []
    for i in range(n):
        if cu is None:
            out.append((i, int(lengths[i]) - 1))
            continue
        b = [j for j in range(len(lengths)) if cu[j] <= i < cu[j + 1]]
        out.append((b[0], int(lengths[b[0]]) - int(cu[b[0] + 1]) + i) if b else (-1, -1))
    return out


def codes(packed) -> np.ndarray:
    p = np.asarray(packed).astype(np.int64)
    c = np.stack([p & 15, p >> 4], -1).reshape(*p.shape[:-1], -1)
    return np.where(c > 7, c - 16, c).astype(np.float64)


def tokens(cache, table_row, ps, upto, which):
    """(codes [upto, Hkv, d], scales [upto, Hkv]) of a sequence's first tokens; a page that is not there: None."""
    q, s = cache[2 * which], cache[2 * which + 1]
    t = np.arange(upto)
    page = np.asarray(table_row)[t // ps]
    return codes(q[page, :, t % ps]), s[page, :, t % ps].astype(np.float64)


def attn(q, cache, table, lengths, cu, ps, shared=0, sm_scale=None, unrotate=False):
    """(out, tol) [N, Hq, d]; tol: how far a kernel may be before its output is rounded.

    The kernels hold the rotated query in pieces that are off by at most 2^-14 of its largest element, so a score is off by
    delta <= sm_scale 2^-14 max|q~| sum|k^| and a probability by 2 delta of itself; probabilities and values are rounded to
    11 bits or more (2^-11 each, together 2^-10), or held in pieces of 8 bits that leave 2^-12 of a value and 2^-17 of the
    largest one, with codes read as 0 .. 15.
    """
    n, hq, d = q.shape
    hkv = cache[0].shape[1]
    grp, h = hq // hkv, hadamard(d)
    sm = 1.0 / np.sqrt(d) if not sm_scale or sm_scale <= 0 else sm_scale
    out, tol = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    for i, (b, pos) in enumerate(places(lengths, cu, n)):
        if b < 0 or pos < 0:
            continue
        own = [tokens(cache, table[b], ps, pos + 1, w) for w in (0, 1)]
        if shared:
            m = min(shared, pos + 1)
            first = [tokens(cache, table[0], ps, m, w) for w in (0, 1)]
            own = [tuple(np.concatenate([f[j], o[j][m:]]) for j in (0, 1)) for f, o in zip(first, own)]
        (kc, ks), (vc, vs) = own
        qr = q[i].astype(np.float64) @ h
        for hh in range(hq):
            g = hh // grp
            x = sm * (kc[:, g] @ qr[hh]) * ks[:, g]
            p = np.exp(x - x.max())
            p /= p.sum()
            w = p * vs[:, g]
            delta = sm * 2.0 ** -14 * np.abs(qr[hh]).max() * (np.abs(kc[:, g]).sum(1) * ks[:, g])
            mag = np.abs(vc[:, g])
            o = w @ vc[:, g]
            t = (w * (2 * delta.max() + 2.0 ** -10)) @ (mag + 2) + 2.0 ** -17 * 15 * len(p) * w.max()
            if unrotate:
                o = o @ h
                t = np.full(d, np.sqrt((t * t).sum()))
            out[i, hh], tol[i, hh] = o, t
    return out, tol


def attn_rows(q, cache, table, lengths, cu, ps, few, eps, shared=0, sm_scale=None):
    """(norms, bounds) [N, Hq]: the norm of each row of attn(), and how far, in norm, a kernel's row may be from it, in either
    basis.  few: up to 16 rows that see the same keys; eps: torch.finfo(output type).eps.

    The output's rounding is at most half a step of each element.  Everything else is many small roundings, each anywhere
    within its half step (its deviation a root of 3 less), whose sum is bounded by six deviations:
      - probabilities, 2^-11 of themselves (few: of themselves times the value scale, and 2^-23 of the largest of these at
        least; else 2^-25 of the largest), and where the rows are many also values, 2^-11;
      - the rotated query's elements, 2^-15 of the largest one, which move all scores together;
      - scores, 2^-22 of 15 sum|q~| times the key scale: sums in fp32 with the codes read as 0 .. 15;
    and the outputs' sums in fp32, one for every 32 tokens, leave 2^-24 of 15 sum w an element each (all one way).
    """
    n, hq, d = q.shape
    hkv = cache[0].shape[1]
    grp, h = hq // hkv, hadamard(d)
    sm = 1.0 / np.sqrt(d) if not sm_scale or sm_scale <= 0 else sm_scale
    norms, bounds = np.zeros((n, hq)), np.zeros((n, hq))
    for i, (b, pos) in enumerate(places(lengths, cu, n)):
        if b < 0 or pos < 0:
            continue
        own = [tokens(cache, table[b], ps, pos + 1, w) for w in (0, 1)]
        if shared:
            m = min(shared, pos + 1)
            first = [tokens(cache, table[0], ps, m, w) for w in (0, 1)]
            own = [tuple(np.concatenate([f[j], o[j][m:]]) for j in (0, 1)) for f, o in zip(first, own)]
        (kc, ks), (vc, vs) = own
        qr = q[i].astype(np.float64) @ h
        for hh in range(hq):
            g = hh // grp
            k, c = kc[:, g] * ks[:, g, None], vc[:, g]
            x = sm * (k @ qr[hh])
            p = np.exp(x - x.max())
            p /= p.sum()
            w = p * vs[:, g]
            o = w @ c
            length2 = (c * c).sum(1)
            least = 2.0 ** -23 * w.max() if few else 2.0 ** -25 * p.max() * vs[:, g]
            var = ((2.0 ** -22 * w * w * (1 if few else 2) + least * least) * length2).sum()
            pull = p[:, None] * (vs[:, g, None] * c - o)  # of a score on the output
            var += (sm * 2.0 ** -15 * np.abs(qr[hh]).max() * np.linalg.norm(k.T @ pull)) ** 2
            var += ((sm * 2.0 ** -22 * 15 * np.abs(qr[hh]).sum() * ks[:, g]) ** 2 * (pull * pull).sum(1)).sum()
            norms[i, hh] = np.linalg.norm(o)
            sums = 2.0 ** -24 * np.ceil(len(p) / 32) * 15 * w.sum() * np.sqrt(d)
            bounds[i, hh] = eps / 2 * norms[i, hh] + 2.0 ** -25 * np.sqrt(d) + 6 * np.sqrt(var / 3) + sums
    return norms, bounds
