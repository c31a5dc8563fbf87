"""The bounds that attention's rows are held to: near enough to the rounding of the output that a row off by a hundredth
fails, whatever the length."""
import numpy as np
import pytest

from oracle import paged_oracle as O


def _batch(T, d, Hkv=1, ps=64, seed=0):
    rng = np.random.default_rng(seed)
    P = -(-T // ps)
    codes = lambda: rng.integers(0, 256, (P, Hkv, ps, d // 2), dtype=np.uint8)  # noqa: E731
    scales = lambda a, b: np.exp(rng.uniform(a, b, (P, Hkv, ps))).astype(np.float16)  # noqa: E731
    return [codes(), scales(-4.0, -1.0), codes(), scales(-3.0, 1.0)], rng.permutation(P)[None], np.array([T])


@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("T,d", [(1, 128), (5, 64), (40, 128), (513, 128), (2300, 64), (20000, 128)])
def test_a_hundredth_is_out_of_bounds(T, d, few):
    cache, table, lengths = _batch(T, d)
    q = np.random.default_rng(1).standard_normal((1, 4, d)).astype(np.float16)
    norms, bounds = O.attn_rows(q, cache, table, lengths, None, 64, few, 2.0 ** -10)
    want, _ = O.attn(q, cache, table, lengths, None, 64)
    assert np.allclose(np.linalg.norm(want, axis=-1), norms, rtol=1e-12)
    assert (bounds >= 2.0 ** -11 * norms).all() and (bounds < 0.01 * norms).all(), (bounds / norms).max()


def test_bounds_hold_for_the_roundings_they_count():
    """Attention in float64 with each rounding made: queries off by 2^-15 of their largest element, probabilities and values
    in fp16, the output in fp16."""
    cache, table, lengths = _batch(700, 128, Hkv=2, seed=3)
    rng = np.random.default_rng(2)
    q = rng.standard_normal((1, 8, 128)).astype(np.float16)
    norms, bounds = O.attn_rows(q, cache, table, lengths, None, 64, False, 2.0 ** -10)
    want, _ = O.attn(q, cache, table, lengths, None, 64)
    (kc, ks), (vc, vs) = (O.tokens(cache, table[0], 64, 700, w) for w in (0, 1))
    for _ in range(20):
        for hh in range(8):
            x = q[0, hh].astype(np.float64) @ O.hadamard(128)
            x = x + rng.uniform(-1, 1, 128) * 2.0 ** -15 * np.abs(x).max()
            s = (kc[:, hh // 4] @ x) * ks[:, hh // 4] / np.sqrt(128)
            p = np.exp(s - s.max())
            v = (vc[:, hh // 4] * vs[:, hh // 4, None]).astype(np.float16).astype(np.float64)
            o = (p.astype(np.float16).astype(np.float64) @ v / p.sum()).astype(np.float16)
            assert np.linalg.norm(o - want[0, hh]) <= bounds[0, hh]
