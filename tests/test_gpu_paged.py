"""Rotary positions and the paged 4-bit cache on the GPU against their float64 forms.

Rotary positions: angles are exact to 2^-25 of a half turn, cos and sin to a few steps of fp32; a product with them and a
sum are off by at most 2^-21 of |a| + |b|, then half a step of the output's type.

Append: the transform's 2 + log2(d) additions and products (3 more where positions turn) each leave 2^-24 of the sum of
magnitudes; a scale is within half a step of fp16 of the largest value's 7th, a code within half a scale of its value.

Attention: oracle/paged_oracle.py derives the bound beside the float64 form.
"""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as O
from oracle import quarot_oracle as Q
from test_gpu_parity import DEV, q  # noqa: F401  (q: fixture)

pytestmark = pytest.mark.gpu

FP16, BF16 = torch.float16, torch.bfloat16


def _np(t):
    return t.detach().double().cpu().numpy()


def _raw(t):
    return t.detach().cpu().numpy()


def _half_step(ref, dtype):
    eps = torch.finfo(dtype).eps / 2
    return np.maximum(eps * np.abs(ref), torch.finfo(dtype).tiny * eps)


def _freqs(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2) / rot)


def _gpu64(a):
    return torch.from_numpy(np.asarray(a, dtype=np.float64)).to(DEV)


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- rotary positions
def _rope_tol(x, inv_freq, interleaved, scale, ref, dtype):
    y = np.abs(_np(x))
    half = len(inv_freq)
    lo = np.arange(half) * 2 if interleaved else np.arange(half)
    hi = lo + 1 if interleaved else lo + half
    own = np.zeros_like(y)
    own[..., lo] = own[..., hi] = (y[..., lo] + y[..., hi]) * abs(scale) * 2.0 ** -21
    return own * (1 + 2.0 ** -7) + _half_step(ref, dtype)


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N,Hq,Hk,d,rot", [(1, 1, 0, 16, 16), (1, 32, 8, 128, 128), (3, 5, 1, 64, 48), (7, 3, 2, 80, 32),
                                           (33, 2, 2, 128, 96), (129, 4, 1, 256, 256), (1000, 6, 3, 64, 16), (2, 1, 1, 1024, 512),
                                           (5, 7, 7, 128, 0), (4000, 9, 2, 128, 112)])
def test_rope(q, dtype, interleaved, N, Hq, Hk, d, rot):
    g = torch.Generator().manual_seed(N + d)
    wide = torch.randn((N, Hq + 2 * Hk + 1, d), generator=g).to(dtype).to(DEV)
    x, k = wide[:, :Hq], wide[:, Hq:Hq + Hk] if Hk else None
    pos = torch.randint(-1000, 2_000_000, (N,), generator=g, dtype=torch.int32)
    pos[0], pos[-1] = 0, 2 ** 31 - 1
    f = _freqs(rot) if rot else np.zeros(0)
    scale = 1.0 if N % 2 else 1.25
    before = wide.clone()
    yq, yk = q.quarot_rope(x, k, pos.to(DEV), _gpu64(f) if rot else None, interleaved, scale)
    assert torch.equal(wide, before)
    for a, y in ((x, yq), (k, yk)):
        if a is None:
            assert y is None
            continue
        ref = O.rope(_np(a), pos.numpy(), f, interleaved, scale)
        err, tol = np.abs(_np(y) - ref), _rope_tol(a, f, interleaved, scale, ref, dtype)
        # positions near 2^31 move an angle by position * 2^-54 turns in the float64 form too
        assert (err <= tol * (1 + 2.0 ** -10) + 2.0 ** -19 * np.abs(_np(a)).max() * (np.abs(pos.numpy())[:, None, None] > 1e8)).all(), \
            float((err / tol).max())
        assert torch.equal(y[..., rot:], a[..., rot:])
    # in place, on a slice: the rest of the tensor stays
    q.quarot_rope(x, k, pos.to(DEV), _gpu64(f) if rot else None, interleaved, scale, q_out=x, k_out=k)
    assert torch.equal(x, yq) and (k is None or torch.equal(k, yk)) and torch.equal(wide[:, Hq + Hk:], before[:, Hq + Hk:])


def test_rope_object_and_refusals(q):
    r = q.QuarotRope(64, scaling="yarn", factor=8.0, original_len=2048, interleaved=True)
    x = torch.randn(5, 4, 128, device=DEV, dtype=FP16)
    pos = _i32([0, 1, 2047, 2048, 16383])
    y, none = r(x, None, pos)
    ref = O.rope(_np(x), _raw(pos), _np(r.inv_freq), True, r.scale)
    assert none is None and (np.abs(_np(y) - ref) <= _rope_tol(x, _np(r.inv_freq), True, r.scale, ref, FP16)).all()
    f = r.inv_freq
    for bad in (lambda: q.quarot_rope(x.float(), None, pos, f), lambda: q.quarot_rope(x, x.bfloat16(), pos, f),
                lambda: q.quarot_rope(x, None, pos.long(), f), lambda: q.quarot_rope(x, None, pos[:4], f),
                lambda: q.quarot_rope(x, None, pos, f.float()), lambda: q.quarot_rope(x, x[:4], pos, f),
                lambda: q.quarot_rope(x.transpose(0, 1), None, pos, f), lambda: q.quarot_rope(x[:, :, :64], None, pos, f),
                lambda: q.quarot_rope(x, None, pos, f[:12]), lambda: q.quarot_rope(x, None, pos, _gpu64(np.zeros(128))),
                lambda: q.quarot_rope(x, None, pos, f, k_out=x), lambda: q.quarot_rope(x, None, pos, f, q_out=x[:4]),
                lambda: q.quarot_rope(x, None, pos.cpu(), f), lambda: q.quarot_rope(x.cpu(), None, pos, f)):
        with pytest.raises(q.QuarotError):
            bad()
    assert q.quarot_rope(x[:0], None, pos[:0], f)[0].shape == (0, 4, 128)


# ---------------------------------------------------------------- batches
class Case:
    """A batch in scattered pages: lengths, new tokens of each sequence (None: one each), pages shared by all."""

    def __init__(self, lengths, ps, Hkv, d, new=None, shared=0, seed=0, spare=3):
        self.lengths, self.ps, self.shared = np.asarray(lengths), ps, shared
        self.cu = None if new is None else np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        self.N = len(lengths) if new is None else int(self.cu[-1])
        rng = np.random.default_rng(seed)
        common = shared // ps
        each = max(0, -(-max(int(max(lengths)) - common * ps, 0) // ps))
        P = common + len(lengths) * each
        order = rng.permutation(P + spare)
        self.n_pages = P + spare
        self.table = np.concatenate([np.tile(order[:common], (len(lengths), 1)),
                                     order[common:P].reshape(len(lengths), each)], 1).astype(np.int64)
        shape = (self.n_pages, Hkv, ps)
        g = torch.Generator().manual_seed(seed)
        codes = lambda: torch.randint(0, 256, shape + (d // 2,), generator=g, dtype=torch.uint8).to(DEV)  # noqa: E731
        scales = lambda a, b: torch.exp(torch.rand(shape, generator=g) * (b - a) + a).half().to(DEV)  # noqa: E731
        self.cache = [codes(), scales(-4.0, -1.0), codes(), scales(-3.0, 1.0)]

    @property
    def where(self):
        return _i32(self.table.reshape(len(self.lengths), -1)), _i32(self.lengths), None if self.cu is None else _i32(self.cu)

    def np_cache(self):
        return [_raw(t) for t in self.cache]


def _queries(N, Hq, d, dtype, seed, strided=True):
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn((N, Hq + 2, d), generator=g).to(dtype).to(DEV)
    return wide[:, :Hq] if strided else wide[:, :Hq].contiguous()


def _check_attn(out, x, c, **kw):
    ref, tol = O.attn(_np(x), c.np_cache(), c.table, c.lengths, c.cu, c.ps, shared=c.shared, **kw)
    err = np.abs(_np(out) - ref)
    bound = tol + _half_step(ref + np.sign(ref) * tol, out.dtype)
    assert np.isfinite(_np(out)).all()
    assert (err <= bound).all(), (float((err / bound).max()), np.argwhere(err > bound)[:4].tolist())


# ---------------------------------------------------------------- append and read
def _check_append(c, cache, k, v, freqs, interleaved, scale):
    """Codes and scales of the batch's new tokens against the values they have to stand for."""
    d = k.shape[-1]
    h = O.hadamard(d)
    pl = O.places(c.lengths, c.cu, c.N)
    pos = np.array([max(p, 0) for _, p in pl])
    turned = O.rope(_np(k), pos, freqs, interleaved, scale)
    for which, x in ((0, turned), (1, _np(v))):
        y = x @ h
        own = np.abs(x).sum(-1) / np.sqrt(d) * (5 + np.log2(d)) * 2.0 ** -24 + (np.abs(x).max(-1) * 2.0 ** -20 * np.sqrt(d) if which == 0 else 0)
        for i, (b, p) in enumerate(pl):
            if b < 0 or p < 0:
                continue
            page, slot = c.table[b, p // c.ps], p % c.ps
            code, s = O.codes(cache[2 * which][page, :, slot]), cache[2 * which + 1][page, :, slot].astype(np.float64)
            want = np.maximum(np.abs(y[i]).max(-1), 1e-5) / 7
            assert (np.abs(s - want) <= want * 2.0 ** -11 + 2.0 ** -25 + own[i] / 7).all()
            off = np.abs(y[i] - code * s[:, None])
            clipped = (code == 7) & (y[i] > 0) | (code == -8) & (y[i] < 0)
            assert ((off <= (s[:, None] / 2) * (1 + 2.0 ** -20) + own[i][:, None]) | clipped).all()
            assert (off <= s[:, None] / 2 + 7 * s[:, None] * 2.0 ** -10 + 2.0 ** -22 + own[i][:, None]).all()


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lengths,new,ps,Hkv,Hq,d,rot", [
    ([1], None, 16, 1, 1, 128, 128), ([37, 0, 64, 65], None, 64, 8, 32, 128, 128), ([5, 17, 40], [5, 0, 23], 16, 3, 9, 64, 48),
    ([100, 200, 7], [100, 33, 7], 48, 2, 0, 128, 32), ([300], [300], 256, 16, 16, 64, 64), ([9, 3], [9, 5], 32, 5, 20, 128, 112),
    ([70] * 33, None, 32, 80, 80, 64, 16), ([130, 1], [130, 1], 128, 1, 7, 128, 0)])
def test_append_and_read(q, dtype, interleaved, lengths, new, ps, Hkv, Hq, d, rot):
    c = Case(lengths, ps, Hkv, d, new, seed=len(lengths) + ps)
    pad = 2 if new is not None else 0  # tokens behind the last sequence
    g = torch.Generator().manual_seed(d + rot)
    wide = torch.randn((c.N + pad, max(Hq, 1) + 2 * Hkv, d), generator=g)
    wide[..., 3] *= 20.0
    wide = wide.to(dtype).to(DEV)
    x, k, v = wide[:, :Hq] if Hq else None, wide[:, -2 * Hkv:-Hkv], wide[:, -Hkv:]
    f = _freqs(rot) if rot else np.zeros(0)
    before = c.np_cache()
    q_out = torch.full((c.N + pad, Hq, d), 7.0, dtype=dtype, device=DEV) if Hq else None
    got = q.quarot_paged_append(k, v, *c.cache, *c.where, q=x, inv_freq=_gpu64(f) if rot else None, interleaved=interleaved,
                                scale=1.125, q_out=q_out)
    q.quarot_check_error()
    after = c.np_cache()
    scale = 1.125 if rot else 1.0
    _check_append(c, after, k[:c.N], v[:c.N], f, interleaved, scale)
    # nothing else was written
    kept = np.ones((c.n_pages, ps), bool)
    pl = O.places(c.lengths, c.cu, c.N)
    for b, p in pl:
        if p >= 0:
            kept[c.table[b, p // ps], p % ps] = False
    for a, b in zip(before, after):
        assert np.array_equal(np.moveaxis(a, 2, 1)[kept], np.moveaxis(b, 2, 1)[kept], equal_nan=True)
    pos = np.array([p for _, p in pl])
    if Hq:
        assert got is q_out and (got[c.N:] == 7.0).all() and (got[:c.N][torch.from_numpy(pos < 0).to(DEV)] == 0).all()
        there = pos >= 0
        ref = O.rope(_np(x)[:c.N][there], pos[there], f, interleaved, scale)
        err = np.abs(_np(got)[:c.N][there] - ref)
        assert (err <= _rope_tol(x[:c.N][torch.from_numpy(there).to(DEV)], f, interleaved, scale, ref, dtype)).all()
        q.quarot_paged_append(k, v, *c.cache, *c.where, q=x, inv_freq=_gpu64(f) if rot else None, interleaved=interleaved,
                              scale=1.125, q_out=x)  # in place, the same cache again
        assert torch.equal(x[:c.N], got[:c.N]) and all(np.array_equal(a, b, equal_nan=True) for a, b in zip(after, c.np_cache()))
    else:
        assert got is None
    # reading back: values of the codes
    for back in (False, True):
        outs = [torch.full((c.N + pad, Hkv, d), 5.0, dtype=dtype, device=DEV) for _ in range(2)]
        kk, vv = q.quarot_paged_read(*c.cache, *c.where, n=c.N + pad, unrotate=back, out_dtype=dtype, k_out=outs[0], v_out=outs[1])
        for which, y in ((0, kk), (1, vv)):
            assert (y[c.N:] == 5.0).all()
            for i, (b, p) in enumerate(pl):
                if p < 0:
                    assert (y[i] == 0).all()
                    continue
                page, slot = c.table[b, p // ps], p % ps
                val = O.codes(after[2 * which][page, :, slot]) * after[2 * which + 1][page, :, slot].astype(np.float64)[:, None]
                own = np.abs(val).sum(-1, keepdims=True) * np.sqrt(d) * 2.0 ** -52  # what d float64 additions, 2^-53 each, and the rounded 1 / sqrt(d) leave of a sum that is 0: below d 2^-53 sum|val| / sqrt(d)
                if back:
                    val = val @ O.hadamard(d)
                err = np.abs(_np(y[i]) - val)
                assert (err <= _half_step(val, dtype) * (1 + 2.0 ** -12) + np.abs(val) * 2.0 ** -22 + own).all()


def test_append_without_rotation_stores_what_the_contiguous_cache_holds(q):
    """The same codes and scales, bit for bit, as quarot_kv_write's."""
    B, T, H, d, ps = 3, 150, 4, 128, 32
    k, v = (torch.randn(B, T, H, d, device=DEV, dtype=FP16) for _ in range(2))
    flat = q.new_kv_cache(B, H, T, d, torch.device(DEV))
    q.quarot_kv_write(k, v, 0, *flat)
    c = Case([T] * B, ps, H, d, [T] * B)
    q.quarot_paged_append(k.view(-1, H, d), v.view(-1, H, d), *c.cache, *c.where)
    at = torch.from_numpy(c.table).to(DEV)
    for a, p in zip(flat, c.cache):
        rows = p[at]  # [B, pages, H, ps, ...]
        rows = rows.movedim(2, 1).flatten(2, 3)[:, :, :T]
        assert torch.equal(rows, a)


def test_append_edge_values(q):
    """Zeros, the largest values, one loud element, infinities: as quarot_kv_write."""
    d, H = 64, 2
    k = torch.zeros(6, H, d, dtype=FP16)
    k[1] = 65504.0
    k[2, :, 5] = 65504.0
    k[3] = -1e-7
    k[4, 0, 3] = float("inf")
    k[5, 1] = torch.linspace(-3, 3, d).half()
    k = k.to(DEV)
    flat = q.new_kv_cache(1, H, 6, d, torch.device(DEV))
    q.quarot_kv_write(k[None].contiguous(), k[None].contiguous(), 0, *flat)
    c = Case([6], 16, H, d, [6])
    q.quarot_paged_append(k, k, *c.cache, *c.where)
    for a, p in zip(flat, c.cache):
        got, want = p[int(c.table[0, 0])][:, :6], a[0]
        rows = [0, 1, 2, 3, 5]
        assert torch.equal(got[:, rows], want[:, rows])


# ---------------------------------------------------------------- attention
ATTN = [
    # lengths, new, ps, Hkv, Hq, d, shared
    ([1], None, 16, 1, 1, 128, 0),
    ([37, 0, 64, 65, 129], None, 64, 2, 8, 128, 0),
    ([1000], None, 16, 1, 4, 64, 0),
    ([15, 16, 17, 127, 128, 129, 255, 256, 257], None, 16, 2, 4, 128, 0),
    ([300, 5, 211], None, 48, 3, 9, 64, 0),
    ([2300, 1], None, 256, 1, 8, 128, 0),
    ([700, 333], None, 32, 2, 32, 128, 0),                        # groups of 16
    ([260, 300], None, 64, 2, 10, 128, 0),                        # groups of 5
    ([260, 300], None, 64, 2, 14, 64, 0),                         # groups of 7
    ([500, 0, 460, 411], None, 64, 2, 8, 128, 400),               # a prefix that ends inside a page
    ([400, 401, 402], None, 16, 2, 4, 128, 400),                  # one token behind the prefix, or none
    ([90] * 40, None, 32, 2, 8, 128, 64),                         # more rows than a tile
    ([1100 + 7 * i for i in range(20)], None, 128, 1, 8, 64, 1030),
    ([5, 17, 40], [5, 0, 23], 16, 2, 4, 64, 0),
    ([100, 200, 7], [100, 33, 7], 48, 2, 4, 128, 0),
    ([700, 600], [130, 1], 64, 1, 4, 128, 500),
    ([300], [300], 64, 2, 2, 128, 0),
    ([9, 3, 20], [2, 3, 1], 16, 2, 8, 128, 0),                    # drafts of a few tokens
    ([9, 3, 2000], [2, 5, 4], 16, 2, 8, 128, 0),                  # a sequence shorter than its new tokens
    ([0, 200, 130], [70, 40, 140], 64, 2, 4, 128, 0),             # whole tiles of rows that see nothing
    ([2000, 900], [150, 3], 64, 2, 4, 64, 333),                   # units of several CTAs, a prefix among them
]


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("hint", ["few", "many"])
@pytest.mark.parametrize("lengths,new,ps,Hkv,Hq,d,shared", ATTN)
def test_attn(q, dtype, hint, lengths, new, ps, Hkv, Hq, d, shared):
    c = Case(lengths, ps, Hkv, d, new, shared, seed=ps + Hq)
    x = _queries(c.N, Hq, d, dtype, 5)
    for un in (False, True):
        out = torch.full((c.N, Hq + 1, d), 3.0, dtype=dtype, device=DEV)
        y = q.quarot_paged_attn(x, *c.cache, *c.where, max_q=1 if hint == "few" else 4096, shared_len=shared, unrotate_out=un,
                                out=out[:, :Hq])
        q.quarot_check_error()
        _check_attn(y, x, c, unrotate=un)
        assert (out[:, Hq] == 3.0).all()


@pytest.mark.parametrize("new", [None, [1, 1, 3, 1]])
def test_attn_loud_scores_and_scales(q, new):
    """Scores of +-100 and more, one token that takes all, scales from fp16's smallest to large ones."""
    c = Case([513, 40, 300, 129], 64, 2, 128, new, seed=3)
    c.cache[1][:, :, 1] *= 20.0
    c.cache[1][:, :, 5] = 2.0 ** -24
    c.cache[3][:, :, 2] = 2.0 ** -24
    c.cache[3][:, :, 7] = 0.0
    c.cache[3][:, :, 9] = 500.0
    x = _queries(c.N, 8, 128, FP16, 1) * 4
    x[1, 2] = 0.0  # all scores equal
    out = q.quarot_paged_attn(x, *c.cache, *c.where, max_q=3)
    _check_attn(out, x, c)
    out = q.quarot_paged_attn(x, *c.cache, *c.where, max_q=3, sm_scale=0.5)
    _check_attn(out, x, c, sm_scale=0.5)


@pytest.mark.parametrize("max_q", [1, 1000])
@pytest.mark.parametrize("shared", [0, 100])
def test_attn_does_not_look_behind_the_lengths(q, max_q, shared):
    """Slots behind a sequence's end, and pages of nobody, may hold anything."""
    new = None if max_q == 1 else [3, 1, 0, 20]
    c = Case([130, 101, 0, 259], 64, 2, 128, new, shared, seed=8)
    x = _queries(c.N, 8, 128, BF16, 2)
    want = q.quarot_paged_attn(x, *c.cache, *c.where, max_q=max_q, shared_len=shared)
    used = torch.zeros((c.n_pages, c.ps), dtype=torch.bool)
    for b, n in enumerate(c.lengths):
        for t in range(int(n)):
            used[c.table[0 if t < shared else b, t // c.ps], t % c.ps] = True
    for i in (1, 3):
        c.cache[i].transpose(1, 2)[~used.to(DEV)] = float("nan")
    for i in (0, 2):
        c.cache[i].transpose(1, 2)[~used.to(DEV)] = 0x88
    got = q.quarot_paged_attn(x, *c.cache, *c.where, max_q=max_q, shared_len=shared)
    assert torch.equal(want, got)


@pytest.mark.parametrize("max_q", [1, 1000])
def test_attn_leaves_rows_behind_the_last_sequence(q, max_q):
    c = Case([50, 80], 16, 2, 64, [3, 4], seed=4)
    x = _queries(12, 6, 64, FP16, 2)
    x[7:] = float("nan")
    out = torch.full((12, 6, 64), 9.0, dtype=FP16, device=DEV)
    q.quarot_paged_attn(x, *c.cache, *c.where, max_q=max_q, shared_len=32, out=out)
    c.shared = 32
    _check_attn(out[:7], x[:7], c)
    assert (out[7:] == 9.0).all()


@pytest.mark.parametrize("max_q", [1, 1000])
@pytest.mark.parametrize("where", [0, 77, 199])
def test_infinite_values_stay_with_the_tokens_that_see_them(q, max_q, where):
    """A value of infinite elements, and the largest scales: rows before it are what they are without it."""
    new = 200
    c = Case([new + 30], 32, 2, 128, [new], seed=8)
    x, out = _queries(new, 8, 128, FP16, 3), []
    page, slot = int(c.table[0, (where + 30) // 32]), (where + 30) % 32
    v = torch.randn(1, 2, 128, device=DEV).half()
    v[:, :, 5] = float("inf")
    pool = [t.clone() for t in c.cache]
    q.quarot_paged_append(v, v, *pool, _i32(c.table[:, :]), _i32([where + 31]))  # one token, at position where + 30
    assert torch.isfinite(pool[3][page, :, slot]).all() and (pool[3][page, :, slot] > 8188).all()
    for scale in (None, 65504.0):
        if scale:
            pool[1][page, :, slot] = pool[3][page, :, slot] = scale
        y = q.quarot_paged_attn(x, *pool, *c.where, max_q=max_q)
        q.quarot_check_error()
        out.append(y[:where])
    ref, tol = O.attn(_np(x), c.np_cache(), c.table, c.lengths, c.cu, c.ps)
    ref, tol = ref[:where], np.broadcast_to(tol, ref.shape)[:where]
    for y in out:
        assert torch.isfinite(y).all()
        assert (np.abs(_np(y) - ref) <= tol + _half_step(ref + np.sign(ref) * tol, FP16)).all()


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at,pitch", [(0, 0), (8, 0), (0, 8), (8, 8)])
def test_attn_outputs_at_every_alignment(q, dtype, d, at, pitch):
    """Outputs whose first row or whose pitch is a multiple of 16 bytes, not of 32."""
    c = Case([300, 150], 32, 2, d, [260, 41], seed=d)
    x = _queries(c.N, 8, d, dtype, 6)
    flat = torch.full((at + c.N * (8 * d + pitch) + 64,), 3.0, dtype=dtype, device=DEV)
    out = flat.as_strided((c.N, 8, d), (8 * d + pitch, d, 1), at)
    for un in (False, True):
        q.quarot_paged_attn(x, *c.cache, *c.where, max_q=260, unrotate_out=un, out=out)
        q.quarot_check_error()
        _check_attn(out, x, c, unrotate=un)
    kept = torch.ones_like(flat, dtype=torch.bool)
    kept.as_strided((c.N, 8, d), (8 * d + pitch, d, 1), at)[:] = False
    assert (flat[kept] == 3.0).all()


@pytest.mark.parametrize("max_q", [1, 1000])
def test_pages_that_are_not_there(q, max_q):
    """A table entry outside the cache and a length past the table are errors that quarot_check_error reports; the other
    sequences' results stay right."""
    c = Case([200, 150, 90], 64, 2, 128, seed=6)
    x = _queries(3, 8, 128, FP16, 2)
    table, lens, _ = c.where
    good = q.quarot_paged_attn(x, *c.cache, table, lens, max_q=max_q)
    for bad in (-1, c.n_pages, 2 ** 31 - 1):
        t = table.clone()
        t[1, 1] = bad
        out = q.quarot_paged_attn(x, *c.cache, t, lens, max_q=max_q)
        with pytest.raises(q.QuarotError) as e:
            q.quarot_check_error()
        assert e.value.status == 1
        assert torch.equal(out[[0, 2]], good[[0, 2]]) and torch.isfinite(out).all()
        kv = torch.randn(3, 2, 128, device=DEV, dtype=FP16)
        t[1, 2] = bad
        before = [a.clone() for a in c.cache]
        q.quarot_paged_append(kv, kv, *[a.clone() for a in c.cache], t, lens)
        with pytest.raises(q.QuarotError):
            q.quarot_check_error()
        k, _ = q.quarot_paged_read(*c.cache, t, lens)
        assert (k[1] == 0).all() and (k[0] != 0).any()
        with pytest.raises(q.QuarotError):
            q.quarot_check_error()
        assert all(torch.equal(a, b) for a, b in zip(before, c.cache))
    lens2 = lens.clone()
    lens2[1] = 10 ** 6
    out = q.quarot_paged_attn(x, *c.cache, table, lens2, max_q=max_q)
    with pytest.raises(q.QuarotError):
        q.quarot_check_error()
    assert torch.equal(out[[0, 2]], good[[0, 2]])
    q.quarot_check_error()


def test_attn_refusals(q):
    c = Case([50, 80], 16, 2, 64)
    x = _queries(2, 4, 64, FP16, 2)
    table, lens, _ = c.where
    call = lambda x=x, cache=c.cache, t=table, n=lens, **kw: q.quarot_paged_attn(x, *cache, t, n, **kw)  # noqa: E731
    call()
    for bad in (lambda: call(x=x.float()), lambda: call(x=x[:, :3]), lambda: call(x=x[..., :32]), lambda: call(t=table.long()),
                lambda: call(t=table[:1]), lambda: call(n=lens.long()), lambda: call(n=lens[:1]), lambda: call(x=x[:1]),
                lambda: call(cu_q=_i32([0, 1])), lambda: call(cu_q=lens), lambda: call(max_q=0), lambda: call(shared_len=-1),
                lambda: call(shared_len=10 ** 6), lambda: call(sm_scale=float("nan")), lambda: call(out=x[:1]),
                lambda: call(out=x.bfloat16()), lambda: call(workspace=torch.empty(1, dtype=torch.uint8, device=DEV)),
                lambda: call(cache=[t.float() for t in c.cache]), lambda: call(cache=c.cache[:1] + c.cache[2:] + c.cache[:1]),
                lambda: call(cache=[t[:, :1] for t in c.cache]), lambda: call(x=x.transpose(1, 2).contiguous().transpose(1, 2)),
                lambda: q.quarot_paged_read(*c.cache, table, lens, _i32([0, 1, 2])),
                lambda: q.quarot_paged_read(*c.cache, table, lens, out_dtype=torch.float32),
                lambda: q.quarot_paged_append(x, x, *c.cache, table, lens),
                lambda: q.quarot_paged_append(x[:, :2], x[:, :2].bfloat16(), *c.cache, table, lens),
                lambda: q.quarot_paged_append(x[:, :2], x[:, :2], *c.cache, table, lens, q_out=x)):
        with pytest.raises(q.QuarotError):
            bad()
    empty = q.quarot_paged_attn(x[:0], *c.cache, table[:0], lens[:0])
    assert empty.shape == (0, 4, 64)


# ---------------------------------------------------------------- as they would be used
def test_serving_run(q):
    """Prompts in chunks behind a shared prefix, then decoding: append, attend and read through QuarotPagedKVCache, against
    the float64 forms over what the pages hold."""
    B, Hq, Hkv, d, ps, S = 3, 8, 2, 128, 32, 80
    rope = q.QuarotRope(64, scaling="linear", factor=4.0)
    cache = q.QuarotPagedKVCache(40, Hkv, ps, d, rope=rope)
    rng = np.random.default_rng(0)
    order = rng.permutation(40)
    table = np.stack([np.concatenate([order[:2], order[2 + 7 * b:9 + 7 * b]]) for b in range(B)])
    t = _i32(table)
    lengths = np.zeros(B, np.int64)
    tok = lambda n: [torch.randn(n, h, d, device=DEV).to(BF16) for h in (Hq, Hkv, Hkv)]  # noqa: E731

    def step(new, tables=t, shared=0):
        lens, cu = _i32(lengths), _i32(np.concatenate([[0], np.cumsum(new)]))
        x, k, v = tok(int(sum(new)))
        turned = cache.append(k, v, tables, lens, cu, q=x)
        out = cache.attend(turned, tables, lens, cu, max_q=int(max(new)), shared_len=shared)
        q.quarot_check_error()
        c = Case.__new__(Case)
        c.cache, c.table, c.lengths, c.cu, c.ps, c.shared = cache.tensors, _raw(tables), lengths, _raw(cu), ps, shared
        _check_attn(out, turned, c)
        return k, v

    # the prefix, by the first sequence alone: 80 tokens; the third page is each sequence's own
    lengths[0] = S
    k, v = step([S, 0, 0])
    kk, vv = cache.read(t[:1], _i32([S]), _i32([0, S]), n=S, unrotate=True, out_dtype=BF16)
    pos = np.arange(S)
    for got, want in ((kk, O.rope(_np(k), pos, _np(rope.inv_freq))), (vv, _np(v))):
        # rotated elements are off by half a scale, the largest one's 14th; the rotation keeps a vector's length; bf16 out
        scale = np.abs(want @ O.hadamard(d)).max(-1) / 7
        err, norm = np.linalg.norm(_np(got) - want, axis=-1), np.linalg.norm(want, axis=-1)
        assert (err <= (np.sqrt(d) * scale / 2 + norm * 2.0 ** -8) * 1.01).all()
    for a in cache.tensors:
        a[table[1:, 2]] = a[table[0, 2]].clone()
    lengths[:] = S
    for new in ([50, 1, 7], [20, 33, 1], [1, 1, 1], [1, 1, 1]):
        lengths += np.asarray(new)
        step(new, shared=S)
    # a decode step without cu_q
    lengths += 1
    lens = _i32(lengths)
    x, k, v = tok(B)
    turned = cache.append(k, v, t, lens, q=x)
    a = cache.attend(turned, t, lens, shared_len=S)
    b = cache.attend(turned, t, lens)
    assert float((a.float() - b.float()).norm() / b.float().norm()) < 2.0 ** -7


def test_attn_agrees_with_the_contiguous_decode(q):
    B, T, Hkv, Hq, d, ps = 4, 777, 2, 8, 128, 64
    k, v = (torch.randn(B, T, Hkv, d, device=DEV, dtype=FP16) for _ in range(2))
    flat = q.QuarotKVCache(B, Hkv, T)
    flat.append(k, v)
    c = Case([T] * B, ps, Hkv, d, [T] * B)
    q.quarot_paged_append(k.view(-1, Hkv, d), v.view(-1, Hkv, d), *c.cache, *c.where)
    x = torch.randn(B, Hq, d, device=DEV, dtype=FP16)
    table, lens, _ = c.where
    for un in (False, True):
        a, b = flat.decode(x, unrotate_out=un), q.quarot_paged_attn(x, *c.cache, table, lens, unrotate_out=un)
        assert float((a.float() - b.float()).norm() / a.float().norm()) < 1e-3


@pytest.mark.parametrize("max_q,shared", [(1, 0), (1, 96), (64, 0)])
def test_replay_follows_the_batch(q, max_q, shared):
    """A captured step replayed after lengths, table and inputs changed gives what an eager call gives."""
    B, Hkv, Hq, d, ps, cap = 5, 2, 8, 128, 32, 16
    new = None if max_q == 1 else [3, 64, 1, 9, 2]
    N = B if new is None else sum(new)
    rng = np.random.default_rng(1)
    n_pages = B * cap + 4
    rope = q.QuarotRope(128)
    cache = q.QuarotPagedKVCache(n_pages, Hkv, ps, d, rope=rope)
    cu = None if new is None else _i32(np.concatenate([[0], np.cumsum(new)]))

    def batch():
        order = rng.permutation(n_pages)
        t = order[:B * cap].reshape(B, cap)
        t[:, :shared // ps] = t[0, :shared // ps]
        return t, rng.integers(130, cap * ps, B)

    t, n = batch()
    table, lens = _i32(t), _i32(n)
    x, k, v = (torch.randn(N, h, d, device=DEV).half() for h in (Hq, Hkv, Hkv))
    for a in cache.tensors:
        a.copy_(torch.randint(0, 256, a.shape, dtype=torch.uint8, device=DEV) if a.dtype == torch.uint8 else torch.rand(a.shape, device=DEV))
    body = lambda: cache.attend(cache.append(k, v, table, lens, cu, q=x), table, lens, cu, max_q=max_q, shared_len=shared)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        body()
    torch.cuda.current_stream().wait_stream(s)
    graphs, outs = [], []
    for _ in range(2):  # two graphs, each with scratch of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(body())
        graphs.append(g)
    for _ in range(3):
        t, n = batch()
        table.copy_(_i32(t))
        lens.copy_(_i32(n))
        x.normal_()
        k.normal_()
        for g in graphs:
            g.replay()
        want = body()
        torch.cuda.synchronize()
        q.quarot_check_error()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_calls_on_other_streams_at_once(q):
    """Calls on several streams side by side, and on a stream that is not current, give what they give alone."""
    cases = [Case([900 + 31 * i, 400], 64, 2, 128, None, 128 if i % 2 else 0, seed=i) for i in range(4)]
    xs = [_queries(2, 8, 128, FP16, i) for i in range(4)]
    args = [c.where for c in cases]
    want = [q.quarot_paged_attn(x, *c.cache, *a, shared_len=c.shared) for x, c, a in zip(xs, cases, args)]
    big = Case([600], 64, 2, 128, [600], seed=9)
    xb, ab = _queries(600, 8, 128, FP16, 7), big.where
    want_b = q.quarot_paged_attn(xb, *big.cache, *ab, max_q=600)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(5)]
    for _ in range(20):
        got = [q.quarot_paged_attn(x, *c.cache, *a, shared_len=c.shared, stream=s) for x, c, a, s in zip(xs, cases, args, streams)]
        got_b = q.quarot_paged_attn(xb, *big.cache, *ab, max_q=600, stream=streams[4])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.equal(want_b, got_b)
    q.quarot_check_error()


# ---------------------------------------------------------------- sizes
@pytest.mark.parametrize("hint", [1, 4096])
def test_more_sequences_than_threads(q, hint):
    """A batch whose sequences no block of threads holds at once; many are empty or all but."""
    rng = np.random.default_rng(2)
    B = 1000
    lengths = rng.integers(0, 40, B)
    lengths[rng.random(B) < 0.3] = 0
    new = np.minimum(lengths, rng.integers(0, 4, B))
    c = Case(lengths, 16, 1, 64, new, seed=5)
    x = _queries(c.N, 2, 64, BF16, 3)
    _check_attn(q.quarot_paged_attn(x, *c.cache, *c.where, max_q=hint), x, c)
    kv = torch.randn(c.N, 1, 64, device=DEV).half()
    q.quarot_paged_append(kv, kv, *c.cache, *c.where)
    _check_append(c, c.np_cache(), kv, kv, np.zeros(0), False, 1.0)
    k, v = q.quarot_paged_read(*c.cache, *c.where, n=c.N)
    assert torch.equal(k, v)
    q.quarot_check_error()


def test_offsets_past_32_bits(q):
    """Pages whose codes lie more than 4 GB into the cache."""
    H, ps, d, T = 8, 64, 128, 150
    n_pages = 2 ** 32 // (H * ps * d // 2) + 40
    cache = [torch.empty((n_pages, H, ps, d // 2), dtype=torch.uint8, device=DEV), torch.empty((n_pages, H, ps), dtype=FP16, device=DEV)]
    cache += [torch.empty_like(cache[0]), torch.empty_like(cache[1])]
    small = Case([T, T], ps, H, d, [T, T])
    kv = [torch.randn(2 * T, H, d, device=DEV).half() for _ in range(2)]
    x = _queries(2 * T, 2 * H, d, FP16, 1)
    table, lens, cu = small.where
    far = table + (n_pages - small.n_pages)
    one = _i32([0, T]), _i32([T, 2 * T])
    for tab, c in ((table, small.cache), (far, cache)):
        q.quarot_paged_append(*kv, *c, tab, lens, cu)
    for a, b in zip(q.quarot_paged_read(*small.cache, table, lens, cu, n=2 * T), q.quarot_paged_read(*cache, far, lens, cu, n=2 * T)):
        assert torch.equal(a, b)
    for max_q in (1, 300):
        a, b = (q.quarot_paged_attn(x, *c, tab, lens, cu, max_q=max_q) for tab, c in ((table, small.cache), (far, cache)))
        assert torch.equal(a, b)
    del one
    q.quarot_check_error()


@pytest.mark.parametrize("new,shared", [(None, 0), (None, 500), ([200, 1, 90], 0)])
def test_the_same_bits_every_time(q, new, shared):
    c = Case([1500, 700, 933], 32, 4, 128, new, shared, seed=2)
    x = _queries(c.N, 32, 128, FP16, 4)
    args = c.where
    first = q.quarot_paged_attn(x, *c.cache, *args, max_q=None if new is None else 200, shared_len=shared)
    for _ in range(100):
        out = q.quarot_paged_attn(x, *c.cache, *args, max_q=None if new is None else 200, shared_len=shared)
        assert torch.equal(out, first)
    _check_attn(first, x, c)
    q.quarot_check_error()


# ---------------------------------------------------------------- the compiled calls
def test_compiled_and_general_path_agree(q, monkeypatch):
    c = Case([300, 70, 20], 32, 2, 128, [40, 1, 20], seed=7)
    wide = torch.randn(c.N, 12, 128, device=DEV).half()
    x, k, v = wide[:, :8], wide[:, 8:10], wide[:, 10:]
    f = _gpu64(_freqs(64))
    pos = _i32(np.arange(c.N) * 1000)
    table, lens, cu = c.where
    assert not isinstance(q._calls, q._GeneralOnly)

    def all_calls():
        cache = [t.clone() for t in c.cache]
        turned = q.quarot_paged_append(k, v, *cache, table, lens, cu, q=x, inv_freq=f, interleaved=True, scale=0.5)
        out = torch.empty(c.N, 8, 128, device=DEV, dtype=FP16)
        ws = torch.empty(q.quarot_paged_workspace_bytes(c.N, 3, 8, 2, 128, 40, 10), dtype=torch.uint8, device=DEV)
        got = q.quarot_paged_attn(turned, *cache, table, lens, cu, max_q=40, shared_len=10, sm_scale=0.1, out=out, workspace=ws)
        assert got is out
        return [*q.quarot_rope(x, k, pos, f), q.quarot_rope(x, None, pos, f, True, 2.0)[0], turned, *cache, out,
                q.quarot_paged_attn(turned, *cache, table, lens, cu, unrotate_out=True),
                *q.quarot_paged_read(*cache, table, lens, cu, n=c.N), *q.quarot_paged_read(*cache, table, lens, out_dtype=BF16, unrotate=True)]

    fast = all_calls()
    assert q._calls.rope(x, k, pos, f, False, 1.0, None, None) is not None
    for none in (q._calls.rope(x, k, pos.long(), f, False, 1.0, None, None), q._calls.rope(x, k, pos, f[:12], False, 1.0, None, None),
                 q._calls.append(k, v.float(), *c.cache, table, lens, cu, None, None, False, 1.0, None),
                 q._calls.append(k, v, *c.cache, table, lens, cu, None, None, False, 1.0, x),
                 q._calls.read(*c.cache, table, lens, cu, None, False, 0, None, None),
                 q._calls.read(*c.cache, table, lens, cu, c.N, False, 7, None, None),
                 q._calls.attn(x, *c.cache, table, lens, cu, 40, -1, 0.0, False, None, None),
                 q._calls.attn(x[:, :3], *c.cache, table, lens, cu, 40, 0, 0.0, False, None, None),
                 q._calls.attn(x, *c.cache[:3], c.cache[0], table, lens, cu, 40, 0, 0.0, False, None, None)):
        assert none is None
    monkeypatch.setattr(q, "_calls", q._GeneralOnly())
    for a, b in zip(fast, all_calls()):
        assert a.dtype == b.dtype and torch.equal(a, b)
    q.quarot_check_error()
