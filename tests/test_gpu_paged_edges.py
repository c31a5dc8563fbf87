"""The paged cache at the edges of its range: long and unequal sequences, loud and missing values, pages that change hands."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as O
from test_gpu_paged import ATTN, BF16, FP16, Case, _check_attn, _i32, _np, _queries, _raw
from test_gpu_parity import DEV, q  # noqa: F401  (q: fixture)

pytestmark = pytest.mark.gpu


def _row_errors(out, ref):
    """Norm of each row's difference over its own norm."""
    return np.linalg.norm(_np(out) - ref, axis=-1) / np.linalg.norm(ref, axis=-1)


# ---------------------------------------------------------------- precision
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_one_loud_token_among_many_small_ones(q, dtype):
    """A token that outweighs each of 32767 others 2^24 times, with a CTA that has all of them (38 sequences x 16 heads are
    608 units).  Rows: the loud token's probability and the output are rounded, half a step of fp16 and of the output's
    type; sums of 1024 products of 32 tokens, 2^-24 each of values 15 / |o| times as large; the small tokens' share."""
    B, H, d, ps, L = 38, 16, 64, 64, 32768
    rng = np.random.default_rng(5)
    pages = L // ps
    shape = (pages, H, ps)
    kq, vq = (rng.integers(0, 256, shape + (d // 2,), dtype=np.uint8) for _ in range(2))
    ks, vs = np.full(shape, 0.35, np.float16), rng.uniform(0.2, 0.4, shape).astype(np.float16)
    x = (rng.standard_normal((1, H, d)) * 0.05).astype(np.float32)
    x = torch.from_numpy(x).to(dtype).to(DEV).expand(B, H, d).contiguous()
    turned = _np(x[0]) @ O.hadamard(d)
    c = np.round(turned / np.abs(turned).max(-1, keepdims=True) * 7).astype(np.int64)  # a key along each head's query
    kq[0, :, 5] = ((c[:, 0::2] & 15) | ((c[:, 1::2] & 15) << 4)).astype(np.uint8)
    ks[0, :, 5] = (24 * np.log(2) / ((c * turned).sum(-1) / np.sqrt(d))).astype(np.float16)
    cache = [torch.from_numpy(a).to(DEV) for a in (kq, ks, vq, vs)]
    table = np.tile(np.arange(pages), (B, 1))
    out = q.quarot_paged_attn(x, *cache, _i32(table), _i32([L] * B), max_q=1)
    q.quarot_check_error()
    (kc, ksd), (vc, vsd) = (O.tokens([kq, ks, vq, vs], table[0], ps, L, w) for w in (0, 1))
    half = torch.finfo(dtype).eps / 2
    for h in range(H):
        s = (kc[:, h] @ turned[h]) * ksd[:, h] / np.sqrt(d)
        p = np.exp(s - s.max())
        p /= p.sum()
        assert p[5] > 0.99 and np.median(p) < 2.0 ** -22.5
        v = (p * vsd[:, h])[:, None] * vc[:, h]
        ref = v.sum(0)
        err = np.linalg.norm(_np(out[:, h]) - ref, axis=-1)
        small = np.linalg.norm(ref - v[5])
        sums = L / 32 * 2.0 ** -24 * 15 * (p * vsd[:, h]).sum() * np.sqrt(d)
        assert (err <= (half + 2.0 ** -11) * np.linalg.norm(ref) + small + sums).all(), (h, err.max() / np.linalg.norm(ref))


# ---------------------------------------------------------------- nothing to see
@pytest.mark.parametrize("hint", [1, 1000])
@pytest.mark.parametrize("new", [None, [1, 40, 0]])
def test_a_table_without_columns(q, hint, new):
    """Sequences with tokens and a table that has room for none: zeros, and an error that quarot_check_error reports."""
    lengths, N = [1, 50, 7], 3 if new is None else 41
    cache = [torch.ones((4, 2, 16, 64), dtype=torch.uint8, device=DEV), torch.ones((4, 2, 16), dtype=FP16, device=DEV)] * 2
    where = torch.empty((3, 0), dtype=torch.int32, device=DEV), _i32(lengths), None if new is None else _i32([0, 1, 41, 41])
    x = torch.randn(N, 8, 128, device=DEV).half()
    out = torch.full_like(x, 3.0)
    q.quarot_paged_attn(x, *cache, *where, max_q=hint, out=out)
    with pytest.raises(q.QuarotError) as e:
        q.quarot_check_error()
    assert e.value.status == 1 and (out == 0).all()
    k, v = q.quarot_paged_read(*cache, *where, n=N)
    with pytest.raises(q.QuarotError):
        q.quarot_check_error()
    assert (k == 0).all() and (v == 0).all()
    q.quarot_check_error()


@pytest.mark.parametrize("hint", [1, 1000])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1e-30, 1e-35, 1e-37, 1e-38, 1e-40, 0.0])
def test_queries_near_nothing(q, hint, d, size):
    """bf16 queries down to the type's subnormals: all scores are 0, and a row is the mean of the values that it sees.  Between
    them rows of ordinary size stay what they are."""
    c = Case([300, 70], 32, 2, d, [40, 33], seed=d)
    x = _queries(c.N, 8, d, BF16, 4)
    x[::2] *= size
    assert (x[::2] != 0).any() == (size > 0)
    for un in (False, True):
        out = q.quarot_paged_attn(x, *c.cache, *c.where, max_q=hint, unrotate_out=un)
        q.quarot_check_error()
        _check_attn(out, x, c, unrotate=un)


# ---------------------------------------------------------------- loud values
@pytest.mark.parametrize("hint", [1, 1000])
@pytest.mark.parametrize("d,new,shared", [(128, [40, 1, 70], 0), (64, [40, 1, 70], 0), (128, None, 0), (128, [9, 1, 3], 100)])
def test_every_value_scale_counts_as_it_is(q, hint, d, new, shared):
    """Value scales up to 65504 in many places, seen and unseen: the same outputs whatever the kernel."""
    c = Case([300, 131, 260], 32, 2, d, new, shared, seed=d)
    g = torch.Generator().manual_seed(1)
    pick = torch.rand(c.cache[3].shape, generator=g).to(DEV)
    for lo, hi, s in ((0.0, 0.02, 20000.0), (0.02, 0.03, 65504.0), (0.03, 0.04, 8188.0), (0.04, 0.05, 8192.0), (0.05, 0.06, 2.0 ** -24)):
        c.cache[3][(pick >= lo) & (pick < hi)] = s
    x = _queries(c.N, 8, d, BF16, 4)
    for un in (False, True):
        out = q.quarot_paged_attn(x, *c.cache, *c.where, max_q=hint, shared_len=shared, unrotate_out=un)
        q.quarot_check_error()
        _check_attn(out, x, c, unrotate=un)
        ref, _ = O.attn(_np(x), c.np_cache(), c.table, c.lengths, c.cu, c.ps, shared=shared, unrotate=un)
        assert _row_errors(out, ref).max() < 2.0 ** -7  # the output's half step is 2^-8 of an element at the most


@pytest.mark.parametrize("hint", [1, 1000])
@pytest.mark.parametrize("at", [0, 77, 199])
def test_rows_from_a_loud_token_on_see_all_of_it(q, hint, at):
    """A value of infinite elements, which the cache holds at its largest scale: rows from it on have that value's weight."""
    new = 200
    c = Case([new + 30], 32, 2, 128, [new], seed=8)
    page, slot = int(c.table[0, (at + 30) // 32]), (at + 30) % 32
    v = torch.randn(1, 2, 128, device=DEV).bfloat16()
    v[:, :, 5] = float("inf")
    q.quarot_paged_append(v, v, *c.cache, _i32(c.table), _i32([at + 31]))
    assert (c.cache[3][page, :, slot] == 65504.0).all()
    c.cache[1][page, :, slot] = 0.25
    x = _queries(new, 8, 128, BF16, 3)
    out = q.quarot_paged_attn(x, *c.cache, *c.where, max_q=hint)
    q.quarot_check_error()
    _check_attn(out, x, c)
    ref, _ = O.attn(_np(x), c.np_cache(), c.table, c.lengths, c.cu, c.ps)
    assert _row_errors(out, ref)[at:].max() < 2.0 ** -7


@pytest.mark.parametrize("hint", [1, 1000])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_scales_that_are_not_finite(q, hint, bad):
    """Among drafts of several tokens: rows before such a token are what they are without it; from it on a value scale counts
    as 65504, in either kernel."""
    c = Case([140, 37], 16, 2, 128, [12, 9], seed=3)
    x = _queries(c.N, 8, 128, BF16, 6)
    page, slot = int(c.table[0, 133 // 16]), 133 % 16  # position 133: rows 0 .. 4 of the first sequence are before it
    clean = [t.clone() for t in c.cache]
    keep = [0, 1, 2, 3, 4] + list(range(12, 21))
    want = q.quarot_paged_attn(x, *c.cache, *c.where, max_q=hint)
    c.cache[1][page, :, slot] = c.cache[3][page, :, slot] = bad
    got = q.quarot_paged_attn(x, *c.cache, *c.where, max_q=hint)
    assert torch.equal(got[keep], want[keep])
    c.cache[1][page, :, slot] = clean[1][page, :, slot]
    got = q.quarot_paged_attn(x, *c.cache, *c.where, max_q=hint)
    assert torch.equal(got[keep], want[keep])
    c.cache[3][page, :, slot] = 65504.0
    _check_attn(got, x, c)
    assert torch.equal(got, q.quarot_paged_attn(x, *c.cache, *c.where, max_q=hint))
    q.quarot_check_error()


# ---------------------------------------------------------------- rows, in norm
def _check_rows(q, c, x, hint):
    """Both bases: rotated rows within attn_rows' bound, unrotated ones those times H but for the two outputs' roundings."""
    both = [q.quarot_paged_attn(x, *c.cache, *c.where, max_q=hint, shared_len=c.shared, unrotate_out=un) for un in (False, True)]
    q.quarot_check_error()
    eps = torch.finfo(x.dtype).eps
    kinds = [O.attn_rows(_np(x), c.np_cache(), c.table, c.lengths, c.cu, c.ps, few, eps, shared=c.shared)
             for few in ([True, False] if c.shared and hint == 1 else [hint == 1])]  # a prefix may be worked on as many rows
    ref, _ = O.attn(_np(x), c.np_cache(), c.table, c.lengths, c.cu, c.ps, shared=c.shared)
    err = np.linalg.norm(_np(both[0]) - ref, axis=-1)
    bound = np.maximum.reduce([b for _, b in kinds])
    assert (err <= bound).all(), (float((err / bound).max()), float((err / kinds[0][0]).max()))
    d = x.shape[-1]
    turned = _np(both[0]) @ O.hadamard(d)
    off = np.linalg.norm(turned - _np(both[1]), axis=-1)
    # half a step of each, and 2^-20 for the transform in fp32
    assert (off <= (eps + 2.0 ** -20) * np.linalg.norm(turned, axis=-1) * 1.01 + 2.0 ** -24 * np.sqrt(d)).all()


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("hint", [1, 4096])
@pytest.mark.parametrize("lengths,new,ps,Hkv,Hq,d,shared", ATTN)
def test_rows_in_both_bases(q, dtype, hint, lengths, new, ps, Hkv, Hq, d, shared):
    c = Case(lengths, ps, Hkv, d, new, shared, seed=ps + Hq)
    _check_rows(q, c, _queries(c.N, Hq, d, dtype, 5), hint)


@pytest.mark.parametrize("hint", [1, 4096])
@pytest.mark.parametrize("lengths,new,ps,Hkv,Hq,d,shared", [
    ([20000, 9001], [3, 1], 64, 1, 4, 128, 0), ([33333], [2], 16, 1, 8, 64, 0), ([40000, 39000, 17000], None, 128, 1, 4, 128, 16384),
    ([65536 + 77], None, 256, 2, 2, 64, 0), ([9000, 9100], [5, 4], 48, 1, 16, 128, 8192)])
def test_rows_of_long_sequences(q, hint, lengths, new, ps, Hkv, Hq, d, shared):
    c = Case(lengths, ps, Hkv, d, new, shared, seed=ps)
    _check_rows(q, c, _queries(c.N, Hq, d, FP16, 5), hint)


@pytest.mark.parametrize("new", [[130, 700, 3], [1000]])
def test_rows_of_units_cut_between_ctas(q, new):
    """More tiles than CTAs, so that units end in another CTA than they begin in: joined states beside direct results."""
    c = Case([n + 500 for n in new], 32, 4, 64, new, seed=1)
    _check_rows(q, c, _queries(c.N, 8, 64, FP16, 5), 4096)


# ---------------------------------------------------------------- as they would be used
def test_pages_that_change_hands(q):
    """Four slots over one pool: sequences come, decode, draft, leave; another takes the pages of the one that left."""
    Hq, Hkv, d, ps, slots, cap = 8, 2, 128, 32, 4, 12
    rope = q.QuarotRope(128, base=50000.0)
    pool = q.QuarotPagedKVCache(30, Hkv, ps, d, rope=rope)
    free, owned = list(np.random.default_rng(4).permutation(30)), [[] for _ in range(slots)]
    lengths = np.zeros(slots, np.int64)
    gen = torch.Generator(device=DEV).manual_seed(9)
    tok = lambda n, h: torch.randn(n, h, d, device=DEV, generator=gen).to(BF16)  # noqa: E731
    held = {}  # what the pool has to hold of each slot: keys and values before they were quantized

    def step(new):
        for b, n in enumerate(new):
            lengths[b] += n
            while len(owned[b]) * ps < lengths[b]:
                owned[b].append(free.pop())
        table = np.zeros((slots, cap), np.int64)
        for b in range(slots):
            table[b, :len(owned[b])] = owned[b]
        one_each = all(n == 1 or lengths[b] == 0 for b, n in enumerate(new))
        cu = None if one_each else np.concatenate([[0], np.cumsum(new)])
        N = slots if one_each else int(cu[-1])
        x, k, v = tok(N, Hq), tok(N, Hkv), tok(N, Hkv)
        where = _i32(table), _i32(lengths), None if cu is None else _i32(cu)
        turned = pool.append(k, v, *where, q=x)
        out = pool.attend(turned, *where, max_q=max(max(new), 1))
        q.quarot_check_error()
        c = Case.__new__(Case)
        c.cache, c.table, c.lengths, c.cu, c.ps, c.shared = pool.tensors, table, lengths.copy(), cu, ps, 0
        _check_attn(out, turned, c)
        for i, (b, p) in enumerate(O.places(lengths, cu, N)):
            if p < 0:
                assert (out[i] == 0).all() and (turned[i] == 0).all()
            else:
                held[b, p] = k[i], v[i]
        return where

    def leave(b):
        free.extend(owned[b])
        owned[b], lengths[b] = [], 0
        for key in [key for key in held if key[0] == b]:
            del held[key]

    step([70, 33, 0, 0])
    step([1, 1, 100, 0])     # a prompt beside decoding sequences
    step([3, 1, 2, 0])       # drafts
    left = set(owned[0])
    leave(0)
    step([0, 1, 1, 0])       # one token each, an empty slot among them
    step([0, 1, 1, 90])      # a prompt in another slot
    assert left & set(owned[3])
    step([0, 1, 1, 1])
    step([64, 1, 1, 1])      # and one in the slot that was left
    where = step([1, 1, 1, 1])
    # what the pool holds of everyone, against the tokens themselves
    cu = np.concatenate([[0], np.cumsum(lengths)])
    kk, vv = pool.read(where[0], where[1], _i32(cu), n=int(cu[-1]), unrotate=True, out_dtype=BF16)
    assert len(held) == cu[-1]
    for i, (b, p) in enumerate(O.places(lengths, cu, int(cu[-1]))):
        k, v = (_np(t)[None] for t in held[b, p])
        for got, want in ((kk[i], O.rope(k, [p], _np(rope.inv_freq))[0]), (vv[i], v[0])):
            # rotated elements are off by half a scale, a 14th of the largest one; the rotation keeps the norm; bf16 out
            scale = np.abs(want @ O.hadamard(d)).max(-1) / 7
            err, norm = np.linalg.norm(_np(got) - want, axis=-1), np.linalg.norm(want, axis=-1)
            assert (err <= (np.sqrt(d) * scale / 2 + norm * 2.0 ** -8) * 1.01).all()


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("d", [64, 128])
def test_append_of_edge_values(q, dtype, d):
    """The type's largest and smallest values, zeros, one loud element; beside them an infinite and a NaN element, whose
    vectors get a finite scale and leave the other heads alone."""
    H, n = 2, 8
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).tiny
    k = torch.zeros(n, H, d, dtype=torch.float64)
    k[1] = min(big, 1e30)
    k[2, :, 5] = 65504.0
    k[3] = -tiny
    k[4, 1] = torch.linspace(-3, 3, d)
    k[5, 0, 3], k[5, 1] = float("inf"), torch.linspace(-3, 3, d)
    k[6, 0, 9], k[6, 1] = float("nan"), torch.linspace(-3, 3, d)
    k[7] = torch.linspace(2.0 ** -14, 2.0 ** -13, d)
    k = k.to(dtype).to(DEV)
    c = Case([n], 16, H, d, [n])
    q.quarot_paged_append(k, k, *c.cache, *c.where)
    q.quarot_check_error()
    cache, x, h = c.np_cache(), _np(k), O.hadamard(d)
    for which in (0, 1):
        code, s = (a[c.table[0, 0]][:, :n] for a in (cache[2 * which], cache[2 * which + 1].astype(np.float64)))
        assert np.isfinite(s).all() and (s > 0).all()
        code = O.codes(code)
        for i in range(n):
            for hh in range(H):
                if not np.isfinite(x[i, hh]).all():
                    continue
                y = x[i, hh] @ h
                top = np.abs(y).max()
                want = min(max(top, 1e-5) / 7, 65504.0)
                own = np.abs(x[i, hh]).sum() / np.sqrt(d) * (5 + np.log2(d)) * 2.0 ** -24  # as for ordinary values
                assert abs(s[hh, i] - want) <= want * 2.0 ** -11 + 2.0 ** -25 + own / 7
                near = np.clip(y / s[hh, i], -8, 7)
                assert (np.abs(code[hh, i] - near) <= 0.5 + 2.0 ** -12 + own / s[hh, i]).all()
        assert (code[1, 5] == code[1, 4]).all() and (code[1, 6] == code[1, 4]).all()
        assert s[1, 5] == s[1, 4] == s[1, 6]
    assert (cache[0][c.table[0, 0]][:, 0] == 0).all()


def test_read_refuses_numbers_of_tokens(q):
    """Before anything is allocated."""
    c = Case([5, 9], 16, 2, 64, [2, 3])
    for n, status in ((-1, 1), (-2 ** 40, 1), (2 ** 24 + 1, 2), (2 ** 40, 2)):
        with pytest.raises(q.QuarotError) as e:
            q.quarot_paged_read(*c.cache, *c.where, n=n)
        assert e.value.status == status
    assert q.quarot_paged_read(*c.cache, *c.where, n=0)[0].shape == (0, 2, 64)


@pytest.mark.parametrize("hint", [1, 4096])
@pytest.mark.parametrize("lengths,new,ps,Hkv,Hq,d,shared", [
    ([500, 100, 399, 400, 401, 0], None, 32, 2, 8, 128, 400), ([500, 100, 399, 400, 401], [3, 9, 1, 2, 30], 16, 2, 8, 64, 400),  # shorter than the prefix
    ([300, 77], [2, 1], 16, 1, 33, 128, 0), ([200, 5], None, 16, 1, 160, 64, 0), ([130], [2], 32, 1, 1024, 64, 100)])  # groups wider than a tile
def test_rows_of_short_sequences_and_wide_groups(q, hint, lengths, new, ps, Hkv, Hq, d, shared):
    c = Case(lengths, ps, Hkv, d, new, shared, seed=Hq)
    _check_rows(q, c, _queries(c.N, Hq, d, FP16, 5), hint)


@pytest.mark.parametrize("Hq", [0, 2])
def test_quotients_of_a_half_go_to_the_even_code(q, Hq):
    """Codes of bf16 values with heads of 64, whose transform is exact in fp32 and whose quotients meet a half again and
    again; and of keys that are turned by nothing (position 0), so that they go through the turn as they are."""
    d, H, n, ps = 64, 8, 8192, 64
    gen = torch.Generator().manual_seed(11)
    v = torch.randn((n, H, d), generator=gen)
    v[..., 7] *= 20
    v = v.to(BF16).to(DEV)
    table = torch.randperm(n, generator=gen).to(torch.int32)[:, None].to(DEV)  # a page a sequence
    cache = [torch.zeros((n, H, 16, d // 2), dtype=torch.uint8, device=DEV), torch.zeros((n, H, 16), dtype=FP16, device=DEV)]
    cache += [torch.zeros_like(t) for t in cache]
    f = torch.full((16,), 0.25, dtype=torch.float64, device=DEV) if Hq else None
    ones = torch.ones(n, dtype=torch.int32, device=DEV)
    q.quarot_paged_append(v, v, *cache, table, ones, inv_freq=f)
    q.quarot_check_error()
    h = torch.from_numpy(O.hadamard(d)).to(DEV)
    y = v.double() @ h
    met = 0
    for which in (0, 1):
        code, s = cache[2 * which][table[:, 0].long(), :, 0], cache[2 * which + 1][table[:, 0].long(), :, 0]
        code = torch.from_numpy(O.codes(_raw(code))).to(DEV)
        u = y / s.double()[..., None]
        want = u.round().clamp(-8, 7)  # half to even
        # fp32 leaves 2^-18 of a step where the transform is not exact
        sure = ((u - u.floor() - 0.5).abs() > 2.0 ** -18) | (u - u.floor() == 0.5)
        met += int((u - u.floor() == 0.5).sum())
        wrong = (code != want) & sure
        assert not wrong.any(), (which, int(wrong.sum()), int(((code != want) & ~sure).sum()))
    assert met > 10


@pytest.mark.parametrize("d", [64, 128])
def test_unturned_fp16_vectors_are_quarot_kv_writes(q, d):
    """17 million codes and more, bit for bit."""
    B, T, H, ps = 4, 2048, 8, 64
    table = torch.arange(B * T // ps, dtype=torch.int32, device=DEV).view(B, -1)
    for seed in range(2048 * 128 // (T * d)):
        g = torch.Generator(device=DEV).manual_seed(seed)
        k, v = (torch.randn(B, T, H, d, device=DEV, generator=g).half() for _ in range(2))
        flat = q.new_kv_cache(B, H, T, d, torch.device(DEV))
        q.quarot_kv_write(k, v, 0, *flat)
        pool = [torch.zeros((B * T // ps, H, ps) + a.shape[3:], dtype=a.dtype, device=DEV) for a in flat]
        q.quarot_paged_append(k.view(-1, H, d), v.view(-1, H, d), *pool, table, _i32([T] * B), _i32(np.arange(B + 1) * T))
        for a, p in zip(flat, pool):
            assert torch.equal(p.view((B, T // ps, H, ps) + a.shape[3:]).movedim(2, 1).flatten(2, 3), a)
    q.quarot_check_error()


@pytest.mark.parametrize("hint", [1, 1000])
@pytest.mark.parametrize("d", [64, 128])
def test_small_values_beside_a_loud_one(q, hint, d):
    """Values of 10^-5 and a token at the largest scale among them: rows that do not see it are right to 2^-22, beside the
    roundings of probabilities, values (2^-11 each) and of the output; those further on than its 32 tokens' group and
    before it have no more than these."""
    new, at = 200, 101  # the group: tokens 96 .. 127
    c = Case([new], 32, 2, d, [new], seed=d)
    g = torch.Generator().manual_seed(7)
    c.cache[3][:] = torch.exp(torch.rand(c.cache[3].shape, generator=g) * 3 - 13.4).half().to(DEV)  # from append's smallest scale up
    x = _queries(new, 8, d, BF16, 3)
    want = q.quarot_paged_attn(x, *c.cache, *c.where, max_q=hint)
    ref, _ = O.attn(_np(x), c.np_cache(), c.table, c.lengths, c.cu, c.ps)
    top = float(8 * c.cache[3].max())
    c.cache[3][int(c.table[0, at // 32]), :, at % 32] = 65504.0
    got = q.quarot_paged_attn(x, *c.cache, *c.where, max_q=hint)
    q.quarot_check_error()
    assert torch.equal(got[:96], want[:96])
    err = np.abs(_np(got)[:at] - ref[:at])
    assert (err <= 2.0 ** -22 + 2.0 ** -10 * top + np.abs(ref[:at]) * 2.0 ** -8).all(), err.max()
    loud, _ = O.attn(_np(x), c.np_cache(), c.table, c.lengths, c.cu, c.ps)
    assert _row_errors(got, loud)[at:].max() < 2.0 ** -7
