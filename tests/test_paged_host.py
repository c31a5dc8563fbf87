"""Rotary positions and the paged cache on the host: refusals before any launch, the binding's checks, QuarotRope's
frequencies, and pins of the float64 forms."""
import ctypes
import math

import numpy as np
import pytest
import torch

import __graft_entry__
import w4a4_rotated_quantized_gb300 as q
from oracle import paged_oracle as O
from oracle import quarot_oracle as Q

P = ctypes.c_void_p
FAKE = P(0x10000)  # never dereferenced: every call below is refused, or has nothing to do
OFF2, OFF4, OFF8, ODD = P(0x10002), P(0x10004), P(0x10008), P(0x10001)


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return q.load()


def test_rope_validation(lib):
    def f(x=FAKE, Hq=4, ld=512, y=FAKE, ld_y=512, k=FAKE, Hk=2, ld_k=256, ko=FAKE, ld_ko=256, dt=0, N=3, d=128, pos=FAKE,
          fr=FAKE, rot=128, inter=0, scale=1.0):
        return lib.quarot_rope(x, Hq, ld, y, ld_y, k, Hk, ld_k, ko, ld_ko, dt, N, d, pos, fr, rot, inter, scale, None)

    assert f(N=0) == 0 and f(N=0, x=None, y=None, k=None, ko=None, pos=None) == 0
    assert f(dt=2) == 1 and f(N=-1) == 1 and f(Hq=0) == 1 and f(Hk=-1) == 1 and f(d=0) == 1 and f(inter=2) == 1
    assert f(scale=math.inf) == 1 and f(scale=math.nan) == 1
    assert f(rot=144) == 1 and f(rot=-16) == 1 and f(fr=None) == 1
    assert f(d=120, ld=480, rot=64) == 2 and f(d=2048, ld=8192, rot=64) == 2 and f(rot=24) == 2 and f(N=(1 << 24) + 1) == 2
    assert f(Hq=3000, ld=384000, ld_y=384000) == 2
    assert f(x=None) == 1 and f(y=None) == 1 and f(k=None) == 1 and f(ko=None) == 1 and f(pos=None) == 1
    assert f(ld=504) == 1 and f(ld_y=504) == 1 and f(ld_k=248) == 1 and f(ld_ko=248) == 1
    assert f(ld=516) == 3 and f(x=OFF8) == 3 and f(y=OFF8) == 3 and f(k=OFF2) == 3 and f(ko=OFF8) == 3
    assert f(pos=OFF2) == 3 and f(fr=OFF4) == 3
    assert f(N=0, Hk=0, k=None, ko=None, ld_k=0, ld_ko=0) == 0


def _append(lib, k=FAKE, ld_k=256, v=FAKE, ld_v=256, qq=FAKE, Hq=4, ld_q=512, qo=FAKE, ld_qo=512, dt=0, N=3, Hkv=2, d=128,
            fr=FAKE, rot=128, inter=0, scale=1.0, kq=FAKE, ks=FAKE, vq=FAKE, vs=FAKE, pages=9, ps=64, tab=FAKE, B=3, mp=4,
            lens=FAKE, cu=None):
    return lib.quarot_paged_append(k, ld_k, v, ld_v, qq, Hq, ld_q, qo, ld_qo, dt, N, Hkv, d, fr, rot, inter, scale, kq, ks, vq,
                                   vs, pages, ps, tab, B, mp, lens, cu, None)


def test_append_validation(lib):
    f = lambda **a: _append(lib, **a)  # noqa: E731
    assert f(N=0, B=0) == 0 and f(N=0, B=0, k=None, v=None, qq=None, Hq=0) == 0 and f(N=0, cu=FAKE) == 0
    assert f(dt=3) == 1 and f(N=-1, B=-1) == 1 and f(Hkv=0) == 1 and f(d=0) == 1 and f(pages=-1) == 1 and f(ps=0) == 1
    assert f(N=4) == 1  # one token a sequence without cu_q
    assert f(Hq=0) == 1 and f(qq=None) == 1 and f(qo=None) == 1
    assert f(inter=-1) == 1 and f(rot=144) == 1 and f(fr=None) == 1 and f(scale=math.nan) == 1
    assert f(d=96, ld_k=192, ld_v=192, rot=96) == 2 and f(d=256, ld_k=512, ld_v=512) == 2 and f(rot=24) == 2
    assert f(ps=24) == 2 and f(ps=65536 + 16) == 2 and f(mp=1 << 26) == 2 and f(N=(1 << 24) + 1, cu=FAKE) == 2
    assert f(Hkv=2000, ld_k=256000, ld_v=256000) == 2
    for a in ("k", "v", "kq", "ks", "vq", "vs", "tab", "lens"):
        assert f(**{a: None}) == 1, a
        assert f(**{a: ODD}) == 3, a
    for a in ("k", "v", "qq", "qo", "kq", "vq"):
        assert f(**{a: OFF8}) == 3, a
    assert f(ld_k=248) == 1 and f(ld_v=248) == 1 and f(ld_q=504) == 1 and f(ld_qo=504) == 1
    assert f(ld_k=260) == 3 and f(ld_q=516) == 3 and f(cu=OFF2) == 3 and f(fr=OFF4) == 3


def test_read_validation(lib):
    def f(kq=FAKE, ks=FAKE, vq=FAKE, vs=FAKE, pages=9, ps=64, Hkv=2, d=128, tab=FAKE, B=3, mp=4, lens=FAKE, cu=None, N=3,
          un=0, ko=FAKE, vo=FAKE, dt=0):
        return lib.quarot_paged_read(kq, ks, vq, vs, pages, ps, Hkv, d, tab, B, mp, lens, cu, N, un, ko, vo, dt, None)

    assert f(N=0, B=0) == 0 and f(N=0, B=0, ko=None, vo=None, kq=None) == 0
    assert f(dt=2) == 1 and f(un=2) == 1 and f(N=2) == 1 and f(d=96) == 2 and f(ps=8) == 2
    for a in ("kq", "ks", "vq", "vs", "tab", "lens", "ko", "vo"):
        assert f(**{a: None}) == 1 and f(**{a: ODD}) == 3, a
    assert f(ko=OFF8) == 3 and f(vo=OFF8) == 3 and f(lens=OFF2) == 3


def test_attn_validation(lib):
    def f(x=FAKE, ld=512, dt=0, N=3, Hq=4, Hkv=2, d=128, kq=FAKE, ks=FAKE, vq=FAKE, vs=FAKE, pages=9, ps=64, tab=FAKE, B=3, mp=4,
          lens=FAKE, cu=None, mq=1, shared=0, sm=0.0, un=0, y=FAKE, ld_y=512, ws=FAKE, wb=1 << 40):
        return lib.quarot_paged_attn(x, ld, dt, N, Hq, Hkv, d, kq, ks, vq, vs, pages, ps, tab, B, mp, lens, cu, mq, shared, sm,
                                     un, y, ld_y, ws, wb, None)

    assert f(N=0, B=0) == 0 and f(N=0, B=0, x=None, y=None, ws=None, wb=0) == 0
    assert f(dt=2) == 1 and f(N=2) == 1 and f(Hq=3) == 1 and f(Hq=0) == 1 and f(mq=0) == 1 and f(shared=-1) == 1
    assert f(shared=257) == 1  # more than the table's pages
    assert f(un=3) == 1 and f(sm=math.nan) == 1 and f(sm=math.inf) == 1
    assert f(d=96, ld=384) == 2 and f(ps=40) == 2 and f(Hq=2000, ld=256000, ld_y=256000) == 2
    for a in ("x", "y", "kq", "ks", "vq", "vs", "tab", "lens", "ws"):
        assert f(**{a: None}) == 1, a
        assert f(**{a: ODD}) == 3, a
    assert f(x=OFF8) == 3 and f(y=OFF8) == 3 and f(ld=516) == 3 and f(ld_y=504) == 1 and f(ws=P(0x10080)) == 3


def test_workspace_bytes_of_invalid_sizes(lib):
    assert q.quarot_paged_workspace_bytes(0, 1, 8, 8, 128) == 0
    assert q.quarot_paged_workspace_bytes(1, 1, 8, 8, 96) == 0
    assert q.quarot_paged_workspace_bytes(1, 1, 9, 8, 128) == 0
    assert q.quarot_paged_workspace_bytes(1, 1, 8, 8, 128, 0) == 0
    assert q.quarot_paged_workspace_bytes(1, 1, 8, 8, 128, 1, -1) == 0


def test_binding_takes_gpu_tensors_only():
    x = torch.zeros(2, 4, 128, dtype=torch.float16)
    cache = (torch.zeros(3, 4, 16, 64, dtype=torch.uint8), torch.zeros(3, 4, 16, dtype=torch.float16)) * 2
    where = (torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32))
    for call in (lambda: q.quarot_rope(x, x, where[1], torch.zeros(64, dtype=torch.float64)),
                 lambda: q.quarot_paged_append(x, x, *cache, *where), lambda: q.quarot_paged_read(*cache, *where),
                 lambda: q.quarot_paged_attn(x, *cache, *where)):
        with pytest.raises(q.QuarotError) as e:
            call()
        assert e.value.status == 1


def test_rope_frequencies():
    f = q.QuarotRope(64, device="cpu").inv_freq
    assert f.dtype == torch.float64 and f.shape == (32,) and f[0] == 1.0
    assert torch.allclose(f, 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32))
    assert torch.equal(q.QuarotRope(64, scaling="linear", factor=8.0, device="cpu").inv_freq, f / 8)
    ntk = q.QuarotRope(64, scaling="ntk", factor=4.0, device="cpu").inv_freq
    assert ntk[0] == 1.0 and math.isclose(float(ntk[-1]), float(f[-1]) / 4, rel_tol=1e-12)  # the slowest pair: the factor
    for kind in ("yarn", "smooth"):
        r = q.QuarotRope(64, scaling=kind, factor=16.0, original_len=4096, device="cpu")
        ratio = f / r.inv_freq
        assert ratio[0] == 1.0 and math.isclose(float(ratio[-1]), 16.0) and (ratio.diff() >= -1e-12).all()
        assert r.scale == (0.1 * math.log(16.0) + 1.0 if kind == "yarn" else 1.0)
    # yarn: pairs that turn more than 32 times in 4096 positions stay, those that turn less than once are divided
    turns = 4096 * f / (2 * math.pi)
    r = q.QuarotRope(64, scaling="yarn", factor=16.0, original_len=4096, device="cpu")
    step = 10000.0 ** (1 / 32)
    assert torch.equal(r.inv_freq[turns > 32 * step], f[turns > 32 * step])
    assert torch.allclose(r.inv_freq[turns < 1 / step], f[turns < 1 / step] / 16)
    for bad in (dict(rot=24), dict(rot=0), dict(rot=64, base=1.0), dict(rot=64, factor=0.5), dict(rot=64, scaling="other"),
                dict(rot=64, scaling="yarn", factor=2.0)):
        with pytest.raises(q.QuarotError):
            q.QuarotRope(device="cpu", **bad)
    with pytest.raises(q.QuarotError):
        q.QuarotPagedKVCache(4, 2, page_size=24)
    with pytest.raises(q.QuarotError):
        q.QuarotPagedKVCache(4, 2, d=96)


def test_float64_forms_agree_with_the_contiguous_oracle():
    rng = np.random.default_rng(3)
    B, T, H, d, ps = 2, 37, 2, 128, 16
    k, v = (rng.standard_normal((B, T, H, d)).astype(np.float16) for _ in range(2))
    flat = [np.zeros((B, H, T, d // 2), np.uint8), np.zeros((B, H, T), np.float16), np.zeros((B, H, T, d // 2), np.uint8),
            np.zeros((B, H, T), np.float16)]
    Q.kv_write(k, v, 0, *flat)
    table = np.array([[4, 1, 5], [0, 3, 2]])
    paged = [np.zeros((6, H, ps) + a.shape[3:], a.dtype) for a in flat]
    for b in range(B):
        for t in range(T):
            for a, p in zip(flat, paged):
                p[table[b, t // ps], :, t % ps] = a[b, :, t]
    x = rng.standard_normal((B, 6, d)).astype(np.float16)
    want = Q.decode_attn(x, *flat, T=T)
    got, tol = O.attn(x, paged, table, np.array([T, T]), None, ps)
    assert np.abs(got - want).max() < 1e-9 and (tol > 0).all()
    # several tokens at once: the last one sees what the only one saw
    got, _ = O.attn(np.concatenate([x[:1], x[:1], x[1:]]), paged, table, np.array([T, T]), np.array([0, 2, 3]), ps)
    assert np.abs(got[1:] - want).max() < 1e-9
    cut, _ = O.attn(x, paged, table, np.array([T - 1, T]), None, ps)
    assert np.abs(got[0] - cut[0]).max() < 1e-9


def test_float64_rope_turns_pairs():
    x = np.zeros((1, 1, 16))
    x[0, 0, 1] = 1.0
    f = np.array([0.0, math.pi / 2, 0.0, 0.0])
    y = O.rope(x, [1], f)  # pair 1 is (1, 5)
    assert abs(y[0, 0, 5] - 1.0) < 1e-12 and abs(y[0, 0, 1]) < 1e-12
    y = O.rope(x, [1], np.array([math.pi / 2] + [0.0] * 3), interleaved=True)  # pair 0 is (0, 1)
    assert abs(y[0, 0, 0] + 1.0) < 1e-12


def test_the_version_tells_of_the_paged_cache(lib):
    assert q.quarot_version() >> 16 == 1 and q.quarot_version() & 0xFFFF >= 3
    import os
    with open(os.path.join(os.path.dirname(q.__file__), os.pardir, "include", "quarot.h")) as f:
        told = " ".join(f.read().split("1.3 adds")[1].split("*/")[0].replace("*", " ").split())
    for name in ("rope", "paged_append", "paged_read", "paged_workspace_bytes", "paged_attn"):
        assert f"quarot_{name}" in told
    for name in ("rope", "append", "read", "attn"):
        assert getattr(q._GeneralOnly(), name)(1, 2, 3) is None


def test_compiled_calls_take_nothing_on_the_cpu(lib):
    x = torch.zeros(2, 4, 128, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    cache = (torch.zeros(3, 4, 16, 64, dtype=torch.uint8), torch.zeros(3, 4, 16, dtype=torch.float16)) * 2
    where = (torch.zeros(2, 3, dtype=torch.int32), i, None)
    assert q._calls.rope(x, x, i, None, False, 1.0, None, None) is None
    assert q._calls.append(x, x, *cache, *where, None, None, False, 1.0, None) is None
    assert q._calls.read(*cache, *where, None, False, 0, None, None) is None
    assert q._calls.attn(x, *cache, *where, 1, 0, 0.0, False, None, None) is None
