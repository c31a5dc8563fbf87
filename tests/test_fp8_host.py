"""The 8-bit entry points on the host: refusals before any launch, the
binding's checks, and pins of the float64 forms the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

import __graft_entry__
import w4a4_rotated_quantized_gb300 as q
from oracle import fp8_oracle as F

P = ctypes.c_void_p
FAKE = P(0x10000)  # never dereferenced: every call below is refused, or has nothing to do
OFF4, OFF8, OFF2 = P(0x10004), P(0x10008), P(0x10002)


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return q.load()


@pytest.mark.parametrize("name", ["quarot_quant_fp8", "quarot_quant_fp8_block"])
def test_quant_validation(lib, name):
    f = getattr(lib, name)
    assert f(FAKE, 0, 0, 4096, 4096, FAKE, FAKE, None) == 0  # nothing to do
    assert f(None, 1, 0, 4096, 4096, None, None, None) == 0
    assert f(FAKE, 2, 4, 4096, 4096, FAKE, FAKE, None) == 1  # dtype
    assert f(FAKE, -1, 4, 4096, 4096, FAKE, FAKE, None) == 1
    assert f(FAKE, 0, -1, 4096, 4096, FAKE, FAKE, None) == 1
    assert f(FAKE, 0, 4, 0, 4096, FAKE, FAKE, None) == 1
    assert f(FAKE, 0, 4, 4096, 4080, FAKE, FAKE, None) == 1  # ld < d
    assert f(FAKE, 0, 4, 4104, 4104, FAKE, FAKE, None) == 2  # d % 16
    assert f(FAKE, 0, 4, (1 << 20) + 16, (1 << 20) + 16, FAKE, FAKE, None) == 2
    assert f(FAKE, 0, (1 << 31) - 100, 16, 16, FAKE, FAKE, None) == 2
    assert f(FAKE, 0, 4, 4096, 4100, FAKE, FAKE, None) == 3  # ld % 8
    assert f(None, 0, 4, 4096, 4096, FAKE, FAKE, None) == 1
    assert f(FAKE, 0, 4, 4096, 4096, None, FAKE, None) == 1
    assert f(FAKE, 0, 4, 4096, 4096, FAKE, None, None) == 1
    assert f(OFF8, 0, 4, 4096, 4096, FAKE, FAKE, None) == 3
    assert f(FAKE, 0, 4, 4096, 4096, OFF8, FAKE, None) == 3
    assert f(FAKE, 0, 4, 4096, 4096, FAKE, OFF2, None) == 3


def test_norm_validation(lib):
    def f(x=FAKE, ld=4096, r=FAKE, ld_r=4096, w=FAKE, dt=0, M=4, d=4096, eps=1e-6, h=FAKE, ld_h=4096, qo=FAKE, s=FAKE):
        return lib.quarot_add_rmsnorm_quant_fp8(x, ld, r, ld_r, w, dt, M, d, eps, h, ld_h, qo, s, None)

    assert f(M=0) == 0
    for eps in (0.0, -1.0, math.inf, math.nan):
        assert f(eps=eps) == 1
    assert f(dt=7) == 1
    assert f(ld=4080) == 1 and f(ld_r=4080) == 1 and f(ld_h=4080) == 1
    assert f(d=4090, ld=4096) == 2
    assert f(ld=4100) == 3 and f(ld_r=4100) == 3 and f(ld_h=4100) == 3
    assert f(x=None) == 1 and f(qo=None) == 1 and f(s=None) == 1
    assert f(x=OFF8) == 3 and f(r=OFF8) == 3 and f(w=OFF4) == 3 and f(h=OFF8) == 3 and f(qo=OFF4) == 3 and f(s=OFF2) == 3
    # strides of absent tensors are not looked at
    assert f(M=0, r=None, ld_r=0, h=None, ld_h=0) == 0


def test_gemm_validation(lib):
    def f(a=FAKE, sa=FAKE, w=FAKE, sw=FAKE, M=4, N=4096, K=4096, y=FAKE, dt=0):
        return lib.quarot_fp8_gemm(a, sa, w, sw, M, N, K, y, dt, None)

    assert f(M=0) == 0 and f(N=0) == 0 and f(M=0, a=None, y=None) == 0
    assert f(dt=2) == 1
    assert f(M=-1) == 1 and f(N=-1) == 1 and f(K=0) == 1
    assert f(K=4104) == 2 and f(K=(1 << 20) + 16) == 2 and f(M=(1 << 31) - 1) == 2 and f(N=(1 << 31) - 1) == 2
    for arg in ("a", "sa", "w", "sw", "y"):
        assert f(**{arg: None}) == 1
        assert f(**{arg: OFF2}) == 3
    for arg in ("a", "w", "y"):
        assert f(**{arg: OFF8}) == 3


def test_gated_validation(lib):
    def f(a=FAKE, sa=FAKE, g=FAKE, sg=FAKE, u=FAKE, su=FAKE, M=4, I=4096, K=4096, qo=FAKE, s=FAKE):
        return lib.quarot_fp8_gated_gemm(a, sa, g, sg, u, su, M, I, K, qo, s, None)

    assert f(M=0) == 0 and f(I=0) == 0
    assert f(M=-1) == 1 and f(I=-16) == 1 and f(K=-16) == 1
    assert f(K=4104) == 2 and f(I=4104) == 2
    for arg in ("a", "sa", "g", "sg", "u", "su", "qo", "s"):
        assert f(**{arg: None}) == 1
        assert f(**{arg: OFF2}) == 3
    for arg in ("a", "g", "u", "qo"):
        assert f(**{arg: OFF8}) == 3


def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 128), dtype=torch.float16)
    c, s = torch.zeros((4, 128), dtype=torch.float8_e4m3fn), torch.zeros((1, 4))
    for call in (lambda: q.quarot_quant_fp8(x), lambda: q.quarot_quant_fp8_block(x), lambda: q.quarot_quant_fp8(x.float()),
                 lambda: q.quarot_add_rmsnorm_quant_fp8(x, x), lambda: q.quarot_fp8_gemm(c, s, c, s),
                 lambda: q.quarot_fp8_gated_gemm(c, s, c, s, c, s), lambda: q.QuarotFp8Linear(x)):
        with pytest.raises(q.QuarotError):
            call()


# ---------------------------------------------------------------- the float64 forms
def test_e4m3_grid():
    t = F.e4m3_table()
    assert t[0x7E] == 448.0 and t[0x01] == 2.0 ** -9 and t[0x08] == 2.0 ** -6 and t[0x38] == 1.0 and t[0xB8] == -1.0
    assert np.isnan(t[0x7F]) and np.isnan(t[0xFF])
    mine = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, mine, equal_nan=True)


def test_round_e4m3_against_torch():
    rng = np.random.default_rng(3)
    v = np.concatenate([rng.normal(size=4000) * 2.0 ** rng.integers(-12, 8, 4000), F.e4m3_table()[:127]])
    pos = F.e4m3_table()[:127]
    v = np.concatenate([v, (pos[1:] + pos[:-1]) / 2, -(pos[1:] + pos[:-1]) / 2])  # every tie
    v = v[np.abs(v) <= 448].astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(F.round_e4m3(v), want)
    assert np.array_equal(F.e4m3_table()[F.e4m3_bytes(want)], want)


def test_quantizer_worked():
    """m = 7: v * 64; 0.21875 * 64 = 14, 0.2265625 * 64 = 14.5 (a tie of 14 and 15: the even fraction, 14)."""
    v = np.zeros((1, 144))
    v[0, :4] = [7.0, -0.21875, 0.2265625, 0.2421875]  # 0.2421875 * 64 = 15.5 -> 16
    v[0, 130] = -2.0
    codes, scale = F.quant_tokens(v)
    assert codes[0, :4].tolist() == [448.0, -14.0, 14.0, 16.0] and codes[0, 130] == -448.0
    assert scale.shape == (2, 1) and scale[0, 0] == 7.0 / 448 and scale[1, 0] == 2.0 / 448
    assert F.quant_tokens(np.zeros((1, 16)))[1][0, 0] == 1e-12 / 448


def test_norm_scales_carry_the_root_mean_square():
    rng = np.random.default_rng(4)
    h, w = rng.normal(size=(3, 272)), rng.normal(size=272)
    codes, scale = F.norm_quant(h, w, 1e-6)
    y = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + 1e-6) * w
    err = np.abs(F.token_values(codes, scale) - y)
    step = np.repeat(scale.T, 128, axis=1)[:, :272]
    assert (err <= np.maximum(np.abs(y) * 2.0 ** -4, step * 2.0 ** -10) * (1 + 1e-12)).all()
    c2, s2 = F.quant_tokens(y)  # the same codes as quantizing the normed values
    assert np.array_equal(c2, codes) and np.allclose(s2, scale, rtol=1e-14)


def test_product_brute_force():
    rng = np.random.default_rng(5)
    M, N, K = 2, 130, 272
    a, w = F.round_e4m3(rng.normal(size=(M, K))), F.round_e4m3(rng.normal(size=(N, K)))
    sa, sw = rng.uniform(0.5, 2, (3, M)), rng.uniform(0.5, 2, (2, 3))
    y, mag = F.product(a, sa, w, sw)
    for i, j in ((0, 0), (1, 127), (0, 128), (1, 129)):
        want = sum(sa[k // 128, i] * sw[j // 128, k // 128] * a[i, k] * w[j, k] for k in range(K))
        assert math.isclose(y[i, j], want, rel_tol=1e-12) and mag[i, j] >= abs(want)


def test_compiled_calls_leave_what_they_do_not_take(lib):
    c = q._calls
    x = torch.zeros(4, 256, dtype=torch.float16)
    e = x.to(torch.float8_e4m3fn)
    s = torch.ones(2, 4)
    for bad in (x, None, 7, "x", np.zeros((4, 256), np.float16), torch.zeros(4, 256, dtype=torch.float16, device="meta")):
        assert c.quant(bad, None, None, False) is None and c.quant(bad, None, None, True) is None
        assert c.norm(bad, None, None, 1e-6, None, None, None) is None
        assert c.gemm(bad, s, e, s, None, 0) is None and c.gated(bad, s, e, s, e, s, None, None) is None
    assert c.quant(x) is None and c.norm() is None and c.gemm(e, s, e, s, None) is None and c.gated(e) is None
    with pytest.raises(TypeError):
        c.bind(1, 2)
    with pytest.raises(TypeError):
        c.bind(1, 2, 3, 4, "x")
