"""The 8-bit operators on the GPU against their float64 forms.

Quantizers: the codes of fp16 and bf16 inputs are exact (16-bit values times
448 are exact in fp32, and the kernels keep ties of the quotient), scales are
one or two fp32 roundings from the float64 ones.

Products: a block's 128 products of codes are exact; their fp32 sum, in an
order and with an alignment that the tensor cores choose, is off by at most
128 * 2^-23 of the sum of magnitudes; scaling and summing nb blocks adds
(nb + 3) * 2^-24; the output's rounding half a step.
"""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as F
from test_gpu_parity import DEV, q  # noqa: F401  (q: fixture)

pytestmark = pytest.mark.gpu

FP16, BF16 = torch.float16, torch.bfloat16
E4M3 = torch.float8_e4m3fn


def _np(t):
    return t.detach().double().cpu().numpy()


def _rand(shape, dtype, seed, loud=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if loud:
        x[:, torch.randint(0, shape[1], (max(1, shape[1] // 300),), generator=g)] *= 30.0
    return x.to(dtype).to(DEV)


def _operand(rows, K, seed, weights):
    """Random codes and scales in the layout of tokens or weights."""
    g = torch.Generator().manual_seed(seed)
    codes = (torch.randn((rows, K), generator=g) * 100).clamp(-448, 448).to(E4M3).to(DEV)
    nb = -(-K // 128)
    shape = (-(-rows // 128), nb) if weights else (nb, rows)
    scale = torch.exp2(torch.rand(shape, generator=g) * 6 - 9).to(DEV)
    return codes, scale


def _rel_bound(K):
    return 128 * 2.0 ** -23 + (-(-K // 128) + 3) * 2.0 ** -24


def _check_product(y, a, sa, w, sw):
    ref, mag = F.product(_np(a), _np(sa), _np(w), _np(sw))
    half = torch.finfo(y.dtype).eps / 2
    err = np.abs(_np(y) - ref)
    tol = _rel_bound(a.shape[1]) * mag * (1 + half) + np.maximum(half * np.abs(ref), 2.0 ** -25)
    bad = err > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5].tolist(), float((err / tol).max()))


def _check_gated(codes, scale, a, sa, g, sg, u, su):
    z, lin, own = F.gated(_np(a), _np(sa), _np(g), _np(sg), _np(u), _np(su))
    dz = lin * _rel_bound(a.shape[1]) + own
    c, s = _np(codes), _np(scale)
    M, I = z.shape
    nb = -(-I // 128)
    pad = lambda v: np.pad(v, ((0, 0), (0, nb * 128 - I))).reshape(M, nb, 128)  # noqa: E731
    amax, damax = np.maximum(pad(np.abs(z)).max(-1), 1e-12).T, pad(dz).max(-1).T
    assert (np.abs(s * 448 - amax) <= damax + amax * 2.0 ** -23).all()
    step = np.repeat(s.T, 128, axis=1)[:, :I]
    err = np.abs(F.token_values(c, s) - z)
    tol = np.maximum((np.abs(z) + dz) * 2.0 ** -4, step * 2.0 ** -10) * (1 + 2.0 ** -20) + dz
    assert (err <= tol).all(), float((err / tol).max())


# ---------------------------------------------------------------- quantizers
def _check_quant(codes, scale, v, weights=False):
    want_c, want_s = (F.quant_block if weights else F.quant_tokens)(_np(v))
    assert codes.dtype == E4M3 and scale.dtype == torch.float32 and tuple(scale.shape) == want_s.shape
    assert np.array_equal(_np(codes), want_c, equal_nan=True)
    assert np.array_equal(_np(scale), want_s.astype(np.float32).astype(np.float64), equal_nan=True)


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("M,d", [(1, 16), (1, 4096), (3, 128), (5, 144), (33, 1008), (130, 4096), (37, 12288), (2, 65552)])
def test_quant_tokens(q, dtype, M, d):
    x = _rand((M, d), dtype, M + d)
    codes, scale = q.quarot_quant_fp8(x)
    _check_quant(codes, scale, x)
    wide = torch.full((M + 1, d + 24), 9.0, dtype=dtype, device=DEV)
    wide[:M, 8:8 + d] = x
    c2, s2 = q.quarot_quant_fp8(wide[:M, 8:8 + d])
    assert torch.equal(c2.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(s2, scale)


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("N,K", [(1, 16), (127, 128), (129, 272), (300, 4096), (4097, 144), (256, 12288)])
def test_quant_block(q, dtype, N, K):
    w = _rand((N, K), dtype, N + K)
    codes, scale = q.quarot_quant_fp8_block(w)
    _check_quant(codes, scale, w, weights=True)
    wide = torch.full((N, K + 8), 9.0, dtype=dtype, device=DEV)
    wide[:, :K] = w
    c2, s2 = q.quarot_quant_fp8_block(wide[:, :K])
    assert torch.equal(c2.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(s2, scale)


def _edge_rows(dtype, d):
    f = torch.finfo(dtype)
    x = torch.zeros((10, d), dtype=dtype)
    x[1, 3] = f.max
    x[1, 5] = f.tiny
    x[2] = f.max
    x[3, ::2] = -f.tiny
    x[3, 1] = f.smallest_normal * f.eps  # the smallest subnormal
    x[4, 7] = float("inf")
    x[5, 9] = float("nan")
    x[6, 2] = -float("inf")
    x[7, :] = torch.arange(d).to(dtype) - d // 2
    x[8] = 1e-7
    x[9, :120] = torch.arange(120) / 8.0  # many exact ties under an abs-max of 448 / 2^k
    x[9, 120] = 14.0
    return x.to(DEV)


@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_quant_edge_values(q, dtype):
    x = _edge_rows(dtype, 272)
    codes, scale = q.quarot_quant_fp8(x)
    _check_quant(codes, scale, x)
    assert torch.isnan(codes[4, :128].float()).all() and torch.isfinite(codes[4, 128:].float()).all()
    wcodes, wscale = q.quarot_quant_fp8_block(x)
    _check_quant(wcodes, wscale, x, weights=True)


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("M,d", [(1, 16), (1, 4096), (3, 272), (5, 1008), (130, 4096), (17, 12288), (2, 65552),
                                 (1025, 272), (1030, 2064), (5, 8208)])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("weighted", [True, False])
def test_norm(q, dtype, M, d, residual, weighted):
    x = _rand((M, d), dtype, 1 + M + d)
    r = _rand((M, d), dtype, 2 + M + d) if residual else None
    w = (1 + 0.3 * _rand((1, d), torch.float32, 3 + d, loud=False)[0]).to(dtype) if weighted else None
    codes, scale, h = q.quarot_add_rmsnorm_quant_fp8(x, r, w, eps=1e-5)
    want_h = (x.float() + r.float()).to(dtype) if residual else x
    assert torch.equal(h, want_h)
    _check_norm(codes, scale, h, w, 1e-5)


def _check_norm(codes, scale, h, w, eps):
    """The mean square of d fp32 squares: at most d roundings in sequence, in fact about d / 512; 64 are granted
    (half of their relative size reaches the root), and four more roundings of the scale."""
    want_c, want_s = F.norm_quant(_np(h), None if w is None else _np(w), eps)
    got = _np(codes)
    if w is None:
        assert np.array_equal(got, want_c, equal_nan=True)
    else:
        # the product h * w is exact in fp32, times 448 it may take one rounding: a quotient within 2^-22 of a tie can fall either way
        v = _np(h) * _np(w)
        s = np.repeat(want_s.T, 128, axis=1)[:, :v.shape[1]] * np.sqrt((_np(h) ** 2).mean(1, keepdims=True) + eps)
        t = v / s
        near = np.abs(F.round_e4m3(t * (1 + 2.0 ** -22)) - F.round_e4m3(t * (1 - 2.0 ** -22))) > 0
        assert np.array_equal(got[~near], want_c[~near])
        assert near.mean() < 1e-2 + 2 / near.size
    assert (np.abs(_np(scale) - want_s) <= want_s * (32 + 4) * 2.0 ** -24).all()


@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_norm_in_place_and_strided(q, dtype):
    M, d = 19, 528
    x, r = _rand((M, d), dtype, 5), _rand((M, d), dtype, 6)
    codes, scale, h = q.quarot_add_rmsnorm_quant_fp8(x, r)
    wide = torch.full((M, 3, d + 16), 7.0, dtype=dtype, device=DEV)
    xs, rs, hs = (wide[:, i, :d] for i in range(3))
    xs.copy_(x)
    rs.copy_(r)
    c2, s2, h2 = q.quarot_add_rmsnorm_quant_fp8(xs, rs, residual_out=hs)
    assert h2.data_ptr() == hs.data_ptr() and torch.equal(hs, h) and (wide[:, :, d:] == 7.0).all()
    assert torch.equal(c2.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(s2, scale)
    for target in (rs, xs):  # the residual updated where it stands, or written over x
        xs.copy_(x)
        rs.copy_(r)
        c2, s2, _ = q.quarot_add_rmsnorm_quant_fp8(xs, rs, residual_out=target)
        assert torch.equal(target, h)
        assert torch.equal(c2.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(s2, scale)
    out = torch.empty_like(x)
    c3, s3, h3 = q.quarot_add_rmsnorm_quant_fp8(x, None, residual_out=out)
    assert h3 is out and torch.equal(out, x)


@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_norm_edge_rows(q, dtype):
    x = _edge_rows(dtype, 272)
    codes, scale, _ = q.quarot_add_rmsnorm_quant_fp8(x)
    s = _np(scale)
    assert np.isnan(s[:, 5]).all()              # NaN anywhere in the row: its root mean square is NaN
    assert np.isnan(s[0, 4]) and s[1, 4] == 0   # infinity: NaN in its block, zero in the others
    if dtype == FP16:
        rows = [0, 1, 2, 3, 7, 8, 9]
        _check_norm(codes[rows], scale[:, rows], x[rows], None, 1e-6)
    else:  # the square of the largest bf16 values passes the fp32 range: an infinite root, scales of zero
        assert (s[:, 2] == 0).all()
        rows = [0, 3, 7, 8, 9]
        _check_norm(codes[rows], scale[:, rows], x[rows], None, 1e-6)


# ---------------------------------------------------------------- products
GEMM = [(1, 1, 16), (1, 4096, 4096), (2, 127, 144), (5, 129, 128), (8, 1000, 12288), (17, 64, 272), (33, 4100, 1008),
        (64, 256, 256), (65, 300, 528), (100, 129, 4096), (128, 128, 384), (129, 1025, 640), (200, 777, 2064),
        (256, 512, 512), (257, 2048, 1040), (513, 1031, 272), (1000, 257, 4096), (1500, 2500, 400),
        (2600, 2100, 144), (2601, 2101, 1168), (20000, 300, 128), (150, 40000, 272),
        (300, 8, 256), (4000, 1, 16), (3000, 24, 4096), (100, 25000, 272), (70, 40001, 400)]


@pytest.mark.parametrize("M,N,K", GEMM)
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_gemm(q, M, N, K, dtype):
    a, sa = _operand(M, K, M + N + K, False)
    w, sw = _operand(N, K, M + N + K + 1, True)
    guard = torch.full((M * N + 64,), 5.0, dtype=dtype, device=DEV)
    y = guard[:M * N].view(M, N)
    assert q.quarot_fp8_gemm(a, sa, w, sw, y=y) is y
    q.quarot_check_error()
    _check_product(y, a, sa, w, sw)
    assert (guard[M * N:] == 5.0).all()


@pytest.mark.parametrize("M,N,K", [(3, 200, 12288), (130, 384, 4096), (700, 520, 1024)])
def test_gemm_exact_integers(q, M, N, K):
    """Codes of -8 .. 8 and scales of 1 and 2 keep every partial sum an integer below 2^24: y is the exact sum rounded once."""
    g = torch.Generator().manual_seed(M)
    a = torch.randint(-8, 9, (M, K), generator=g)
    w = torch.randint(-8, 9, (N, K), generator=g)
    nb = K // 128
    sa = torch.randint(1, 3, (nb, M), generator=g)
    sw = torch.randint(1, 3, (-(-N // 128), nb), generator=g)
    A = a * sa.t().repeat_interleave(128, 1)
    W = w * sw.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
    want = (A.double() @ W.double().t()).to(BF16)
    y = q.quarot_fp8_gemm(a.float().to(E4M3).to(DEV), sa.float().to(DEV), w.float().to(E4M3).to(DEV), sw.float().to(DEV),
                          out_dtype=BF16)
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_gemm_nan_stays_in_its_row_and_column(q, M):
    N, K = 260, 272
    a, sa = _operand(M, K, 1, False)
    w, sw = _operand(N, K, 2, True)
    clean = q.quarot_fp8_gemm(a, sa, w, sw)
    sa[1, 1] = float("nan")
    w[200, 271] = float("nan")
    y = q.quarot_fp8_gemm(a, sa, w, sw)
    assert torch.isnan(y[1]).all() and torch.isnan(y[:, 200]).all()
    keep = torch.ones((M, N), dtype=torch.bool, device=DEV)
    keep[1] = False
    keep[:, 200] = False
    assert torch.equal(y[keep], clean[keep])


GATED = [(1, 16, 16), (1, 4096, 4096), (3, 144, 272), (7, 272, 128), (16, 1040, 4096), (33, 400, 1008), (64, 256, 512),
         (65, 656, 528), (130, 1024, 640), (257, 272, 1040), (333, 1040, 2064), (600, 784, 400),
         (2600, 1040, 144), (2601, 1168, 1296), (20000, 144, 128), (150, 20000, 272), (70, 12304, 272), (100, 20000, 400)]


@pytest.mark.parametrize("M,I,K", GATED)
def test_gated(q, M, I, K):
    a, sa = _operand(M, K, M + I + K, False)
    g, sg = _operand(I, K, M + I + K + 1, True)
    u, su = _operand(I, K, M + I + K + 2, True)
    sg.mul_(2.0 ** -8 * (12.0 / K ** 0.5))  # gate values of a few units
    guard = torch.full((M * I + 64,), 0x55, dtype=torch.uint8, device=DEV)
    qo = guard[:M * I].view(E4M3).view(M, I)
    codes, scale = q.quarot_fp8_gated_gemm(a, sa, g, sg, u, su, q_out=qo)
    q.quarot_check_error()
    assert codes is qo and (guard[M * I:] == 0x55).all()
    _check_gated(codes, scale, a, sa, g, sg, u, su)


def test_gated_extremes(q):
    """Zero tokens quantize to zeros under the floor; large gates of either sign give u and 0; NaN stays in its row."""
    M, I, K = 6, 144, 128
    a, sa = _operand(M, K, 1, False)
    g, sg = _operand(I, K, 2, True)
    u, su = _operand(I, K, 3, True)
    g[:] = 1.0
    sa[:] = 1.0
    a[0] = 0.0
    a[1] = 200.0    # g = 200 * 128: silu(g) = g
    a[2] = -200.0   # exp overflows: silu(g) = -0
    a[3] = 1.0
    sa[0, 4] = float("inf")
    sg[:] = 1.0
    codes, scale = q.quarot_fp8_gated_gemm(a, sa, g, sg, u, su)
    c, s = codes.float(), scale
    assert (c[0] == 0).all() and (s[:, 0] == np.float32(1e-12) / np.float32(448)).all()
    assert (c[2] == 0).all() and (s[:, 2] == s[:, 0]).all()
    assert torch.isnan(c[4]).all() and torch.isnan(s[:, 4]).all()
    rows = [1, 3]
    _check_gated(codes[rows], scale[:, rows], a[rows], sa[:, rows], g, sg, u, su)


@pytest.mark.parametrize("M", [3, 70, 3000])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_gated_gates_near_the_largest_float(q, M, sign):
    """silu(g) is g for g = 2.8e38, whose multiple by log2 e overflows, and 0 for -2.8e38."""
    I, K = 1152, 128
    a, sa = _operand(M, K, 1, False)
    u, su = _operand(I, K, 2, True)
    a[:], sa[:] = 1.0, 2.0 ** 60
    g, sg = torch.full((I, K), sign, device=DEV).to(E4M3), torch.full((9, 1), 1.9e18, device=DEV)
    su.mul_(2.0 ** -110)
    codes, scale = q.quarot_fp8_gated_gemm(a, sa, g, sg, u, su)
    q.quarot_check_error()
    if sign > 0:
        _check_gated(codes, scale, a, sa, g, sg, u, su)
    else:
        assert (codes.float() == 0).all()


# ---------------------------------------------------------------- as they are used
def _weights(N, K, seed):
    return (_rand((N, K), FP16, seed, loud=False).float() * K ** -0.5).to(FP16)


def _values(codes, scale):
    return F.token_values(_np(codes), _np(scale))


@pytest.mark.parametrize("M", [1, 20, 150, 400])
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_feed_forward_block(q, M, dtype):
    """Norm, gated product and down projection in a row: each step against the float64 form of its own inputs, and
    the block within the quantization error of the unquantized one."""
    K, I = 528, 784
    wg, wu, wd = _weights(I, K, 1).to(dtype), _weights(I, K, 2).to(dtype), _weights(K, I, 3).to(dtype)
    nw = (1 + 0.1 * _rand((1, K), torch.float32, 4, loud=False)[0]).to(dtype)
    x, r = _rand((M, K), dtype, 5, loud=False), _rand((M, K), dtype, 6, loud=False)
    mlp = q.QuarotFp8GatedMLP(wg, wu, wd, nw)
    y, h = mlp(x, r)
    q.quarot_check_error()
    assert y.dtype == dtype and torch.equal(h, (x.float() + r.float()).to(dtype))
    a, sa, _ = q.quarot_add_rmsnorm_quant_fp8(x, r, nw)
    z, sz = q.quarot_fp8_gated_gemm(a, sa, mlp.gate_q, mlp.gate_scale, mlp.up_q, mlp.up_scale)
    _check_gated(z, sz, a, sa, mlp.gate_q, mlp.gate_scale, mlp.up_q, mlp.up_scale)
    _check_product(y, z, sz, mlp.down.w_q, mlp.down.w_scale)
    hn = _np(h)
    n = hn / np.sqrt((hn * hn).mean(1, keepdims=True) + 1e-6) * _np(nw)
    full = (F.silu(n @ _np(wg).T) * (n @ _np(wu).T)) @ _np(wd).T
    # every e4m3 value is off by at most 2^-4, about 0.026 of its size in the root mean square; five operands' errors, independent
    assert np.linalg.norm(_np(y) - full) / np.linalg.norm(full) < 5 ** 0.5 * 0.026 * 2
    y3, h3 = mlp(x.view(1, M, K))
    assert y3.shape == (1, M, K) and torch.equal(h3.view(M, K), x)


def test_linear(q):
    w = _weights(300, 400, 7)
    lin = q.QuarotFp8Linear(w)
    x = _rand((18, 400), FP16, 8).view(2, 9, 400)
    y = lin(x)
    a, sa = q.quarot_quant_fp8(x.view(18, 400))
    assert y.shape == (2, 9, 300) and torch.equal(y.view(18, 300), q.quarot_fp8_gemm(a, sa, lin.w_q, lin.w_scale))
    assert lin(x.to(BF16)).dtype == BF16
    with pytest.raises(q.QuarotError):
        lin(x[..., :384])


@pytest.mark.parametrize("M", [1, 40, 300])
def test_capture_streams_and_repeats(q, M):
    """The block captured into a graph and replayed on new inputs, eager calls between the replays, two streams at once,
    and a hundred repeats: always the same bits."""
    K, I = 512, 640
    mlp = q.QuarotFp8GatedMLP(_weights(I, K, 1), _weights(I, K, 2), _weights(K, I, 3))
    xs = [_rand((M, K), FP16, 10 + i) for i in range(3)]
    want = [mlp(x, xs[0])[0].clone() for x in xs]
    x, r = xs[0].clone(), xs[0].clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        mlp(x, r)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y, _ = mlp(x, r)
        graphs.append(g)
        outs.append(y)
    for i, xi in enumerate(xs):
        x.copy_(xi)
        graphs[0].replay()
        eager = mlp(xi, xs[0])[0]
        graphs[1].replay()
        assert torch.equal(outs[0], want[i]) and torch.equal(outs[1], want[i]) and torch.equal(eager, want[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(50):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(mlp(xs[k + 1], xs[0], stream=s)[0])
    torch.cuda.synchronize()
    q.quarot_check_error()
    for k in range(2):
        assert all(torch.equal(y, want[k + 1]) for y in got[k])


@pytest.mark.parametrize("M", [1, 40, 129, 700])
def test_calls_in_a_row_wait_for_one_another(q, M):
    """Each call reads what the one before wrote, into buffers that the one before that still read."""
    K, I = 1024, 1536
    w = [_operand(n, k, 90 + i, True) for i, (n, k) in enumerate([(I, K), (I, K), (K, I)])]
    w = [(c, s * 2.0 ** -12) for c, s in w]
    weight = _rand((1, K), FP16, 93, loud=False)[0]
    x0 = _rand((M, K), FP16, 94)
    y, h = torch.empty_like(x0), torch.empty_like(x0)
    a, sa = q.quarot_quant_fp8(x0)
    z, sz = torch.empty((M, I), dtype=E4M3, device=DEV), torch.empty((I // 128, M), device=DEV)

    def layers(n, pause):
        y.copy_(x0)
        h.copy_(x0)
        for _ in range(n):
            q.quarot_add_rmsnorm_quant_fp8(y, h, weight, residual_out=h, q_out=a, scale_out=sa)
            pause()
            q.quarot_fp8_gated_gemm(a, sa, *w[0], *w[1], q_out=z, scale_out=sz)
            pause()
            q.quarot_fp8_gemm(z, sz, *w[2], y=y)
            pause()
            q.quarot_quant_fp8(y, q_out=a, scale_out=sa)
            pause()
        return [t.clone() for t in (y, h, a.view(torch.uint8), sa, z.view(torch.uint8), sz)]

    want = layers(12, torch.cuda.synchronize)
    assert torch.isfinite(want[0].float()).all() and want[0].abs().max() > 0
    for _ in range(3):
        assert all(torch.equal(p, r) for p, r in zip(layers(12, lambda: None), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layers(12, lambda: None)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, r) for p, r in zip(got, want))
    q.quarot_check_error()


def test_a_given_streams_memory_is_its_own(q):
    """What a call on a given stream allocates is not what work still queued on the current stream writes."""
    x = _rand((64, 512), FP16, 20)
    lin = q.QuarotFp8Linear(_weights(512, 512, 21))
    mlp = q.QuarotFp8GatedMLP(_weights(512, 512, 21), _weights(512, 512, 22), _weights(512, 512, 23))
    side = torch.cuda.Stream()

    def all_of(stream):
        a, sa = q.quarot_quant_fp8(x, stream=stream)
        return [a.view(torch.uint8), sa, q.quarot_fp8_gemm(a, sa, lin.w_q, lin.w_scale, stream=stream),
                lin(x, stream=stream), *mlp(x, x, stream=stream)]

    want = all_of(None)
    torch.cuda.synchronize()
    old = [torch.empty_like(t) for t in want for _ in range(4)]
    torch.cuda._sleep(20_000_000)  # about 10 ms
    for t in old:
        t.fill_(7)
    del old, t
    got = all_of(side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, r) for p, r in zip(got, want))
    with pytest.raises(q.QuarotError):
        q.quarot_quant_fp8(x.cpu(), stream=side)


@pytest.mark.parametrize("M", [1, 129, 600])
def test_forked_and_joined_streams(q, M):
    """Calls that follow an event of another stream, two kernels at once, a fill or a copy, eagerly and as graph nodes."""
    K, N = 768, 640
    w = [_operand(N, K, 60 + i, True) for i in range(2)]
    d, sd = _operand(K, N, 62, True)
    x = _rand((M, K), BF16, 63)
    side = torch.cuda.Stream()

    def passes():
        here = torch.cuda.current_stream()
        h = torch.zeros_like(x)
        for _ in range(4):
            a, sa = q.quarot_quant_fp8(x)            # after a fill, and after the join below
            side.wait_stream(here)
            with torch.cuda.stream(side):
                y1 = q.quarot_fp8_gemm(a, sa, *w[1], out_dtype=BF16)
                c1, s1 = q.quarot_quant_fp8(y1)
            y0 = q.quarot_fp8_gemm(a, sa, *w[0], out_dtype=BF16)
            c0, s0 = q.quarot_quant_fp8(y0)
            here.wait_stream(side)                   # both quantizers are what the next call follows
            g = q.quarot_fp8_gemm(c1, s1, d, sd, out_dtype=BF16)
            c, s, h = q.quarot_add_rmsnorm_quant_fp8(g, h)
            h = h.clone()
            for t in (a, sa, y1, c1, s1):
                t.record_stream(side)
        return [y0, c0.view(torch.uint8), s0, g, c.view(torch.uint8), s, h]

    want = [t.clone() for t in passes()]
    torch.cuda.synchronize()
    assert all(torch.equal(p, r) for p, r in zip(passes(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = passes()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, r) for p, r in zip(got, want))
    q.quarot_check_error()


@pytest.mark.parametrize("M,N,K", [(4200, 2304, 1040), (4096, 1536, 128), (700, 4000, 2064)])
def test_many_tokens_repeat(q, M, N, K):
    """Several tiles for each pair of CTAs, launch after launch and beside small calls of another stream: the same bits."""
    a, sa = _operand(M, K, 70, False)
    w, sw = _operand(N, K, 71, True)
    u, su = _operand(N, K, 72, True)
    sw.mul_(2.0 ** -8)
    b, sb = _operand(9, K, 73, False)
    want = q.quarot_fp8_gemm(a, sa, w, sw), *q.quarot_fp8_gated_gemm(a, sa, w, sw, u, su), q.quarot_fp8_gemm(b, sb, w, sw)
    rows = torch.randint(0, M, (64,), generator=torch.Generator().manual_seed(74)).to(DEV)
    _check_product(want[0][rows], a.view(torch.uint8)[rows].view(E4M3), sa[:, rows], w, sw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(25):
        small = [q.quarot_fp8_gemm(b, sb, w, sw, stream=side) for _ in range(3)]
        got = q.quarot_fp8_gemm(a, sa, w, sw), *q.quarot_fp8_gated_gemm(a, sa, w, sw, u, su)
        torch.cuda.synchronize()
        assert all(torch.equal(g.view(torch.uint8), v.view(torch.uint8)) for g, v in zip(got, want))
        assert all(torch.equal(y, want[3]) for y in small)
    q.quarot_check_error()


class _Sub(torch.Tensor):
    """A subclass, which the compiled form leaves to the general one."""


def test_compiled_and_general_forms_agree(q):
    M, K, N = 21, 272, 144
    x, r, w = _rand((M, K), BF16, 40), _rand((M, K), BF16, 41), _rand((1, K), BF16, 42, loud=False)[0]
    wt, wu = _weights(N, K, 43), _weights(N, K, 44)
    wq, ws = q.quarot_quant_fp8_block(wt)
    uq, us = q.quarot_quant_fp8_block(wu)

    def all_of(x, r, wt):
        a, sa, h = q.quarot_add_rmsnorm_quant_fp8(x, r, w)
        b, sb, h0 = q.quarot_add_rmsnorm_quant_fp8(x)
        assert h0 is x
        b, sb, h1 = q.quarot_add_rmsnorm_quant_fp8(x, residual_out=torch.empty_like(r.as_subclass(torch.Tensor)))
        a2, s2 = q.quarot_quant_fp8(x)
        w2, ws2 = q.quarot_quant_fp8_block(wt)
        like = (lambda t: t.as_subclass(_Sub)) if type(x) is _Sub else lambda t: t
        y = q.quarot_fp8_gemm(like(a), sa, wq, ws, out_dtype=BF16)
        z, sz = q.quarot_fp8_gated_gemm(like(a), sa, wq, ws, uq, us)
        return a, sa, h, b, sb, h1, a2, s2, w2, ws2, y, z, sz

    raw = lambda t: t.as_subclass(torch.Tensor).contiguous().view(torch.uint8)  # noqa: E731
    got = all_of(x, r, wt)
    want = all_of(x.as_subclass(_Sub), r.as_subclass(_Sub), wt.as_subclass(_Sub))
    assert all(g.dtype == v.dtype and g.shape == v.shape and torch.equal(raw(g), raw(v)) for g, v in zip(got, want))
    out = torch.empty((M, N), dtype=FP16, device=DEV)
    assert q.quarot_fp8_gemm(got[0], got[1], wq, ws, y=out) is out
    assert q.quarot_fp8_gemm(got[0].as_subclass(_Sub), got[1], wq, ws, y=out) is out


def test_refusals(q):
    a, sa = _operand(4, 256, 1, False)
    w, sw = _operand(130, 256, 2, True)
    x = _rand((4, 256), FP16, 1)
    bad = [
        lambda: q.quarot_fp8_gemm(a, sa.t().contiguous(), w, sw),             # scales laid out the other way
        lambda: q.quarot_fp8_gemm(a, sa[:1], w, sw),                          # too few scales
        lambda: q.quarot_fp8_gemm(a, sa, w, sw[:1]),
        lambda: q.quarot_fp8_gemm(a, sa, w[:, :128].contiguous(), sw[:, :1].contiguous()),  # another depth
        lambda: q.quarot_fp8_gemm(a.view(torch.uint8), sa, w, sw),
        lambda: q.quarot_fp8_gemm(a, sa.half(), w, sw),
        lambda: q.quarot_fp8_gemm(a[:, ::2], sa[:1], w, sw),
        lambda: q.quarot_fp8_gemm(a, sa, w, sw, out_dtype=torch.float32),
        lambda: q.quarot_fp8_gemm(a, sa, w, sw, y=torch.empty((4, 128), dtype=FP16, device=DEV)),
        lambda: q.quarot_fp8_gated_gemm(a, sa, w, sw, w[:128], sw[:1]),
        lambda: q.quarot_fp8_gated_gemm(a, sa, w, sw, w, sw),                 # 130 columns: not a multiple of 16
        lambda: q.quarot_quant_fp8(x.float()),
        lambda: q.quarot_quant_fp8(x[:, :200]),                               # 200 % 16
        lambda: q.quarot_quant_fp8(x.t()),
        lambda: q.quarot_quant_fp8(x, q_out=torch.empty((4, 128), dtype=E4M3, device=DEV)),
        lambda: q.quarot_add_rmsnorm_quant_fp8(x, x.to(BF16)),
        lambda: q.quarot_add_rmsnorm_quant_fp8(x, x[:2]),
        lambda: q.quarot_add_rmsnorm_quant_fp8(x, x, torch.ones(128, dtype=FP16, device=DEV)),
        lambda: q.quarot_add_rmsnorm_quant_fp8(x, x, eps=0.0),
        lambda: q.QuarotFp8GatedMLP(x, x, x),
    ]
    for call in bad:
        with pytest.raises(q.QuarotError):
            call()


def test_empty(q):
    w, sw = _operand(130, 256, 2, True)
    x = torch.empty((0, 256), dtype=FP16, device=DEV)
    a, sa = q.quarot_quant_fp8(x)
    assert a.shape == (0, 256) and sa.shape == (2, 0)
    assert q.quarot_fp8_gemm(a, sa, w, sw).shape == (0, 130)
    c, s, h = q.quarot_add_rmsnorm_quant_fp8(x, x)
    assert c.shape == (0, 256) and h.shape == (0, 256)
