"""The 8-bit operators with block scales: what is measured, and their plain forms.

  quant   tokens [M, d] to e4m3 codes with one fp32 scale for each token and block of 128 columns, or
          weights [N, K] with one scale for each 128 x 128 block
  norm    residual addition, root-mean-square norm and the token quantizer
  gemm    codes x codes with both operands' block scales, to fp16 or bf16
  gated   silu(a Wg^T) * (a Wu^T) of such codes, quantized again

`run` computes them with elementary torch operations, or, where `own` is true, with the framework's calls.
"""
import math

import torch

own = False

BLOCK = 128
MAX_CODE = 448.0   # the largest e4m3 value
FLOOR = 1e-12      # the smallest abs-max a scale is made from
EPS = 1e-6
DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one decoded token between two layers: latency
        {"name": "norm 1 x 4096 fp16", "op": "norm", "M": 1, "d": 4096, "t": "fp16", "weight": True},
        # a ragged prompt, the learned scale absorbed into the next weights
        {"name": "norm 509 x 12288 bf16", "op": "norm", "M": 509, "d": 12288, "t": "bf16", "weight": False},
        # a batch of long prompts
        {"name": "norm 8192 x 12288 fp16", "op": "norm", "M": 8192, "d": 12288, "t": "fp16", "weight": True},
        # the feed-forward's activations before an 8-bit down projection
        {"name": "quant tokens 2048 x 12288 bf16", "op": "quant", "M": 2048, "d": 12288, "t": "bf16", "block": False},
        # a weight matrix at load time
        {"name": "quant weight 12288 x 4096 fp16", "op": "quant", "M": 12288, "d": 4096, "t": "fp16", "block": True},
        # the down projection for one decoded token: weight traffic
        {"name": "gemm 1 x 4096 x 12288 fp16", "op": "gemm", "M": 1, "N": 4096, "K": 12288, "t": "fp16"},
        # an odd decode batch
        {"name": "gemm 37 x 12288 x 4096 bf16", "op": "gemm", "M": 37, "N": 12288, "K": 4096, "t": "bf16"},
        # the down projection of one prompt
        {"name": "gemm 2048 x 4096 x 12288 fp16", "op": "gemm", "M": 2048, "N": 4096, "K": 12288, "t": "fp16"},
        # a batch of prompts
        {"name": "gemm 8192 x 12288 x 4096 bf16", "op": "gemm", "M": 8192, "N": 12288, "K": 4096, "t": "bf16"},
        # the gated half of a feed-forward block: four sequences decoding, an odd prompt, a batch of prompts
        {"name": "gated 4 x 12288 x 4096", "op": "gated", "M": 4, "I": 12288, "K": 4096},
        {"name": "gated 333 x 4096 x 4096", "op": "gated", "M": 333, "I": 4096, "K": 4096},
        {"name": "gated 4096 x 12288 x 4096", "op": "gated", "M": 4096, "I": 12288, "K": 4096},
    ]


def _spread(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v // step * step))


def draw(rng):
    """Another case of the same ranges: any number of tokens and output columns, depths that are multiples of 16."""
    op = rng.choice(["norm", "quant", "gemm", "gemm", "gated"])
    t = rng.choice(["fp16", "bf16"])
    M, K = _spread(rng, 1, 8192), _spread(rng, 256, 12288, 16)
    if op == "norm":
        return {"op": op, "M": M, "d": K, "t": t, "weight": rng.random() < 0.5}
    if op == "quant":
        block = rng.random() < 0.4
        return {"op": op, "M": _spread(rng, 100, 12288) if block else M, "d": K, "t": t, "block": block}
    if op == "gemm":
        N = _spread(rng, 100, 12288)
        while M * N * K > 8192 * 12288 * 4096:
            M = M // 2
        return {"op": op, "M": M, "N": N, "K": K, "t": t}
    I = _spread(rng, 128, 12288, 16)
    while 2 * M * I * K > 8192 * 12288 * 4096:
        M = M // 2
    return {"op": op, "M": M, "I": I, "K": K}


def _tokens(g, M, d, t):
    """Activations: normal, with a few channels that carry large values in every token."""
    x = torch.randn((M, d), generator=g, device=DEV)
    loud = torch.randint(0, d, (max(1, d // 512),), generator=g, device=DEV)
    x[:, loud] *= 30.0
    return x.to(t)


def _codes(g, M, K):
    return _quant_tokens(_tokens(g, M, K, torch.bfloat16).float())


def _weight(g, N, K):
    w = (torch.randn((N, K), generator=g, device=DEV) * 0.02).to(torch.float16)
    return _quant_block(w.float())


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op == "norm":
        t = TYPES[case["t"]]
        s["x"] = torch.randn((case["M"], case["d"]), generator=g, device=DEV).to(t)
        s["residual"] = _tokens(g, case["M"], case["d"], t)
        s["weight"] = (1.0 + 0.2 * torch.randn((case["d"],), generator=g, device=DEV)).to(t) if case["weight"] else None
    elif op == "quant":
        t = TYPES[case["t"]]
        if case["block"]:
            s["x"] = (torch.randn((case["M"], case["d"]), generator=g, device=DEV) * 0.02).to(t)
        else:
            s["x"] = _tokens(g, case["M"], case["d"], t)
    elif op == "gemm":
        s["a"], s["a_scale"] = _codes(g, case["M"], case["K"])
        s["w"], s["w_scale"] = _weight(g, case["N"], case["K"])
    else:
        s["a"], s["a_scale"] = _codes(g, case["M"], case["K"])
        s["wg"], s["wg_scale"] = _weight(g, case["I"], case["K"])
        s["wu"], s["wu_scale"] = _weight(g, case["I"], case["K"])
    return s


# ---------------------------------------------------------------- plain forms (32 bits)
def _blocks(v, rows):
    """v [M, d] padded with zeros and seen as [M / rows, rows, d / 128, 128]."""
    M, d = v.shape
    p = torch.zeros(-(-M // rows) * rows, -(-d // BLOCK) * BLOCK, dtype=v.dtype, device=v.device)
    p[:M, :d] = v
    return p.view(p.shape[0] // rows, rows, p.shape[1] // BLOCK, BLOCK)


def _quant(v, rows):
    M, d = v.shape
    b = _blocks(v, rows)
    amax = b.abs().amax(dim=(1, 3), keepdim=True).clamp(min=FLOOR)
    # 16-bit values: b * 448 is exact and a tie of the quotient is a tie in fp32 too
    codes = (b * MAX_CODE / amax).to(torch.float8_e4m3fn)
    codes = codes.view(b.shape[0] * rows, -1)[:M, :d].contiguous()
    return codes, (amax / MAX_CODE)[:, 0, :, 0]


def _quant_tokens(v):
    codes, scale = _quant(v, 1)
    return codes, scale.t().contiguous()


def _quant_block(v):
    codes, scale = _quant(v, BLOCK)
    return codes, scale.contiguous()


def _token_values(codes, scale):
    K = codes.shape[1]
    return codes.to(scale.dtype) * scale.t().repeat_interleave(BLOCK, 1)[:, :K]


def _block_values(codes, scale):
    N, K = codes.shape
    return codes.to(scale.dtype) * scale.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        h = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
        hf = h.float()
        rms = torch.sqrt(hf.square().mean(dim=1) + EPS)
        # the row's 1 / rms is a common factor of all its blocks: it goes into their scales
        codes, scale = _quant_tokens(hf if s["weight"] is None else hf * s["weight"].float())
        return {"codes": codes, "scale": scale / rms, "residual": h}
    if op == "quant":
        codes, scale = (_quant_block if case["block"] else _quant_tokens)(s["x"].float())
        return {"codes": codes, "scale": scale}
    a = _token_values(s["a"], s["a_scale"])
    if op == "gemm":
        return {"y": (a @ _block_values(s["w"], s["w_scale"]).t()).to(TYPES[case["t"]])}
    g = a @ _block_values(s["wg"], s["wg_scale"]).t()
    u = a @ _block_values(s["wu"], s["wu_scale"]).t()
    codes, scale = _quant_tokens(g / (1.0 + torch.exp(-g)) * u)
    return {"codes": codes, "scale": scale}


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import w4a4_rotated_quantized_gb300 as q

    case = s["case"]
    op = case["op"]
    if op == "norm":
        codes, scale, h = q.quarot_add_rmsnorm_quant_fp8(s["x"], s["residual"], s["weight"], eps=EPS)
        return {"codes": codes, "scale": scale, "residual": h}
    if op == "quant":
        codes, scale = (q.quarot_quant_fp8_block if case["block"] else q.quarot_quant_fp8)(s["x"])
        return {"codes": codes, "scale": scale}
    if op == "gemm":
        return {"y": q.quarot_fp8_gemm(s["a"], s["a_scale"], s["w"], s["w_scale"], out_dtype=TYPES[case["t"]])}
    codes, scale = q.quarot_fp8_gated_gemm(s["a"], s["a_scale"], s["wg"], s["wg_scale"], s["wu"], s["wu_scale"])
    return {"codes": codes, "scale": scale}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- minimum work
def work(case):
    op = case["op"]
    blocks = lambda n: -(-n // BLOCK)  # noqa: E731
    if op == "norm":
        M, d = case["M"], case["d"]
        return {"bytes": 7 * M * d + 4 * M * blocks(d) + (2 * d if case["weight"] else 0), "flops": 8 * M * d}
    if op == "quant":
        M, d = case["M"], case["d"]
        return {"bytes": 3 * M * d + 4 * (blocks(M) if case["block"] else M) * blocks(d), "flops": 3 * M * d}
    M, K = case["M"], case["K"]
    a = M * K + 4 * M * blocks(K)
    if op == "gemm":
        N = case["N"]
        return {"bytes": a + N * K + 4 * blocks(N) * blocks(K) + 2 * M * N, "flops": 2 * M * N * K}
    I = case["I"]
    return {"bytes": a + 2 * I * K + 8 * blocks(I) * blocks(K) + M * I + 4 * M * blocks(I), "flops": 4 * M * I * K}


# ---------------------------------------------------------------- the definition in 64 bits
def _round_e4m3(v):
    """Nearest e4m3 value, ties to even: 3 fraction bits above 2^-6, steps of 2^-9 below, at most 448."""
    e = torch.frexp(v)[1].clamp(min=-5).double() - 4.0
    return (torch.round(v * torch.exp2(-e)) * torch.exp2(e)).clamp(-MAX_CODE, MAX_CODE)


def _exact_quant(v, rows=1):
    M, d = v.shape
    codes = torch.empty_like(v)
    nb = -(-d // BLOCK)
    scale = torch.empty((-(-M // rows), nb), dtype=v.dtype, device=v.device)
    rep = lambda c: c.repeat_interleave(rows, 0)[:M, None]  # noqa: E731
    for b in range(nb):
        part = v[:, b * BLOCK:(b + 1) * BLOCK]
        m = part.abs().max(dim=1).values
        if rows > 1:
            m = torch.nn.functional.pad(m, (0, -M % rows)).view(-1, rows).max(dim=1).values
        m = m.clamp(min=FLOOR)
        scale[:, b] = m / MAX_CODE
        codes[:, b * BLOCK:(b + 1) * BLOCK] = _round_e4m3(part * MAX_CODE / rep(m))
    return codes, scale if rows > 1 else scale.t().contiguous()


def _exact_product(a, a_scale, w, w_scale):
    n, k = (torch.arange(m, device=DEV) // BLOCK for m in w.shape)
    A = a.double() * a_scale.double()[k].t()
    return A @ (w.double() * w_scale.double()[n[:, None], k[None, :]]).t()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double() + s["residual"].double()
        r = h.to(s["x"].dtype).double()  # the stored sum is what is normed
        inv = 1.0 / torch.sqrt((r * r).sum(dim=1) / r.shape[1] + EPS)
        codes, scale = _exact_quant(r * s["weight"].double() if s["weight"] is not None else r)
        return {"codes": codes, "scale": scale * inv, "residual": h}
    if op == "quant":
        codes, scale = _exact_quant(s["x"].double(), BLOCK if case["block"] else 1)
        return {"codes": codes, "scale": scale}
    if op == "gemm":
        return {"y": _exact_product(s["a"], s["a_scale"], s["w"], s["w_scale"])}
    g = _exact_product(s["a"], s["a_scale"], s["wg"], s["wg_scale"])
    u = _exact_product(s["a"], s["a_scale"], s["wu"], s["wu_scale"])
    codes, scale = _exact_quant(g * torch.sigmoid(g) * u)
    return {"codes": codes, "scale": scale}
