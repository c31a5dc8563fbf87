"""Operators of a paged, rotated INT4 KV cache: what is measured, and their plain forms.

  rope    rotary positions of queries and keys: half or interleaved pairs, part of the head, any frequencies
  append  new keys (positions rotated on the way) and values into 4-bit pages, the queries rotated beside them;
          what was stored is read back as the values that the codes stand for
  attn    attention over the pages: one token a sequence or several, a prefix that all sequences share, or none
  read    cached tokens back in 16 bits, in the rotated basis or the original one

`run` computes them with elementary torch operations, or, where `own` is true, with the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # the query and key heads of one decoded token: latency
        {"name": "rope 1 token 32+8 heads bf16", "op": "rope", "N": 1, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128, "pairs": False, "far": 4096, "t": "bf16"},
        # a batch of prompts in a long context, three quarters of each head rotated, neighbouring elements paired
        {"name": "rope 8192 tokens 32+8 heads fp16", "op": "rope", "N": 8192, "Hq": 32, "Hkv": 8, "d": 128, "rot": 96, "pairs": True, "far": 1000000, "t": "fp16"},
        # sixteen sequences decode one token each
        {"name": "append 16 x 1 bf16", "op": "append", "B": 16, "Q": 1, "ragged": False, "L": 4096, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128, "pairs": False, "ps": 64, "t": "bf16"},
        # ragged prompts of small heads, half of each rotated
        {"name": "append 5 x 700 d64 fp16", "op": "append", "B": 5, "Q": 700, "ragged": True, "L": 2000, "Hq": 16, "Hkv": 16, "d": 64, "rot": 32, "pairs": True, "ps": 16, "t": "fp16"},
        # a batch of prompts
        {"name": "append 4 x 2048 fp16", "op": "append", "B": 4, "Q": 2048, "ragged": False, "L": 2048, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128, "pairs": False, "ps": 64, "t": "fp16"},
        # one sequence decodes over an odd context: latency
        {"name": "attn 1 x 4097 fp16", "op": "attn", "B": 1, "Q": 1, "ragged": False, "S": 0, "L": 4097, "Hq": 32, "Hkv": 8, "d": 128, "ps": 64, "t": "fp16"},
        # a decode batch without a common prefix: cache traffic
        {"name": "attn 16 x 4096 fp16", "op": "attn", "B": 16, "Q": 1, "ragged": False, "S": 0, "L": 4096, "Hq": 32, "Hkv": 8, "d": 128, "ps": 64, "t": "fp16"},
        # answers of many lengths to one system prompt
        {"name": "attn 64 sharing 8000 + 500 bf16", "op": "attn", "B": 64, "Q": 1, "ragged": True, "S": 8000, "L": 500, "Hq": 32, "Hkv": 8, "d": 128, "ps": 32, "t": "bf16"},
        # many questions about one long document
        {"name": "attn 256 sharing 32768 + 300 fp16", "op": "attn", "B": 256, "Q": 1, "ragged": True, "S": 32768, "L": 300, "Hq": 32, "Hkv": 8, "d": 128, "ps": 128, "t": "fp16"},
        # prompts over their own pages
        {"name": "attn 4 x 2048 tokens fp16", "op": "attn", "B": 4, "Q": 2048, "ragged": False, "S": 0, "L": 2048, "Hq": 32, "Hkv": 8, "d": 128, "ps": 64, "t": "fp16"},
        # one short sequence leaves the pages
        {"name": "read 1 x 333 fp16", "op": "read", "B": 1, "Q": 333, "ragged": False, "L": 333, "Hkv": 8, "d": 128, "ps": 16, "back": True, "t": "fp16"},
        # a whole batch does
        {"name": "read 16 x 4096 bf16", "op": "read", "B": 16, "Q": 4096, "ragged": False, "L": 4096, "Hkv": 8, "d": 128, "ps": 64, "back": False, "t": "bf16"},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Another case of the same ranges: 1 to 16 cached heads, groups of 1 to 8, heads of 64 or 128, pages of 16 to 128."""
    op = rng.choice(["rope", "append", "attn", "attn", "attn", "read"])
    Hkv, d, ps, t = _spread(rng, 1, 16), rng.choice([64, 128, 128]), rng.choice([16, 32, 48, 64, 128]), rng.choice(["fp16", "bf16"])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 4, 5, 8])
    rot, pairs = rng.randrange(16, d + 1, 16), rng.random() < 0.5
    if op == "rope":
        N = _spread(rng, 1, 8192 * 40 // (Hq + Hkv))
        return {"op": op, "N": min(N, 16384), "Hq": Hq, "Hkv": Hkv, "d": d, "rot": rot, "pairs": pairs, "far": _spread(rng, 100, 2000000), "t": t}
    B = _spread(rng, 1, 256)
    if op == "append":
        Q = _spread(rng, 1, max(1, 8192 * 40 // ((Hq + Hkv) * B)))
        return {"op": op, "B": B, "Q": min(Q, 8192), "ragged": rng.random() < 0.5, "L": min(Q, 8192) + rng.randrange(0, 500), "Hq": Hq, "Hkv": Hkv, "d": d,
                "rot": rot, "pairs": pairs, "ps": ps, "t": t}
    if op == "read":
        Q = min(_spread(rng, 1, max(1, 16 * 4096 * 8 // (Hkv * B))), 32768)
        return {"op": op, "B": B, "Q": Q, "ragged": rng.random() < 0.5, "L": Q + rng.randrange(0, 100), "Hkv": Hkv, "d": d, "ps": ps, "back": rng.random() < 0.5, "t": t}
    kind = rng.random()
    if kind < 0.3:  # prompts or drafts: several tokens of a sequence at once, over a cached part of any length
        B = _spread(rng, 1, 16)
        Q = _spread(rng, 2, max(2, min(2048, 8192 * 32 // (Hq * B))))
        S = rng.choice([0, _spread(rng, 1, 4096)])
        return {"op": op, "B": B, "Q": Q, "ragged": rng.random() < 0.5, "S": S, "L": Q + rng.choice([0, _spread(rng, 1, 1000)]), "Hq": Hq, "Hkv": Hkv, "d": d, "ps": ps, "t": t}
    S = 0 if kind < 0.6 else _spread(rng, 16, max(16, min(32768, 256 * 32768 * 32 // (Hq * B))))
    L = _spread(rng, 1, max(1, min(32768, 16 * 4096 * 8 // (Hkv * B))))
    return {"op": op, "B": B, "Q": 1, "ragged": rng.random() < 0.5, "S": S, "L": L, "Hq": Hq, "Hkv": Hkv, "d": d, "ps": ps, "t": t}


def _frequencies(rot):
    """Inverse frequencies of a context stretched eight times: the slow half of the pairs turns eight times slower."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    f = 10000.0 ** (-2.0 * i / rot)
    return torch.where(f > 0.01, f, f / 8.0)


def _lengths(case):
    """New tokens of each sequence, and all of them behind the shared ones: the case's own, whatever the values."""
    B, Q, L = case["B"], case["Q"], case["L"]
    g = torch.Generator()
    g.manual_seed(B + 1000 * Q + 7000 * L)
    new = torch.full((B,), Q, dtype=torch.int64)
    total = torch.full((B,), L, dtype=torch.int64)
    if case["ragged"]:
        r = torch.rand((2, B), generator=g)
        new = (1 + r[0] * (Q - 1)).round().long().clamp(1, Q)
        total = torch.maximum(new, (1 + r[1] * (L - 1)).round().long())
        new[0], total[0] = Q, L
    return new, total


def _codes(g, shape):
    """Packed codes of rotated, nearly normal vectors."""
    lo, hi = ((torch.randn(shape, generator=g, device=DEV, dtype=torch.float16) * 2.6).round().clamp(-8, 7).to(torch.int8) for _ in range(2))
    return ((lo & 15) | (hi << 4)).view(torch.uint8)


def _scales(g, shape, mean):
    """One scale a vector; a few tokens are several times louder than the others."""
    r = torch.rand(shape, generator=g, device=DEV)
    return (mean * (0.7 + 0.6 * r) * torch.where(r > 0.995, 4.0, 1.0)).to(torch.float16)


def prepare(case, seed):
    g, c = torch.Generator(device=DEV), torch.Generator()
    g.manual_seed(int(seed))
    c.manual_seed(int(seed))
    op, d, Hkv, t = case["op"], case["d"], case["Hkv"], TYPES[case["t"]]
    s = {"case": case}
    if op == "rope":
        s["positions"] = torch.randint(0, case["far"], (case["N"],), generator=g, device=DEV, dtype=torch.int32)
        s["inv_freq"] = _frequencies(case["rot"])
        # slices of one projection's output
        qkv = torch.randn((case["N"], case["Hq"] + 2 * Hkv, d), generator=g, device=DEV).to(t)
        s["q"], s["k"] = qkv[:, :case["Hq"]], qkv[:, case["Hq"]:case["Hq"] + Hkv]
        return s
    new, total = _lengths(case)
    B, ps, S = case["B"], case["ps"], case.get("S", 0)
    lengths = total + S
    # pages lie scattered; the shared ones stand in every sequence's table
    common = S // ps
    each = -(-(int(lengths.max()) - common * ps) // ps)
    P = common + B * each
    order = torch.randperm(P + 3, generator=c, dtype=torch.int32)[:P]
    table = torch.cat([order[:common].expand(B, common), order[common:].view(B, each)], 1)
    s["table"], s["lengths"] = table.contiguous().to(DEV), lengths.to(torch.int32).to(DEV)
    s["cu"] = None if case["Q"] == 1 else torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)]).to(torch.int32).to(DEV)
    s["n"] = N = int(new.sum())  # a scheduler knows it without asking the GPU
    if op == "append":
        shape = (P + 3, Hkv, ps)
        s["cache"] = [torch.zeros(shape + (d // 2,), dtype=torch.uint8, device=DEV), torch.zeros(shape, dtype=torch.float16, device=DEV),
                      torch.zeros(shape + (d // 2,), dtype=torch.uint8, device=DEV), torch.zeros(shape, dtype=torch.float16, device=DEV)]
        qkv = torch.randn((N, case["Hq"] + 2 * Hkv, d), generator=g, device=DEV)
        qkv[:, case["Hq"]:, torch.randint(0, d, (2,), generator=g, device=DEV)] *= 20.0  # the loud channels that the Hadamard rotation spreads
        s["q"], s["k"], s["v"] = qkv.to(t).split([case["Hq"], Hkv, Hkv], 1)
        s["inv_freq"] = _frequencies(case["rot"])
        return s
    shape = (P + 3, Hkv, ps)
    s["cache"] = [_codes(g, shape + (d // 2,)), _scales(g, shape, 0.35), _codes(g, shape + (d // 2,)), _scales(g, shape, 0.3)]
    if op == "attn":
        s["q"] = torch.randn((N, case["Hq"], d), generator=g, device=DEV).to(t)
    return s


# ---------------------------------------------------------------- plain forms (32 bits)
def _hadamard(x):
    """x times the Sylvester matrix over the root of its size: entry (i, j) is minus one to the number of ones that i and j share."""
    d = x.shape[-1]
    i = torch.arange(d, device=DEV)
    b = i[:, None] & i[None, :]
    b = b ^ (b >> 4)
    b = b ^ (b >> 2)
    b = (b ^ (b >> 1)) & 1
    return x @ ((1 - 2 * b).to(x.dtype) / math.sqrt(d))


def _rope(x, positions, inv_freq, pairs):
    """The first 2 len(inv_freq) elements of each head turned; angles in 64 bits."""
    rot = 2 * inv_freq.numel()
    a = positions.double()[:, None] * inv_freq[None, :]
    c, n = a.cos().to(x.dtype)[:, None, :], a.sin().to(x.dtype)[:, None, :]
    u, w = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, w = u * c - w * n, w * c + u * n
    y = torch.stack([u, w], -1).flatten(-2) if pairs else torch.cat([u, w], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _places(s):
    """(sequence, position) of every new token."""
    L, B = s["lengths"].long(), s["lengths"].numel()
    if s["cu"] is None:
        return torch.arange(B, device=DEV), L - 1
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), n)
    return seq, L[seq] - n[seq] + torch.arange(seq.numel(), device=DEV) - cu[seq]


def _values(codes, scale, dtype=torch.float32):
    """Values of packed codes [..., d / 2] and their scales [...]."""
    lo, hi = codes & 15, codes >> 4
    v = torch.stack([lo, hi], -1).flatten(-2).to(torch.int8)
    return torch.where(v > 7, v - 16, v).to(dtype) * scale.to(dtype)[..., None]


def _fetch(s, seq, pos, which):
    """Keys (0) or values (1) of tokens: [..., Hkv, d]; places past the table's end are the last page's."""
    ps = s["case"]["ps"]
    page = s["table"].long()[seq, (pos // ps).clamp(max=s["table"].shape[1] - 1)]
    codes, scale = s["cache"][2 * which], s["cache"][2 * which + 1]
    return _values(codes.transpose(1, 2)[page, pos % ps], scale.transpose(1, 2)[page, pos % ps])


def _store(s, x, page, slot, which):
    """The 4-bit quantizer with one scale a vector, into the pages; the values that were stored."""
    scale = (x.abs().amax(-1).clamp(min=1e-5) / 7.0).clamp(max=65504.0).to(torch.float16)
    q = torch.round(x / scale.float()[..., None]).clamp(-8, 7).to(torch.int8)
    s["cache"][2 * which].transpose(1, 2)[page, slot] = ((q[..., 0::2] & 15) | (q[..., 1::2] << 4)).view(torch.uint8)
    s["cache"][2 * which + 1].transpose(1, 2)[page, slot] = scale
    return (q.float() * scale.float()[..., None]).to(torch.float16)


def _attend(s):
    case = s["case"]
    q, S, Hkv, d = s["q"], case["S"], case["Hkv"], case["d"]
    N, Hq, _ = q.shape
    B, G = case["B"], Hq // Hkv
    seq, pos = _places(s)
    i = torch.zeros_like(seq) if s["cu"] is None else torch.arange(N, device=DEV) - s["cu"].long()[seq]
    Q = case["Q"]
    # queries in rows of their sequence: [B, Hkv, Q * G, d]
    rows = torch.zeros((B, Q, Hkv, G, d), device=DEV)
    rows[seq, i] = _hadamard(q.float()).view(N, Hkv, G, d) / math.sqrt(d)
    rows = rows.permute(0, 2, 1, 3, 4).reshape(B, Hkv, Q * G, d)
    last = torch.full((B, Q), -1, dtype=torch.int64, device=DEV)
    last[seq, i] = pos
    last = last[:, None, :, None, None].expand(B, 1, Q, G, 1).reshape(B, 1, Q * G, 1)
    t = torch.arange(S + case["L"], device=DEV)
    zero = torch.zeros((), dtype=torch.int64, device=DEV)
    k0, v0 = _fetch(s, zero, t[:S], 0), _fetch(s, zero, t[:S], 1)
    b = torch.arange(B, device=DEV)[:, None]
    k1, v1 = _fetch(s, b, t[None, S:], 0), _fetch(s, b, t[None, S:], 1)
    # the shared keys once for all rows: [Hkv, B * Q * G, S]
    shared = rows.transpose(0, 1).reshape(Hkv, B * Q * G, d) @ k0.permute(1, 2, 0)
    shared = shared.view(Hkv, B, Q * G, S).transpose(0, 1)
    each = rows @ k1.permute(0, 2, 3, 1)
    x = torch.cat([shared, each], -1)
    x = torch.where(t <= last, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p[..., :S].transpose(0, 1).reshape(Hkv, B * Q * G, S) @ v0.transpose(0, 1)).view(Hkv, B, Q * G, d).transpose(0, 1)
    o = (o + p[..., S:] @ v1.transpose(1, 2)) / torch.where(total == 0.0, 1.0, total)
    o = o.view(B, Hkv, Q, G, d).permute(0, 2, 1, 3, 4)[seq, i]
    return {"out": o.reshape(N, Hq, d).to(q.dtype)}


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "rope":
        return {n: _rope(s[n].float(), s["positions"], s["inv_freq"], case["pairs"]).to(s[n].dtype) for n in ("q", "k")}
    if op == "attn":
        return _attend(s)
    seq, pos = _places(s)
    if op == "read":
        back = _hadamard if case["back"] else lambda x: x
        return {n: back(_fetch(s, seq, pos, w)).to(TYPES[case["t"]]) for w, n in enumerate("kv")}
    page, slot = s["table"].long()[seq, pos // case["ps"]], pos % case["ps"]
    turn = lambda n: _rope(s[n].float(), pos, s["inv_freq"], case["pairs"])  # noqa: E731
    return {"q": turn("q").to(s["q"].dtype), "k": _store(s, _hadamard(turn("k")), page, slot, 0), "v": _store(s, _hadamard(s["v"].float()), page, slot, 1)}


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import w4a4_rotated_quantized_gb300 as qr

    case = s["case"]
    op = case["op"]
    if op == "rope":
        q, k = qr.quarot_rope(s["q"], s["k"], s["positions"], s["inv_freq"], interleaved=case["pairs"])
        return {"q": q, "k": k}
    where = (s["table"], s["lengths"], s["cu"])
    if op == "append":
        q = qr.quarot_paged_append(s["k"], s["v"], *s["cache"], *where, q=s["q"], inv_freq=s["inv_freq"], interleaved=case["pairs"])
        k, v = qr.quarot_paged_read(*s["cache"], *where, n=s["n"])
        return {"q": q, "k": k, "v": v}
    if op == "read":
        k, v = qr.quarot_paged_read(*s["cache"], *where, n=s["n"], unrotate=case["back"], out_dtype=TYPES[case["t"]])
        return {"k": k, "v": v}
    return {"out": qr.quarot_paged_attn(s["q"], *s["cache"], *where, max_q=case["Q"], shared_len=case["S"])}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- minimum work
def work(case):
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    if op == "rope":
        v = case["N"] * (case["Hq"] + Hkv)
        return {"bytes": 4 * v * d, "flops": 3 * v * case["rot"]}
    share = 0.5 if case["ragged"] else 1.0  # ragged numbers of tokens are half the largest on average
    B, Q, L = case["B"], case["Q"], case["L"]
    tokens = B * max(1.0, Q * (share if Q > 1 else 1.0))
    vec = d / 2 + 2
    steps = int(math.log2(d))
    if op == "append":
        return {"bytes": tokens * (4 * case["Hq"] * d + 2 * Hkv * (2 * d + vec + 2 * d)), "flops": tokens * (3 * (case["Hq"] + Hkv) * case["rot"] + 2 * Hkv * d * (steps + 4))}
    if op == "read":
        return {"bytes": tokens * 2 * Hkv * (vec + 2 * d), "flops": tokens * 2 * Hkv * d * (1 + (steps if case["back"] else 0))}
    cached = max(Q, L * share)
    seen = (cached - Q) + (Q + 1) / 2 + case["S"]
    return {"bytes": 2 * Hkv * vec * (case["S"] + B * cached) + 4 * tokens * case["Hq"] * d, "flops": 4 * tokens * case["Hq"] * seen * d}


# ---------------------------------------------------------------- the definition in 64 bits
def _sylvester(d):
    h = torch.ones((1, 1), dtype=torch.float64, device=DEV)
    while h.shape[0] < d:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(d)


def _turned(x, positions, inv_freq, pairs):
    x, half = x.double().clone(), inv_freq.numel()
    for j in range(half):
        u, w = (2 * j, 2 * j + 1) if pairs else (j, j + half)
        a = positions.double() * inv_freq[j]
        z = torch.complex(x[:, :, u], x[:, :, w]) * torch.polar(torch.ones_like(a), a)[:, None]
        x[:, :, u], x[:, :, w] = z.real, z.imag
    return x


def _numbers(codes, scale):
    n = codes.to(torch.int64)
    n = torch.stack([n % 16, n // 16], -1).reshape(*codes.shape[:-1], -1)
    return (n - 16 * (n >= 8)).double() * scale.double().unsqueeze(-1)


def _sequence(s, b, upto, which):
    """Tokens 0 .. upto - 1 of sequence b: [upto, Hkv, d]."""
    pages = s["table"][b, :-(-upto // s["case"]["ps"])].long()
    x = _numbers(s["cache"][2 * which][pages], s["cache"][2 * which + 1][pages])
    return x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])[:upto]


def _spans(s):
    lengths = s["lengths"].tolist()
    ends = list(range(1, len(lengths) + 1)) if s["cu"] is None else s["cu"].tolist()[1:]
    return [(b, lengths[b], (ends[b - 1] if b else 0), ends[b]) for b in range(len(lengths))]


def exact(case, seed):
    s = prepare(case, seed)
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    if op == "rope":
        return {n: _turned(s[n], s["positions"], s["inv_freq"], case["pairs"]) for n in ("q", "k")}
    spans, h = _spans(s), _sylvester(d)
    if op == "append":
        pos = torch.cat([torch.arange(n - (z - a), n, device=DEV) for _, n, a, z in spans])
        r = {"q": _turned(s["q"], pos, s["inv_freq"], case["pairs"])}
        for n, x in (("k", _turned(s["k"], pos, s["inv_freq"], case["pairs"])), ("v", s["v"].double())):
            x = x @ h
            scale = torch.clamp(x.abs().max(-1, keepdim=True).values, min=1e-5).div(7).clamp(max=65504).half().double()
            r[n] = torch.clamp(torch.round(x / scale), -8, 7) * scale
        return r
    if op == "read":
        r = [torch.cat([_sequence(s, b, n, w)[n - (z - a):] for b, n, a, z in spans]) for w in (0, 1)]
        return dict(zip("kv", (x @ h if case["back"] else x for x in r)))
    S, G = case["S"], case["Hq"] // Hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    first = [_sequence(s, 0, S, w) for w in (0, 1)] if S else None
    for b, n, a, z in spans:
        k, v = (_sequence(s, b, n, w) for w in (0, 1))
        if S:
            k, v = (torch.cat([f, x[S:]]) for f, x in zip(first, (k, v)))
        q = (s["q"][a:z].double() @ h).view(z - a, Hkv, G, d)
        hidden = torch.arange(n, device=DEV)[None, :] > torch.arange(n - (z - a), n, device=DEV)[:, None]
        for g in range(Hkv):
            x = torch.einsum("ihd,td->hit", q[:, g], k[:, g]) / math.sqrt(d)
            x = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
            out[a:z, g * G:(g + 1) * G] = torch.einsum("hit,td->ihd", x, v[:, g])
    return {"out": out}
