"""The operators around a cache that is held in 4 bits, as cases to time.

A decode step over such a cache picks its Top-k tokens by a cheap score over
index keys (``select``), assembles their 4-bit rows in the hot buffer, and
attends over them (``attend``); rows get into the cache by rounding bf16 rows
to 4 bits (``pack``) and are read back as bf16 (``unpack``).

A case is one call of one operator.  ``run`` computes it either in plain torch
operations (``own`` false) or with the library's calls (``own`` true).

Packed row of 576 values, 336 bytes: 288 bytes of e2m1 codes (value 2j in the
low half of byte j), 36 bytes of e4m3 scales (one for 16 values), one byte with
the row's exponent + 127, 11 bytes of zeros.
"""
import math

import torch

own = False

DIM, GROUP, GROUPS, V_DIM, HEADS = 576, 16, 36, 512, 128
ROW, CODES, EXP_AT = 336, 288, 324


# --------------------------------------------------------------------- cases
def listed():
    return [
        # pack: the rows that one decode step of a batch of 192 requests x 8 layers adds
        {"name": "pack step 1536 rows", "op": "pack", "n": 1536, "stride": DIM},
        # pack: one short prompt of odd length whose rows lie in a wider buffer
        {"name": "pack 4099 wide rows", "op": "pack", "n": 4099, "stride": 640},
        # pack: a prompt of 16K tokens x 8 layers
        {"name": "pack prompt 16K x 8", "op": "pack", "n": 131072, "stride": DIM},
        # unpack: one layer's Top-k rows of one request
        {"name": "unpack 2048 rows", "op": "unpack", "n": 2048},
        # unpack: a prompt's rows of 8 layers, read back
        {"name": "unpack prompt 16K x 8", "op": "unpack", "n": 131072},
        # attend: one request, one layer (one call of a layer-by-layer step with nothing batched)
        {"name": "attend one unit", "op": "attend", "B": 1, "L": 1, "T": 2560, "k": 2048, "pad": 0, "empty": False},
        # attend: a small batch, odd sizes, padded selections and one that selects nothing
        {"name": "attend 21 odd units", "op": "attend", "B": 7, "L": 3, "T": 1900, "k": 1337, "pad": 130, "empty": True},
        # attend: batch 192 x 8 layers, k = 2048
        {"name": "attend 192 x 8", "op": "attend", "B": 192, "L": 8, "T": 2560, "k": 2048, "pad": 0, "empty": False},
        # select: the smallest configuration: 4 requests, one layer, 4K tokens
        {"name": "select 4 x 4K", "op": "select", "B": 4, "L": 1, "ctx": 4096, "ragged": 0.5, "k": 256, "heads": 64,
         "dim": 128, "block": 1, "first": 0, "last": 0, "relu": True},
        # select: blocks of 64 tokens, one summary key each, the ends of the context always taken
        {"name": "select blocks 32 x 4 x 128K", "op": "select", "B": 32, "L": 4, "ctx": 131072, "ragged": 0.3, "k": 2048,
         "heads": 16, "dim": 64, "block": 64, "first": 1, "last": 4, "relu": False},
        # select: 4 requests x 4 layers of 1M tokens
        {"name": "select 4 x 4 x 1M", "op": "select", "B": 4, "L": 4, "ctx": 1048576, "ragged": 0.0, "k": 2048, "heads": 64,
         "dim": 128, "block": 1, "first": 0, "last": 0, "relu": True},
        # select: batch 192 x 8 layers of 16K tokens
        {"name": "select 192 x 8 x 16K", "op": "select", "B": 192, "L": 8, "ctx": 16384, "ragged": 0.1, "k": 2048,
         "heads": 64, "dim": 128, "block": 1, "first": 0, "last": 0, "relu": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["pack", "unpack", "attend", "attend", "select", "select"])
    if op == "pack":
        return {"op": op, "n": _log(rng, 1, 131072), "stride": DIM + 8 * rng.choice([0, 0, 1, 8, 24])}
    if op == "unpack":
        return {"op": op, "n": _log(rng, 1, 131072)}
    if op == "attend":
        L = rng.randint(1, 8)
        B = _log(rng, 1, 192)
        k = _log(rng, 16, 4096)
        while B * L * k > 1536 * 2048:
            B = (B + 1) // 2
        return {"op": op, "B": B, "L": L, "T": k + rng.randint(0, 600), "k": k, "pad": rng.choice([0, 1, k // 8, k // 2]),
                "empty": rng.random() < 0.3}
    block = rng.choice([1, 1, 2, 16, 64])
    ctx = _log(rng, 64, 1 << 20)
    L = rng.randint(1, 8)
    B = _log(rng, 1, 192)
    while B * L * ctx > 24 << 20:
        if B == 1:
            L = (L + 1) // 2
        B = (B + 1) // 2
    nb = rng.randint(4, max(4, min(2048, 4096 // block)))
    return {"op": op, "B": B, "L": L, "ctx": ctx, "ragged": rng.choice([0.0, 0.1, 0.5, 0.99]), "k": nb * block,
            "heads": rng.choice([1, 8, 16, 37, 64, 64]), "dim": rng.choice([64, 128]), "block": block,
            "first": rng.choice([0, 0, 1, 2]), "last": rng.choice([0, 0, 1, 2]), "relu": rng.random() < 0.7}


def _lens(case):
    """Tokens of each request: ctx, less up to `ragged` of it, spread over the batch."""
    return [max(1, case["ctx"] - int(case["ctx"] * case["ragged"] * ((b * 0.6180339887) % 1.0))) for b in range(case["B"])]


def work(case):
    if case["op"] == "pack":  # bf16 rows in; packed rows and the values they stand for out
        return {"bytes": case["n"] * (2 * DIM + ROW + 2 * DIM), "flops": case["n"] * DIM * 3}
    if case["op"] == "unpack":
        return {"bytes": case["n"] * (ROW + 2 * DIM), "flops": case["n"] * DIM}
    if case["op"] == "attend":
        units = case["B"] * case["L"]
        rows = (units - (1 if case["empty"] else 0)) * (case["k"] - case["pad"])
        return {"bytes": rows * ROW + units * (HEADS * (2 * DIM + 2 * V_DIM + 4) + case["k"] * 4),
                "flops": 2 * HEADS * (DIM + V_DIM) * rows}
    units = case["B"] * case["L"]
    keys = case["L"] * sum(-(-n // case["block"]) for n in _lens(case))
    return {"bytes": keys * case["dim"] * 2 + units * (case["heads"] * (case["dim"] * 2 + 4) + case["k"] * 4),
            "flops": 2 * keys * case["heads"] * case["dim"]}


# -------------------------------------------------------------------- inputs
def _rows(n, g, width=DIM):
    """bf16 KV rows: a normalised latent of 512 with a few louder channels, 64 rope values of a wider range; each row
    has a size of its own."""
    gain = torch.exp2(2 * torch.rand(width, generator=g, device="cuda") - 1)
    gain[512:DIM] *= 3
    size = torch.exp2(4 * torch.rand(n, 1, generator=g, device="cuda") - 2)
    return (torch.randn(n, width, generator=g, device="cuda") * gain * size).to(torch.bfloat16)


def _grid(shape, g):
    """Index values on the grid that an 8-bit index holds: multiples of 1/8 up to 4."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return x.mul_(8).round_().clamp_(-32, 32).mul_(0.125)


def _context(**kw):
    from sparse_attention_kv_skv_gb300 import Config, Context
    return Context(Config(**kw))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "pack":
        s["rows"] = _rows(case["n"], g, case["stride"])
        if own:
            s["ctx"] = _context(max_requests=1, num_layers=1, max_context=1, topk=1, hot_slots=1, max_batch=1, row_bytes=ROW)
            s["packed"] = torch.empty((case["n"], ROW), dtype=torch.uint8, device="cuda")
            s["values"] = torch.empty((case["n"], DIM), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "unpack":
        s["packed"] = _packed_rows(_rows(case["n"], g))
        if own:
            s["ctx"] = _context(max_requests=1, num_layers=1, max_context=1, topk=1, hot_slots=1, max_batch=1, row_bytes=ROW)
            s["values"] = torch.empty((case["n"], DIM), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "attend":
        B, L, T, k = case["B"], case["L"], case["T"], case["k"]
        s["rows"] = torch.stack([_packed_rows(_rows(L * T, g)).view(L, T, ROW) for _ in range(B)])
        # distinct tokens in no order, -1 in places of their own
        topk = torch.rand((B, L, T), generator=g, device="cuda").argsort(-1)[..., :k].to(torch.int32)
        if case["pad"]:
            at = torch.rand((B, L, k), generator=g, device="cuda").argsort(-1)[..., :case["pad"]]
            topk.scatter_(-1, at, -1)
        if case["empty"]:
            topk[0, 0] = -1
        s["topk"] = topk
        s["q"] = torch.randn((B * L, HEADS, DIM), generator=g, device="cuda").to(torch.bfloat16)
        s["scale"] = 1.0 / 24.0
        if own:
            ctx = s["ctx"] = _context(max_requests=B, num_layers=L, max_context=T, topk=k, hot_slots=k, max_batch=B, row_bytes=ROW)
            s["req"] = torch.tensor([ctx.publish(T, rows=s["rows"][b]) for b in range(B)], dtype=torch.int32, device="cuda")
            s["slots"] = torch.empty_like(topk)
            count = torch.empty((2, B, L), dtype=torch.int32, device="cuda")
            ctx.assemble(s["req"], topk, s["slots"], count[0], count[1])
            s["out"] = torch.empty((B * L, HEADS, V_DIM), dtype=torch.bfloat16, device="cuda")
            s["lse"] = torch.empty((B * L, HEADS), device="cuda")
    else:
        B, L, block = case["B"], case["L"], case["block"]
        n = -(-case["ctx"] // block)
        s["keys"] = _grid((B, L, n, case["dim"]), g)
        s["q"] = _grid((B, L, case["heads"], case["dim"]), g)
        s["w"] = torch.randint(-16, 65, (B, L, case["heads"]), generator=g, device="cuda").float() / 64
        s["len"] = torch.tensor(_lens(case), device="cuda")
        if own:
            from sparse_attention_kv_skv_gb300 import Index
            # a select reads a context's request table alone, so this one holds the shortest rows there are
            ctx = s["ctx"] = _context(max_requests=B, num_layers=L, max_context=case["ctx"], topk=case["k"], hot_slots=case["k"],
                                      max_batch=B, row_bytes=16)
            s["req"] = torch.tensor([ctx.publish(t) for t in _lens(case)], dtype=torch.int32, device="cuda")
            s["index"] = Index(s["keys"], block=block, first=case["first"], last=case["last"], relu=case["relu"])
            s["out"] = torch.empty((B, L, case["k"]), dtype=torch.int32, device="cuda")
            s["workspace"] = torch.empty(ctx.select_workspace(s["index"], B), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------- runs
def run(s):
    op = s["op"]
    if own:
        if op == "pack":
            s["ctx"].pack_rows(s["rows"][:, :DIM], s["packed"], s["values"])
            return s["values"]
        if op == "unpack":
            s["ctx"].unpack_rows(s["packed"], s["values"])
            return s["values"]
        if op == "attend":
            s["ctx"].attend_q4(s["req"], s["q"], s["slots"], s["out"], s["lse"], sm_scale=s["scale"])
            return {"out": s["out"], "lse": s["lse"]}
        s["ctx"].select(s["index"], s["req"], s["q"], s["w"], s["out"], s["workspace"])
        return s["out"]
    if op == "pack":
        return _round4(s["rows"][:, :DIM])[0].to(torch.bfloat16)
    if op == "unpack":
        return _values(s["packed"]).to(torch.bfloat16)
    return _plain_attend(s) if op == "attend" else _plain_select(s)


def _ldexp(x, e):
    """x * 2^e in two exact factors (a single one can pass the range of 32 bits)."""
    half = torch.div(e, 2, rounding_mode="floor")
    return x * torch.exp2(half.float()) * torch.exp2((e - half).float())


def _nearest(x, bits, low, most):
    """x >= 0 to the nearest value of `bits` fraction bits and exponent >= low (ties to even), at most `most`."""
    e = (torch.frexp(x)[1] - 1).clamp(min=low) - bits
    return _ldexp(torch.round(_ldexp(x, -e)), e).clamp(max=most)


def _round4(rows):
    """bf16 rows [n][576] -> the values their packed rows stand for (32 bits), the codes' sizes, the groups' scales and
    the rows' exponents."""
    x = rows.float().view(-1, GROUPS, GROUP)
    size = x.abs()
    bad = ~torch.isfinite(x).all(-1)
    top = size.amax(-1).masked_fill(bad, 0.0)
    m, e = torch.frexp(top.amax(-1))
    e = (e - 12 + (m > 0.65625).int()).clamp(-100, 116)  # the least e with 2688 * 2^e >= the row's largest size
    e = torch.where(m > 0, e, torch.full_like(e, -100))
    scale = _nearest(_ldexp(top, -e[:, None]) / 6, 3, -6, 448)
    codes = _nearest(_ldexp(size, -e[:, None, None]) / scale[..., None], 1, 0, 6).masked_fill((scale == 0)[..., None], 0.0)
    scale = scale.masked_fill(bad, math.nan)
    v = _ldexp(torch.copysign(codes, x) * scale[..., None], e[:, None, None].expand_as(x))
    return v.view(-1, DIM), codes, scale, e


def _packed_rows(rows):
    """The packed rows [n][336] of bf16 rows [n][576]."""
    out = torch.zeros((rows.shape[0], ROW), dtype=torch.uint8, device=rows.device)
    step = 1 << 19
    for a in range(0, rows.shape[0], step):
        part = rows[a:a + step]
        v, codes, scale, e = _round4(part)
        # 0 .5 1 1.5 2 3 4 6 -> 0..7
        code = torch.where(codes < 2, codes * 2, torch.where(codes < 4, codes + 2, codes / 2 + 4)).to(torch.uint8)
        code |= (torch.signbit(part.float()).view_as(code) & (scale != 0)[..., None]).to(torch.uint8) << 3
        code = code.view(-1, DIM // 2, 2)
        out[a:a + step, :CODES] = code[..., 0] | (code[..., 1] << 4)
        out[a:a + step, CODES:EXP_AT] = scale.to(torch.float8_e4m3fn).view(torch.uint8)
        out[a:a + step, EXP_AT] = (e + 127).to(torch.uint8)
    return out


def _values(packed):
    """Packed rows [..., 336] -> the values they stand for, in 32 bits."""
    b = packed[..., :CODES]
    code = torch.stack((b & 15, b >> 4), -1).flatten(-2)
    size, power = (code & 1).float(), (code >> 1) & 3
    size = torch.where(power == 0, size * 0.5, (1 + 0.5 * size) * torch.exp2(power.float() - 1))
    size = torch.where(code > 7, -size, size)
    sb = packed[..., CODES:EXP_AT]
    frac, power = (sb & 7).float(), ((sb >> 3) & 15).float()
    scale = torch.where(power == 0, frac * 2.0 ** -9, (8 + frac) * torch.exp2(power - 10)).masked_fill((sb & 127) == 127, math.nan)
    v = size.unflatten(-1, (GROUPS, GROUP)) * scale[..., None]
    return _ldexp(v, packed[..., EXP_AT, None, None].int() - 127).flatten(-2)


def _plain_attend(s):
    topk = s["topk"].flatten(0, 1).long()
    rows = s["rows"].flatten(0, 1)
    picked = rows.gather(1, topk.clamp(min=0)[..., None].expand(-1, -1, ROW))
    keys = _values(picked)
    x = torch.matmul(s["q"].float(), keys.transpose(1, 2)) * s["scale"]
    x = x.masked_fill((topk < 0)[:, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, keys[..., :V_DIM]) / total.clamp(min=1e-30)
    return {"out": out.to(torch.bfloat16), "lse": (top + torch.log(total))[..., 0]}


def _plain_select(s):
    block, k, n = s["block"], s["k"], s["keys"].shape[2]
    dots = torch.matmul(s["keys"].float(), s["q"].float().transpose(-1, -2))  # [B][L][n][heads]
    if s["relu"]:
        dots = dots.clamp_(min=0)
    score = torch.matmul(dots, s["w"][..., None])[..., 0]
    have = ((s["len"] + block - 1) // block)[:, None, None]  # index keys of each request
    j = torch.arange(n, device=score.device)
    score = score.masked_fill((j < s["first"]) | (j >= have - s["last"]), math.inf).masked_fill(j >= have, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :k // block]
    best = torch.where(best < have, best, n).sort(-1)[0]
    token = (best[..., None] * block + torch.arange(block, device=score.device)).flatten(-2)
    token = torch.where(token < s["len"][:, None, None], token, -1).to(torch.int32)
    return torch.nn.functional.pad(token, (0, k - token.shape[-1]), value=-1)


# --------------------------------------------------------- the definitions
def exact(case, seed):
    """The outputs in 64 bits, from the definitions."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "pack":
        return _exact_round(s["rows"][:, :DIM])
    if case["op"] == "unpack":
        return _exact_values(s["packed"])
    return _exact_attend(s) if case["op"] == "attend" else _exact_select(s)


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _e4m3():
    return [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (p - 10) for p in range(1, 16) for m in range(8)][:-1]


def _closest(x, grid):
    """The grid's value nearest to each x; of two as near, the one at the even place."""
    g = torch.tensor(grid, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(g, x).clamp(1, len(grid) - 1)
    lo = hi - 1
    a, b = x - g[lo], g[hi] - x
    return g[torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)]


def _exact_round(rows):
    x = rows.double().view(-1, GROUPS, GROUP)
    fine = torch.isfinite(x).all(-1)
    top = torch.where(fine, x.abs().amax(-1), 0.0)
    e = torch.ceil(torch.log2(top.amax(-1).clamp(min=2.0 ** -200) / 2688)).clamp(-100, 116)
    unit = torch.exp2(e)[:, None]
    scale = _closest(top / unit / 6, _e4m3()) * unit
    code = _closest(x.abs() / torch.where(scale > 0, scale, 1.0)[..., None], _E2M1) * (scale > 0)[..., None]
    return (torch.where(fine, scale, math.nan)[..., None] * code * torch.sign(x)).view(-1, DIM)


def _exact_values(packed):
    codes = torch.tensor(_E2M1 + [-v for v in _E2M1], dtype=torch.float64, device=packed.device)
    scales = torch.tensor((_e4m3() + [math.nan]) * 2, dtype=torch.float64, device=packed.device)
    p = packed.long()
    v = codes[torch.stack((p[..., :CODES] % 16, p[..., :CODES] // 16), -1)].flatten(-2)
    scale = scales[p[..., CODES:EXP_AT]].repeat_interleave(GROUP, -1)
    return v * scale * torch.exp2(p[..., EXP_AT:EXP_AT + 1].double() - 127)


def _exact_attend(s):
    B, L = s["topk"].shape[:2]
    out = torch.zeros((B * L, HEADS, V_DIM), dtype=torch.float64, device="cuda")
    lse = torch.full((B * L, HEADS), -math.inf, dtype=torch.float64, device="cuda")
    for u in range(B * L):
        token = s["topk"][u // L, u % L]
        token = token[token >= 0].long()
        if token.numel():
            keys = _exact_values(s["rows"][u // L, u % L][token])
            x = s["q"][u].double() @ keys.T * s["scale"]
            lse[u] = torch.logsumexp(x, -1)
            out[u] = torch.exp(x - lse[u][:, None]) @ keys[:, :V_DIM]
    return {"out": out, "lse": lse}


def _exact_select(s):
    B, L, n, _ = s["keys"].shape
    k, block = s["k"], s["block"]
    out = torch.full((B, L, k), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        tokens = int(s["len"][b])
        have = -(-tokens // block)
        for l in range(L):
            x = torch.einsum("hd,nd->hn", s["q"][b, l].double(), s["keys"][b, l, :have].double())
            score = torch.einsum("h,hn->n", s["w"][b, l].double(), torch.relu(x) if s["relu"] else x)
            score[:min(s["first"], have)] = math.inf
            score[max(0, have - s["last"]):] = math.inf
            if have > k // block:
                least = torch.topk(score, k // block)[0][-1]
                above, ties = score > least, score == least
                taken = above | (ties & (ties.cumsum(0) <= k // block - above.sum()))
                blocks = taken.nonzero()[:, 0]
            else:
                blocks = torch.arange(have, device="cuda")
            token = (blocks[:, None] * block + torch.arange(block, device="cuda")).flatten()
            token = token[token < tokens]
            out[b, l, :token.numel()] = token.to(torch.int32)
    return out
