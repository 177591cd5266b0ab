"""The operators around a prefix that a whole batch shares, as cases to time.

A batch whose requests all start with the same long text (a system prompt, a
tool description) keeps that text's KV rows once, in device memory.  A decode
step attends over them for the whole batch at once (``attend``) and joins the
result with each request's attention over its own tokens (``join``); the weight
that each of the prefix's tokens receives is accumulated (``weigh``), and when
the prefix has to shrink, its lightest tokens leave it (``evict``).

A case is one call of one operator.  ``run`` computes it either in plain torch
operations (``own`` false) or with the library's calls (``own`` true).

Rows are 576 bf16 wide (a latent of 512, whose values are also what the
attention returns, and 64 rope dims); ``heads`` is what one rank holds.
"""
import math

import torch

own = False

DIM, V_DIM = 576, 512
SCALE = 1.0 / 24.0
CHUNK = 1 << 28  # scores that a plain form holds at once


# --------------------------------------------------------------------- cases
def listed():
    return [
        # attend: two requests of one layer that share a short instruction
        {"name": "attend 2 x 1000", "op": "attend", "B": 2, "L": 1, "heads": 128, "n": 1000, "stride": DIM},
        # attend: a rank with 16 of the heads, odd batch and length, rows that lie in a wider buffer
        {"name": "attend 7 x 3 x 5003, 16 heads", "op": "attend", "B": 7, "L": 3, "heads": 16, "n": 5003, "stride": 640},
        # attend: eight requests over one long document
        {"name": "attend 8 x 128K", "op": "attend", "B": 8, "L": 1, "heads": 128, "n": 131072, "stride": DIM},
        # attend: batch 192 over a prefix of 16K tokens, two layers at once
        {"name": "attend 192 x 2 x 16K", "op": "attend", "B": 192, "L": 2, "heads": 128, "n": 16384, "stride": DIM},
        # join: one layer of a small odd batch, the prefix and the own tokens, some requests without one of them
        {"name": "join 21 units", "op": "join", "units": 21, "heads": 128, "parts": 2, "empty": 0.2},
        # join: batch 192 x 8 layers
        {"name": "join 192 x 8", "op": "join", "units": 1536, "heads": 128, "parts": 2, "empty": 0.0},
        # weigh: four requests over a prefix of 4K tokens
        {"name": "weigh 4 x 4K", "op": "weigh", "B": 4, "L": 1, "heads": 128, "n": 4096, "stride": DIM},
        # weigh: odd sizes, 40 heads a rank
        {"name": "weigh 5 x 3 x 10007, 40 heads", "op": "weigh", "B": 5, "L": 3, "heads": 40, "n": 10007, "stride": 640},
        # weigh: batch 192 over a prefix of 16K tokens, two layers at once
        {"name": "weigh 192 x 2 x 16K", "op": "weigh", "B": 192, "L": 2, "heads": 128, "n": 16384, "stride": DIM},
        # evict: one layer of a short prefix cut to a quarter
        {"name": "evict 4K", "op": "evict", "L": 1, "n": 4096, "keep": 1024, "first": 4, "last": 64, "stride": DIM},
        # evict: odd sizes, eight layers of 16K tokens, a third stays
        {"name": "evict 8 x 16001", "op": "evict", "L": 8, "n": 16001, "keep": 5333, "first": 16, "last": 255, "stride": 640},
        # evict: two layers of a prefix of 1M tokens cut to a quarter
        {"name": "evict 2 x 1M", "op": "evict", "L": 2, "n": 1048576, "keep": 262144, "first": 64, "last": 1024, "stride": DIM},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "join", "weigh", "weigh", "evict"])
    stride = DIM + 8 * rng.choice([0, 0, 1, 8, 24])
    if op == "join":
        return {"op": op, "units": _log(rng, 1, 1536), "heads": rng.choice([16, 40, 128, 128]), "parts": rng.randint(2, 4),
                "empty": rng.choice([0.0, 0.2, 0.9])}
    if op == "evict":
        L, n = rng.randint(1, 8), _log(rng, 1, 1 << 20)
        while L * n > 2 << 20:
            L -= 1
        keep = max(1, int(n * rng.choice([0.02, 0.25, 0.5, 0.97])))
        first = rng.randint(0, min(64, keep))
        return {"op": op, "L": L, "n": n, "keep": keep, "first": first, "last": rng.randint(0, min(1024, keep - first)),
                "stride": stride}
    L, B, n = rng.randint(1, 4), _log(rng, 1, 192), _log(rng, 1, 1 << 18)
    heads = rng.choice([1, 8, 16, 37, 64, 128, 128, 128])
    while B * L * heads * n > 192 * 2 * 128 * 16384:
        if B > 1:
            B = (B + 1) // 2
        else:
            n = (n + 1) // 2
    return {"op": op, "B": B, "L": L, "heads": heads, "n": n, "stride": stride}


def work(case):
    if case["op"] == "join":
        rows = case["units"] * case["heads"]
        return {"bytes": rows * (case["parts"] + 1) * (2 * V_DIM + 4), "flops": rows * case["parts"] * 2 * V_DIM}
    if case["op"] == "evict":
        return {"bytes": case["L"] * (case["n"] * 4 + case["keep"] * (2 * (2 * DIM + 4) + 4)), "flops": case["L"] * case["n"]}
    rows = case["B"] * case["L"] * case["heads"]
    if case["op"] == "attend":
        return {"bytes": case["L"] * case["n"] * 2 * DIM + rows * (2 * DIM + 2 * V_DIM + 4),
                "flops": 2 * rows * case["n"] * (DIM + V_DIM)}
    return {"bytes": case["L"] * case["n"] * (2 * DIM + 8) + rows * (2 * DIM + 4), "flops": 2 * rows * case["n"] * DIM}


# -------------------------------------------------------------------- inputs
def _rows(shape, g):
    """bf16 KV rows: a normalised latent of 512 with a few louder channels, 64 rope values of a wider range; rows differ
    in size, and the first few draw attention."""
    width = shape[-1]
    gain = torch.exp2(2 * torch.rand(width, generator=g, device="cuda") - 1)
    gain[V_DIM:DIM] *= 2
    size = torch.exp2(2 * torch.rand(*shape[:-1], 1, generator=g, device="cuda") - 1.5)
    size[:, :4] *= 2
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return x.mul_(gain.to(torch.bfloat16)).mul_(size.to(torch.bfloat16))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "join":
        shape = (case["units"], case["heads"])
        s["outs"] = [torch.randn(*shape, V_DIM, generator=g, device="cuda").to(torch.bfloat16) for _ in range(case["parts"])]
        s["lses"] = [5 + 2 * torch.randn(shape, generator=g, device="cuda") for _ in range(case["parts"])]
        for o, e in zip(s["outs"], s["lses"]):  # what an attention without a key returns
            none = torch.rand(case["units"], generator=g, device="cuda") < case["empty"]
            o[none] = 0
            e[none] = -math.inf
    else:
        L, n = case["L"], case["n"]
        s["rows"] = _rows((L, n, case["stride"]), g)[..., :DIM]
        if op == "evict":
            # accumulated weights: most tokens light, a few heavy
            s["weights"] = torch.exp(3 * torch.randn((L, n), generator=g, device="cuda"))
        else:
            s["q"] = torch.randn((case["B"] * L, case["heads"], DIM), generator=g, device="cuda").to(torch.bfloat16)
        if op == "weigh":
            # the prefix's part of the softmax is about a half
            s["lse"] = _plain_scores(s, lambda x, rows, l: torch.logsumexp(x, -1)) + torch.rand((), generator=g, device="cuda") + 0.3
            s["before"] = torch.exp(2 * torch.randn((L, n), generator=g, device="cuda"))
    if own:
        from sparse_attention_kv_skv_gb300 import Config, Context, Prefix
        ctx = s["ctx"] = Context(Config(max_requests=1, num_layers=case.get("L", 1), max_context=1, topk=1, hot_slots=1,
                                        max_batch=case.get("B", 1)))
        if op == "join":
            s["out"], s["joined"] = torch.empty_like(s["outs"][0]), torch.empty_like(s["lses"][0])
        else:
            s["prefix"] = Prefix(s["rows"])
        if op == "evict":
            s["kept"] = torch.empty((L, case["keep"]), dtype=torch.int32, device="cuda")
            s["kept_rows"] = torch.empty((L, case["keep"], DIM), dtype=torch.bfloat16, device="cuda")
            s["kept_weights"] = torch.empty((L, case["keep"]), device="cuda")
            s["workspace"] = torch.empty(ctx.evict_prefix_workspace(s["prefix"]), dtype=torch.uint8, device="cuda")
        elif op == "attend":
            s["out"] = torch.empty((case["B"] * L, case["heads"], V_DIM), dtype=torch.bfloat16, device="cuda")
            s["lse"] = torch.empty((case["B"] * L, case["heads"]), device="cuda")
            s["workspace"] = torch.empty(ctx.attend_prefix_workspace(s["prefix"], case["B"], case["heads"]), dtype=torch.uint8,
                                         device="cuda")
        elif op == "weigh":
            s["after"] = torch.empty_like(s["before"])
            s["workspace"] = torch.empty(ctx.weigh_prefix_workspace(s["prefix"], case["B"], case["heads"]), dtype=torch.uint8,
                                         device="cuda")
    return s


# ---------------------------------------------------------------------- runs
def run(s):
    op = s["op"]
    if own:
        ctx = s["ctx"]
        if op == "attend":
            ctx.attend_prefix(s["prefix"], s["q"], s["out"], s["lse"], s["workspace"], sm_scale=SCALE)
            return {"out": s["out"], "lse": s["lse"]}
        if op == "join":
            ctx.join(s["outs"], s["lses"], s["out"], s["joined"])
            return {"out": s["out"], "lse": s["joined"]}
        if op == "weigh":
            ctx.weigh_prefix(s["prefix"], s["q"], s["lse"], s["before"], s["after"], s["workspace"], sm_scale=SCALE)
            return s["after"]
        ctx.evict_prefix(s["prefix"], s["weights"], s["kept"], s["kept_rows"], s["kept_weights"], s["workspace"],
                         first=s["first"], last=s["last"])
        return {"kept": s["kept"], "rows": s["kept_rows"], "weights": s["kept_weights"]}
    if op == "attend":
        return _plain_attend(s)
    if op == "join":
        return _plain_join(s)
    return _plain_weigh(s) if op == "weigh" else _plain_evict(s)


def _plain_scores(s, f):
    """f(scores [entries][heads][n] in 32 bits, the layer's rows, the layer) of some entries of a layer at a time, put
    together as [units][heads]..."""
    B, L, heads, n = s["B"], s["L"], s["heads"], s["n"]
    q = s["q"].view(B, L, heads, DIM)
    step = max(1, CHUNK // (heads * n))
    whole = []
    for l in range(L):
        rows = s["rows"][l].float()
        whole.append(torch.cat([f(torch.matmul(q[b:b + step, l].float(), rows.T) * SCALE, rows, l) for b in range(0, B, step)]))
    return torch.stack(whole, 1).flatten(0, 1)


def _plain_attend(s):
    def part(x, rows, l):
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x.sub_(top))
        total = p.sum(-1, keepdim=True)
        return torch.cat((torch.matmul(p, rows[:, :V_DIM]) / total, top + torch.log(total)), -1)

    both = _plain_scores(s, part)
    return {"out": both[..., :V_DIM].to(torch.bfloat16), "lse": both[..., V_DIM].contiguous()}


def _plain_join(s):
    lse = torch.stack(s["lses"])
    top = lse.amax(0)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    w = torch.exp(lse - top)
    total = w.sum(0)
    out = sum(wi[..., None] * o.float() for wi, o in zip(w, s["outs"])) / total.clamp(min=1e-30)[..., None]
    return {"out": out.to(torch.bfloat16), "lse": top + torch.log(total)}


def _plain_weigh(s):
    B, L, heads, n = s["B"], s["L"], s["heads"], s["n"]
    q, lse = s["q"].view(B, L, heads, DIM), s["lse"].view(B, L, heads)
    step = max(1, CHUNK // (heads * n))
    after = s["before"].clone()
    for l in range(L):
        rows = s["rows"][l].float()
        for b in range(0, B, step):
            x = torch.matmul(q[b:b + step, l].float(), rows.T) * SCALE
            after[l] += torch.exp(x.sub_(lse[b:b + step, l, :, None])).sum((0, 1))
    return after


def _plain_evict(s):
    n, keep = s["n"], s["keep"]
    j = torch.arange(n, device="cuda")
    score = s["weights"].masked_fill((j < s["first"]) | (j >= n - s["last"]), math.inf)
    kept = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :keep].sort(-1)[0]
    return {"kept": kept.to(torch.int32), "rows": s["rows"].gather(1, kept[..., None].expand(-1, -1, DIM)),
            "weights": s["weights"].gather(1, kept)}


# --------------------------------------------------------- the definitions
def exact(case, seed):
    """The outputs in 64 bits, from the definitions."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "join":
        return _exact_join(s)
    if case["op"] == "evict":
        return _exact_evict(s)
    B, L, heads, n = case["B"], case["L"], case["heads"], case["n"]
    weigh = case["op"] == "weigh"
    out = torch.empty((B * L, heads, V_DIM), dtype=torch.float64, device="cuda") if not weigh else None
    lse = torch.empty((B * L, heads), dtype=torch.float64, device="cuda")
    after = s["before"].double() if weigh else None
    for l in range(L):
        rows = s["rows"][l].double()
        for b in range(B):
            u = b * L + l
            x = torch.einsum("hd,nd->hn", s["q"][u].double(), rows) * SCALE
            if weigh:
                after[l] += torch.exp(x - s["lse"][u].double()[:, None]).sum(0)
            else:
                lse[u] = torch.logsumexp(x, -1)
                out[u] = torch.softmax(x, -1) @ rows[:, :V_DIM]
    return after if weigh else {"out": out, "lse": lse}


def _exact_join(s):
    lse = torch.stack([e.double() for e in s["lses"]], -1)
    both = torch.logsumexp(lse, -1)
    share = torch.where(lse == -math.inf, 0.0, torch.exp(lse - both[..., None]))
    return {"out": torch.einsum("uhp,puhd->uhd", share, torch.stack([o.double() for o in s["outs"]])), "lse": both}


def _exact_evict(s):
    n, keep, first, last = s["n"], s["keep"], s["first"], s["last"]
    kept = []
    for w in s["weights"].double():
        always = torch.zeros(n, dtype=torch.bool, device="cuda")
        always[:first] = True
        always[n - last:] = True
        more = keep - int(always.sum())
        taken = always
        if more > 0:
            free = torch.where(always, -math.inf, w)
            least = torch.topk(free, more)[0][-1]
            ties = free == least
            taken = always | (free > least) | (ties & (ties.cumsum(0) <= more - (free > least).sum()))
        kept.append(taken.nonzero()[:, 0])
    kept = torch.stack(kept)
    at = torch.arange(len(kept), device="cuda")[:, None]
    return {"kept": kept.to(torch.int32), "rows": s["rows"][at, kept].double(), "weights": s["weights"][at, kept].double()}
