"""Operators of a step that takes in the prompts of many requests, next to the packed linear layers, as cases to be measured.

A served model takes prompts in whole or in chunks, several requests at once, and requests may bring low-rank adapters of
their own for the shared, packed projections.  Such a step runs the prefill GEMM, then the adapters of its requests, and
attention over all tokens of the prompts:

  prompt     causal attention of packed sequences of new tokens (one to thousands each) over their cached prefixes and over
             themselves, with grouped heads, on the pages of the cache (bf16 or e4m3)
  adapters   what a projection's low-rank adapters add to its output, each request with its own adapter and rank, for whole
             prompts and for single tokens

``run`` computes them in elementary torch operations, or, with ``own`` set, with this repository's kernels.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
BF = torch.bfloat16
F8 = torch.float8_e4m3fn
# (query heads, key/value heads, head dim): 5120 wide with 40 heads of 128, and generic groupings of 1 to 8
HEADS = ((40, 8, 128), (32, 8, 128), (16, 2, 256), (64, 8, 64), (16, 16, 128), (20, 4, 256), (28, 4, 128), (12, 12, 64))
# (inputs, outputs) of a projection: the framework's MLP matrices, its attention's width, and smaller ones
SIZES = ((5120, 17408), (17408, 5120), (5120, 5120), (5120, 7168), (4096, 1024), (1024, 2048), (2048, 1000), (520, 264))


def listed():
    return [
        # a short prompt by itself: the latency of one layer's attention
        dict(name="prompt short", op="prompt", batch=1, tokens=100, ctx=0, hq=40, hkv=8, d=128, page=16, f8=False,
             ragged=False),
        # prompts of a served batch, packed, some with a cached prefix
        dict(name="prompt ragged batch", op="prompt", batch=16, tokens=2000, ctx=700, hq=40, hkv=8, d=128, page=16, f8=False,
             ragged=True),
        # one long document in a single pass: bound by the products
        dict(name="prompt long", op="prompt", batch=1, tokens=16384, ctx=0, hq=32, hkv=8, d=128, page=64, f8=False,
             ragged=False),
        # a chunk of a long prompt whose beginning is cached in e4m3, heads of 256: few rows against a long axis
        dict(name="prompt chunk e4m3", op="prompt", batch=1, tokens=512, ctx=60001, hq=16, hkv=2, d=256, page=64, f8=True,
             ragged=False),
        # prompts with small heads over an e4m3 cache: half the products per score
        dict(name="prompt small heads e4m3", op="prompt", batch=5, tokens=3001, ctx=128, hq=64, hkv=8, d=64, page=32, f8=True,
             ragged=True),
        # one token of one request: latency, paid once per projection and layer
        dict(name="adapters 1 token", op="adapters", batch=1, tokens=1, ids=1, rank=16, mixed=False, k=5120, n=5120,
             ragged=False),
        # the next tokens of a batch, most requests with an adapter of their own: bound by the adapters' bytes
        dict(name="adapters batch of tokens", op="adapters", batch=64, tokens=1, ids=40, rank=64, mixed=True, k=5120, n=17408,
             ragged=False),
        # a long prompt of one request: bound by the projection's input and output
        dict(name="adapters prompt", op="adapters", batch=1, tokens=4096, ids=1, rank=16, mixed=False, k=5120, n=17408,
             ragged=False),
        # packed prompts of odd lengths with adapters of many ranks, some requests without one
        dict(name="adapters ragged prompts", op="adapters", batch=9, tokens=1001, ids=6, rank=128, mixed=True, k=17408, n=5120,
             ragged=True),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    op = rng.choice(("prompt", "adapters"))
    top = [work(x) for x in listed() if x["op"] == op]
    most = {key: max(w[key] for w in top) for key in ("bytes", "flops")}
    while True:
        if op == "prompt":
            hq, hkv, d = rng.choice(HEADS)
            c = dict(op=op, batch=_log_int(rng, 1, 32), tokens=_log_int(rng, 1, 16384),
                     ctx=rng.choice((0, _log_int(rng, 1, 65536))), hq=hq, hkv=hkv, d=d, page=rng.choice((16, 32, 64, 128)),
                     f8=rng.random() < 0.4, ragged=rng.random() < 0.7)
        else:
            k, n = rng.choice(SIZES)
            c = dict(op=op, batch=_log_int(rng, 1, 200), tokens=_log_int(rng, 1, 4096), ids=_log_int(rng, 1, 64),
                     rank=rng.choice((8, 16, 32, 64, 128)), mixed=rng.random() < 0.5, k=k, n=n, ragged=rng.random() < 0.5)
        w = work(c)
        if all(w[key] <= most[key] for key in most):
            return c


# ---------------------------------------------------------------- the shapes that follow from a case

def _counts(c, rng):
    """New tokens of each sequence: plain numbers of the case, not of the seed."""
    if not c["ragged"]:
        return [c["tokens"]] * c["batch"]
    return [c["tokens"]] + [rng.randint(1, c["tokens"]) for _ in range(c["batch"] - 1)]


def _prompt_shape(c):
    """Cached positions and new tokens of each sequence."""
    rng = random.Random(c["ctx"] * 131 + c["batch"] * 7 + c["tokens"])
    toks = _counts(c, rng)
    lens = [c["ctx"]] * c["batch"]
    if c["ragged"]:
        lens = [c["ctx"]] + [rng.choice((0, rng.randint(0, c["ctx"]))) for _ in range(c["batch"] - 1)]
    return lens, toks


def _adapter_shape(c):
    """Tokens and adapter (-1: none) of each request, and the rank of each adapter."""
    rng = random.Random(c["batch"] * 57 + c["ids"] * 3 + c["rank"])
    toks = _counts(c, rng)
    # every adapter in use while there are requests for it, then any; of eight or more requests some have none
    which = [b if b < c["ids"] else rng.randrange(c["ids"]) for b in range(c["batch"])]
    if c["batch"] >= 8:
        which[5] = -1
    rng.shuffle(which)
    ranks = [rng.choice([r for r in (4, 8, 16, 32, 64, 128) if r <= c["rank"]]) if c["mixed"] else c["rank"]
             for _ in range(c["ids"])]
    return toks, which, ranks


def work(c):
    if c["op"] == "prompt":
        lens, toks = _prompt_shape(c)
        elem, n = (1 if c["f8"] else 2), sum(toks)
        b = sum((p + t) * 2 * c["hkv"] * c["d"] * elem + 4 * -(-(p + t) // c["page"]) for p, t in zip(lens, toks))
        b += n * c["hq"] * (c["d"] * 4 + 4)
        return {"bytes": b, "flops": sum(4 * t * c["hq"] * c["d"] * (p + (t + 1) / 2) for p, t in zip(lens, toks))}
    toks, which, ranks = _adapter_shape(c)
    used = {a for a in which if a >= 0}
    with_one = sum(t for t, a in zip(toks, which) if a >= 0)
    b = 2 * sum(ranks[a] for a in used) * (c["k"] + c["n"]) + 2 * with_one * c["k"] + 4 * sum(toks) * c["n"] + 8 * c["batch"]
    return {"bytes": b, "flops": sum(2 * t * ranks[a] * (c["k"] + c["n"]) for t, a in zip(toks, which) if a >= 0)}


# ---------------------------------------------------------------- inputs

def _gen(seed, salt=0):
    return torch.Generator(device=DEV).manual_seed(seed * 1000003 + salt)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def _starts(toks):
    start = [0]
    for t in toks:
        start.append(start[-1] + t)
    return start


def _prepare_prompt(c, seed):
    g, (lens, toks) = _gen(seed), _prompt_shape(c)
    held = [-(-(p + t) // c["page"]) for p, t in zip(lens, toks)]
    shape = (1, sum(held) + 2, 2, c["hkv"], c["page"], c["d"])
    pool, scales = torch.randn(shape, generator=g, device=DEV, dtype=BF), None
    if c["f8"]:
        pool = (pool * 40).to(F8)
        scales = torch.rand((1, 2, c["hkv"]), generator=g, device=DEV) * 0.01 + 0.02
    order = torch.randperm(sum(held) + 2, generator=g, device=DEV).int()
    table = torch.full((c["batch"], max(held)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    n, start = sum(toks), _starts(toks)
    return dict(q=(torch.randn((n, c["hq"], c["d"]), generator=g, device=DEV) * 1.5).to(BF), pool=pool, scales=scales,
                layer=0, table=table, prefix=_ints(lens), q_start=_ints(start), max_tokens=max(toks), lens=lens, toks=toks,
                scale=c["d"] ** -0.5, out=torch.empty((n, c["hq"], c["d"]), dtype=BF, device=DEV),
                lse=torch.empty((n, c["hq"]), device=DEV))


def _prepare_adapters(c, seed):
    g, (toks, which, ranks) = _gen(seed), _adapter_shape(c)
    n, start = sum(toks), _starts(toks)
    a = (torch.randn((c["ids"], c["rank"], c["k"]), generator=g, device=DEV) * c["k"] ** -0.5).to(BF)
    b = (torch.randn((c["ids"], c["n"], c["rank"]), generator=g, device=DEV) * 0.3).to(BF)
    return dict(x=torch.randn((n, c["k"]), generator=g, device=DEV).to(BF),
                y=torch.randn((n, c["n"]), generator=g, device=DEV).to(BF), a=a, b=b,
                scales=torch.rand(c["ids"], generator=g, device=DEV) + 0.5, ranks=_ints(ranks), adapter=_ints(which),
                q_start=_ints(start), start=start, which=which, rank_of=ranks, count=n,
                out=torch.empty((n, c["n"]), dtype=BF, device=DEV))


_PREPARE = {"prompt": _prepare_prompt, "adapters": _prepare_adapters}


def prepare(case, seed):
    s = _PREPARE[case["op"]](case, seed)
    s["op"] = case["op"]
    if own:
        # what a serving program keeps between calls: the cache's, the adapters' and the step's descriptions, and workspaces
        from trellis_coded_weight_gb300 import binding as tb
        if case["op"] == "prompt":
            s["cache"] = tb.PagedCache(s["pool"], s["scales"])
            s["batch"] = tb.DraftBatch(s["table"], s["prefix"], s["q_start"], s["max_tokens"], n=s["q"].shape[0])
            s["workspace"] = tb.new_prompt_workspace(s["cache"], s["batch"], case["hq"])
        else:
            s["adapters"] = tb.Adapters(s["a"], s["b"], s["ranks"], s["scales"])
            # tokens by adapter: made once for a step, used by each of its projections in all layers
            s["plan"] = tb.AdapterPlan(s["adapter"], s["q_start"], s["count"])
            tb.adapter_plan(s["plan"])
    return s


# ---------------------------------------------------------------- the plain forms

def _plain_prompt(s):
    pool, table = s["pool"][s["layer"]], s["table"]
    n, hq, d = s["q"].shape
    hkv, page = pool.shape[2], pool.shape[3]
    group, first = hq // hkv, 0
    outs, lses = [], []
    for b, (p, t) in enumerate(zip(s["lens"], s["toks"])):
        held = -(-(p + t) // page)
        kv = pool[table[b, :held].long()].float()  # [pages, 2, hkv, page, d]
        if s["scales"] is not None:
            kv = kv * s["scales"][s["layer"]][None, :, :, None, None]
        k, v = (kv[:, i].transpose(0, 1).flatten(1, 2) for i in (0, 1))  # [hkv, positions, d]
        step = max(16, (1 << 27) // (hq * (p + t)))  # tokens at a time, by the memory of their scores
        for at in range(0, t, step):
            c = min(step, t - at)
            upto = p + at + c
            q = s["q"][first + at:first + at + c].float().unflatten(1, (hkv, group)).permute(1, 0, 2, 3).flatten(1, 2)
            x = (q @ k[:, :upto].transpose(1, 2) * s["scale"]).unflatten(1, (c, group))  # [hkv, c, group, upto]
            pos = torch.arange(upto, device=DEV)
            x = x.masked_fill((pos[None] > p + at + torch.arange(c, device=DEV)[:, None])[None, :, None], -math.inf)
            m = x.amax(-1, keepdim=True)
            e = torch.exp(x - m)
            z = e.sum(-1, keepdim=True)
            o = (e.flatten(1, 2) @ v[:, :upto]).unflatten(1, (c, group)) / z
            outs.append(o.permute(1, 0, 2, 3).flatten(1, 2).to(BF))
            lses.append((m + torch.log(z)).squeeze(-1).permute(1, 0, 2).flatten(1, 2))
        first += t
    return torch.cat(outs), torch.cat(lses)


def _plain_adapters(s):
    out = s["y"].clone()
    for b, a in enumerate(s["which"]):
        if a < 0:
            continue
        rows, r = slice(s["start"][b], s["start"][b + 1]), s["rank_of"][a]
        h = s["x"][rows].float() @ s["a"][a, :r].float().T
        out[rows] = (s["y"][rows].float() + (h @ s["b"][a, :, :r].float().T) * s["scales"][a]).to(BF)
    return out


_PLAIN = {"prompt": _plain_prompt, "adapters": _plain_adapters}


def _own(s):
    from trellis_coded_weight_gb300 import binding as tb
    if s["op"] == "prompt":
        return tb.prompt_attention(s["q"], s["cache"], s["layer"], s["batch"], s["workspace"], s["scale"], s["out"], s["lse"])
    return tb.adapter_add(s["x"], s["y"], s["adapters"], s["plan"], s["out"])


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_prompt(s, c):
    lens, toks = _prompt_shape(c)
    group = c["hq"] // c["hkv"]
    n = sum(toks)
    out = torch.zeros((n, c["hq"], c["d"]), dtype=torch.float64, device=DEV)
    lse = torch.zeros((n, c["hq"]), dtype=torch.float64, device=DEV)
    first = 0
    for b, (p, t) in enumerate(zip(lens, toks)):
        positions = torch.arange(p + t, device=DEV)
        pages, offs = s["table"][b].long()[positions // c["page"]], positions % c["page"]
        for h in range(c["hkv"]):
            k, v = (s["pool"][0, pages, i, h, offs].double() for i in (0, 1))
            if s["scales"] is not None:
                k, v = k * s["scales"][0, 0, h].double(), v * s["scales"][0, 1, h].double()
            for lo in range(0, t, 1024):
                hi = min(t, lo + 1024)
                future = positions[None, :p + hi] > p + torch.arange(lo, hi, device=DEV)[:, None]
                for g in range(h * group, (h + 1) * group):
                    x = s["q"][first + lo:first + hi, g].double() @ k[:p + hi].T * s["scale"]
                    x[future] = -math.inf
                    norm = torch.logsumexp(x, 1)
                    lse[first + lo:first + hi, g] = norm
                    out[first + lo:first + hi, g] = torch.exp(x - norm[:, None]) @ v[:p + hi]
        first += t
    return out, lse


def _exact_adapters(s, c):
    toks, which, ranks = _adapter_shape(c)
    out = s["y"].double()
    for a in range(c["ids"]):
        mine = [i for b, w in enumerate(which) if w == a for i in range(sum(toks[:b]), sum(toks[:b + 1]))]
        if mine:
            rows = torch.tensor(mine, device=DEV)
            low = torch.einsum("tk,rk->tr", s["x"][rows].double(), s["a"][a, :ranks[a]].double())
            out[rows] += s["scales"][a].double() * torch.einsum("tr,nr->tn", low, s["b"][a, :, :ranks[a]].double())
    return out


def exact(case, seed):
    if case["op"] == "prompt" and work(case)["flops"] > 3e12:
        return None  # too long in 64 bits
    s = _PREPARE[case["op"]](case, seed)
    return _exact_prompt(s, case) if case["op"] == "prompt" else _exact_adapters(s, case)
