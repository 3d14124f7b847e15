"""The operators of a speculative decoding step next to the packed linear layers, as cases to be measured.

A step of a served model drafts a small tree of tokens per sequence and runs the model once over all of them.  Its
projections are the packed matvecs and the prefill GEMM; between and after them come the operators here:

  norm_rope   RMS norms of queries and keys for each head, the position rotation, and the write of keys and values
              into the pages of a cache, in one pass
  attention   attention of each sequence's drafted tree (one to 64 tokens) over its pages and over itself
  fork        pages of a cache: rows of the page table forked, grown and freed, partly filled pages copied
  commit      the accepted drafts of each sequence moved next to its prefix
  compact     live pages moved to the front of the pool
  logprobs    log probabilities of given tokens with the entropy and the top alternatives of their rows

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
F8_MAX = 448.0
# (query heads, key/value heads, head dim): 5120 wide with 40 heads of 128, and generic groupings of 1 to 8
HEADS = ((40, 8, 128), (32, 8, 128), (16, 2, 256), (64, 8, 64), (16, 16, 128), (20, 4, 256), (28, 4, 128))


def listed():
    return [
        # one token of one sequence: the latency of a plain decode step, once per layer
        dict(name="norm_rope 1 token", op="norm_rope", n=1, hq=40, hkv=8, d=128, rot=128, interleaved=False, page=16,
             f8=False, max_pos=4096),
        # a prompt of odd length written into an e4m3 cache, a quarter of each head rotated
        dict(name="norm_rope prompt e4m3", op="norm_rope", n=4099, hq=16, hkv=2, d=256, rot=64, interleaved=True,
             page=64, f8=True, max_pos=32768),
        # one token against an ordinary context: few rows, the work has to be split along the context
        dict(name="attention 1 token", op="attention", batch=1, tokens=1, ctx=4095, hq=40, hkv=8, d=128, page=16,
             f8=False, ragged=False),
        # a served batch with short drafts, ragged contexts (one of them empty) and an e4m3 cache, heads of 256
        dict(name="attention batch e4m3", op="attention", batch=32, tokens=4, ctx=8200, hq=16, hkv=2, d=256, page=64,
             f8=True, ragged=True),
        # a tree of 16 drafts over a long document: bound by the bytes of the cache
        dict(name="attention long", op="attention", batch=1, tokens=16, ctx=131072, hq=32, hkv=8, d=128, page=64,
             f8=False, ragged=False),
        # the widest trees: enough rows for the products to matter as much as the bytes
        dict(name="attention wide trees", op="attention", batch=4, tokens=64, ctx=16384, hq=40, hkv=8, d=128, page=32,
             f8=False, ragged=False),
        # beams or samples forked from a few sequences, with room for the next drafts
        dict(name="fork", op="fork", parents=5, pairs=40, width=24, layers=16, hkv=8, d=128, page=64, f8=False, room=17),
        # the accepted drafts of a batch, in all layers
        dict(name="commit", op="commit", batch=48, tokens=24, width=5, layers=32, hkv=8, d=128, page=16, f8=False),
        # a half empty pool made dense
        dict(name="compact", op="compact", pages=1021, live=0.5, rows=64, layers=8, hkv=8, d=128, page=32, f8=True),
        # one row sampled or verified: latency
        dict(name="logprobs 1 row", op="logprobs", n=1, vocab=50257, cands=1, top=5, bf16=True, temp=1.0),
        # the rows of one drafted tree in 32 bits
        dict(name="logprobs tree f32", op="logprobs", n=61, vocab=128256, cands=4, top=8, bf16=False, temp=0.7),
        # the drafts of a batch, or the tokens of a prompt to be scored
        dict(name="logprobs batch", op="logprobs", n=256, vocab=151936, cands=8, top=20, bf16=True, temp=1.0),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    op = rng.choice(("norm_rope", "attention", "attention", "fork", "commit", "compact", "logprobs", "logprobs"))
    hq, hkv, d = rng.choice(HEADS)
    page, f8 = rng.choice((16, 32, 64, 128)), rng.random() < 0.4
    if op == "norm_rope":
        rot = rng.choice([r for r in (32, 64, 128, 256) if r <= d])
        c = dict(op=op, n=_log_int(rng, 1, 4096), hq=hq, hkv=hkv, d=d, rot=rot, interleaved=rng.random() < 0.5,
                 page=page, f8=f8, max_pos=rng.randint(2000, 33000))
    elif op == "attention":
        while True:
            c = dict(op=op, batch=_log_int(rng, 1, 64), tokens=_log_int(rng, 1, 64), ctx=_log_int(rng, 1, 131072), hq=hq,
                     hkv=hkv, d=d, page=page, f8=f8, ragged=rng.random() < 0.7)
            w, top = work(c), [work(x) for x in listed() if x["op"] == op]
            # the padded form of a ragged batch has to fit too
            if w["bytes"] <= max(x["bytes"] for x in top) and w["flops"] <= max(x["flops"] for x in top) and \
                    c["batch"] * c["ctx"] * hkv * d <= 1 << 28 and c["batch"] * c["tokens"] * hq * c["ctx"] <= 1 << 29:
                break
    elif op == "fork":
        c = dict(op=op, parents=rng.randint(1, 6), pairs=_log_int(rng, 1, 40), width=rng.randint(2, 24),
                 layers=rng.randint(1, 16), hkv=hkv, d=d, page=min(page, 64), f8=f8, room=rng.randint(0, 40))
    elif op == "commit":
        t = _log_int(rng, 1, 64)
        c = dict(op=op, batch=_log_int(rng, 1, 48), tokens=t, width=rng.randint(5, 9) if page == 16 else 5,
                 layers=rng.randint(1, 32), hkv=hkv, d=d, page=page if page < 128 else 16, f8=f8)
    elif op == "compact":
        c = dict(op=op, pages=_log_int(rng, 40, 1000), live=rng.choice((0.1, 0.3, 0.5, 0.8)), rows=rng.randint(1, 64),
                 layers=rng.randint(1, 8), hkv=hkv, d=d, page=min(page, 32), f8=f8)
    else:
        c = dict(op=op, n=_log_int(rng, 1, 256), vocab=_log_int(rng, 1000, 151936), cands=rng.randint(1, 16),
                 top=rng.randint(1, 32), bf16=rng.random() < 0.6, temp=rng.choice((1.0, 0.7, 1.3)))
        if not c["bf16"]:
            c["n"] = min(c["n"], 128)
    # not a width of this framework's models
    return {k: v + 1 if type(v) is int and v == 3072 else v for k, v in c.items()}


# ---------------------------------------------------------------- the shapes that follow from a case

def _batch_shape(c):
    """Prefix lengths and drafted tokens of each sequence: plain numbers of the case, not of the seed."""
    rng = random.Random(c["ctx"] * 131 + c["batch"] * 7 + c["tokens"])
    lens, toks = [c["ctx"]] * c["batch"], [c["tokens"]] * c["batch"]
    if c["ragged"]:
        lens = [c["ctx"]] + [rng.randint(0, c["ctx"]) for _ in range(c["batch"] - 1)]
        toks = [c["tokens"]] + [rng.randint(1, c["tokens"]) for _ in range(c["batch"] - 1)]
        if c["batch"] >= 4:
            lens[1] = 0
    return lens, toks


def _fork_shape(c):
    """Lengths of the parents; the kinds of the pairs: fork, and where there is room for it one grown and one freed row."""
    rng = random.Random(c["pairs"] * 37 + c["width"])
    most = c["width"] * c["page"] - c["room"]
    lens = [max(1, rng.randint(max(1, most // 2), max(1, most))) for _ in range(c["parents"])]
    kinds = ["fork"] * c["pairs"]
    if c["pairs"] >= 8:
        kinds[3], kinds[5] = "grow", "free"
    return lens, kinds


def _accepted(c):
    rng = random.Random(c["batch"] * 31 + c["tokens"])
    return [rng.randint(0, min(c["tokens"], 9)) for _ in range(c["batch"])]


def _moves(c):
    """Pages of the pool that are live (by the case, not the seed), as truth values, and how many compacting moves."""
    rng = random.Random(c["pages"] * 17 + int(c["live"] * 10))
    live = [rng.random() < c["live"] for _ in range(c["pages"])]
    n = sum(live)
    return live, sum(live[n:])


def _page_bytes(c):
    return 2 * c["hkv"] * c["page"] * c["d"] * (1 if c["f8"] else 2)


def work(c):
    op = c["op"]
    if op == "norm_rope":
        n, heads, kv = c["n"], c["hq"] + c["hkv"], (1 if c["f8"] else 2)
        b = n * ((heads + c["hkv"]) * c["d"] * 2 + c["hq"] * c["d"] * 2 + 2 * c["hkv"] * c["d"] * kv + c["rot"] * 4 + 12)
        return {"bytes": b, "flops": 8 * n * heads * c["d"]}
    if op == "attention":
        lens, toks = _batch_shape(c)
        elem, n = (1 if c["f8"] else 2), sum(toks)
        b = sum((p + t) * 2 * c["hkv"] * c["d"] * elem + 4 * -(-(p + t) // c["page"]) for p, t in zip(lens, toks))
        b += n * c["hq"] * (c["d"] * 4 + 4) + 8 * n
        return {"bytes": b, "flops": sum(4 * t * c["hq"] * c["d"] * (p + (t + 1) / 2) for p, t in zip(lens, toks))}
    if op == "fork":
        lens, kinds = _fork_shape(c)
        tails = sum(k == "fork" and lens[i % c["parents"]] % c["page"] > 0 for i, k in enumerate(kinds))
        return {"bytes": 2 * tails * c["layers"] * _page_bytes(c) + 8 * c["pairs"] * c["width"], "flops": 0}
    if op == "commit":
        row = 2 * c["hkv"] * c["d"] * (1 if c["f8"] else 2) * c["layers"]
        return {"bytes": 2 * row * max(1, sum(max(0, a - 1) for a in _accepted(c))) + 8 * c["batch"] * c["tokens"], "flops": 0}
    if op == "compact":
        return {"bytes": 2 * _moves(c)[1] * c["layers"] * _page_bytes(c) + 8 * c["pages"], "flops": 0}
    b = c["n"] * (c["vocab"] * (2 if c["bf16"] else 4) + c["cands"] * 8 + c["top"] * 8 + 8)
    return {"bytes": b, "flops": 6 * c["n"] * c["vocab"]}


# ---------------------------------------------------------------- inputs

def _gen(seed, salt=0):
    return torch.Generator(device=DEV).manual_seed(seed * 1000003 + salt)


def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV) * std


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def _pool(g, layers, pages, c):
    """A cache pool [layers, pages, 2, heads, page, d] of normal keys and values, and for e4m3 the scales [layers, 2, heads]."""
    shape = (layers, pages, 2, c["hkv"], c["page"], c["d"])
    if not c["f8"]:
        return torch.randn(shape, generator=g, device=DEV, dtype=BF), None
    pool = torch.empty(shape, dtype=F8, device=DEV)
    for layer in range(layers):
        pool[layer] = (torch.randn(shape[1:], generator=g, device=DEV, dtype=BF) * 40).to(F8)
    return pool, torch.rand((layers, 2, c["hkv"]), generator=g, device=DEV) * 0.01 + 0.02


def _prepare_norm_rope(c, seed):
    g, n, hq, hkv, d = _gen(seed), c["n"], c["hq"], c["hkv"], c["d"]
    # q, k and v are slices of one projection's rows, as a fused projection leaves them
    qkv = _normal(g, (n, (hq + 2 * hkv) * d)).to(BF)
    pages = -(-n // c["page"]) + 3
    pool, scales = _pool(g, 2, pages, c)
    slots = torch.randperm(pages * c["page"], generator=g, device=DEV)[:n]
    half = torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64)
    angle = torch.arange(c["max_pos"], device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (-2 * half / c["rot"])
    return dict(q=qkv[:, :hq * d].unflatten(1, (hq, d)), k=qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
                v=qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)), pool=pool, scales=scales, slots=slots, layer=1,
                rope=torch.cat([angle.cos(), angle.sin()], 1).float(),
                positions=torch.randint(0, c["max_pos"], (n,), generator=g, device=DEV).int(),
                wq=(1 + _normal(g, (d,), 0.1)).to(BF), wk=(1 + _normal(g, (d,), 0.1)).to(BF),
                out=torch.empty((n, hq, d), dtype=BF, device=DEV))


def _tree_masks(toks, rng):
    """A random tree per sequence: each draft sees itself and its ancestors; bit j of a mask is draft j."""
    masks = []
    for t in toks:
        own_masks = []
        for i in range(t):
            parent = rng.randint(-1, i - 1)
            own_masks.append((own_masks[parent] if parent >= 0 else 0) | 1 << i)
        masks += own_masks
    return [m - (1 << 64) if m >> 63 else m for m in masks]


def _prepare_attention(c, seed):
    g, (lens, toks) = _gen(seed), _batch_shape(c)
    held = [-(-(p + t) // c["page"]) for p, t in zip(lens, toks)]
    pool, scales = _pool(g, 1, sum(held) + 2, c)
    order = torch.randperm(sum(held) + 2, generator=g, device=DEV).int()
    table = torch.full((c["batch"], max(held)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    n, start = sum(toks), [0]
    for t in toks:
        start.append(start[-1] + t)
    return dict(q=_normal(g, (n, c["hq"], c["d"]), 1.5).to(BF), pool=pool, scales=scales, layer=0, table=table,
                prefix=_ints(lens), q_start=_ints(start), max_tokens=c["tokens"],
                mask=_ints(_tree_masks(toks, random.Random(seed)), torch.int64), scale=c["d"] ** -0.5,
                out=torch.empty((n, c["hq"], c["d"]), dtype=BF, device=DEV), lse=torch.empty((n, c["hq"]), device=DEV))


def _prepare_fork(c, seed):
    g, (lens, kinds) = _gen(seed), _fork_shape(c)
    page, rows = c["page"], c["parents"] + c["pairs"]
    held = [-(-x // page) for x in lens]
    room = -(-(c["room"] + page) // page)
    pages = sum(held) + 2 * c["pairs"] * (room + 1) + 4
    pool, _ = _pool(g, c["layers"], pages, c)
    order = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.full((rows, c["width"]), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    refs[order[:at].long()] = 1
    child = list(range(c["parents"], rows))
    parent = [i % c["parents"] for i in range(c["pairs"])]
    for i, kind in enumerate(kinds):
        if kind == "grow":
            parent[i] = child[i] = 0
        elif kind == "free":
            parent[i] = -1
    return dict(pool=pool, table=table, lens=_ints(lens + [0] * c["pairs"]), refs=refs, parent=_ints(parent),
                child=_ints(child), room=c["room"], status=torch.empty(c["pairs"], dtype=torch.int32, device=DEV))


def _prepare_commit(c, seed):
    g, rng, acc = _gen(seed), random.Random(seed), _accepted(c)
    pages = c["batch"] * c["width"]
    pool, _ = _pool(g, c["layers"], pages, c)
    path = torch.full((c["batch"], c["tokens"]), -1, dtype=torch.int32)
    for b, a in enumerate(acc):
        path[b, :a] = torch.tensor(sorted(rng.sample(range(c["tokens"]), a)), dtype=torch.int32)
    room = c["width"] * c["page"] - c["tokens"]
    prefix = [rng.randint(0, max(0, min(room, 2 * c["page"]))) for _ in acc]
    return dict(pool=pool, table=torch.randperm(pages, generator=g, device=DEV).int().view(c["batch"], c["width"]),
                prefix=_ints(prefix), path=path.to(DEV), accepted=_ints(acc),
                lens=torch.empty(c["batch"], dtype=torch.int32, device=DEV))


def _prepare_compact(c, seed):
    g, (live, _) = _gen(seed), _moves(c)
    pool, _ = _pool(g, c["layers"], c["pages"], c)
    at = [i for i, x in enumerate(live) if x]
    order = torch.tensor(at, device=DEV)[torch.randperm(len(at), generator=g, device=DEV)] if at else torch.zeros(0, device=DEV)
    width = max(1, -(-len(at) // c["rows"]) + 2)
    table = torch.full((c["rows"], width), -1, dtype=torch.int32, device=DEV)
    per = max(1, -(-len(at) // c["rows"]))
    for r in range(c["rows"]):
        mine = order[r * per:(r + 1) * per].int()
        table[r, :mine.numel()] = mine
    refs = _ints([int(x) for x in live])
    # two more holders of every seventh live page, as shared prefixes have
    refs[order[::7].long()] += 2
    return dict(pool=pool, table=table, refs=refs, out_table=torch.empty_like(table), out_refs=torch.empty_like(refs))


def _prepare_logprobs(c, seed):
    g, n, v = _gen(seed), c["n"], c["vocab"]
    x = _normal(g, (n, v), 2.5)
    # a few likely tokens per row; the last columns are padding of the vocabulary and banned
    x.scatter_add_(1, torch.randint(0, v, (n, 12), generator=g, device=DEV), torch.rand((n, 12), generator=g, device=DEV) * 12)
    x[:, v - 7:] = -math.inf
    outs = tuple(torch.empty(shape, dtype=dtype, device=DEV) for shape, dtype in (
        ((n, c["cands"]), torch.float32), ((n,), torch.float32), ((n,), torch.float32), ((n, c["top"]), torch.int32),
        ((n, c["top"]), torch.float32)))
    return dict(logits=x.to(BF) if c["bf16"] else x, top=c["top"], temp=c["temp"], outs=outs,
                tokens=torch.randint(0, v - 7, (n, c["cands"]), generator=g, device=DEV).int())


_PREPARE = {"norm_rope": _prepare_norm_rope, "attention": _prepare_attention, "fork": _prepare_fork,
            "commit": _prepare_commit, "compact": _prepare_compact, "logprobs": _prepare_logprobs}


def prepare(case, seed):
    s = _PREPARE[case["op"]](case, seed)
    s["op"] = case["op"]
    s["interleaved"] = case.get("interleaved")
    if own:
        # what a serving program keeps between calls: the cache's and the step's descriptions, and workspaces
        from trellis_coded_weight_gb300 import binding as tb
        op = case["op"]
        if "pool" in s:
            s["cache"] = tb.PagedCache(s["pool"], s.get("scales"))
        if op == "norm_rope":
            s["norm"] = tb.NormRope(s["wq"], s["wk"], s["rope"], case["hq"], case["hkv"], interleaved=case["interleaved"])
        elif op == "attention":
            s["batch"] = tb.DraftBatch(s["table"], s["prefix"], s["q_start"], s["max_tokens"], s["mask"])
            s["workspace"] = tb.new_tree_workspace(s["cache"], s["batch"], case["hq"])
        elif op in ("fork", "compact"):
            s["workspace"] = tb.new_cache_workspace(s["cache"], s["table"], case.get("pairs", 0))
        elif op == "logprobs":
            s["workspace"] = tb.new_logprobs_workspace(case["n"], case["vocab"], case["top"], DEV)
    return s


# ---------------------------------------------------------------- the plain forms

def _rotated(x, cos, sin, interleaved):
    r = 2 * cos.shape[-1]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    p, q = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([p, q], -1).flatten(-2) if interleaved else torch.cat([p, q], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_norm_rope(s):
    rope = s["rope"][s["positions"].long()]
    cos, sin = rope[:, None, :rope.shape[1] // 2], rope[:, None, rope.shape[1] // 2:]
    q, k = s["q"].float(), s["k"].float()
    q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + 1e-6) * s["wq"].float()
    k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + 1e-6) * s["wk"].float()
    q, k = _rotated(q, cos, sin, s["interleaved"]), _rotated(k, cos, sin, s["interleaved"])
    pool, layer = s["pool"], s["layer"]
    kv = torch.stack([k, s["v"].float()], 1)
    if s["scales"] is not None:
        kv = (kv / s["scales"][layer][None, :, :, None]).clamp(-F8_MAX, F8_MAX)
    page, off = s["slots"] // pool.shape[4], s["slots"] % pool.shape[4]
    pool[layer][page, :, :, off] = kv.to(pool.dtype)
    return q.to(BF), pool


def _plain_attention(s):
    pool, table, prefix, start = s["pool"][s["layer"]], s["table"], s["prefix"].long(), s["q_start"].long()
    n, hq, d = s["q"].shape
    hkv, t = pool.shape[2], s["max_tokens"]
    kv = pool[table.clamp(min=0).long()].float()  # [B, W, 2, hkv, page, d]
    if s["scales"] is not None:
        kv = kv * s["scales"][s["layer"]][None, None, :, :, None, None]
    k, v = (kv[:, :, i].transpose(1, 2).flatten(2, 3) for i in (0, 1))  # [B, hkv, L, d]
    count = start[1:] - start[:-1]
    tok = torch.arange(t, device=DEV)
    row = (start[:-1, None] + tok).clamp(max=n - 1)  # [B, t]
    q = s["q"].float()[row].unflatten(2, (hkv, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, hkv, t*g, d]
    x = (q @ k.transpose(2, 3) * s["scale"]).unflatten(2, (t, hq // hkv))  # [B, hkv, t, g, L]
    pos = torch.arange(k.shape[2], device=DEV)
    j = pos[None] - prefix[:, None]
    drafts = ((s["mask"][row][:, :, None] >> j.clamp(0, 63)[:, None]) & 1).bool() & (j >= 0)[:, None] & (j < count[:, None])[:, None]
    seen = (j < 0)[:, None] | drafts  # [B, t, L]
    x = x.masked_fill(~seen[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    o = (e / z).flatten(2, 3) @ v  # [B, hkv, t*g, d]
    o = o.unflatten(2, (t, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    lse = (m + torch.log(z)).squeeze(-1).permute(0, 2, 1, 3).flatten(2, 3)
    used = tok < count[:, None]
    return o[used].to(BF), lse[used]


def _plain_fork(s):
    table, lens, refs, parent, child, pool = s["table"], s["lens"], s["refs"], s["parent"].long(), s["child"].long(), s["pool"]
    page, width, n = pool.shape[4], table.shape[1], refs.numel()
    at = torch.arange(width, device=DEV)
    keep, drop = parent == child, parent < 0
    src = parent.clamp(min=0)
    plen, prow, old = lens[src].long(), table[src], table[child]
    held = (old >= 0).cumprod(1).sum(1)
    full = torch.where(drop, 0, torch.where(keep, held, plen // page))
    need = torch.where(drop, 0, torch.maximum(full, (plen + s["room"] + page - 1) // page))
    fits = need <= width
    fresh = torch.where(fits, need - full, 0)
    upto = fresh.cumsum(0)
    spare = torch.argsort((refs != 0).int(), stable=True)
    ok = fits & ((fresh == 0) | (upto <= (refs == 0).sum()))
    new = torch.where(at < full[:, None], prow, -1)
    taken = (at >= full[:, None]) & (at < need[:, None]) & ok[:, None]
    new = torch.where(taken, spare[((upto - fresh)[:, None] + at - full[:, None]).clamp(0, n - 1)].int(), new)
    new = torch.where(ok[:, None], new, torch.where(keep[:, None], old, -1))
    gone = ~keep[:, None] & (at < held[:, None])
    shared = (~keep & ok & ~drop)[:, None] & (at < full[:, None])
    refs.index_add_(0, old[gone].long(), torch.full_like(old[gone], -1))
    refs.index_add_(0, torch.cat([prow[shared], new[taken]]).long(), torch.ones_like(torch.cat([prow[shared], new[taken]])))
    tail = ~keep & ok & ~drop & (plen % page > 0)
    where = full.clamp(max=width - 1)[:, None]
    pool[:, new.gather(1, where)[tail, 0].long()] = pool[:, prow.gather(1, where)[tail, 0].long()]
    table[child] = new
    lens[child] = torch.where(keep, lens[child].long(), torch.where(ok & ~drop, plen, 0)).int()
    return table, lens, refs, (~ok).int(), _as_ints(pool)


def _as_ints(pool):
    """The bits of a pool: what is moved has to arrive as it is."""
    return pool.view(torch.int8 if pool.dtype == F8 else torch.int16)


def _plain_commit(s):
    pool, table, prefix, path, acc = s["pool"], s["table"].long(), s["prefix"].long(), s["path"].long(), s["accepted"].long()
    page, i = pool.shape[4], torch.arange(path.shape[1], device=DEV)
    use = (i < acc[:, None]) & (path != i)
    src, dst = (prefix[:, None] + path).clamp(min=0), (prefix[:, None] + i).clamp(max=table.shape[1] * page - 1)
    row = torch.arange(path.shape[0], device=DEV)[:, None].expand_as(path)[use]
    src, dst = src[use], dst[use]
    bits = _as_ints(pool)
    bits[:, table[row, dst // page], :, :, dst % page] = bits[:, table[row, src // page], :, :, src % page]
    return _as_ints(pool), (prefix + acc).int()


def _plain_compact(s):
    pool, table, refs = s["pool"], s["table"], s["refs"]
    at = torch.arange(refs.numel(), device=DEV)
    live = refs > 0
    n = live.sum()
    high, holes = at[live & (at >= n)], at[~live & (at < n)]
    to = at.clone()
    to[high] = holes
    bits = _as_ints(pool)
    bits[:, holes] = bits[:, high]
    out = torch.zeros_like(refs)
    out[to[live]] = refs[live]
    return torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table), out, bits


def _plain_logprobs(s):
    x, tokens = s["logits"], s["tokens"].long()
    z = x.float() / s["temp"]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = m + torch.log(total)
    entropy = torch.log(total) - torch.where(e > 0, e * (z - m), 0.0).sum(1, keepdim=True) / total
    ids = x.sort(dim=1, descending=True, stable=True).indices[:, :s["top"]]
    return z.gather(1, tokens) - lse, lse[:, 0], entropy[:, 0], ids.int(), z.gather(1, ids) - lse


_PLAIN = {"norm_rope": _plain_norm_rope, "attention": _plain_attention, "fork": _plain_fork, "commit": _plain_commit,
          "compact": _plain_compact, "logprobs": _plain_logprobs}


def _own(s):
    from trellis_coded_weight_gb300 import binding as tb
    op = s["op"]
    if op == "norm_rope":
        q = tb.qk_norm_rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["norm"], s["cache"], s["layer"], s["out"])
        return q, s["pool"]
    if op == "attention":
        return tb.tree_attention(s["q"], s["cache"], s["layer"], s["batch"], s["workspace"], s["scale"], s["out"], s["lse"])
    if op == "fork":
        tb.cache_fork(s["cache"], s["table"], s["lens"], s["refs"], s["parent"], s["child"], s["status"], s["workspace"], s["room"])
        return s["table"], s["lens"], s["refs"], s["status"], _as_ints(s["pool"])
    if op == "commit":
        lens = tb.cache_commit(s["cache"], s["table"], s["prefix"], s["path"], s["accepted"], s["lens"])
        return _as_ints(s["pool"]), lens
    if op == "compact":
        table, refs = tb.cache_compact(s["cache"], s["table"], s["refs"], s["workspace"], s["out_table"], s["out_refs"])
        return table, refs, _as_ints(s["pool"])
    return tuple(tb.token_logprobs(s["logits"], s["tokens"], s["top"], s["workspace"], s["temp"], s["outs"]))


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_norm_rope(s, c):
    pos = s["positions"].long()
    table = s["rope"].double()
    half = c["rot"] // 2
    turn = torch.complex(table[pos, :half], table[pos, half:])[:, None]

    def one(x, w):
        x = x.double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * w.double()
        even, odd = (slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["interleaved"] else (slice(0, half), slice(half, c["rot"]))
        z = torch.complex(x[..., even].contiguous(), x[..., odd].contiguous()) * turn
        x[..., even], x[..., odd] = z.real, z.imag
        return x

    pool, layer = s["pool"].double(), s["layer"]
    for i, x in enumerate((one(s["k"], s["wk"]), s["v"].double())):
        if s["scales"] is not None:
            x = (x / s["scales"][layer, i].double()[:, None]).clamp(-F8_MAX, F8_MAX)
        pool[layer, s["slots"] // c["page"], i, :, s["slots"] % c["page"]] = x
    return one(s["q"], s["wq"]), pool


def _exact_attention(s, c):
    lens, toks = _batch_shape(c)
    pool, hkv, group = s["pool"][s["layer"]], c["hkv"], c["hq"] // c["hkv"]
    outs, lses, first = [], [], 0
    for b, (p, t) in enumerate(zip(lens, toks)):
        held = -(-(p + t) // c["page"])
        rows = pool[s["table"][b, :held].long()].double()
        bits = torch.tensor([[m >> j & 1 for j in range(t)] for m in s["mask"][first:first + t].tolist()], device=DEV, dtype=torch.bool)
        seen = torch.cat([torch.ones((t, p), dtype=torch.bool, device=DEV), bits], 1)
        o = torch.zeros((t, c["hq"], c["d"]), dtype=torch.float64, device=DEV)
        lse = torch.zeros((t, c["hq"]), dtype=torch.float64, device=DEV)
        for h in range(hkv):
            k, v = (rows[:, i, h].reshape(-1, c["d"])[:p + t] for i in (0, 1))
            if s["scales"] is not None:
                k, v = k * s["scales"][s["layer"], 0, h].double(), v * s["scales"][s["layer"], 1, h].double()
            for g in range(h * group, (h + 1) * group):
                x = (s["q"][first:first + t, g].double() @ k.T * s["scale"]).masked_fill(~seen, -math.inf)
                lse[:, g] = torch.logsumexp(x, 1)
                o[:, g] = torch.softmax(x, 1) @ v
        outs.append(o)
        lses.append(lse)
        first += t
    return torch.cat(outs), torch.cat(lses)


def _exact_logprobs(s, c):
    lp = torch.log_softmax(s["logits"].double() / c["temp"], 1)
    x = s["logits"].double() / c["temp"]
    p = lp.exp()
    return (lp.gather(1, s["tokens"].long()), torch.logsumexp(x, 1), -(p * lp.masked_fill(p == 0, 0.0)).sum(1), None,
            lp.topk(c["top"], 1).values)


def exact(case, seed):
    if case["op"] not in ("norm_rope", "attention", "logprobs"):
        return None  # whole numbers and moved bits
    s = _PREPARE[case["op"]](case, seed)
    return {"norm_rope": _exact_norm_rope, "attention": _exact_attention, "logprobs": _exact_logprobs}[case["op"]](s, case)
