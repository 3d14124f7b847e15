"""Prompts of several requests, each with its own low-rank adapter, taken in whole and continued together, on a small model
with random weights.

    python examples/adapter_prompts.py

The packed projections are shared.  A step groups its tokens by adapter once (adapter_plan); per layer it runs the packed qkv
projection and adds the adapters' part (adapter_add), then qk_norm_rope_append, attention, and the packed MLP, whose down
projection has adapters too.  Attention is prompt_attention over the packed prompts, and tree_attention for the single tokens that
continue them."""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import speculative_decode as base  # noqa: E402
from speculative_decode import DIM, HIDDEN, INNER, KV_HEADS, LAYERS, PAGE, Q_HEADS, VOCAB, rms, tb  # noqa: E402

RANKS = [8, 16, 5]  # of the adapters
I32 = dict(dtype=torch.int32, device="cuda")


def make_adapters(g, k: int, n: int):
    a = torch.randn((len(RANKS), max(RANKS), k), generator=g, device="cuda") * k ** -0.5
    b = torch.randn((len(RANKS), n, max(RANKS)), generator=g, device="cuda") * 0.3
    return tb.Adapters(a.bfloat16(), b.bfloat16(), torch.tensor(RANKS, **I32), torch.tensor([1.0, 0.5, 2.0], device="cuda"))


class Model(base.Model):
    def __init__(self, dtype=torch.bfloat16):
        super().__init__(dtype)
        g = torch.Generator(device="cuda").manual_seed(11)
        self.adapters = [{"qkv": make_adapters(g, HIDDEN, (Q_HEADS + 2 * KV_HEADS) * DIM), "down": make_adapters(g, INNER, HIDDEN)}
                         for _ in range(LAYERS)]

    def __call__(self, tokens, positions, slots, batch, plan):
        """Log probabilities and alternatives of the tokens that follow the last of each sequence's tokens."""
        x, n = self.embed[tokens.long()], tokens.shape[0]
        if batch.max_tokens > 64:
            ws, attention = tb.new_prompt_workspace(self.cache, batch, Q_HEADS), tb.prompt_attention
        else:
            ws, attention = tb.new_tree_workspace(self.cache, batch, Q_HEADS), tb.tree_attention
        for i, (w, ad) in enumerate(zip(self.layers, self.adapters)):
            y = rms(x)
            qkv = tb.adapter_add(y, w["qkv"](y), ad["qkv"], plan).view(n, Q_HEADS + 2 * KV_HEADS, DIM)
            q, k, v = qkv.split([Q_HEADS, KV_HEADS, KV_HEADS], 1)
            q = tb.qk_norm_rope_append(q, k, v, positions, slots, self.norm, self.cache, i)
            a, _ = attention(q, self.cache, i, batch, ws, lse=False)
            x = x + rms(w["out"](a.view(n, -1)))
            y = rms(x)
            h = torch.nn.functional.silu(w["gate"](y)) * w["up"](y)
            x = x + rms(tb.adapter_add(h, w["down"](h), ad["down"], plan))
        last = batch.q_start[1:].long() - 1
        logits = self.head(rms(x[last]))
        return tb.token_logprobs(logits, torch.zeros((len(last), 1), **I32), 4, self.logprobs_ws)


def step(model, seqs, rows, new, which):
    """One step over tokens new[i] of row rows[i] with adapter which[i]; all of them are kept."""
    seqs.fork(rows, rows, max(len(t) for t in new))
    lens = seqs.lens.tolist()
    starts = [0]
    for t in new:
        starts.append(starts[-1] + len(t))
    at = torch.tensor([lens[r] + j for r, t in zip(rows, new) for j in range(len(t))], device="cuda")
    row = torch.tensor([r for r, t in zip(rows, new) for _ in t], device="cuda")
    slots = seqs.table[row, at // PAGE].long() * PAGE + at % PAGE
    pick = torch.tensor(rows, device="cuda")
    batch = tb.DraftBatch(seqs.table[pick].contiguous(), seqs.lens[pick].contiguous(), torch.tensor(starts, **I32),
                          max(len(t) for t in new), n=starts[-1])
    plan = tb.adapter_plan(tb.AdapterPlan(torch.tensor(which, **I32), batch.q_start, batch.n))
    got = model(torch.tensor([t for ts in new for t in ts], **I32), at.int(), slots, batch, plan)
    seqs.lens[pick] += torch.tensor([len(t) for t in new], **I32)
    return got


def generate(model, prompts, which, length, chunk=10 ** 6):
    """Continues the prompts together, each by its most likely tokens; `chunk`: most tokens of a prompt in one step."""
    seqs = base.Sequences(model.cache)
    rows = list(range(len(prompts)))
    first = [None] * len(prompts)  # what follows a prompt: the results of the step that took its last chunk
    for at in range(0, max(len(p) for p in prompts), chunk):
        here = [r for r in rows if at < len(prompts[r])]
        got = step(model, seqs, here, [prompts[r][at:at + chunk] for r in here], [which[r] for r in here])
        for i, r in enumerate(here):
            first[r] = (got.top_ids[i], got.top_logprobs[i])
    ids, lp = (torch.stack(t) for t in zip(*first))
    tokens, logprobs = [], []
    for _ in range(length):
        tokens.append(ids[:, 0].tolist())
        logprobs.append(lp)
        got = step(model, seqs, rows, [[t] for t in tokens[-1]], which)
        ids, lp = got.top_ids, got.top_logprobs
    return tokens, torch.stack(logprobs)


def run(dtype=torch.bfloat16, length=6):
    model = Model(dtype)
    g = torch.Generator().manual_seed(5)
    prompts = [torch.randint(0, VOCAB, (n,), generator=g).tolist() for n in (150, 67, 211)]
    which = [1, -1, 2]
    return dict(model=model, prompts=prompts, which=which, together=generate(model, prompts, which, length),
                alone=[generate(model, [p], [a], length) for p, a in zip(prompts, which)],
                chunks=[generate(model, [p], [a], length, chunk=64) for p, a in zip(prompts, which)],
                others=generate(model, prompts, [0, -1, -1], length))


if __name__ == "__main__":
    r = run()
    tokens, lp = r["together"]
    for i, w in enumerate(r["which"]):
        print(f"request {i} (adapter {w}):", [t[i] for t in tokens], "alone:", [t[0] for t in r["alone"][i][0]],
              "other adapter:", [t[i] for t in r["others"][0]])
