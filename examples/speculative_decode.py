"""Speculative decoding with packed projections and the serving calls, on a small model with random weights.

    python examples/speculative_decode.py

A prompt is taken in chunks and continued twice: token by token, and by verifying trees of drafts.  A step of either kind runs,
per layer, the packed qkv projection, qk_norm_rope_append, tree_attention and the packed MLP, then token_logprobs on the
logits; cache_commit keeps the accepted drafts, cache_fork gives sequences their pages (and makes a second continuation that
shares them), cache_compact moves what is left to the front of the pool.  The drafts come from a stand-in for a draft model:
the plain continuation with every fourth token replaced, and a side branch."""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from trellis_coded_weight_gb300 import binding as tb  # noqa: E402
from trellis_coded_weight_gb300 import inputs  # noqa: E402

HIDDEN, INNER, VOCAB = 1024, 2048, 4096
Q_HEADS, KV_HEADS, DIM, LAYERS = 8, 2, 128, 2
PAGE, PAGES, ROWS, WIDTH = 16, 64, 3, 16  # pool and page table
MOST = 64                                 # tokens of a sequence in one step


class Packed:
    """A trellis-coded projection [outputs, inputs], k = 3, with random codes."""

    def __init__(self, outputs: int, inputs_: int, seed: int):
        codes, scales, _ = inputs.make_linear(outputs, inputs_, 3, 1, seed_codes=seed, seed_scales=seed + 1)
        self.g = tb.Geometry(3, 16, 256, 1, outputs, inputs_)
        self.codes = torch.from_numpy(codes.view(np.int32)).cuda()
        self.scales = torch.from_numpy(scales.view(np.int16)).view(torch.float16).cuda()

    def __call__(self, x):
        return tb.gemm_prefill(self.codes, self.scales, x.contiguous(), self.g)


def rms(x):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Model:
    def __init__(self, dtype=torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(7)
        self.embed = torch.randn((VOCAB, HIDDEN), generator=g, device="cuda").bfloat16()
        sizes = [("qkv", (Q_HEADS + 2 * KV_HEADS) * DIM, HIDDEN), ("out", HIDDEN, Q_HEADS * DIM), ("gate", INNER, HIDDEN),
                 ("up", INNER, HIDDEN), ("down", HIDDEN, INNER)]
        self.layers = [{name: Packed(r, c, 100 * i + 2 * j) for j, (name, r, c) in enumerate(sizes)} for i in range(LAYERS)]
        self.head = Packed(VOCAB, HIDDEN, 9000)
        angle = torch.arange(PAGE * WIDTH).double()[:, None] / 10000.0 ** (torch.arange(0, DIM, 2).double() / DIM)
        rope = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        ones = torch.ones(DIM, dtype=torch.bfloat16, device="cuda")
        self.norm = tb.NormRope(ones, ones, rope, Q_HEADS, KV_HEADS)
        self.cache = tb.PagedCache.new(LAYERS, PAGES, KV_HEADS, PAGE, DIM, "cuda", dtype)
        self.logprobs_ws = tb.new_logprobs_workspace(MOST * ROWS, VOCAB, 4, "cuda")
        self.tree_ws = None

    def __call__(self, tokens, positions, slots, batch):
        """Log probabilities and alternatives of the tokens that follow each of the batch's tokens."""
        if self.tree_ws is None:
            most = tb.DraftBatch(batch.table, batch.prefix, batch.q_start, MOST, n=batch.n)
            self.tree_ws = tb.new_tree_workspace(self.cache, most, Q_HEADS)
        x, n = self.embed[tokens.long()], tokens.shape[0]
        for i, w in enumerate(self.layers):
            qkv = w["qkv"](rms(x)).view(n, Q_HEADS + 2 * KV_HEADS, DIM)
            q, k, v = qkv.split([Q_HEADS, KV_HEADS, KV_HEADS], 1)
            q = tb.qk_norm_rope_append(q, k, v, positions, slots, self.norm, self.cache, i)
            a, _ = tb.tree_attention(q, self.cache, i, batch, self.tree_ws, lse=False)
            x = x + rms(w["out"](a.view(n, -1)))
            y = rms(x)
            x = x + rms(w["down"](torch.nn.functional.silu(w["gate"](y)) * w["up"](y)))
        logits = self.head(rms(x))
        return tb.token_logprobs(logits, torch.zeros((n, 1), dtype=torch.int32, device="cuda"), 4, self.logprobs_ws)


class Sequences:
    """The page table's rows, their lengths, and the pages' reference counts."""

    def __init__(self, cache):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.cache = cache
        self.table, self.lens = torch.full((ROWS, WIDTH), -1, **i32), torch.zeros(ROWS, **i32)
        self.refs = torch.zeros(PAGES, **i32)
        self.ws = tb.new_cache_workspace(cache, self.table, ROWS)

    def fork(self, parent, child, room=0):
        i32 = dict(dtype=torch.int32, device="cuda")
        status = torch.empty(len(parent), **i32)
        tb.cache_fork(self.cache, self.table, self.lens, self.refs, torch.tensor(parent, **i32), torch.tensor(child, **i32),
                      status, self.ws, room)
        if status.any():
            raise RuntimeError(f"no pages: {status.tolist()}")

    def batch(self, rows, trees):
        """The tokens of one step: trees[i] = (tokens, parents) of row rows[i], parents before their children (-1: the
        prefix).  Returns tokens, positions (by depth), slots (in the order of the drafts) and the DraftBatch."""
        lens = self.lens.tolist()
        tokens, positions, masks, places, seqs, starts = [], [], [], [], [], [0]
        for r, (toks, parents) in zip(rows, trees):
            depth, seen = [], []
            for j, parent in enumerate(parents):
                depth.append(0 if parent < 0 else depth[parent] + 1)
                seen.append((0 if parent < 0 else seen[parent]) | 1 << j)
            tokens += toks
            positions += [lens[r] + d for d in depth]
            places += [lens[r] + j for j in range(len(toks))]
            seqs += [r] * len(toks)
            masks += seen
            starts.append(len(tokens))
        i32 = dict(dtype=torch.int32, device="cuda")
        at, seq = torch.tensor(places, device="cuda"), torch.tensor(seqs, device="cuda")
        slots = self.table[seq, at // PAGE].long() * PAGE + at % PAGE
        mask = torch.from_numpy(np.array(masks, dtype=np.uint64).view(np.int64)).cuda()
        pick = torch.tensor(rows, device="cuda")
        batch = tb.DraftBatch(self.table[pick].contiguous(), self.lens[pick].contiguous(), torch.tensor(starts, **i32),
                              max(len(t) for t, _ in trees), mask)
        return torch.tensor(tokens, **i32), torch.tensor(positions, **i32), slots, batch

    def commit(self, rows, paths, batch):
        """Keeps the drafts `paths` of each row."""
        i32 = dict(dtype=torch.int32, device="cuda")
        path = torch.zeros((len(rows), max(len(p) for p in paths)), **i32)
        for i, p in enumerate(paths):
            path[i, :len(p)] = torch.tensor(p, **i32)
        kept = tb.cache_commit(self.cache, batch.table, batch.prefix, path, torch.tensor([len(p) for p in paths], **i32))
        self.lens[torch.tensor(rows, device="cuda")] = kept


def step(model, seqs, row, tokens, parents=None):
    """One step of one sequence; parents None: a chain, all of which is kept.  Returns (log probabilities, path)."""
    chain = parents is None
    parents = list(range(-1, len(tokens) - 1)) if chain else parents
    seqs.fork([row], [row], len(tokens))
    toks, positions, slots, batch = seqs.batch([row], [(tokens, parents)])
    got = model(toks, positions, slots, batch)
    path = list(range(len(tokens)))
    if not chain:  # greedy: from the root, the child that is the most likely next token
        best, path = got.top_ids[:, 0].tolist(), [0]
        while True:
            follow = [j for j, p in enumerate(parents) if p == path[-1] and tokens[j] == best[path[-1]]]
            if not follow:
                break
            path.append(follow[0])
    seqs.commit([row], [path], batch)
    return got, path


def drafts_after(known, at, rng):
    """A tree: the known next token, a chain of four guesses after it, and a side branch of two."""
    guess = [t if (at + 1 + i) % 4 else (t + 1) % VOCAB for i, t in enumerate(known[at + 1:at + 5])]
    tokens, parents = [known[at]], [-1]
    for t in guess:
        tokens.append(t)
        parents.append(len(tokens) - 2)
    for parent in (0, len(tokens)):
        tokens.append(int(rng.integers(VOCAB)))
        parents.append(parent)
    return tokens, parents


def run(dtype=torch.bfloat16, length=40):
    model = Model(dtype)
    seqs = Sequences(model.cache)
    rng = np.random.default_rng(3)
    prompt = rng.integers(0, VOCAB, 90).tolist()
    for row in (0, 1):
        for at in range(0, len(prompt), MOST):
            got, path = step(model, seqs, row, prompt[at:at + MOST])
    first = int(got.top_ids[path[-1], 0])

    plain, margins, token = [], [], first  # row 0: token by token
    for _ in range(length + 6):
        plain.append(token)
        got, _ = step(model, seqs, 0, [token])
        token = int(got.top_ids[0, 0])
        margins.append(float(got.top_logprobs[0, 0] - got.top_logprobs[0, 1]))

    spec, accepted = [], []                # row 1: trees of drafts
    while len(spec) < length:
        tokens, parents = drafts_after(plain[:len(spec)] + [first] + plain[len(spec) + 1:], len(spec), rng)
        got, path = step(model, seqs, 1, tokens, parents)
        spec += [tokens[j] for j in path]
        accepted.append(len(path))
        first = int(got.top_ids[path[-1], 0])

    seqs.fork([1], [2])                    # row 2: the same sequence, its full pages shared; row 0 gives up its pages
    seqs.fork([-1], [0])
    seqs.fork([1, 2], [1, 2], 2)
    before = model(*seqs.batch([1, 2], [([first, 5], [-1, 0])] * 2))
    tb.cache_compact(model.cache, seqs.table, seqs.refs, seqs.ws)
    after = model(*seqs.batch([1, 2], [([first, 5], [-1, 0])] * 2))
    return dict(plain=plain, spec=spec, margins=margins, accepted=accepted, before=before, after=after, seqs=seqs)


if __name__ == "__main__":
    r = run()
    same = sum(a == b for a, b in zip(r["plain"], r["spec"]))
    print(f"{len(r['spec'])} tokens in {len(r['accepted'])} steps ({np.mean(r['accepted']):.2f} a step), {same} of them as by single tokens")
    print("live pages at the front:", int((r["seqs"].refs > 0).sum()), "of", PAGES)
    print("log probabilities of the next tokens unchanged by compaction:",
          bool(torch.equal(r["before"].top_logprobs, r["after"].top_logprobs)))
