"""Serving calls directly behind one another on a stream.  Their kernels may be scheduled while the one ahead still runs, and some
read through caches of an SM; each has to see all that the call ahead has written, in buffers whose earlier contents the same SMs
have read before.  Chains without any wait on the host, and as a graph, against the same calls with a wait after each: equal bits."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from trellis_coded_weight_gb300 import binding as tb

pytestmark = pytest.mark.gpu
I32 = torch.int32
ROUNDS = 24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from trellis_coded_weight_gb300 import build
    build.build()
    tb.load()


def same_with_and_without_waits(setup, step, outputs):
    """setup() makes a fresh state, step(state, i) issues round i's calls, outputs(state, i) names the buffers that round i filled."""
    slow = setup()
    for i in range(ROUNDS):
        step(slow, i)
    torch.cuda.synchronize()
    for s in ("calls", "graph"):
        if s == "calls":
            fast = setup()
            torch.cuda.synchronize()
            for _ in range(2):
                for i in range(ROUNDS):
                    step(fast, i)
        else:
            fast = setup()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                for i in range(ROUNDS):
                    step(fast, i)
            for _ in range(3):
                graph.replay()
        torch.cuda.synchronize()
        for i in range(ROUNDS):
            for a, b in zip(outputs(slow, i), outputs(fast, i)):
                assert torch.equal(a, b), (s, i)


class Waits:
    """A state whose calls are followed by a wait on the host, or not."""

    made = 0

    def __init__(self):
        self.wait = Waits.made % 3 == 0  # setup() is called for the slow run first, then for the two fast ones
        Waits.made += 1

    def done(self):
        if self.wait:
            torch.cuda.synchronize()


@pytest.mark.parametrize("n,heads,top", [(2, 200, 5), (9, 40, 0), (64, 120, 20), (700, 16, 3)])
def test_logits_written_by_the_call_ahead(n, heads, top):
    """token_logprobs of a buffer that qk_norm_rope_append has just overwritten, round after round."""
    d, g = 128, torch.Generator(device="cuda").manual_seed(n)
    qs = torch.randn((ROUNDS, n, heads, d), generator=g, device="cuda").bfloat16()
    k = torch.randn((n, 1, d), generator=g, device="cuda").bfloat16()
    ones = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    norm, cache = tb.NormRope(ones, ones, None, heads, 1), tb.PagedCache.new(1, 2, 1, 16, d, "cuda")
    pos, slots = torch.zeros(n, dtype=I32, device="cuda"), torch.full((n,), -1, device="cuda")
    tokens = torch.randint(0, heads * d, (n, 2), generator=g, device="cuda").int()
    f = dict(dtype=torch.float32, device="cuda")

    def setup():
        s = Waits()
        s.x = torch.zeros((n, heads, d), dtype=torch.bfloat16, device="cuda")
        s.out = [(torch.empty((n, 2), **f), torch.empty(n, **f), torch.empty(n, **f), torch.empty((n, top), dtype=I32, device="cuda"),
                  torch.empty((n, top), **f)) for _ in range(ROUNDS)]
        s.ws = tb.new_logprobs_workspace(n, heads * d, top, "cuda")
        return s

    def step(s, i):
        tb.qk_norm_rope_append(qs[i], k, k, pos, slots, norm, cache, 0, out=s.x)
        s.done()
        tb.token_logprobs(s.x.view(n, -1), tokens, top, s.ws, 1.0, s.out[i])
        s.done()

    Waits.made = 0
    same_with_and_without_waits(setup, step, lambda s, i: s.out[i])


SHAPES = [(4, 1, 8, 2, 128, False), (3, 4, 8, 2, 64, True), (4, 9, 16, 2, 128, False), (3, 12, 16, 2, 128, True),
          (3, 3, 8, 2, 256, True), (2, 40, 8, 2, 64, False), (2, 5, 8, 2, 256, False)]


@pytest.mark.parametrize("batch,toks,hq,hkv,d,f8", SHAPES)
def test_a_cache_and_queries_written_by_the_call_ahead(batch, toks, hq, hkv, d, f8):
    """tree_attention of queries, keys and values that qk_norm_rope_append has just written, to the same places every round."""
    page, width, n = 16, 6, batch * toks
    g = torch.Generator(device="cuda").manual_seed(d + toks)
    qkv = torch.randn((ROUNDS, n, hq + 2 * hkv, d), generator=g, device="cuda").bfloat16()
    pool = torch.randn((1, batch * width, 2, hkv, page, d), generator=g, device="cuda").to(ref.F8 if f8 else torch.bfloat16)
    ones = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    norm = tb.NormRope(ones, ones, None, hq, hkv)
    table = torch.randperm(batch * width, generator=g, device="cuda").int().view(batch, width)
    prefix = torch.arange(batch, device="cuda").int() * 11 + 3
    at = (prefix[:, None] + torch.arange(toks, device="cuda")).long()
    slots = (table.gather(1, at // page).long() * page + at % page).view(-1)
    pos = torch.zeros(n, dtype=I32, device="cuda")

    def setup():
        s = Waits()
        s.cache = tb.PagedCache(pool.clone())
        s.drafts = tb.DraftBatch(table, prefix, torch.arange(batch + 1, device="cuda").int() * toks, toks, n=n)
        s.ws = tb.new_tree_workspace(s.cache, s.drafts, hq)
        s.q = torch.zeros((n, hq, d), dtype=torch.bfloat16, device="cuda")
        s.out = [(torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda"), torch.empty((n, hq), device="cuda")) for _ in range(ROUNDS)]
        return s

    def step(s, i):
        q, k, v = qkv[i].split([hq, hkv, hkv], 1)
        tb.qk_norm_rope_append(q, k, v, pos, slots, norm, s.cache, 0, out=s.q)
        s.done()
        tb.tree_attention(s.q, s.cache, 0, s.drafts, s.ws, out=s.out[i][0], lse=s.out[i][1])
        s.done()

    Waits.made = 0
    same_with_and_without_waits(setup, step, lambda s, i: s.out[i])


@pytest.mark.parametrize("batch,toks,hq,hkv,d,f8", SHAPES)
def test_lengths_tables_and_pages_written_by_the_call_ahead(batch, toks, hq, hkv, d, f8):
    """tree_attention behind cache_commit (lengths in place), behind cache_fork (tables, copied pages) and behind cache_compact
    (renamed tables, moved pages)."""
    page, width, n, rows = 16, 8, batch * toks, 2 * batch
    pages = 3 * rows * width
    rng = np.random.default_rng(d + toks)
    g = torch.Generator(device="cuda").manual_seed(d + toks)
    raw = torch.randn((1, pages, 2, hkv, page, d), generator=g, device="cuda").to(ref.F8 if f8 else torch.bfloat16)
    q = torch.randn((n, hq, d), generator=g, device="cuda").bfloat16()
    i32 = lambda a: torch.as_tensor(np.asarray(a), dtype=I32).cuda()  # noqa: E731
    start_table = np.full((rows, width), -1)
    start_table[:, :2] = rng.permutation(pages)[:2 * rows].reshape(rows, 2)
    refs = np.zeros(pages, int)
    refs[start_table[:, :2]] = 1
    accepted = [i32(rng.integers(0, 2, batch)) for _ in range(ROUNDS)]
    path = i32(np.tile(np.arange(1, 3), (batch, 1)))[:, :1].contiguous()
    # the second half of the rows become copies of some of the first
    parent = [i32(rng.integers(0, batch, batch)) for _ in range(ROUNDS)]
    child = i32(range(batch, rows))

    def setup():
        s = Waits()
        s.cache = tb.PagedCache(raw.clone())
        s.table, s.lens, s.refs = i32(start_table), i32([17 + b % 5 for b in range(rows)]), i32(refs)
        s.status = torch.zeros(batch, dtype=I32, device="cuda")
        s.live = tb.DraftBatch(s.table[:batch], s.lens[:batch], torch.arange(batch + 1, device="cuda").int() * toks, toks, n=n)
        s.copies = tb.DraftBatch(s.table[batch:].view(batch, width), s.lens[batch:], torch.arange(batch + 1, device="cuda").int() * toks, toks, n=n) \
            if batch % 4 == 0 else None  # (its arrays begin on 16-byte boundaries)
        s.fork_ws, s.ws = tb.new_cache_workspace(s.cache, s.table, rows), tb.new_tree_workspace(s.cache, s.live, hq)
        s.self = i32(range(rows))
        s.grown = torch.zeros(rows, dtype=I32, device="cuda")
        s.start = [s.table.clone(), s.lens.clone(), s.refs.clone(), s.cache.pool.view(torch.uint8).clone()]
        new = lambda: (torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda"), torch.empty((n, hq), device="cuda"))  # noqa: E731
        s.out = [[new() for _ in range(4)] for _ in range(ROUNDS)]
        return s

    def step(s, i):
        if i == 0:  # every run of the chain begins alike
            for t, was in zip((s.table, s.lens, s.refs, s.cache.pool.view(torch.uint8)), s.start):
                t.copy_(was)
            tb.cache_fork(s.cache, s.table, s.lens, s.refs, s.self, s.self, s.grown, s.fork_ws, toks + ROUNDS)
            s.done()
        look = lambda k, b: tb.tree_attention(q, s.cache, 0, b, s.ws, out=s.out[i][k][0], lse=s.out[i][k][1])  # noqa: E731
        tb.cache_commit(s.cache, s.table[:batch], s.lens[:batch], path, accepted[i], s.lens[:batch])
        s.done()
        look(0, s.live)
        s.done()
        tb.cache_fork(s.cache, s.table, s.lens, s.refs, parent[i], child, s.status, s.fork_ws, toks)
        s.done()
        look(1, s.copies or s.live)
        s.done()
        tb.cache_compact(s.cache, s.table, s.refs, s.fork_ws)
        s.done()
        look(2, s.live)
        s.done()
        tb.cache_copy(s.cache, s.table[0, :1].clone(), i32_last)  # pages nobody holds
        look(3, s.copies or s.live)
        s.done()

    i32_last = i32([pages - 1])
    Waits.made = 0
    same_with_and_without_waits(setup, step, lambda s, i: [t for pair in s.out[i] for t in pair])
