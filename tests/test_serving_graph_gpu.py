"""The serving calls captured once in a CUDA graph and replayed over changed device data: lengths, tables, masks, tokens and
positions are read by each replay, workspaces are as the call before left them.  A replay has to give the bits that the same calls give
outside a graph, and those are compared with the 64-bit definitions elsewhere (attention also here)."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from test_tree_attention_gpu import Step
from trellis_coded_weight_gb300 import binding as tb

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from trellis_coded_weight_gb300 import build
    build.build()
    tb.load()


def captured(call):
    """A graph of `call`, which has run once before (function attributes are set by then)."""
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    return graph, out


@pytest.mark.parametrize("f8,d,hq,hkv,most", [(False, 128, 8, 2, 3), (True, 64, 8, 2, 3), (False, 128, 16, 2, 16),
                                              (True, 128, 16, 2, 16), (True, 256, 8, 2, 6)])
def test_attention_replayed_over_other_lengths(f8, d, hq, hkv, most):
    batch, width, page = 6, 80, 32
    pages = batch * width
    g = torch.Generator(device="cuda").manual_seed(d + most)
    pool = torch.randn((1, pages, 2, hkv, page, d), generator=g, device="cuda").to(ref.F8 if f8 else torch.bfloat16)
    scales = torch.rand((1, 2, hkv), generator=g, device="cuda") + 0.5 if f8 else None
    cache = tb.PagedCache(pool, scales)
    n = batch * most
    q, out = torch.zeros((n, hq, d), dtype=torch.bfloat16, device="cuda"), torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((n, hq), device="cuda")
    table, prefix = torch.zeros((batch, width), dtype=I32, device="cuda"), torch.zeros(batch, dtype=I32, device="cuda")
    q_start, mask = torch.zeros(batch + 1, dtype=I32, device="cuda"), torch.zeros(n, dtype=torch.int64, device="cuda")
    drafts = tb.DraftBatch(table, prefix, q_start, most, mask)
    ws = tb.new_tree_workspace(cache, drafts, hq)
    graph, _ = captured(lambda: tb.tree_attention(q, cache, 0, drafts, ws, out=out, lse=lse))
    rng = np.random.default_rng(most)
    for lens, toks in (([0] * batch, [most] * batch), ([2500, 0, 7, 300, 64, 1], [1, most, 0, 2, most, 1]),
                       ([31, 31, 32, 33, 2000, 0], [most] * batch), ([0] * batch, [0] * batch),
                       ([2400] * batch, [1] * batch)):
        s = Step(lens, toks, hq, hkv, d, page, f8, seed=3, garbage=False)  # its masks and queries; pages of this pool
        s.pool, s.scales = pool, scales
        s.table = rng.permutation(pages).reshape(batch, width)
        m = np.array(s.masks + [0] * (n - s.n), dtype=np.uint64).view(np.int64)
        table.copy_(torch.as_tensor(s.table))
        prefix.copy_(torch.as_tensor(lens))
        q_start.copy_(torch.as_tensor(s.q_start))
        mask.copy_(torch.as_tensor(m))
        q[:s.n].copy_(s.q)
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        got = out.clone(), lse.clone()
        assert (got[0][s.n:] == 7.0).all() and (got[1][s.n:] == 7.0).all()  # tokens of no sequence
        out.fill_(7.0)
        lse.fill_(7.0)
        tb.tree_attention(q, cache, 0, drafts, ws, out=out, lse=lse)
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)
        s.check(*got)
    assert tb.device_error() == 0


def test_a_step_replayed_token_by_token():
    """Room for a token, its norms and append, attention, the commit, and the alternatives, as one graph: sixty replays of two
    sequences, one of which grows over pages, against the same calls one by one on a cache of their own."""
    layers, pages, hq, hkv, d, page, rows, width, vocab = 2, 24, 8, 2, 128, 16, 2, 8, 5000
    g = torch.Generator(device="cuda").manual_seed(1)
    ones = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    angle = torch.arange(width * page, device="cuda")[:, None] / 10000.0 ** (torch.arange(0, d, 2, device="cuda") / d)
    norm = tb.NormRope(ones, ones, torch.cat([angle.cos(), angle.sin()], 1).float(), hq, hkv)
    qkv = torch.empty((rows, hq + 2 * hkv, d), dtype=torch.bfloat16, device="cuda")
    logits = torch.empty((rows, vocab), dtype=torch.bfloat16, device="cuda")
    tokens = torch.zeros((rows, 1), dtype=I32, device="cuda")

    class Side:
        def __init__(self):
            i32 = dict(dtype=I32, device="cuda")
            self.cache = tb.PagedCache.new(layers, pages, hkv, page, d, "cuda")
            self.table, self.refs = torch.full((rows, width), -1, **i32), torch.zeros(pages, **i32)
            self.lens = torch.tensor([0, 13], **i32)
            self.pair, self.status = torch.arange(rows, **i32), torch.full((rows,), 9, **i32)
            self.path, self.one = torch.zeros((rows, 1), **i32), torch.ones(rows, **i32)
            self.batch = tb.DraftBatch(self.table, self.lens, torch.arange(rows + 1, **i32), 1, n=rows)
            self.fork_ws = tb.new_cache_workspace(self.cache, self.table, rows)
            self.tree_ws = tb.new_tree_workspace(self.cache, self.batch, hq)
            self.top_ws = tb.new_logprobs_workspace(rows, vocab, 6, "cuda")

        def step(self):
            tb.cache_fork(self.cache, self.table, self.lens, self.refs, self.pair, self.pair, self.status, self.fork_ws, 1)
            at = self.lens.long()
            slots = self.table.gather(1, (at // page)[:, None])[:, 0].long() * page + at % page
            outs = []
            for layer in range(layers):
                q, k, v = qkv.split([hq, hkv, hkv], 1)
                q = tb.qk_norm_rope_append(q, k, v, self.lens, slots, norm, self.cache, layer)
                outs += tb.tree_attention(q, self.cache, layer, self.batch, self.tree_ws)
            tb.cache_commit(self.cache, self.table, self.lens, self.path, self.one, self.lens)
            return outs + list(tb.token_logprobs(logits, tokens, 6, self.top_ws))

        def state(self):
            return [self.table, self.lens, self.refs, self.status, self.cache.pool.view(torch.int16)]

    a, b = Side(), Side()
    start = [t.clone() for t in a.state()]
    graph, out = captured(a.step)
    for t, was in zip(a.state(), start):  # the run before the capture is taken back
        t.copy_(was)
    for _ in range(60):
        qkv.normal_(generator=g)
        logits.normal_(generator=g)
        graph.replay()
        want = b.step()
        assert all(torch.equal(x, y) for x, y in zip(out, want))
        assert all(torch.equal(x, y) for x, y in zip(a.state(), b.state()))
    assert a.lens.tolist() == [60, 73] and a.status.tolist() == [0, 0] and int((a.refs > 0).sum()) == 4 + 5


def test_forks_and_compactions_replayed():
    rng = np.random.default_rng(2)
    rows, width, page, pages, pairs = 9, 7, 16, 60, 5
    raw = torch.randint(0, 256, (2, pages, 2, 1, page, 128), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(torch.uint8)
    cache = tb.PagedCache(raw.view(torch.bfloat16))
    i32 = lambda a: torch.as_tensor(np.asarray(a), dtype=I32).cuda()  # noqa: E731
    table, lens, refs = np.full((rows, width), -1), np.zeros(rows, int), np.zeros(pages, int)
    table[0, :3], lens[0], refs[[50, 7, 31]] = [50, 7, 31], 45, 1
    t, le, r, parent, child, status = i32(table), i32(lens), i32(refs), i32([0] * pairs), i32(range(pairs)), i32([0] * pairs)
    keep = [x.clone() for x in (t, le, r, raw)]
    ws = tb.new_cache_workspace(cache, t, pairs)

    def call():
        tb.cache_fork(cache, t, le, r, parent, child, status, ws, 5)
        tb.cache_compact(cache, t, r, ws)

    graph, _ = captured(call)
    for x, was in zip((t, le, r, raw), keep):
        x.copy_(was)
    for _ in range(25):
        ch = rng.permutation(rows)[:pairs]
        pa = np.array([rng.choice([-1, c, rng.integers(0, rows)]) for c in ch])
        parent.copy_(torch.as_tensor(pa))
        child.copy_(torch.as_tensor(ch))
        want_raw = raw.clone()
        table, lens, refs, st, copies = ref.fork(table, lens, refs, pa, ch, page, 5)
        for src, dst in copies:
            want_raw[:, dst] = want_raw[:, src]
        table, refs, moves = ref.compact(table, refs)
        for src, dst in moves:
            want_raw[:, dst] = want_raw[:, src]
        graph.replay()
        for got, w in ((t, table), (le, lens), (r, refs), (status, st)):
            assert np.array_equal(got.cpu().numpy(), w)
        assert torch.equal(raw, want_raw)
