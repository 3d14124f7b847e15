"""trellis_prompt_attention against the 64-bit definition.

Tolerance, per output with w the softmax weights, A = sum w |v| and X = max over the keys of scale * sum |q k|:
  one rounding to bf16 (half a unit)              2^-8 |out|
  weights rounded to bf16                         2^-8 A
  scores summed in fp32 (up to 256 products in steps of 16, some kept to 2^-23 of the largest): 2^-18 X in the
  exponent, on weights and sum                     2 * 2^-18 X A
each with a tenth more.  lse: 2^-18 X + 1e-5 (the sum, and the approximate exponentials of 2^-22)."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from trellis_coded_weight_gb300 import binding as tb

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from trellis_coded_weight_gb300 import build
    build.build()
    tb.load()


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=I32).cuda()


class Prompts:
    """A cache with the pages of some sequences, and their new tokens' queries.  Rows past the ends, and pages nobody holds,
    hold NaN."""

    def __init__(self, lens, toks, hq, hkv, d, page, f8=False, seed=0, std=1.0, layers=1, layer=0, q_pad=0, out_pad=0, lead=0,
                 tail=0, scale=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.toks, self.layer, self.d, self.page, self.hq, self.hkv, self.f8 = lens, toks, layer, d, page, hq, hkv, f8
        held = [-(-(p + t) // page) for p, t in zip(lens, toks)]
        pages = sum(held) + 2
        pool = torch.randn((layers, pages, 2, hkv, page, d), generator=g, device="cuda")
        self.scales = None
        if f8:
            self.scales = torch.rand((layers, 2, hkv), generator=g, device="cuda") * 0.02 + 0.01
            pool = (pool / self.scales[:, None, :, :, None, None]).clamp(-448, 448)
        self.pool = pool.to(ref.F8 if f8 else torch.bfloat16)
        order = rng.permutation(pages)
        self.table = np.full((len(lens), max(max(held), 1)), -1)
        at = 0
        for b, h in enumerate(held):
            self.table[b, :h] = order[at:at + h]
            at += h
        nan = self.pool.view(torch.uint8)
        for p in order[at:]:
            nan[:, p] = 0x7F if f8 else 0xFF
        for b, (p, t) in enumerate(zip(lens, toks)):
            if (p + t) % page:
                nan[:, self.table[b, held[b] - 1], :, :, (p + t) % page:] = 0x7F if f8 else 0xFF
        self.q_start = lead + np.concatenate([[0], np.cumsum(toks)])
        self.n = lead + sum(toks) + tail
        wide = (torch.randn((max(1, self.n), hq * d + q_pad), generator=g, device="cuda") * std).bfloat16()[:self.n]
        self.q = wide[:, :hq * d].unflatten(1, (hq, d))
        self.out = torch.full((max(1, self.n), hq * d + out_pad), 7.5, dtype=torch.bfloat16,
                              device="cuda")[:self.n, :hq * d].unflatten(1, (hq, d))
        self.lse = torch.full((self.n, hq), 7.5, device="cuda")
        self.scale = d ** -0.5 if scale is None else scale

    def row(self, b, pos):
        """The cache's keys or values of position pos of sequence b: index them with [.., 0 or 1, head]."""
        return self.pool[self.layer, self.table[b, pos // self.page], :, :, pos % self.page]

    def run(self, ws=None, **kw):
        self.cache = tb.PagedCache(self.pool, self.scales)
        self.batch = tb.DraftBatch(i32(self.table), i32(self.lens), i32(self.q_start), max(1, max(self.toks)), None, self.n)
        self.ws = tb.new_prompt_workspace(self.cache, self.batch, self.hq) if ws is None else ws
        return tb.prompt_attention(self.q, self.cache, self.layer, self.batch, self.ws, self.scale,
                                   **{"out": self.out, "lse": self.lse, **kw})

    def keys_values(self, b):
        p, t = self.lens[b], self.toks[b]
        rows = self.pool[self.layer][torch.as_tensor(self.table[b, :-(-(p + t) // self.page)]).long().cuda()]
        rows = rows.float().double().permute(1, 2, 0, 3, 4).reshape(2, self.hkv, -1, self.d)[:, :, :p + t]
        if self.scales is not None:
            rows = rows * self.scales.double()[self.layer][:, :, None, None]
        return rows

    def check(self, out, lse, sequences=None, loud=False):
        """Every number of the given sequences (all finite, or `loud`: any numbers, a row at a time)."""
        group = self.hq // self.hkv
        for b in range(len(self.lens)) if sequences is None else sequences:
            first, t, p = int(self.q_start[b]), self.toks[b], self.lens[b]
            if t == 0:
                continue
            kv = self.keys_values(b)
            for h in range(self.hq):
                q, k, v = self.q[first:first + t, h].double(), kv[0, h // group], kv[1, h // group]
                got, got_l = out[first:first + t, h].double(), lse[first:first + t, h].double()
                if loud:
                    seen = np.arange(p + t)[None] <= p + np.arange(t)[:, None]
                    want, lw, mass, size = (torch.as_tensor(a).cuda() for a in ref.attention(ref.f64(q), ref.f64(k), ref.f64(v), seen, self.scale))
                else:
                    x = q @ k.T * self.scale
                    unseen = torch.arange(p + t, device="cuda")[None] > p + torch.arange(t, device="cuda")[:, None]
                    x[unseen] = -torch.inf
                    lw = torch.logsumexp(x, 1)
                    w = torch.exp(x - lw[:, None])
                    want, mass = w @ v, w @ v.abs()
                    size = (q.abs() @ k.abs().T).masked_fill(unseen, 0).amax(1) * abs(self.scale)
                fine = torch.isfinite(want)
                assert torch.equal(torch.isnan(got), torch.isnan(want)), (b, h)
                assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)])
                tol = 1.1 * (2.0 ** -8 * want.abs() + 2.0 ** -8 * mass + 2.0 ** -17 * size[:, None] * mass) + 1e-30
                off = ((got - want).abs() / tol)[fine]
                assert off.numel() == 0 or bool((off <= 1).all()), (b, h, float(off.max()), torch.nonzero(((got - want).abs() > tol) & fine)[:4].tolist())
                ok = torch.isfinite(lw)
                assert torch.equal(got_l[~ok & ~torch.isnan(lw)], lw[~ok & ~torch.isnan(lw)])
                assert bool(((got_l - lw).abs()[ok] <= 2.0 ** -18 * size[ok] + 1e-5).all()), (b, h, float((got_l - lw).abs()[ok].max()))


HEADS = [(8, 8, 64), (40, 8, 128), (16, 2, 256), (6, 2, 128), (16, 1, 64), (5, 1, 256), (64, 8, 64), (3, 3, 128)]


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_ragged_batch(hq, hkv, d, f8, page):
    p = Prompts([0, 200, 0, 37, 128, 5, 1], [1, 77, 300, 129, 128, 0, 31], hq, hkv, d, page, f8, seed=page + hq)
    out, lse = p.run()
    p.check(out, lse)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,toks", [([0], [1]), ([0], [2]), ([1], [1]), ([0], [63]), ([0], [64]), ([0], [65]), ([0], [127]), ([0], [128]),
                                       ([0], [129]), ([127], [1]), ([128], [1]), ([0], [255]), ([0], [256]), ([0], [257]), ([1000], [513]),
                                       ([4000], [3]), ([63] * 9, [1, 2, 3, 64, 65, 66, 127, 128, 129])])
def test_lengths_around_tiles(lens, toks, d, f8):
    for hq, hkv in ((4, 4), (8, 2), (7, 1)):
        p = Prompts(lens, toks, hq, hkv, d, 16, f8, seed=sum(toks) + d)
        out, lse = p.run()
        p.check(out, lse)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 128), (8, 2, 64), (4, 1, 256), (2, 2, 128)])
@pytest.mark.parametrize("lens,toks", [([0], [3001]), ([9001], [400]), ([20011, 0, 333], [70, 1500, 2]), ([0] * 40, [130] * 40)])
def test_long_and_many(hq, hkv, d, f8, lens, toks):
    p = Prompts(lens, toks, hq, hkv, d, 64, f8, seed=d)
    out, lse = p.run()
    p.check(out, lse)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_long_batch_of_one_head(d, f8):
    p = Prompts([0, 5000], [5003, 2000], 1, 1, d, 128, f8, seed=d + 1)
    out, lse = p.run()
    p.check(out, lse)


def test_batch_of_1024_sequences():
    rng = np.random.default_rng(5)
    lens, toks = rng.integers(0, 40, 1024).tolist(), rng.integers(0, 9, 1024).tolist()
    lens[700], toks[700] = 3000, 500
    p = Prompts(lens, toks, 4, 2, 64, 16, seed=2)
    out, lse = p.run()
    p.check(out, lse, sequences=[0, 1, 2, 255, 256, 257, 511, 512, 699, 700, 701, 1022, 1023])


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_strides_layers_and_rows_of_no_sequence(d, f8):
    p = Prompts([10, 300], [260, 33], 8, 2, d, 32, f8, seed=3, layers=3, layer=1, q_pad=24, out_pad=40, lead=5, tail=9)
    out, lse = p.run()
    p.check(out, lse)
    for a, z in ((0, 5), (p.n - 9, p.n)):
        assert bool((out[a:z] == 7.5).all()) and bool((lse[a:z] == 7.5).all())
    again, none = tb.prompt_attention(p.q, p.cache, p.layer, p.batch, p.ws, p.scale, lse=False)
    assert none is None and torch.equal(again[5:p.n - 9], out[5:p.n - 9])


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["nan", "inf"])
def test_values_that_are_not_finite_reach_who_sees_them(d, f8, kind):
    """A value that is no number (or infinite) at position 150 of the first sequence: tokens before it are as if it were not
    there, in the same tile of keys too."""
    if f8 and kind == "inf":
        pytest.skip("e4m3 has no infinities")
    p = Prompts([20, 0], [300, 260], 4, 2, d, 16, f8, seed=8)
    p.row(0, 150)[1, 1, 3] = float(kind)
    p.row(0, 150)[1, 0, d - 1] = float(kind)
    p.row(1, 259)[1, 1, 0] = float(kind)
    p.row(1, 100)[1, 0, 1] = float(kind)
    out, lse = p.run()
    p.check(out, lse, loud=True)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_keys_that_are_not_finite_reach_who_sees_them(d, f8):
    p = Prompts([20, 0], [300, 130], 4, 2, d, 16, f8, seed=9)
    p.row(0, 200)[0, 1, 3] = float("nan")
    out, lse = p.run()
    at = 200 - 20
    heads = slice(2, 4)
    assert bool(torch.isnan(out[at:300, heads]).all()) and bool(torch.isnan(lse[at:300, heads]).all())
    p.row(0, 200)[0, 1, 3] = 0.5
    want, want_l = out.clone(), lse.clone()
    p.run()
    assert torch.equal(out[:at], want[:at]) and torch.equal(out[300:], want[300:]) and torch.equal(lse[:at], want_l[:at])
    assert torch.equal(out[:300, :2], want[:300, :2])
    p.check(out, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_queries_that_are_not_finite_touch_no_other(d):
    p = Prompts([20, 0], [300, 130], 4, 2, d, 16, seed=10)
    out, lse = p.run()
    want, want_l = out.clone(), lse.clone()
    p.q[57, 1, 5] = float("nan")
    p.q[301, 3, 0] = float("inf")
    p.run()
    keep = torch.ones((p.n, 4), dtype=torch.bool, device="cuda")
    keep[57, 1] = keep[301, 3] = False
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_l[keep])


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 3.0])
def test_scales(d, f8, scale):
    p = Prompts([3, 0], [200, 257], 4, 2, d, 32, f8, seed=11, scale=scale, std=0.3)
    out, lse = p.run()
    p.check(out, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_growing_and_falling_scores(d):
    """Keys that grow, and keys that fall, along the sequence by far more than 2^8 in their weights."""
    for sign in (1, -1):
        p = Prompts([700], [300], 4, 2, d, 32, seed=12)
        ramp = torch.linspace(0, 6, 1000, device="cuda") if sign > 0 else torch.linspace(6, 0, 1000, device="cuda")
        for pos in range(1000):
            p.row(0, pos)[0, :, 0] = float(ramp[pos]) * 8
        p.q[:, :, 0] = 4.0
        out, lse = p.run()
        p.check(out, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_scores_of_minus_infinity(d):
    p = Prompts([0], [140], 2, 1, d, 16, seed=13)
    p.q[:, :, 0] = 1.0
    p.pool[..., 0, :, :, 0] = -float("inf")  # every key's first number
    out, lse = p.run()
    assert bool((out == 0).all()) and bool((lse == -torch.inf).all())
    p.row(0, 100)[0, 0, 0] = 0.25
    out, lse = p.run()
    assert bool((out[:100] == 0).all()) and bool((lse[:100] == -torch.inf).all())
    v = p.row(0, 100)[1, 0]
    assert bool((out[100:] == v).all())


def test_lengths_are_clamped():
    """A prefix past the table's width, more tokens than max_tokens, starts outside n, pages outside the pool."""
    p = Prompts([0, 30], [100, 50], 4, 2, 64, 16, seed=14)
    p.run()
    width = p.table.shape[1]
    batch = tb.DraftBatch(i32(p.table), i32([0, 10 ** 9]), i32([0, 100, 2 ** 30]), 100, None, p.n)
    out, lse = p.out.fill_(7.5), p.lse.fill_(7.5)
    tb.prompt_attention(p.q, p.cache, 0, batch, p.ws, p.scale, out=out, lse=lse)
    p.check(out, lse, sequences=[0])
    assert bool(torch.isfinite(lse[100:]).all() | torch.isnan(lse[100:]).any())
    q = Prompts([0], [width * 16], 4, 2, 64, 16, seed=15)
    q.run()
    short = tb.DraftBatch(i32(q.table), i32([0]), i32([0, q.n]), 40, None, q.n)
    out, lse = q.out.fill_(7.5), q.lse.fill_(7.5)
    tb.prompt_attention(q.q, q.cache, 0, short, q.ws, q.scale, out=out, lse=lse)
    assert bool((out[40:] == 7.5).all())
    q.toks = [40]
    q.check(out, lse)
    wild = q.table.copy()
    wild[0, 1], wild[0, 2] = 10 ** 9, -5
    tb.prompt_attention(q.q, q.cache, 0, tb.DraftBatch(i32(wild), i32([0]), i32([0, q.n]), q.n, None, q.n), q.ws, q.scale, out=out)
    torch.cuda.synchronize()
    assert tb.device_error() == 0


@pytest.mark.parametrize("f8,d", [(False, 128), (True, 128), (False, 256), (True, 64)])
def test_equal_calls_give_equal_bits_and_tokens_do_not_touch_others(f8, d):
    p = Prompts([500, 0, 9000], [300, 1200, 64], 8, 2, d, 64, f8, seed=16)
    out, lse = p.run()
    first, first_l = out.clone(), lse.clone()
    for _ in range(3):
        out.fill_(1), lse.fill_(1)
        p.run(p.ws)
    assert torch.equal(out, first) and torch.equal(lse, first_l)


@pytest.mark.parametrize("f8,d", [(False, 128), (True, 128), (False, 256), (True, 64)])
def test_captured_and_replayed_over_other_lengths(f8, d):
    hq, hkv, page, batch, width, n = 8, 2, 32, 4, 70, 2600
    g = torch.Generator(device="cuda").manual_seed(d)
    pool = torch.randn((1, batch * width, 2, hkv, page, d), generator=g, device="cuda").to(ref.F8 if f8 else torch.bfloat16)
    cache = tb.PagedCache(pool)
    q = torch.randn((n, hq, d), generator=g, device="cuda").bfloat16()
    table = torch.randperm(batch * width, generator=g, device="cuda").int().view(batch, width)
    prefix, starts = torch.zeros(batch, dtype=I32, device="cuda"), torch.zeros(batch + 1, dtype=I32, device="cuda")
    drafts = tb.DraftBatch(table, prefix, starts, 2000, None, n)
    ws = tb.new_prompt_workspace(cache, drafts, hq)
    out, lse = torch.zeros_like(q), torch.zeros((n, hq), device="cuda")
    call = lambda o=out, m=lse, w=ws: tb.prompt_attention(q, cache, 0, drafts, w, out=o, lse=m)  # noqa: E731
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens, toks in (([0] * 4, [500, 1, 0, 2000]), ([2100, 0, 7, 300], [100, 100, 100, 100]), ([0] * 4, [0] * 4), ([0, 0, 0, 2200], [0, 0, 0, 40])):
        prefix.copy_(i32(lens))
        starts.copy_(i32(np.concatenate([[0], np.cumsum(toks)])))
        out.zero_(), lse.zero_()
        graph.replay()
        want, want_l = torch.zeros_like(out), torch.zeros_like(lse)
        call(want, want_l, tb.new_prompt_workspace(cache, drafts, hq))
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_l)
        p = Prompts.__new__(Prompts)
        p.__dict__.update(lens=lens, toks=toks, layer=0, d=d, page=page, hq=hq, hkv=hkv, pool=pool, scales=None, table=table.cpu().numpy(),
                          q_start=starts.cpu().numpy(), q=q, scale=d ** -0.5)
        p.check(out, lse, sequences=[b for b in range(4) if toks[b] <= 500])


@pytest.mark.parametrize("f8,d", [(False, 64), (True, 128), (False, 256)])
def test_agrees_with_the_tree_attention_of_chains(f8, d):
    """Up to 64 tokens of a sequence the tree attention of a chain is the same operator."""
    p = Prompts([100, 0, 3000, 17], [64, 3, 20, 1], 8, 2, d, 16, f8, seed=17)
    out, lse = p.run()
    other, other_l = tb.tree_attention(p.q, p.cache, 0, p.batch, tb.new_tree_workspace(p.cache, p.batch, 8), p.scale)
    p.check(out, lse)
    p.check(other, other_l)


def test_another_stream_and_two_calls_at_once():
    a, b = Prompts([5, 0], [700, 300], 8, 2, 128, 64, seed=18), Prompts([0, 3000], [400, 65], 8, 8, 64, 16, True, seed=19)
    a.run(), b.run()
    want = [x.clone() for x in (a.out, a.lse, b.out, b.lse)]
    for x in (a.out, a.lse, b.out, b.lse):
        x.fill_(1)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s):
            a.run(a.ws)
        with torch.cuda.stream(t):
            b.run(b.ws)
    torch.cuda.synchronize()
    for x, y in zip((a.out, a.lse, b.out, b.lse), want):
        assert torch.equal(x, y)


def test_a_pool_past_32_bits():
    """Pages whose offsets pass 2^32 bytes and 2^31 numbers."""
    d, hkv, page, pages = 128, 8, 128, 9000
    pool = torch.zeros((1, pages, 2, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    assert pool.numel() > 2 ** 31
    p = Prompts([130], [300], 16, hkv, d, page, seed=20)
    held = p.table.shape[1]
    for i in range(held):
        pool[0, pages - 1 - 3 * i] = p.pool[0, p.table[0, i]]
    p.table = np.array([[pages - 1 - 3 * i for i in range(held)]])
    p.pool = pool
    out, lse = p.run()
    p.check(out, lse)


def test_refusals_of_the_binding():
    p = Prompts([0], [70], 4, 2, 64, 16)
    p.run()
    ok = dict(q=p.q, cache=p.cache, layer=0, batch=p.batch, workspace=p.ws, scale=1.0)
    masked = tb.DraftBatch(p.batch.table, p.batch.prefix, p.batch.q_start, 70, torch.zeros(70, dtype=torch.int64, device="cuda"))
    for bad in (dict(q=p.q.float()), dict(q=p.q[:50]), dict(q=p.q.cpu()), dict(q=p.q.transpose(0, 1)), dict(out=p.out[:50]), dict(lse=p.lse.double()),
                dict(batch=masked), dict(workspace=p.ws.cpu())):
        with pytest.raises(ValueError):
            tb.prompt_attention(**{**ok, **bad})
    for bad in (dict(layer=1), dict(layer=-1), dict(scale=float("nan")), dict(workspace=p.ws[:64])):
        with pytest.raises(tb.TrellisError):
            tb.prompt_attention(**{**ok, **bad})
    with pytest.raises(tb.TrellisError):  # three heads over two
        tb.prompt_attention(p.q[:, :3].contiguous(), p.cache, 0, p.batch, p.ws)


@pytest.mark.parametrize("f8,d", [(False, 128), (True, 128), (False, 256), (True, 256), (False, 64), (True, 64)])
def test_bounded_waits_run_out_and_the_next_call_is_right(f8, d):
    p = Prompts([30000, 0], [300, 700], 16, 8, d, 64, f8, seed=21)
    want = [t.clone() for t in p.run()]
    assert tb.device_error(reset=True) == 0
    tb.set_wait_limit(200)
    try:
        p.run(p.ws)
        torch.cuda.synchronize()
        assert tb.device_error(reset=True) != 0
    finally:
        tb.set_wait_limit(0)
    got = p.run(p.ws)
    assert tb.device_error(reset=True) == 0 and all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("hq,hkv,d,f8", [(32, 8, 128, False), (7, 1, 64, False), (16, 2, 256, True), (40, 8, 128, True), (16, 2, 64, True), (6, 6, 256, False)])
def test_many_items_per_block_in_repeated_calls(hq, hkv, d, f8):
    """Rings of tiles and queries that go through many items, of one and of two streams' rows."""
    rng = np.random.default_rng(d + hq)
    lens = [int(x) for x in rng.integers(0, 700, 120)]
    toks = [int(x) for x in rng.integers(1, 300, 120)]
    p = Prompts(lens, toks, hq, hkv, d, 64, f8, seed=22)
    first = [t.clone() for t in p.run()]
    p.check(*first, sequences=range(0, 120, 7))
    for _ in range(20):
        got = p.run(p.ws)
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    assert tb.device_error() == 0


@pytest.mark.parametrize("d", [64, 128, 256])
def test_queries_over_an_e4m3_cache_of_the_whole_range(d):
    """Rows of very different sizes in one block; keys are small enough for scores of a few units at the most."""
    p = Prompts([40], [200], 4, 2, d, 16, True, seed=23, scale=1.0)
    size = torch.exp2(torch.randint(-100, 60, (200, 4, 1), device="cuda").float())
    p.q.copy_((p.q.float() * size).bfloat16())
    p.scales[:, 0] = 2.0 ** -65
    out, lse = p.run()
    p.check(out, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_channel_far_above_the_others_over_an_e4m3_cache(d):
    """A query's numbers below 2^-13 of its row's largest are rounded to within 2^-21 of the largest, so a score is off by at most
    2^-21 max|q| sum|k| besides the rest: e in the exponent, and twice e A on the outputs."""
    p = Prompts([40], [200], 4, 2, d, 16, True, seed=23)
    p.q[:, :, 3] *= 2.0 ** 16
    p.pool.view(torch.uint8)[0, :, 0, :, :, 3] = 0  # keys do not see it
    out, lse = p.run()
    kv = p.keys_values(0)
    for h in range(4):
        q, k, v = p.q[:, h].double(), kv[0, h // 2], kv[1, h // 2]
        unseen = torch.arange(240, device="cuda")[None] > 40 + torch.arange(200, device="cuda")[:, None]
        x = (q @ k.T * p.scale).masked_fill(unseen, -torch.inf)
        lw = torch.logsumexp(x, 1)
        w = torch.exp(x - lw[:, None])
        size = (q.abs() @ k.abs().T).masked_fill(unseen, 0).amax(1) * p.scale
        e = 2.0 ** -21 * q.abs().amax(1) * k.abs().sum(1).amax() * p.scale
        tol = 1.1 * (2.0 ** -8 * (w @ v).abs() + (2.0 ** -8 + 2.0 ** -17 * size + 2 * e)[:, None] * (w @ v.abs())) + 1e-30
        assert bool(((out[:, h].double() - w @ v).abs() <= tol).all())
        assert bool(((lse[:, h].double() - lw).abs() <= 2.0 ** -18 * size + e + 1e-5).all())


def test_one_workspace_in_two_graphs():
    """Two graphs that share a workspace, replayed one after the other in both orders."""
    a, b = Prompts([5, 9000], [300, 100], 8, 2, 128, 64, seed=24), Prompts([0] * 3, [700, 65, 900], 8, 2, 128, 64, seed=25)
    want = [x.clone() for x in (*a.run(), *b.run())]
    graphs = []
    for p in (a, b):
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            p.run(a.ws)
        torch.cuda.current_stream().wait_stream(st)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tb.prompt_attention(p.q, p.cache, p.layer, p.batch, a.ws, p.scale, out=p.out, lse=p.lse)
        graphs.append(g)
    for order in ((0, 1), (1, 0), (1, 1), (0, 0)):
        for x in (a.out, a.lse, b.out, b.lse):
            x.fill_(1)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in order:
            assert torch.equal((a, b)[i].out, want[2 * i]) and torch.equal((a, b)[i].lse, want[2 * i + 1])


def test_counts_of_zero():
    p = Prompts([0], [70], 4, 2, 64, 16)
    p.run()
    none = tb.DraftBatch(p.batch.table[:0], p.batch.prefix[:0], p.batch.q_start[:1].contiguous(), 70, None, 0)
    assert tb.prompt_attention(p.q[:0], p.cache, 0, none, p.ws)[0].numel() == 0
    nothing = tb.DraftBatch(p.batch.table, p.batch.prefix, torch.zeros_like(p.batch.q_start), 70, None, 70)
    out, lse = p.out.fill_(7.5), p.lse.fill_(7.5)
    tb.prompt_attention(p.q, p.cache, 0, nothing, p.ws, out=out, lse=lse)
    assert bool((out == 7.5).all()) and bool((lse == 7.5).all())


@pytest.mark.parametrize("hq,hkv,d,f8,lens,toks", [
    (40, 8, 128, False, [0, 300, 0, 17] * 4, [1300, 900, 500, 1] * 4),  # items of whole blocks, more than there are thread blocks
    (16, 2, 256, True, [0] * 12, [700] * 12),
    (16, 4, 64, True, [0] * 20, [900] * 20),
    (8, 2, 128, False, [9000], [300]),                                  # split ranges, joined
    (8, 2, 128, False, [0], [100])])                                    # an item for each block at most
@pytest.mark.parametrize("fill", [0, 5, 1 << 20, -1, -1000, 0x7FFFFFFF, "floats"])
def test_a_workspace_of_any_contents(hq, hkv, d, f8, lens, toks, fill):
    """A program's scratch memory that other calls have used: the workspace needs no initial state."""
    p = Prompts(lens, toks, hq, hkv, d, 64, f8, seed=26)
    want = [t.clone() for t in p.run()]
    words = p.ws.view(torch.int32)
    if fill == "floats":
        g = torch.Generator(device="cuda").manual_seed(3)
        p.ws.view(torch.float32).copy_(torch.randn(words.shape, generator=g, device="cuda"))
    else:
        words.fill_(fill)
    p.out.fill_(7.5), p.lse.fill_(7.5)
    out, lse = p.run(p.ws)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_one_scratch_buffer_for_tree_and_prompt_attention():
    p = Prompts([500, 0, 100, 40] * 5, [64, 3, 20, 1] * 5, 8, 2, 128, 16, seed=27)
    big = Prompts([0] * 12, [1200, 900, 1, 700] * 3, 40, 8, 128, 64, seed=28)
    want, want_l = [t.clone() for t in big.run()]
    tree = tb.DraftBatch(i32(p.table), i32(p.lens), i32(p.q_start), 64, None, p.n)
    p.run()
    need = max(tb.new_tree_workspace(p.cache, tree, 8).numel(), big.ws.numel())
    scratch = torch.zeros(need, dtype=big.ws.dtype, device="cuda")
    for _ in range(3):
        tb.tree_attention(p.q, p.cache, 0, tree, scratch, p.scale)
        big.out.fill_(7.5), big.lse.fill_(7.5)
        big.run(scratch)
        assert torch.equal(big.out, want) and torch.equal(big.lse, want_l)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["inf", "nan"])
def test_scores_of_minus_infinity_give_zeros_whatever_the_values(d, kind):
    """Tokens whose scores are all minus infinity, over values that are not finite: in whole tiles, at the end of what they see,
    and where an item is split."""
    for lens, toks in (([0], [300]), ([6000], [200])):
        p = Prompts(lens, toks, 2, 1, d, 16, seed=13)
        p.q[:, :, 0] = 1.0
        p.pool[..., 0, :, :, 0] = -float("inf")  # every key's first number
        end = lens[0] + toks[0]
        for pos in (3, lens[0] + 1, lens[0] + 150, end - 1):
            p.row(0, pos)[1, 0, 5] = float(kind)
        out, lse = p.run()
        assert bool((out == 0).all()) and bool((lse == -torch.inf).all())


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_clamped_lengths_and_pages_give_what_the_clamped_ones_give(d, f8):
    """Prefixes past the table's width or below zero, starts outside n, more tokens than max_tokens, pages outside the pool."""
    p = Prompts([0, 30 * 16 - 50], [100, 50], 4, 2, d, 16, f8, seed=14)
    assert p.table.shape[1] == 30
    p.run()

    def call(table, prefix, starts, most):
        p.out.fill_(7.5), p.lse.fill_(7.5)
        batch = tb.DraftBatch(i32(table), i32(prefix), i32(starts), most, None, p.n)
        return tb.prompt_attention(p.q, p.cache, 0, batch, p.ws, p.scale, out=p.out, lse=p.lse)

    for prefix, starts in (([0, 10 ** 9], [0, 100, 2 ** 30]), ([-5, 30 * 16], [-7, 100, 151]), ([0, 30 * 16 - 49], [0, 100, 150])):
        p.check(*call(p.table, prefix, starts, 100))
    out, lse = call(p.table, [0, 30 * 16 - 50], [0, 100, 150], 40)
    assert bool((out[40:100] == 7.5).all()) and bool((lse[40:100] == 7.5).all()) and bool((out[140:] == 7.5).all())
    short = Prompts.__new__(Prompts)
    short.__dict__.update(p.__dict__, toks=[40, 40])
    short.check(out, lse)
    # pages outside the pool are its first or its last one
    last = p.pool.shape[1] - 1
    p.pool.view(torch.uint8)[:, [0, last]] = p.pool.view(torch.uint8)[:, p.table[1, [2, 3]]]  # finite
    wild, kept = p.table.copy(), p.table.copy()
    wild[1, 1], wild[1, 7], wild[0, 2] = 10 ** 9, -5, last + 1
    kept[1, 1], kept[1, 7], kept[0, 2] = last, 0, last
    want = [t.clone() for t in call(kept, p.lens, p.q_start, 100)]
    got = call(wild, p.lens, p.q_start, 100)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    p.table = kept
    p.check(*got)
    assert tb.device_error() == 0


@pytest.mark.parametrize("d", [64, 128, 256])
def test_queries_that_are_not_finite_touch_no_other_over_an_e4m3_cache(d):
    p = Prompts([20, 0], [300, 130], 4, 2, d, 16, True, seed=10)
    out, lse = p.run()
    want, want_l = out.clone(), lse.clone()
    p.q[57, 1, 5] = float("nan")
    p.q[301, 3, 0] = float("inf")
    p.run()
    keep = torch.ones((p.n, 4), dtype=torch.bool, device="cuda")
    keep[57, 1] = keep[301, 3] = False
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_l[keep])


@pytest.mark.parametrize("f8,d", [(False, 128), (True, 128), (False, 256), (True, 64)])
def test_a_sequence_does_not_depend_on_the_others_numbers(f8, d):
    p = Prompts([500, 0, 9000], [300, 1200, 64], 8, 2, d, 64, f8, seed=16)
    first, first_l = (t.clone() for t in p.run())
    bits = p.pool.view(torch.uint8)
    for b in (0, 2):  # other queries, and other pages with other numbers
        p.q[p.q_start[b]:p.q_start[b + 1]] *= -3
        held = p.table[b, :-(-(p.lens[b] + p.toks[b]) // 64)].tolist()
        bits[:, held] = bits[:, held[::-1]].clone()
        p.table[b, :len(held)] = held[::-1]
    p.table[0, [0, 1]] = p.table[0, [1, 0]]
    out, lse = p.run()
    mine = slice(300, 1500)
    assert torch.equal(out[mine], first[mine]) and torch.equal(lse[mine], first_l[mine])
    assert not torch.equal(out[:300], first[:300]) and not torch.equal(out[1500:], first[1500:])
    p.check(out, lse)
