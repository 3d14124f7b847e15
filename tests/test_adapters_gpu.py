"""trellis_adapter_plan and trellis_adapter_add against the 64-bit definition.

Tolerance, per output with h = A x and the sums of absolute values H = |A| |x|, S = |scale| (|B| |h|), T = |scale| (|B| H):
  one rounding to bf16 (half a unit)                     2^-8 |out|
  h summed in fp32 over `in` products                    in 2^-24 T at the most
  h as the sum of two bf16 numbers                       2^-16 S
  the second product, times scale, and y                 (rank + 3) 2^-24 (S + |y|)
each with a tenth more."""
import numpy as np
import pytest
import torch

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


class Step:
    """Sequences with adapters: which[b] of toks[b] tokens; rows past a rank hold NaN."""

    def __init__(self, toks, which, ranks, max_rank, k, n, seed=0, lead=0, tail=0, pad=0, scales=True, nan=True):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.toks, self.which, self.ranks, self.max_rank, self.k, self.n = toks, which, ranks, max_rank, k, n
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        count = len(ranks)
        self.a, self.b = (rand(count, max_rank, k) * k ** -0.5).bfloat16(), rand(count, n, max_rank).bfloat16()
        if nan:
            for i, r in enumerate(ranks):
                self.a[i, max(0, r):] = float("nan")
                self.b[i, :, max(0, r):] = float("nan")
        self.scales = torch.rand(count, generator=g, device="cuda") * 2 - 0.5 if scales else None
        self.starts = lead + np.concatenate([[0], np.cumsum(toks)])
        self.tokens = lead + sum(toks) + tail
        self.x = rand(self.tokens, k + pad).bfloat16()[:, :k]
        self.y = rand(self.tokens, n + pad).bfloat16()[:, :n]
        self.out = torch.full((self.tokens, n + pad), 7.5, dtype=torch.bfloat16, device="cuda")[:, :n]

    def run(self, **kw):
        self.adapters = tb.Adapters(self.a, self.b, i32(self.ranks), self.scales)
        self.plan = tb.adapter_plan(tb.AdapterPlan(i32(self.which), i32(self.starts), self.tokens))
        return tb.adapter_add(self.x, self.y, self.adapters, self.plan, **{"out": self.out, **kw})

    def check(self, out, y=None):
        y = self.y if y is None else y
        for b, (t, a) in enumerate(zip(self.toks, self.which)):
            rows = slice(int(self.starts[b]), int(self.starts[b + 1]))
            r = max(0, min(self.ranks[a], self.max_rank)) if 0 <= a < len(self.ranks) else 0
            if r == 0:
                assert torch.equal(out[rows], y[rows]), b
                continue
            x, A, B = self.x[rows].double(), self.a[a, :r].double(), self.b[a, :, :r].double()
            s = 1.0 if self.scales is None else float(self.scales[a])
            h, big = x @ A.T, x.abs() @ A.abs().T
            want = y[rows].double() + s * (h @ B.T)
            S, T = abs(s) * (h.abs() @ B.abs().T), abs(s) * (big @ B.abs().T)
            tol = 1.1 * (2.0 ** -8 * want.abs() + self.k * 2.0 ** -24 * T + 2.0 ** -16 * S + (r + 3) * 2.0 ** -24 * (S + y[rows].double().abs()))
            off = (out[rows].double() - want).abs() / tol
            assert bool((off <= 1).all()), (b, a, float(off.max()), torch.nonzero(~(off <= 1))[:4].tolist())


@pytest.mark.parametrize("rank", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("k,n", [(5120, 5120), (8, 8), (1024, 2048), (520, 264), (4096, 1000), (2048, 17408)])
@pytest.mark.parametrize("toks", [[1], [3], [17], [1] * 9, [70, 1, 64, 0, 130]])
def test_sizes(rank, k, n, toks):
    count = 3
    which = [(7 * b + 1) % count for b in range(len(toks))]
    s = Step(toks, which, [rank] * count, rank, k, n, seed=rank + k + len(toks))
    s.check(s.run())


@pytest.mark.parametrize("max_rank,ranks", [(8, [0, 1, 5, 8]), (24, [24, 9, 17, 16]), (40, [40, 33, 1, 7]), (64, [4, 64, 63, 16]), (128, [128, 3, 100, 65]),
                                            (104, [104, 97, 90, 80]), (16, [-3, 99, 16, 2])])
def test_mixed_ranks(max_rank, ranks):
    toks = [5, 1, 100, 33, 2, 64, 1, 9]
    s = Step(toks, [0, 1, 2, 3, -1, 2, 1, 3], ranks, max_rank, 640, 1032, seed=max_rank)
    s.check(s.run())


def test_without_ranks_and_scales():
    s = Step([40, 2], [1, 0], [16, 16], 16, 512, 768, scales=False, nan=False)
    adapters = tb.Adapters(s.a, s.b)
    s.run()
    s.check(tb.adapter_add(s.x, s.y, adapters, s.plan, out=torch.empty_like(s.y)))


@pytest.mark.parametrize("toks", [[1] * 30, [130, 1, 40]])
def test_in_place_strides_and_rows_of_no_sequence(toks):
    which = [(b % 5) - 1 for b in range(len(toks))]
    s = Step(toks, which, [16, 8, 4, 12], 16, 776, 1544, seed=4, lead=3, tail=6, pad=16)
    out = s.run()
    s.check(out)
    assert bool((out[:3] == 7.5).all()) and bool((out[-6:] == 7.5).all())
    y = s.y.clone()
    wide = torch.full((s.tokens, s.n + 16), 9.25, dtype=torch.bfloat16, device="cuda")
    wide[:, :s.n] = y
    got = tb.adapter_add(s.x, wide[:, :s.n], s.adapters, s.plan)
    s.check(got, y)
    assert torch.equal(got[:3], y[:3]) and torch.equal(got[-6:], y[-6:]) and bool((wide[:, s.n:] == 9.25).all())
    assert torch.equal(got[3:-6], out[3:-6])


def test_indices_outside_the_adapters():
    s = Step([2, 70, 1, 3, 5], [2, -7, 2 ** 31 - 1, 1, 0], [8, 8], 8, 256, 512, seed=5)
    s.check(s.run())


@pytest.mark.parametrize("batch,most", [(1, 5000), (64, 1), (1024, 7), (300, 300)])
def test_plans(batch, most):
    """Each token of a sequence is in one tile of its adapter; tiles have 1 to 64 tokens."""
    rng = np.random.default_rng(batch)
    toks = rng.integers(0, most + 1, batch) if batch > 1 else np.array([most])
    which = rng.integers(-1, 40, batch)
    starts = 2 + np.concatenate([[0], np.cumsum(toks)])
    n = int(starts[-1]) + 3
    plan = tb.AdapterPlan(i32(which), i32(starts), n)
    plan.plan.fill_(-1)
    tb.adapter_plan(plan)
    words = plan.plan.cpu().numpy()
    tiles, with_one = int(words[0]), int(words[1])
    most_tiles = n // 64 + min(batch, n) + (256 if n >= 32 else 0)
    at = words[4:4 + 4 * tiles].reshape(tiles, 4)
    order = words[4 + 4 * most_tiles:]
    assert tiles <= most_tiles and np.all(at[:, 2] >= 1) and np.all(at[:, 2] <= 64)
    owner = np.full(n, -9)
    for b in range(batch):
        owner[starts[b]:starts[b + 1]] = which[b]
    seen, place = np.zeros(n, bool), 0
    for i, (a, first, count, _) in enumerate(at):
        assert first == place and (a >= 0) == (i < with_one)
        place += count
        mine = order[first:first + count]
        assert np.all(owner[mine] == a) and not seen[mine].any()
        seen[mine] = True
    assert place == toks.sum() and seen.sum() == toks.sum()
    groups = at[:, 0][np.concatenate([[True], at[1:, 0] != at[:-1, 0]])] if tiles else []
    assert list(groups) == sorted(set(groups), key=lambda a: (a < 0, a))
    # as few tiles as the groups' sizes allow, or more of 32 tokens and more
    sizes = [int(toks[which == a].sum()) for a in set(which.tolist())]
    assert sum(-(-s // 64) for s in sizes) <= tiles <= sum(-(-s // 32) for s in sizes)
    # tiles of a group are as long as one another, to within a token
    for a in set(at[:, 0].tolist()):
        assert np.ptp(at[at[:, 0] == a, 2]) <= 1


def test_starts_that_fall_or_leave_the_range():
    """Starts are clamped to [0, n] and taken as ascending; what no sequence has then is left as it is."""
    s = Step([10, 10, 10], [0, 1, 0], [8, 8], 8, 256, 512, seed=6)
    out = s.run()
    want = out.clone()
    out.fill_(7.5)
    plan = tb.adapter_plan(tb.AdapterPlan(i32([0, 1, 0, 1]), i32([-4, 10, 3, 20, 10 ** 9]), 30))  # 0..10, none, 10..20, 20..30
    tb.adapter_add(s.x, s.y, s.adapters, plan, out=out)
    assert torch.equal(out[:10], want[:10])
    s2 = Step([10, 10, 10], [0, 0, 1], [8, 8], 8, 256, 512, seed=6)
    s2.check(out)


def test_rows_do_not_depend_on_others_and_equal_calls_give_equal_bits():
    toks = [1, 1, 40, 1, 100, 7]
    s = Step(toks, [0, 1, 0, 2, 2, 1], [16, 5, 64], 64, 1544, 1288, seed=7)
    first = s.run().clone()
    assert torch.equal(s.run(), first)
    bad = s.x.clone()
    bad[2 + 5] = float("nan")
    keep = torch.ones(s.tokens, dtype=torch.bool, device="cuda")
    keep[2 + 5] = False
    s.x = bad
    got = s.run()
    assert torch.equal(got[keep], first[keep]) and bool(torch.isnan(got[2 + 5]).all())


def test_values_that_are_not_finite():
    s = Step([3, 70], [0, 1], [8, 8], 8, 256, 512, seed=8, scales=False)
    s.y[1, 5], s.y[10, 7] = float("inf"), float("nan")
    s.b[0, 9, 2] = float("nan")
    out = s.run()
    assert out[1, 5] == float("inf") and bool(torch.isnan(out[10, 7])) and bool(torch.isnan(out[:3, 9]).all())
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[1, 5] = bad[10, 7] = True
    bad[:3, 9] = True
    assert bool(torch.isfinite(out[~bad]).all())


def test_large_numbers_keep_their_low_rank_product():
    """Products whose parts cancel: the size of the parts is what errors are relative to."""
    s = Step([20, 1], [0, 1], [64, 64], 64, 2048, 512, seed=9)
    s.x *= 1000
    s.check(s.run())


@pytest.mark.parametrize("toks", [[1] * 40, [300, 2, 64]])
def test_captured_and_replayed_over_other_adapters(toks):
    s = Step(toks, [b % 3 for b in range(len(toks))], [16, 8, 12], 16, 1024, 1032, seed=10)
    s.run()
    which, starts = i32(s.which), i32(s.starts)
    plan = tb.AdapterPlan(which, starts, s.tokens)

    def call():
        tb.adapter_plan(plan)
        return tb.adapter_add(s.x, s.y, s.adapters, plan, out=s.out)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for shift in range(3):
        s.which = [(b + shift) % 4 - 1 for b in range(len(toks))]
        s.toks = [toks[(b + shift) % len(toks)] for b in range(len(toks))]
        s.starts = np.concatenate([[0], np.cumsum(s.toks)])
        which.copy_(i32(s.which)), starts.copy_(i32(s.starts))
        s.out.fill_(7.5)
        graph.replay()
        torch.cuda.synchronize()
        s.check(s.out)


def test_another_stream_and_two_calls_at_once():
    a, b = Step([1] * 50, [i % 7 for i in range(50)], [16] * 7, 16, 2048, 4096, seed=11), Step([700], [0], [64], 64, 4096, 2048, seed=12)
    want = [a.run().clone(), b.run().clone()]
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.out.fill_(1), b.out.fill_(1)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            tb.adapter_add(a.x, a.y, a.adapters, a.plan, out=a.out)
        with torch.cuda.stream(t):
            tb.adapter_add(b.x, b.y, b.adapters, b.plan, out=b.out)
        torch.cuda.synchronize()
        assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])


def test_many_tokens_past_32_bits():
    """Rows whose offsets pass 2^31 numbers."""
    n, wide = 130000, 17408
    assert n * wide > 2 ** 31
    s = Step([3], [0], [16], 16, 256, wide, seed=13)
    s.run()
    x, y = torch.zeros((n, 256), dtype=torch.bfloat16, device="cuda"), torch.zeros((n, wide), dtype=torch.bfloat16, device="cuda")
    x[-3:], y[-3:] = s.x, s.y
    plan = tb.adapter_plan(tb.AdapterPlan(i32([0]), i32([0, n]), n))
    got = tb.adapter_add(x, y, s.adapters, plan)
    assert torch.equal(got[-3:], s.out) and bool((got[:-3] == 0).all())


def test_refusals_of_the_binding():
    s = Step([4, 3], [0, 1], [8, 8], 8, 256, 512)
    s.run()
    ok = dict(x=s.x, y=s.y, adapters=s.adapters, plan=s.plan, out=s.out)
    for bad in (dict(x=s.x.float()), dict(x=s.x[:5]), dict(y=s.y.cpu()), dict(out=s.out.T.contiguous().T), dict(x=s.x[:, :128]), dict(out=s.out[:6])):
        with pytest.raises(ValueError):
            tb.adapter_add(**{**ok, **bad})
    odd = torch.empty((7, 516), dtype=torch.bfloat16, device="cuda")[:, 4:]
    with pytest.raises(tb.TrellisError):  # rows that do not begin at 16 bytes
        tb.adapter_add(**{**ok, "out": odd})
    for a, b in ((s.a[0], s.b[0]), (s.a, s.b.float()), (s.a, s.b[:1]), (s.a.cpu(), s.b)):
        with pytest.raises(ValueError):
            tb.Adapters(a, b)
    with pytest.raises(ValueError):
        tb.AdapterPlan(i32([0]), i32([0, 1, 2]), 2)
    with pytest.raises(ValueError):
        tb.AdapterPlan(i32([0] * 1025), i32([0] * 1026), 2)


def test_counts_of_zero():
    s = Step([4, 3], [0, 1], [8, 8], 8, 256, 512)
    s.run()
    none = tb.adapter_plan(tb.AdapterPlan(i32([]), i32([0]), 0))
    assert tb.adapter_add(s.x[:0], s.y[:0], s.adapters, none).numel() == 0
    empty = tb.adapter_plan(tb.AdapterPlan(i32([0, 1]), i32([0, 0, 0]), 7))
    s.out.fill_(7.5)
    assert bool((tb.adapter_add(s.x, s.y, s.adapters, empty, out=s.out) == 7.5).all())


def test_a_plan_not_made_yet_does_nothing():
    s = Step([4, 3], [0, 1], [8, 8], 8, 256, 512)
    s.run()
    s.out.fill_(7.5)
    fresh = tb.AdapterPlan(i32([0, 1]), i32([0, 4, 7]), 7)
    assert bool((tb.adapter_add(s.x, s.y, s.adapters, fresh, out=s.out) == 7.5).all())


@pytest.mark.parametrize("rank,count", [(16, 90), (40, 90), (16, 300), (128, 50)])
def test_rounds_of_many_adapters(rank, count):
    """More tiles than clusters: whole rounds and a last one that clusters share."""
    rng = np.random.default_rng(count)
    toks = rng.integers(1, 40, count).tolist()
    s = Step(toks, list(range(count)), [int(r) for r in rng.integers(1, rank + 1, count)], rank, 264, 2056, seed=count)
    first = s.run().clone()
    s.check(first)
    assert torch.equal(s.run(), first)


def check_any_numbers(s, out):
    """Every number against the definition, infinities and NaN in their places.  The finite ones are to the tolerance above."""
    with np.errstate(invalid="ignore", over="ignore"):
        for b, (t, a) in enumerate(zip(s.toks, s.which)):
            rows, r = slice(int(s.starts[b]), int(s.starts[b + 1])), s.ranks[a]
            x, A, B, y = (v.double().cpu().numpy() for v in (s.x[rows], s.a[a, :r], s.b[a, :, :r], s.y[rows]))
            # one product after the other: a library's matrix product may pad with zeros
            h, T = (x[:, None] * A[None]).sum(-1), (np.abs(x)[:, None] * np.abs(A)[None]).sum(-1)
            low, S, big = (sum(g[:, i, None] * w[None, :, i] for i in range(r)) for g, w in ((h, B), (np.abs(h), np.abs(B)), (T, np.abs(B))))
            want, got = y + low, out[rows].double().cpu().numpy()
            fine = np.isfinite(want)
            assert np.array_equal(np.isnan(got), np.isnan(want)), (b, r, np.argwhere(np.isnan(got) != np.isnan(want))[:4].tolist())
            assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), (b, r)
            tol = 1.1 * (2.0 ** -8 * np.abs(want) + s.k * 2.0 ** -24 * big + 2.0 ** -16 * S + (r + 3) * 2.0 ** -24 * (S + np.abs(y)))
            assert np.all(np.abs(got - want)[fine] <= tol[fine]), (b, r)


RANKS_OF_ALL_KERNELS = [(8, 1), (8, 5), (8, 8), (16, 16), (24, 17), (32, 32), (40, 3), (64, 40), (64, 64), (128, 9), (128, 100), (128, 128)]


@pytest.mark.parametrize("max_rank,rank", RANKS_OF_ALL_KERNELS)
def test_infinite_numbers_in_b(max_rank, rank):
    """B's infinities are infinite in the outputs, also where the low-rank product is a bf16 number (its low part is zero)."""
    s = Step([3, 70], [0, 1], [rank, rank], max_rank, 264, 520, seed=30 + rank, scales=False)
    s.x[:, :] = 0
    for t in range(s.tokens):  # h is a column of A (exact), twice it, or with a second one what takes more than 8 bits
        s.x[t, (37 * t) % 264] = 1.0 + t % 2
        if t % 3 == 2:
            s.x[t, (37 * t + 5) % 264] = 1.0
    s.b[0, 9, 0], s.b[0, 10, rank - 1], s.b[1, 500, rank // 2] = float("inf"), -float("inf"), -float("inf")
    check_any_numbers(s, s.run())


@pytest.mark.parametrize("max_rank,rank", RANKS_OF_ALL_KERNELS)
def test_infinite_numbers_in_x_and_a(max_rank, rank):
    """Ranks that an adapter does not have take no part, also where a token's numbers are infinite."""
    s = Step([3, 70, 2, 40], [0, 1, 2, 3], [rank] * 4, max_rank, 264, 520, seed=50 + rank, scales=False)
    for i in (0, 1):  # one sign: sums of infinities are infinite
        s.a[i, :rank], s.b[i, :, :rank] = s.a[i, :rank].abs() + 0.01, s.b[i, :, :rank].abs() + 0.01
    s.x[1, 100], s.x[3 + 40, 7], s.x[3 + 69, 263], s.x[75 + 20, 9] = float("inf"), -float("inf"), float("inf"), float("inf")
    s.a[2, 0, 0], s.a[3, rank - 1, 11] = float("inf"), -float("inf")
    s.x[75 + 30, 11] = 0  # times infinity: NaN
    check_any_numbers(s, s.run())


@pytest.mark.parametrize("rank", [8, 32, 64, 128])
@pytest.mark.parametrize("n", [264, 4104])
def test_a_token_does_not_depend_on_who_shares_its_adapter(rank, n):
    """The same token alone, among few and many tokens of its adapter, and beside other adapters: equal bits."""
    k = 1544
    s = Step([64], [0], [rank - 3] + [rank] * 60, rank, k, n, seed=rank + n)
    g = torch.Generator(device="cuda").manual_seed(1)
    more = [torch.randn((200, m), generator=g, device="cuda").bfloat16() for m in (k, n)]
    s.run()
    want = None
    for toks, which in (([1], [0]), ([2], [0]), ([16], [0]), ([17], [0]), ([33], [0]), ([64], [0]), ([1, 3], [0, 1]), ([16, 130], [0, 1]),
                        ([64, 100, 1], [0, 1, 2]), ([64, 100], [0, 0]), ([1] + [2] * 60, [0] + list(range(1, 61))), ([1, 40, 64], [0, -1, 0])):
        total = sum(toks)
        x, y = torch.cat([s.x, more[0]])[:total], torch.cat([s.y, more[1]])[:total]
        plan = tb.adapter_plan(tb.AdapterPlan(i32(which), i32(np.concatenate([[0], np.cumsum(toks)])), total))
        got = tb.adapter_add(x, y, s.adapters, plan, out=torch.empty_like(y))
        want = got[0] if want is None else want
        assert torch.equal(got[0], want), (toks, which)
        assert not torch.equal(got[0], y[0])


@pytest.mark.parametrize("count", [50, 90, 250, 300])
@pytest.mark.parametrize("ranks", ["equal", "mixed"])
def test_rounds_of_adapters_of_equal_and_of_mixed_ranks(count, ranks):
    """More tiles than clusters, each of a token or two, with the same rank or with several."""
    rank = [64] * count if ranks == "equal" else [(i * 11) % 64 + 1 for i in range(count)]
    s = Step([1 + b % 2 for b in range(count)], list(range(count)), rank, 64, 264, 4104, seed=count)
    s.check(s.run())


@pytest.mark.parametrize("toks,rank", [([1], 16), ([1] * 40, 64), ([300, 2, 70], 16), ([300, 2, 70], 32), ([500], 128)])
def test_adapters_written_directly_before_a_call(toks, rank):
    """Requests bring their adapters: what a call reads of them may have been written by the launch ahead, captured or not."""
    count = 3
    steps = [Step(toks, [b % count for b in range(len(toks))], [rank, max(1, rank - 5 * i), rank], rank, 1544, 1288, seed=60 + i, nan=False) for i in range(4)]
    want = []
    for t in steps:
        t.x, t.y = steps[0].x, steps[0].y
        want.append(t.run().clone())
        torch.cuda.synchronize()
    a, b, ranks, scales = (v.clone() for v in (steps[0].a, steps[0].b, i32(steps[0].ranks), steps[0].scales))
    kept = [i32(t.ranks) for t in steps]
    adapters = tb.Adapters(a, b, ranks, scales)
    outs = [torch.empty_like(w) for w in want]

    def calls():
        for t, r, out in zip(steps, kept, outs):
            for to, of in ((ranks, r), (scales, t.scales), (a, t.a), (b, t.b)):
                to.mul_(0).add_(of)
            tb.adapter_add(steps[0].x, steps[0].y, adapters, steps[0].plan, out=out)

    for _ in range(10):
        calls()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        calls()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(10):
        for o in outs:
            o.fill_(1)
        graph.replay()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
