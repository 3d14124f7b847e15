"""trellis_tree_attention against the 64-bit definition.

Tolerance, per output with w the softmax weights, A = sum w |v| and X = max over the keys of scale * sum |q k|:
  one rounding to bf16 (half a unit)              2^-8 |out|
  weights rounded to 16 bits                      2^-8 A  (bf16; fp16 is finer)
  scores summed in fp32 (up to 256 products in steps of 16, some kept to 2^-23 of the largest): 2^-18 X in the
  exponent, on weights and sum                     2 * 2^-18 X A
each with a tenth more.  lse: 2^-18 X + 1e-5 (the sum, and the approximate exponentials of 2^-22)."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from trellis_coded_weight_gb300 import binding as tb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from trellis_coded_weight_gb300 import build
    build.build()
    tb.load()


class Step:
    """A cache with the pages of some sequences, their drafts' masks and queries."""

    def __init__(self, lens, toks, hq, hkv, d, page, f8=False, seed=0, masks="tree", std=1.0, layers=1, layer=0, spare=2,
                 q_pad=0, garbage=True):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.toks, self.layer, self.d, self.page = lens, toks, layer, d, page
        held = [-(-(p + t) // page) for p, t in zip(lens, toks)]
        pages = sum(held) + spare
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
        if garbage:  # rows past the ends, and pages nobody holds, hold NaN
            nan = self.pool.view(torch.uint8)
            for p in order[at:]:
                nan[:, p] = 0xFF if not f8 else 0x7F
            for b, (p, t) in enumerate(zip(lens, toks)):
                if (p + t) % page:
                    nan[:, self.table[b, held[b] - 1], :, :, (p + t) % page:] = 0xFF if not f8 else 0x7F
        self.n = sum(toks)
        self.q_start = np.concatenate([[0], np.cumsum(toks)])
        self.masks = []
        for t in toks:
            mine = []
            for i in range(t):
                if masks == "tree":
                    parent = int(rng.integers(-1, i)) if i else -1
                    mine.append((mine[parent] if parent >= 0 else 0) | 1 << i)
                elif masks == "random":
                    mine.append(int(rng.integers(0, 2 ** 63)) & ((1 << t) - 1))
                elif masks == "none":
                    mine.append(0)
                elif masks == "past":  # bits past the drafts are ignored
                    mine.append(2 ** 64 - 1)
                else:
                    mine.append((2 << i) - 1)
            self.masks += mine
        wide = (torch.randn((max(1, self.n), hq * d + q_pad), generator=g, device="cuda") * std).bfloat16()[:self.n]
        self.q = wide[:, :hq * d].unflatten(1, (hq, d))
        self.hq, self.hkv = hq, hkv
        self.scale = d ** -0.5

    def run(self, ws=None, **kw):
        i32 = lambda a: torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()  # noqa: E731
        self.cache = tb.PagedCache(self.pool, self.scales)
        m = torch.as_tensor(np.array(self.masks, dtype=np.uint64).view(np.int64)).cuda() if self.masks_given else None
        self.batch = tb.DraftBatch(i32(self.table), i32(self.lens), i32(self.q_start), max(1, max(self.toks)), m, self.n)
        ws = tb.new_tree_workspace(self.cache, self.batch, self.hq) if ws is None else ws
        return tb.tree_attention(self.q, self.cache, self.layer, self.batch, ws, self.scale, **kw)

    masks_given = True

    def want(self, b):
        p, t, page = self.lens[b], self.toks[b], self.page
        rows = self.pool[self.layer][torch.as_tensor(self.table[b, :-(-(p + t) // page)]).long().cuda()]
        rows = ref.f64(rows.float()).transpose(1, 2, 0, 3, 4).reshape(2, self.hkv, -1, self.d)[:, :, :p + t]
        if self.scales is not None:
            rows = rows * ref.f64(self.scales)[self.layer][:, :, None, None]
        first = self.q_start[b]
        seen = np.ones((t, p + t), bool)
        for i in range(t):
            seen[i, p:] = [self.masks[first + i] >> j & 1 for j in range(t)]
        q = ref.f64(self.q[first:first + t])
        group = self.hq // self.hkv
        return [ref.attention(q[:, h], rows[0, h // group], rows[1, h // group], seen, self.scale) for h in range(self.hq)]

    def check(self, out, lse, sequences=None):
        for b in range(len(self.lens)) if sequences is None else sequences:
            first, t = self.q_start[b], self.toks[b]
            got_o, got_l = ref.f64(out[first:first + t]), ref.f64(lse[first:first + t])
            for h, (o, lw, mass, size) in enumerate(self.want(b)):
                fine = np.isfinite(o)
                g = got_o[:, h]
                assert np.array_equal(np.isnan(g), np.isnan(o)) and np.array_equal(g[~fine & ~np.isnan(o)], o[~fine & ~np.isnan(o)])
                with np.errstate(invalid="ignore"):
                    tol = 1.1 * (2.0 ** -8 * np.abs(o) + 2.0 ** -8 * mass + 2.0 ** -17 * size[:, None] * mass) + 1e-30
                    assert np.all((np.abs(g - o) <= tol)[fine]), (b, h, np.nanmax(np.abs(g - o) / tol))
                ok = np.isfinite(lw)
                assert np.array_equal(got_l[~ok, h], lw[~ok])
                assert np.all(np.abs(got_l[:, h] - lw)[ok] <= 2.0 ** -18 * size[ok] + 1e-5), (b, h)


HEADS = [(8, 8, 64), (40, 8, 128), (16, 2, 256), (6, 2, 128), (16, 1, 64), (5, 1, 256)]


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("lens,toks,page", [([0], [1], 16), ([300], [1], 16), ([63, 0, 64, 1000], [1, 5, 3, 4], 32),
                                            ([517, 129], [64, 17], 64), ([95], [33], 128)])
def test_sequences(lens, toks, page, hq, hkv, d, f8):
    s = Step(lens, toks, hq, hkv, d, page, f8, seed=len(lens) + d, q_pad=8)
    s.check(*s.run())


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("masks", ["random", "none", "past", "chain"])
def test_masks(masks, f8):
    s = Step([0, 70, 16, 0], [9, 64, 1, 64], 12, 4, 128, 16, f8, seed=4, masks=masks)
    out, lse = s.run()
    if masks == "none":
        assert torch.all(out[:9] == 0) and torch.all(lse[:9] == -torch.inf) and torch.all(out[-64:] == 0)
    s.check(out, lse)


def test_chain_without_a_mask():
    s = Step([5, 200], [64, 3], 8, 2, 64, 32, seed=6, masks="chain")
    s.masks_given = False
    s.check(*s.run())


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_what_is_not_seen_does_not_reach_the_result(d, f8):
    s = Step([40, 3], [12, 30], 8, 2, d, 16, f8, seed=7, masks="chain")
    bad = {0: [3, 7], 1: [29, 11, 0]}  # drafts with keys and values that are not numbers
    raw = s.pool.view(torch.uint8 if f8 else torch.int16)
    kinds = [0x7F, 0xFF] if f8 else [0x7FC0, 0x7F80, -128, 0x7F81]  # NaN, infinities, NaN
    for b, js in bad.items():
        for n, j in enumerate(js):
            p = s.lens[b] + j
            at = (0, int(s.table[b, p // 16]), slice(None), slice(None), p % 16)
            raw[at] = kinds[n % len(kinds)]
        first = int(s.q_start[b])
        for i in range(s.toks[b]):
            s.masks[first + i] = sum(1 << j for j in range(i + 1) if j not in js)
    out, lse = s.run()
    assert out.isfinite().all()
    s.check(out, lse)
    # values that are not numbers in a draft that some rows see: those rows and columns, and no others
    first = int(s.q_start[0])
    p = s.lens[0] + 5
    raw[0, int(s.table[0, p // 16]), 1, :, p % 16, 5] = 0x7F if f8 else 0x7F80
    out, _ = s.run()
    seen = torch.tensor([m >> 5 & 1 for m in s.masks[first:first + s.toks[0]]], device="cuda").bool()
    got = ~out[first:first + s.toks[0]].isfinite()
    assert got[seen][:, :, 5].all() and not got[~seen].any() and int(got[seen].sum()) == int(seen.sum()) * s.hq


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d,hq", [(64, 16), (128, 8), (256, 10)])
def test_odd_values_in_short_sequences_one_after_another(d, hq, f8):
    # every sequence is one short item and has a draft whose values are no numbers: each block has several such items
    count, t = 700, 5
    lens = [int(v) for v in np.random.default_rng(5).integers(0, 40, count)]
    s = Step(lens, [t] * count, hq, 2, d, 16, f8=f8, seed=11)
    bad = s.pool.view(torch.uint8 if f8 else torch.int16)
    at = torch.as_tensor([[s.table[b, (lens[b] + b % t) // 16], (lens[b] + b % t) % 16] for b in range(count)]).cuda()
    bad[0, at[:, 0], 1, :, at[:, 1]] = 0x7F if f8 else 0x7FC0
    out, _ = s.run()
    masks = torch.tensor(s.masks).view(count, t)
    sees = (masks >> (torch.arange(count) % t)[:, None] & 1).bool().view(-1)
    nan = out.isnan().cpu()
    assert nan[sees].all() and not nan[~sees].any()


@pytest.mark.parametrize("f8,d,hq,hkv,toks", [(False, 128, 8, 2, 1), (True, 128, 8, 1, 4), (False, 64, 16, 2, 8),
                                               (False, 128, 16, 2, 33), (True, 256, 4, 1, 16)])
def test_long_contexts_split_over_the_gpu(f8, d, hq, hkv, toks):
    s = Step([20011, 7, 4096], [toks, 1, toks], hq, hkv, d, 64, f8, seed=11, std=3.0)
    s.check(*s.run())


def test_ragged_batch_of_many():
    rng = np.random.default_rng(5)
    lens, toks = [int(x) for x in rng.integers(0, 300, 200)], [int(x) for x in rng.integers(0, 9, 200)]
    s = Step(lens, toks, 4, 2, 64, 16, seed=12)
    out = torch.full((s.n, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    s.check(*s.run(out=out))


def test_peaked_scores_and_a_negative_scale():
    s = Step([3000], [4], 8, 2, 128, 32, seed=13, std=12.0)
    s.check(*s.run())
    s.scale = -0.05
    s.check(*s.run())
    s = Step([3000], [4], 8, 2, 128, 32, True, seed=13, std=12.0)
    s.check(*s.run())


def test_e4m3_queries_far_from_one():
    for std in (1e-20, 1e20):
        s = Step([100], [3], 4, 2, 128, 16, True, seed=14, std=std)
        s.scale = 0.1 / std
        s.check(*s.run())


def test_equal_bits_in_repeated_calls_and_one_workspace_for_all():
    big = Step([9000, 800], [16, 16], 32, 4, 128, 64, seed=15)
    big.run()
    ws = tb.new_tree_workspace(big.cache, big.batch, 32)
    a = [t.clone() for t in big.run(ws)]
    for other in (Step([50] * 40, [1] * 40, 8, 8, 64, 16, seed=16), Step([7000], [2], 8, 1, 128, 16, seed=17)):
        other.check(*other.run(ws))
    b = big.run(ws)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_another_layer_stream_and_no_lse():
    s = Step([200, 31], [3, 2], 8, 2, 128, 32, True, seed=18, layers=3, layer=2)
    out, lse = s.run()
    s.check(out, lse)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        out2, none = s.run(lse=False)
    st.synchronize()
    assert none is None and torch.equal(out, out2)


def test_lengths_and_tables_out_of_range_stay_in_bounds():
    """Lengths past the table, entries past the pool, ranges past the tokens: results are undefined for those sequences
    (nothing outside the arrays is read), and the others are right."""
    s = Step([100, 60, 33], [4, 4, 4], 8, 2, 64, 16, seed=19)
    s.run()
    i32 = lambda a: torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()  # noqa: E731
    table = s.table.copy()
    table[1, 0], table[1, 2] = 1 << 30, -5
    mask = s.batch.mask
    lens = [100, 10 ** 9, 33]
    batch = tb.DraftBatch(i32(table), i32(lens), i32([0, 4, 8, 10 ** 6]), 4, mask, s.n)
    ws = tb.new_tree_workspace(s.cache, batch, 8)
    s.check(*tb.tree_attention(s.q, s.cache, 0, batch, ws, s.scale), sequences=[0, 2])
    batch = tb.DraftBatch(i32(table), i32([100, -7, 33]), i32([0, 4, -3, 12]), 4, mask, s.n)
    s.check(*tb.tree_attention(s.q, s.cache, 0, batch, ws, s.scale), sequences=[0])


def test_cache_past_32_bits_of_elements():
    hkv, d, page, pages = 8, 128, 64, 34000  # 4.5e9 numbers in one layer
    pool = torch.zeros((1, pages, 2, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    s = Step([250, 70], [4, 4], 16, 8, d, page, seed=20, garbage=False)
    used = s.pool.shape[1]
    pool[:, pages - used:] = s.pool
    s.pool, s.table = pool, np.where(s.table >= 0, s.table + pages - used, -1)
    s.check(*s.run())


def test_refusals():
    s = Step([20], [3], 8, 2, 64, 16)
    s.run()
    ws = tb.new_tree_workspace(s.cache, s.batch, 8)
    f = tb.tree_attention
    with pytest.raises(ValueError, match="CUDA tensor"):
        f(s.q.cpu(), s.cache, 0, s.batch, ws)
    with pytest.raises(ValueError, match="shape"):
        f(s.q[:2], s.cache, 0, s.batch, ws)
    with pytest.raises(ValueError, match="dtype"):
        f(s.q.half(), s.cache, 0, s.batch, ws)
    with pytest.raises(ValueError, match="shape"):
        f(s.q, s.cache, 0, s.batch, ws, lse=torch.empty((3, 7), device="cuda"))
    with pytest.raises(tb.TrellisError, match="ESHAPE"):
        f(s.q, s.cache, 1, s.batch, ws)
    with pytest.raises(tb.TrellisError, match="ESHAPE"):  # 7 query heads over 2
        f(s.q[:, :7].contiguous(), s.cache, 0, s.batch, ws)
    with pytest.raises(tb.TrellisError, match="ESHAPE"):
        f(s.q, s.cache, 0, s.batch, ws, scale=float("inf"))
    with pytest.raises(tb.TrellisError, match="EWORKSPACE"):
        f(s.q, s.cache, 0, s.batch, ws[:64].contiguous())
    b = s.batch
    with pytest.raises(tb.TrellisError, match="EM"):
        f(s.q, s.cache, 0, tb.DraftBatch(b.table, b.prefix, b.q_start, 65, b.mask), ws)
    with pytest.raises(ValueError, match="n is needed"):
        tb.DraftBatch(b.table, b.prefix, b.q_start, 3)
    with pytest.raises(ValueError, match="shape"):
        tb.DraftBatch(b.table, b.prefix, b.q_start[:1].contiguous(), 3, b.mask)
    with pytest.raises(ValueError, match="dtype"):
        tb.DraftBatch(b.table, b.prefix.long(), b.q_start, 3, b.mask)
    assert f(s.q[:0], s.cache, 0, tb.DraftBatch(b.table[:0], b.prefix[:0], b.q_start[:1].contiguous(), 3, b.mask[:0]), ws)[0].numel() == 0


def test_bounded_waits_run_out_and_the_next_call_is_right():
    # a cache larger than L2 and few rows: the loads are what the warps wait for
    s = Step([60000, 300], [2, 4], 16, 8, 128, 64, seed=21)
    want = [t.clone() for t in s.run()]
    assert tb.device_error(reset=True) == 0
    tb.set_wait_limit(200)
    try:
        s.run()
        torch.cuda.synchronize()
        assert tb.device_error(reset=True) != 0
    finally:
        tb.set_wait_limit(0)
    got = s.run()
    assert tb.device_error(reset=True) == 0 and all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("hq,hkv,d,toks,f8", [(32, 8, 128, 8, False), (16, 4, 64, 12, False), (40, 2, 128, 12, False),
                                               (16, 2, 256, 4, True), (16, 2, 256, 9, False), (40, 4, 128, 12, True), (16, 2, 64, 20, True)])
def test_many_items_per_block_in_repeated_calls(hq, hkv, d, toks, f8):
    """Rings of tiles that go through many items, of one and of two streams' rows, in both orders."""
    rng = np.random.default_rng(d + toks)
    lens = [int(x) for x in rng.integers(0, 1500, 70)]
    counts = [int(x) for x in rng.integers(1, toks + 1, 70)]
    s = Step(lens, counts, hq, hkv, d, 64, f8, seed=22)
    first = [t.clone() for t in s.run()]
    s.check(*first, sequences=range(0, 70, 3))
    for _ in range(20):
        got = s.run()
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    assert tb.device_error() == 0


@pytest.mark.parametrize("f8", [False, True])
def test_bounded_waits_run_out_with_many_rows(f8):
    s = Step([60000, 300], [16, 4], 32, 8, 128, 64, f8, seed=23)
    want = [t.clone() for t in s.run()]
    assert tb.device_error(reset=True) == 0
    tb.set_wait_limit(200)
    try:
        s.run()
        torch.cuda.synchronize()
        assert tb.device_error(reset=True) != 0
    finally:
        tb.set_wait_limit(0)
    got = s.run()
    assert tb.device_error(reset=True) == 0 and all(torch.equal(a, b) for a, b in zip(want, got))
