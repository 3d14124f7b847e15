"""trellis_tree_attention at the edges of its numbers: keys that are not numbers among what a token sees, queries and scales at the
ends of their ranges, query rows with one channel far above the others.

Where results are finite the tolerances are those of test_tree_attention_gpu.py, derived there from the roundings: Step.check
applies them.  Shapes go through each kernel: up to 16 rows of a key/value head (heads of 64 and 128), more (256 rows a block:
bf16 of those; 128 rows a block: e4m3 of those and heads of 256)."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from test_tree_attention_gpu import Step
from trellis_coded_weight_gb300 import binding as tb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from trellis_coded_weight_gb300 import build
    build.build()
    tb.load()


# query heads, key/value heads, head dim, e4m3 cache, drafts: rows of a key/value head are drafts * query heads / heads
KERNELS = [(4, 2, 64, False, 3), (4, 2, 128, False, 3), (4, 2, 128, True, 3), (4, 2, 64, True, 3),   # up to 16 rows
           (8, 2, 64, False, 9), (8, 2, 128, False, 9), (16, 1, 128, False, 12),                    # 36 and 192 rows, bf16
           (8, 2, 64, True, 9), (8, 2, 128, True, 9), (4, 2, 256, True, 3), (4, 2, 256, False, 3)]  # 128 rows a block


def put(s, b, positions, kv, value, dims=slice(None)):
    """Bits of keys (0) or values (1) of sequence b at some positions, all heads."""
    raw = s.pool.view(torch.uint8 if s.scales is not None else torch.int16)
    for p in positions:
        raw[s.layer, int(s.table[b, p // s.page]), kv, :, p % s.page, dims] = value


@pytest.mark.parametrize("hq,hkv,d,f8,toks", KERNELS)
@pytest.mark.parametrize("prefix,keys", [(0, "own"), (100, "first tile"), (300, "one"), (20000, "one"), (40, "all")])
def test_keys_that_are_not_numbers_make_rows_that_see_them_so(prefix, keys, hq, hkv, d, f8, toks):
    s = Step([prefix, 50], [toks, toks], hq, hkv, d, 64, f8, seed=prefix + d, masks="chain")
    nan = 0x7F if f8 else 0x7FC0
    # a draft's own key alone; the keys of a tile of 64, before one without; one key of the prefix; every key
    at = {"own": [prefix], "first tile": range(64), "one": [prefix // 3], "all": range(prefix + toks)}[keys]
    put(s, 0, at, 0, nan)
    out, lse = s.run()
    # chains of drafts: all of them see the first one, and the prefix
    assert out[:toks].isnan().all() and lse[:toks].isnan().all()
    s.check(out, lse, sequences=[1])


@pytest.mark.parametrize("hq,hkv,d,f8,toks", KERNELS)
def test_rows_that_do_not_see_such_keys_keep_their_results(hq, hkv, d, f8, toks):
    s = Step([0, 70], [toks, toks], hq, hkv, d, 64, f8, seed=5, masks="chain")
    for b in (0, 1):
        put(s, b, [s.lens[b] + 1], 0, 0x7F if f8 else 0x7FC0)
        for i in range(0, toks, 2):  # every other draft does not see it
            s.masks[b * toks + i] &= ~2
    out, lse = s.run()
    sees = torch.tensor([m >> 1 & 1 for m in s.masks], device="cuda").bool()
    assert out[sees].isnan().all() and lse[sees].isnan().all() and out[~sees].isfinite().all()
    put(s, 0, [1], 0, 0)
    put(s, 1, [71], 0, 0)
    want, want_lse = s.run()
    assert torch.equal(out[~sees], want[~sees]) and torch.equal(lse[~sees], want_lse[~sees])


@pytest.mark.parametrize("hq,hkv,d,f8,toks", [k for k in KERNELS if k[3]])
@pytest.mark.parametrize("largest,scale", [((126, 127), 2e-38), ((-126, -128), 2e38)])
def test_e4m3_queries_at_the_ends_of_their_range(largest, scale, hq, hkv, d, f8, toks):
    # rows whose largest number has the largest two exponents of bf16, or its smallest normal one and a subnormal one
    s = Step([70], [toks], hq, hkv, d, 64, f8, seed=d + toks)
    s.scales *= 0.1
    q = s.q.float()
    q /= q.abs().amax(-1, keepdim=True)
    of = torch.where(torch.arange(toks, device="cuda") % 2 == 0, 1.5 * 2.0 ** largest[0], 1.5 * 2.0 ** largest[1]).float()
    s.q, s.scale = (q * of[:, None, None]).bfloat16(), scale
    assert s.q.isfinite().all() and (s.q != 0).any(-1).all()
    s.check(*s.run())


@pytest.mark.parametrize("hq,hkv,d,f8,toks", KERNELS)
def test_zero_queries_weigh_all_alike(hq, hkv, d, f8, toks):
    s = Step([70], [toks], hq, hkv, d, 64, f8, seed=d + toks)
    s.q = torch.zeros_like(s.q)
    s.check(*s.run())


@pytest.mark.parametrize("hq,hkv,d,f8,toks", KERNELS)
def test_small_scales_of_large_queries(hq, hkv, d, f8, toks):
    # scores of about one from queries of 1e36 (their products with the keys stay below the largest number of fp32)
    s = Step([300, 5], [toks, toks], hq, hkv, d, 64, f8, seed=d + toks, std=1e36)
    s.scale = 4e-38
    s.check(*s.run())


@pytest.mark.parametrize("hq,hkv,d,f8,toks", KERNELS)
def test_a_scale_of_zero_weighs_all_alike(hq, hkv, d, f8, toks):
    s = Step([300, 5], [toks, toks], hq, hkv, d, 64, f8, seed=d + toks, masks="random")
    s.scale = 0.0
    s.check(*s.run())


@pytest.mark.parametrize("hq,hkv,d,f8,toks", [k for k in KERNELS if k[3]])
def test_a_cache_scale_that_is_no_number(hq, hkv, d, f8, toks):
    # keys of the first head: its queries' results are NaN, the other heads' are what they were
    s = Step([70], [toks], hq, hkv, d, 64, f8, seed=d + toks)
    want, want_lse = s.run()
    s.scales[0, 0, 0] = float("nan")
    out, lse = s.run()
    mine = hq // hkv
    assert out[:, :mine].isnan().all() and lse[:, :mine].isnan().all()
    assert torch.equal(out[:, mine:], want[:, mine:]) and torch.equal(lse[:, mine:], want_lse[:, mine:])


@pytest.mark.parametrize("hq,hkv,d,f8,toks", KERNELS)
@pytest.mark.parametrize("times", [2.0 ** 6, 2.0 ** 10, 2.0 ** 14])
def test_query_rows_with_one_channel_far_above_the_others(times, hq, hkv, d, f8, toks):
    # in every row another one; the others' part of a score is what separates the keys for which the large one's is alike
    s = Step([600, 30], [toks, toks], hq, hkv, d, 64, f8, seed=d + toks)
    q = s.q.float()
    row = torch.arange(s.n * hq, device="cuda").view(s.n, hq, 1)
    q.scatter_(2, row * 7 % d, torch.where(row % 2 == 0, times, -times))
    s.q = q.bfloat16()
    s.check(*s.run())
