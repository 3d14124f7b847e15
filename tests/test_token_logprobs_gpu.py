"""trellis_token_logprobs against the 64-bit definition.

Tolerance: a sum of V exponentials (2^-22 each) in chains of at most 1024 fp32 additions per thread is within
1024 * 2^-24 = 6.1e-5 of its value, so logarithms are within 7e-5 absolutely; c = log2(e) / t and the products with it
are within 2 * 2^-24 of their size, allowed 2^-21 of the row's range over t.  The entropy's two sums: 2e-4 absolutely.
Indices have to be equal."""
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


def check(x, tokens, top, temp, ws=None, out=None):
    n, vocab = x.shape
    ws = tb.new_logprobs_workspace(max(1, n), vocab, top, "cuda") if ws is None else ws
    got = tb.token_logprobs(x, tokens, top, ws, temp, out)
    x64 = ref.f64(x)
    lp, lse, ent, ids, tlp = ref.logprobs(x64, tokens.cpu().numpy(), top, temp)
    assert np.array_equal(got.top_ids.cpu().numpy(), ids)
    fin = np.where(np.isfinite(x64), x64, 0)
    span = (np.abs(fin).max(1) * 2 / temp if vocab else np.zeros(n))
    for name, g, w, t in (("logprobs", got.logprobs, lp, 7e-5), ("top", got.top_logprobs, tlp, 7e-5),
                          ("lse", got.lse[:, None], lse[:, None], 7e-5), ("entropy", got.entropy[:, None], ent[:, None], 2e-4)):
        g = ref.f64(g)
        fine = np.isfinite(w)
        assert np.array_equal(np.isnan(g), np.isnan(w)), name
        assert np.array_equal(g[~fine & ~np.isnan(w)], w[~fine & ~np.isnan(w)]), name
        tol = np.broadcast_to(t + 2.0 ** -21 * span[:, None], w.shape)
        assert np.all(np.abs(g - w)[fine] <= tol[fine]), (name, np.abs(g - w)[fine].max())
    return got


def logits(n, vocab, bf16, seed, std=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, vocab), generator=g, device="cuda") * std
    return x.bfloat16() if bf16 else x


def toks(n, c, vocab, seed=1):
    return torch.randint(0, vocab, (n, c), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").int()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("n,vocab,cands,top,temp", [
    (1, 1, 1, 1, 1.0), (1, 50257, 1, 5, 1.0), (3, 33, 64, 32, 0.5), (2, 32, 2, 32, 1.0), (5, 1001, 3, 1, 2.0),
    (61, 12345, 4, 8, 0.7), (1, 151936, 0, 20, 1.0), (7, 40000, 5, 0, 1.0), (300, 8191, 2, 32, 1.0), (1200, 257, 1, 3, 1.3),
    (2, 8193, 1, 7, 1.0), (4, 4096, 1, 9, 1.0)])
def test_rows(n, vocab, cands, top, temp, bf16):
    check(logits(n, vocab, bf16, n + vocab), toks(n, cands, vocab), top, temp)


@pytest.mark.parametrize("bf16", [True, False])
def test_many_rows(bf16):
    check(logits(70000, 40, bf16, 3), toks(70000, 1, 40), 4, 1.0)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("kind", ["equal", "two values", "rising", "falling", "one group", "steps", "zeros"])
def test_rows_with_many_equal_or_ordered_numbers(kind, bf16):
    vocab = 30011
    i = torch.arange(vocab, device="cuda", dtype=torch.float32)
    x = {"equal": torch.full_like(i, -1.5), "two values": (i % 7 == 3).float(), "rising": i / 4000, "falling": -i / 4000,
         "one group": torch.where((i >= 9000) & (i < 9040), 5 + (i % 13) / 8, i * 0 - 2), "steps": (i // 3000).float(),
         "zeros": torch.where(i % 2 == 0, 0.0, -0.0)}[kind]
    x = torch.stack([x, x.flip(0)])
    for top in (1, 20, 32):
        check(x.bfloat16() if bf16 else x.contiguous(), toks(2, 3, vocab), top, 1.0)


@pytest.mark.parametrize("bf16", [True, False])
def test_infinities_and_nan(bf16):
    x = logits(8, 9001, bf16, 5)
    inf, low = float("inf"), torch.finfo(x.dtype).min
    x[0, 100:] = -inf          # a hundred tokens left
    x[1] = -inf                # none
    x[2] = -inf
    x[2, 8999] = 3.0           # one
    x[3, 4000] = float("nan")
    x[4, 17] = inf
    x[5, ::2] = low            # the type's lowest value in masked places
    x[6] = low
    x[7, 5:] = -inf            # fewer than top_k
    t = toks(8, 6, 9001)
    t[2, 0], t[1, 1], t[0, 2], t[3, 3], t[5, 4] = 8999, -1, 9001, 2 ** 31 - 1, -2 ** 31
    got = check(x, t, 20, 1.0)
    assert got.logprobs[2, 0] == 0 and got.entropy[2] == 0


@pytest.mark.parametrize("bf16", [True, False])
def test_rows_apart_and_unaligned(bf16):
    base = logits(9, 5200, bf16, 8)
    for stride_extra in (0, 1, 3, 8):
        flat = torch.empty(9 * (5001 + stride_extra) + 16, dtype=base.dtype, device="cuda")
        x = flat.as_strided((9, 5001), (5001 + stride_extra, 1))
        x.copy_(base[:, :5001])
        check(x, toks(9, 2, 5001), 11, 1.0)


def test_numbers_outside_a_row_do_not_reach_it():
    flat = torch.full((5 * 1003,), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((5, 1001), (1003, 1))
    x.copy_(logits(5, 1001, True, 2))
    check(x, toks(5, 2, 1001), 6, 1.0)


def test_one_workspace_for_calls_of_any_sizes_and_equal_bits():
    ws = tb.new_logprobs_workspace(600, 60000, 32, "cuda")
    first = None
    for n, vocab, top in ((1, 60000, 32), (600, 3001, 7), (40, 60000, 20), (2, 700, 3), (1, 60000, 32)):
        got = check(logits(n, vocab, True, n), toks(n, 2, vocab), top, 1.0, ws)
        if n == 1:
            if first is not None:
                assert all(torch.equal(a, b) for a, b in zip(first, got))
            first = got


def test_another_stream_given_outputs_and_no_rows():
    x, t = logits(3, 20000, True, 4), toks(3, 2, 20000)
    f = dict(dtype=torch.float32, device="cuda")
    out = (torch.empty((3, 2), **f), torch.empty(3, **f), torch.empty(3, **f), torch.empty((3, 4), dtype=torch.int32, device="cuda"),
           torch.empty((3, 4), **f))
    ws = tb.new_logprobs_workspace(3, 20000, 4, "cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = tb.token_logprobs(x, t, 4, ws, 1.0, out)
    st.synchronize()
    assert got.lse.data_ptr() == out[1].data_ptr()
    torch.cuda.synchronize()
    check(x, t, 4, 1.0, ws, out)
    tb.token_logprobs(x[:0], t[:0], 4, ws)


def test_large_scale_and_small_temperature():
    check(logits(3, 5000, False, 6, std=300.0), toks(3, 2, 5000), 5, 0.05)
    check(logits(3, 5000, False, 7, std=1e-3), toks(3, 2, 5000), 5, 10.0)


def test_rows_past_32_bits_of_elements():
    n, vocab = 5, (1 << 24)
    stride = (1 << 30) + 8
    flat = torch.zeros(4 * stride + vocab, dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((n, vocab), (stride, 1))
    hit = [5, 77, 123456, 1 << 23, vocab - 1]
    for r, c in enumerate(hit):
        x[r, c] = 30.0
    ws = tb.new_logprobs_workspace(n, vocab, 2, "cuda")
    got = tb.token_logprobs(x, torch.tensor(hit, device="cuda").int()[:, None], 2, ws)
    assert got.top_ids[:, 0].tolist() == hit and got.top_ids[:, 1].tolist() == [0] * n
    lse = np.log(np.exp(30.0) + vocab - 1)
    assert np.allclose(got.lse.cpu().numpy(), lse, atol=7e-5) and np.allclose(got.logprobs[:, 0].cpu().numpy(), 30 - lse, atol=7e-5)


def test_refusals():
    x, t = logits(2, 100, True, 1), toks(2, 1, 100)
    ws = tb.new_logprobs_workspace(2, 100, 5, "cuda")
    with pytest.raises(ValueError, match="CUDA tensor"):
        tb.token_logprobs(x.cpu(), t, 5, ws)
    with pytest.raises(ValueError, match="dtype"):
        tb.token_logprobs(x.half(), t, 5, ws)
    with pytest.raises(ValueError, match="shape"):
        tb.token_logprobs(x, t[:1], 5, ws)
    with pytest.raises(ValueError, match="contiguous"):
        tb.token_logprobs(x.t().contiguous().t(), t, 5, ws)
    with pytest.raises(ValueError, match="dtype"):
        tb.token_logprobs(x, t.long(), 5, ws)
    for bad in (dict(top_k=33), dict(top_k=5, temperature=0.0), dict(top_k=5, temperature=-1.0),
                dict(top_k=5, temperature=float("nan")), dict(top_k=5, temperature=1e-40)):
        with pytest.raises(tb.TrellisError, match="ESHAPE"):
            tb.token_logprobs(x, t, workspace=ws, **bad)
    with pytest.raises(tb.TrellisError, match="ESHAPE"):  # more alternatives than tokens
        tb.token_logprobs(x[:, :4], t, 5, ws)
    with pytest.raises(tb.TrellisError, match="ESHAPE"):
        tb.token_logprobs(x, toks(2, 65, 100), 5, ws)
    with pytest.raises(tb.TrellisError, match="ESHAPE"):  # rows that overlap
        tb.token_logprobs(x.view(-1).as_strided((2, 100), (50, 1)), t, 5, ws)
    with pytest.raises(tb.TrellisError, match="EWORKSPACE"):
        tb.token_logprobs(x, t, 5, ws[:64].contiguous())
    with pytest.raises(tb.TrellisError, match="EALIGN"):
        tb.token_logprobs(x.view(-1)[1:101].view(1, 100), t[:1], 5, ws)
    with pytest.raises(ValueError, match="unsupported"):
        tb.new_logprobs_workspace(2, 100, 40, "cuda")
