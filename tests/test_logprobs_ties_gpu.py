"""trellis_token_logprobs on rows with more numbers at the threshold of the alternatives than a block can list: the ones above
it are counted first, then equal ones are added in the order of their columns.  Indices and log probabilities have to be
those of the 64-bit definition, in every one of many calls (the count is shared by the threads of a block)."""
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


def rows_with(above, vocab, per_group, seed):
    """Rows of equal numbers but for above[r] larger ones, all in columns of the first eight of a block's 64 groups of
    threads (per_group columns each, again every 64 groups): fewer groups than alternatives, so that the threshold is the
    equal number itself."""
    rng = np.random.default_rng(seed)
    cols = np.arange(vocab)
    cols = cols[cols % (64 * per_group) < 8 * per_group]
    x = np.full((len(above), vocab), -1.5)
    for r, a in enumerate(above):
        at = rng.permutation(cols)[:a]
        x[r, at] = rng.integers(1, 40, a) / 8  # exact in bf16, with ties among them
    return x


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("top", [9, 20, 32])
def test_numbers_above_a_threshold_that_many_equal(top, bf16):
    # 700 rows: one block each (a part of a row would not hold so many); above 512 the block takes turns instead of a list
    above = [1, 2, 3, top - 1, top, top + 1, 31, 63, 100, 255, 256, 257, 400, 505, 510, 511, 512, 513, 700, 0]
    above = (above * 35)[:700]
    x64 = rows_with(above, 20000, 32 if bf16 else 16, top)
    x = torch.as_tensor(x64).to(torch.bfloat16 if bf16 else torch.float32).cuda()
    tokens = torch.zeros((700, 1), dtype=torch.int32, device="cuda")
    ws = tb.new_logprobs_workspace(700, 20000, top, "cuda")
    first = [t.clone() for t in tb.token_logprobs(x, tokens, top, ws)]
    lp, lse, ent, ids, tlp = ref.logprobs(x64[:40], np.zeros((40, 1), int), top, 1.0)
    # sums of 20000 exponentials in fp32, as in the other tests of this call: 7e-5 absolutely
    assert np.array_equal(first[3][:40].cpu().numpy(), ids)
    assert np.abs(ref.f64(first[4][:40]) - tlp).max() < 7e-5 and np.abs(ref.f64(first[1][:40]) - lse).max() < 7e-5
    for _ in range(30):
        got = tb.token_logprobs(x, tokens, top, ws)
        assert all(torch.equal(a, b) for a, b in zip(first, got))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("n,vocab", [(1, 9001), (1, 151936), (700, 2500)])
def test_rows_of_nan_alone(n, vocab, bf16):
    # every number orders before all others and is equal to the rest: the first columns, column 0 too
    x = torch.full((n, vocab), float("nan"), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    x[n // 2, vocab - 1] = 1.0
    tokens = torch.zeros((n, 1), dtype=torch.int32, device="cuda")
    got = tb.token_logprobs(x, tokens, 20, tb.new_logprobs_workspace(n, vocab, 20, "cuda"))
    assert got.top_ids.tolist() == [list(range(20))] * n
    assert all(t.isnan().all() for t in (got.logprobs, got.lse, got.entropy, got.top_logprobs))
