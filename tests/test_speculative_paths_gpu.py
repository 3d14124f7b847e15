"""Trees of drafts against single tokens, number by number: both ways of the example are fed the same continuation, and the log
probabilities after every one of its tokens are compared, whatever alternatives come first.

Tolerance: that of the example's own test, 0.1 on log probabilities, for both kinds of cache.  The two ways multiply the same
bf16 numbers in other orders, and both round their logits to bf16 at the end.  Another context gives another row of logits: half
of the differences between neighbouring tokens' numbers are above 0.18 here, so a mask, position or page at fault moves many of the
288 numbers compared by more than the tolerance."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from trellis_coded_weight_gb300 import binding as tb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from trellis_coded_weight_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "speculative_decode.py")
    spec = importlib.util.spec_from_file_location("speculative_decode", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def feed(example, seqs, model, row, tokens, parents, path):
    """One step of one sequence with the given tree, of which the drafts `path` are kept: their log probabilities."""
    seqs.fork([row], [row], len(tokens))
    toks, positions, slots, batch = seqs.batch([row], [(tokens, parents)])
    got = model(toks, positions, slots, batch)
    seqs.commit([row], [path], batch)
    at = torch.tensor(path, device="cuda")
    return torch.cat([got.logprobs[at], got.lse[at, None], got.top_logprobs[at]], 1).double().cpu().numpy(), got.top_ids[at].cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_every_accepted_draft_has_the_numbers_of_a_single_token(example, dtype):
    model = example.Model(dtype)
    seqs = example.Sequences(model.cache)
    rng = np.random.default_rng(8)
    prompt, known = rng.integers(0, example.VOCAB, 70).tolist(), rng.integers(0, example.VOCAB, 48).tolist()
    for row in (0, 1):
        for at in range(0, 70, example.MOST):
            example.step(model, seqs, row, prompt[at:at + example.MOST])
    want, want_ids = (np.concatenate(x) for x in zip(*(feed(example, seqs, model, 0, [t], [-1], [0]) for t in known)))
    got, got_ids, at, steps = [], [], 0, 0
    while at < len(known):
        # the known tokens in a chain, each with a sibling before it that is not kept, so that kept drafts move and masks have holes
        n = min(int(rng.integers(1, 7)), len(known) - at)
        tokens, parents, path = [], [], []
        for i in range(n):
            last = path[-1] if path else -1
            for t in (int(rng.integers(example.VOCAB)), known[at + i]):
                tokens.append(t)
                parents.append(last)
            path.append(len(tokens) - 1)
        a, b = feed(example, seqs, model, 1, tokens, parents, path)
        got.append(a)
        got_ids.append(b)
        at, steps = at + n, steps + 1
    got, got_ids = np.concatenate(got), np.concatenate(got_ids)
    assert steps < len(known) // 2 and got.shape == want.shape == (48, 6)
    assert np.abs(got - want).max() < 0.1, np.abs(got - want).max()
    clear = want[:, 2] - want[:, 3] > 0.2  # the best alternative leads by more than both can be off
    assert np.array_equal(got_ids[clear, 0], want_ids[clear, 0])
    assert seqs.lens.tolist()[:2] == [118, 118]
