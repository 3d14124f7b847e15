"""The example that runs the serving calls together: verified drafts give the continuation of single tokens.

The two ways multiply the same bf16 numbers in other orders (single tokens and trees take other tiles), so a step's log
probabilities agree to a few of bf16's half units (2^-9 of logits of a few units: 0.1 with room).  The continuations are the
same up to the first token whose two best alternatives lie closer than that."""
import importlib.util
import os

import numpy as np
import pytest
import torch

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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_drafts_give_the_continuation_of_single_tokens(example, dtype):
    r = example.run(dtype)
    plain, spec = r["plain"], r["spec"]
    differ = [i for i, (a, b) in enumerate(zip(plain, spec)) if a != b]
    if differ:
        i = differ[0]  # chosen by the step before
        assert i > 0 and r["margins"][i - 1] < 0.1, (i, r["margins"][i - 1])
    assert len(r["accepted"]) < len(spec)
    # the forked row is the same sequence, and compaction moves pages without touching a number
    n = r["before"].lse.shape[0]
    for a, b in zip(r["before"], r["after"]):
        assert torch.equal(a, b)
        assert torch.equal(a[:n // 2], a[n // 2:])
    refs = r["seqs"].refs.cpu().numpy()
    live = int((refs > 0).sum())
    assert np.all(refs[:live] > 0) and np.all(refs[live:] == 0)
    table, lens = r["seqs"].table.cpu().numpy(), r["seqs"].lens.cpu().numpy()
    assert lens[1] == lens[2] == 90 + len(spec) and lens[0] == 0 and np.all(table[0] == -1)
    full = lens[1] // example.PAGE
    assert np.array_equal(table[1, :full], table[2, :full]) and not np.array_equal(table[1], table[2])
    assert np.all(refs[table[1, :full]] == 2)
