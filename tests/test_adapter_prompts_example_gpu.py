"""The example that runs the calls of a prompt step together: packed prompts with adapters of their own give the continuations
that each gives alone, whole or in chunks that the tree attention takes.

The ways multiply the same bf16 numbers in other orders and tiles, so a step's log probabilities agree to a few of bf16's half
units (2^-9 of logits of a few units: 0.1 with room), as long as the tokens before them are the same."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from trellis_coded_weight_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "adapter_prompts.py")
    spec = importlib.util.spec_from_file_location("adapter_prompts", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_requests_together_are_what_they_are_alone(example, dtype):
    r = example.run(dtype)
    tokens, lp = r["together"]
    assert lp.isfinite().all()
    for i in range(len(r["prompts"])):
        for other in (r["alone"][i], r["chunks"][i]):
            for s in range(len(tokens)):
                mine = lp[s, i]
                assert (mine - other[1][s, 0]).abs().max() < 0.1, (i, s)
                if tokens[s][i] != other[0][s][0]:
                    assert mine[0] - mine[1] < 0.1  # two tokens equally likely; what follows differs
                    break
    # another adapter gives another first step, and the request without one keeps its own
    _, changed = r["others"]
    assert (changed[0, 0] - lp[0, 0]).abs().max() > 0.1 and (changed[0, 2] - lp[0, 2]).abs().max() > 0.1
    assert (changed[0, 1] - lp[0, 1]).abs().max() < 0.1


def test_prompts_in_chunks_together_are_what_they_are_whole(example):
    """Prompts of different lengths end in different chunks' steps; each is continued from its own last token's results."""
    model = example.Model()
    g = torch.Generator().manual_seed(6)
    prompts = [torch.randint(0, example.VOCAB, (n,), generator=g).tolist() for n in (150, 67, 211)]
    tokens, lp = example.generate(model, prompts, [1, -1, 2], 4)
    parts, parts_lp = example.generate(model, prompts, [1, -1, 2], 4, chunk=64)
    assert lp.shape == parts_lp.shape
    for i in range(len(prompts)):
        for s in range(len(tokens)):
            assert (lp[s, i] - parts_lp[s, i]).abs().max() < 0.1, (i, s)
            if tokens[s][i] != parts[s][i]:
                assert lp[s, i, 0] - lp[s, i, 1] < 0.1
                break
