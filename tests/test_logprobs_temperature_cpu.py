"""trellis_token_logprobs refuses temperatures whose factor log2(e) / temperature is not finite: differences of logits times it
would not be numbers."""
import ctypes

import pytest

from trellis_coded_weight_gb300 import binding as tb
from trellis_coded_weight_gb300 import build as tbuild

A = 1 << 20  # a 16-byte aligned address that is never dereferenced
ESHAPE = -9


@pytest.mark.parametrize("temperature", [3e-39, 4e-39, 4.2e-39])
def test_temperatures_too_small_for_their_factor(temperature):
    tbuild.build()
    lib = tb._serving_lib()
    assert ctypes.c_float(1.0 / temperature).value < float("inf")  # the reciprocal alone is finite
    need = lib.trellis_logprobs_workspace_bytes(3, 1000, 5)
    got = lib.trellis_token_logprobs(A, 0, 1000, A, 3, 1000, 2, 5, temperature, A, A, A, A, A, A, need, None)
    assert got == ESHAPE
