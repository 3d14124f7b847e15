"""The calls of a prompt step without a GPU: argument errors return their status before any launch, counts of zero are no error."""
import ctypes

import pytest

from test_serving_abi_cpu import A, EALIGN, EM, ENULL, ESHAPE, EWS, cache, drafts
from trellis_coded_weight_gb300 import binding as tb
from trellis_coded_weight_gb300 import build as tbuild


@pytest.fixture(scope="module")
def lib():
    tbuild.build()
    return tb._serving_lib()


def prompts(**kw):
    return drafts(**{"mask": None, **kw})


def attention(lib, c=None, d=None, layer=0, hq=16, scale=0.1, stride=2048, ws=A, ws_bytes=1 << 40, **kw):
    a = dict(q=A, out=2 * A, lse=A)
    a.update(kw)
    return lib.trellis_prompt_attention(a["q"], stride, ctypes.byref(c or cache()), layer, ctypes.byref(d or prompts()), hq, scale,
                                        a["out"], stride, a["lse"], ws, ws_bytes, None)


def test_prompt_attention_errors_before_launch(lib):
    assert attention(lib, d=prompts(batch=0)) == 0 and attention(lib, d=prompts(n=0)) == 0
    assert attention(lib, d=prompts(mask=A)) == ESHAPE
    for kw in (dict(batch=-1), dict(batch=1025), dict(n=-1), dict(n=(1 << 20) + 1), dict(max_tokens=0), dict(max_tokens=(1 << 20) + 1)):
        assert attention(lib, d=prompts(**kw)) == EM, kw
    assert attention(lib, layer=5) == ESHAPE and attention(lib, layer=-1) == ESHAPE
    assert attention(lib, hq=12) == ESHAPE and attention(lib, hq=0) == ESHAPE and attention(lib, hq=1032) == ESHAPE
    assert attention(lib, scale=float("nan")) == ESHAPE and attention(lib, scale=float("inf")) == ESHAPE
    assert attention(lib, d=prompts(width=0)) == ESHAPE and attention(lib, d=prompts(width=1 << 27)) == ESHAPE
    assert attention(lib, stride=2040) == ESHAPE and attention(lib, stride=2052) == ESHAPE
    for kw in (dict(table=None), dict(prefix=None), dict(q_start=None)):
        assert attention(lib, d=prompts(**kw)) == ENULL
    for kw in (dict(table=A + 4), dict(prefix=A + 4), dict(q_start=A + 8)):
        assert attention(lib, d=prompts(**kw)) == EALIGN
    assert attention(lib, q=None) == ENULL and attention(lib, out=None) == ENULL
    assert attention(lib, out=A) == ESHAPE  # out over q
    assert attention(lib, q=A + 2) == EALIGN and attention(lib, out=A + 4) == EALIGN and attention(lib, lse=A + 4) == EALIGN
    assert attention(lib, c=cache(head_dim=96)) == ESHAPE and attention(lib, c=cache(pool=None)) == ENULL
    size = lambda c, hq: lib.trellis_prompt_workspace_bytes(ctypes.byref(c), hq)  # noqa: E731
    assert size(cache(), 12) == 0 and size(cache(), 0) == 0 and size(cache(page_size=8), 16) == 0 and size(cache(), 16) > 0


def adapters(**kw):
    base = dict(a=A, b=A, ranks=A, scales=A, in_=256, out=512, count=4, max_rank=16)
    base.update(kw)
    return tb.TrellisAdapters(*[base[n] for n, _ in tb.TrellisAdapters._fields_])


def add(lib, ad=None, strides=(256, 512, 512), plan=A, plan_bytes=1 << 30, batch=2, n=6, **kw):
    a = dict(x=A, y=A, out=2 * A)
    a.update(kw)
    return lib.trellis_adapter_add(a["x"], strides[0], a["y"], strides[1], a["out"], strides[2], ctypes.byref(ad or adapters()),
                                   plan, plan_bytes, batch, n, None)


def test_adapter_add_errors_before_launch(lib):
    assert add(lib, batch=0) == 0 and add(lib, n=0) == 0
    for kw in (dict(batch=-1), dict(batch=1025), dict(n=-1), dict(n=(1 << 20) + 1)):
        assert add(lib, **kw) == EM, kw
    for kw in (dict(in_=0), dict(in_=260), dict(in_=(1 << 20) + 8), dict(out=4), dict(out=516), dict(count=0), dict(count=(1 << 16) + 1),
               dict(max_rank=0), dict(max_rank=12), dict(max_rank=136)):
        assert add(lib, ad=adapters(**kw)) == ESHAPE, kw
    for strides in ((248, 512, 512), (256, 504, 512), (256, 512, 504), (260, 512, 512), (256, 516, 512), (256, 512, 516)):
        assert add(lib, strides=strides) == ESHAPE, strides
    assert add(lib, strides=(256, 512, 520), out=A) == ESHAPE  # in place with another stride
    assert add(lib, ad=adapters(in_=512), strides=(512, 512, 512), x=2 * A) == ESHAPE  # out over x
    for name in ("x", "y", "out"):
        assert add(lib, **{name: None}) == ENULL
        assert add(lib, **{name: A + 4}) == EALIGN
    for name in ("a", "b"):
        assert add(lib, ad=adapters(**{name: None})) == ENULL
    for name in ("a", "b", "ranks", "scales"):
        assert add(lib, ad=adapters(**{name: A + 8})) == EALIGN
    need = lib.trellis_adapter_plan_bytes(2, 6)
    assert add(lib, plan=None) == EWS and add(lib, plan=A + 4) == EWS and add(lib, plan_bytes=need - 16) == EWS
    assert lib.trellis_adapter_add(A, 256, A, 512, A, 512, None, A, 1 << 30, 2, 6, None) == ENULL


def test_adapter_plan_errors_before_launch(lib):
    plan = lambda ad=A, qs=A, batch=2, n=6, w=A, size=1 << 30: lib.trellis_adapter_plan(ad, qs, batch, n, w, size, None)  # noqa: E731
    assert plan(batch=0) == 0 and plan(n=0) == 0
    assert plan(batch=-1) == EM and plan(batch=1025) == EM and plan(n=-1) == EM and plan(n=(1 << 20) + 1) == EM
    assert plan(ad=None) == ENULL and plan(qs=None) == ENULL and plan(ad=A + 4) == EALIGN and plan(qs=A + 8) == EALIGN
    need = lib.trellis_adapter_plan_bytes(2, 6)
    assert plan(w=None) == EWS and plan(w=A + 8) == EWS and plan(size=need - 16) == EWS
    assert lib.trellis_adapter_plan_bytes(0, 6) == 0 and lib.trellis_adapter_plan_bytes(2, 0) == 0
    assert lib.trellis_adapter_plan_bytes(1025, 6) == 0 and lib.trellis_adapter_plan_bytes(1024, 1 << 20) > 0


def test_mirrors_have_the_size_of_the_structs():
    assert ctypes.sizeof(tb.TrellisAdapters) == 4 * 8 + 2 * 8 + 2 * 4
