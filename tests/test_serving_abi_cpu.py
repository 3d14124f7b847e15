"""The serving calls without a GPU: argument errors return their status before any launch, counts of zero are no error,
host tensors are refused, and the 64-bit definitions that the GPU tests compare with agree with brute force."""
import ctypes

import numpy as np
import pytest
import torch

import serving_ref as ref
from trellis_coded_weight_gb300 import binding as tb
from trellis_coded_weight_gb300 import build as tbuild

A = 1 << 20  # a 16-byte aligned address that is never dereferenced
EGEOM, EM, EALIGN, EWS, ENULL, ESHAPE = -1, -2, -3, -5, -7, -9


@pytest.fixture(scope="module")
def lib():
    tbuild.build()
    return tb._serving_lib()


def cache(**kw):
    base = dict(pool=A, scales=None, pages=100, layers=2, heads=8, page_size=16, head_dim=128, dtype=0, reserved=0)
    base.update(kw)
    return tb.TrellisCache(*[base[n] for n, _ in tb.TrellisCache._fields_])


def norm(**kw):
    base = dict(q_weight=A, k_weight=A, rope=A, max_pos=10, q_heads=16, kv_heads=8, head_dim=128, rotary_dim=64,
                interleaved=0, reserved=0, eps=1e-6, weight_offset=0.0)
    base.update(kw)
    return tb.TrellisNormRope(*[base[n] for n, _ in tb.TrellisNormRope._fields_])


def drafts(**kw):
    base = dict(table=A, prefix=A, q_start=A, mask=A, batch=2, width=8, n=6, max_tokens=4)
    base.update(kw)
    return tb.TrellisDrafts(*[base[n] for n, _ in tb.TrellisDrafts._fields_])


@pytest.mark.parametrize("kw,st", [
    ({}, 0), (dict(dtype=1), 0), (dict(dtype=1, scales=A), 0), (dict(pool=None), ENULL), (dict(scales=A), ESHAPE),
    (dict(page_size=8), ESHAPE), (dict(page_size=48), ESHAPE), (dict(page_size=256), ESHAPE), (dict(head_dim=96), ESHAPE),
    (dict(dtype=2), ESHAPE), (dict(pages=0), ESHAPE), (dict(pages=(1 << 24) + 1), ESHAPE), (dict(layers=0), ESHAPE),
    (dict(heads=0), ESHAPE), (dict(heads=1024, pages=1 << 20), ESHAPE), (dict(reserved=1), ESHAPE), (dict(pool=A + 8), EALIGN)])
def test_cache_rules(lib, kw, st):
    assert lib.trellis_check_cache(ctypes.byref(cache(**kw))) == st


def norm_rope(lib, c=None, p=None, n=3, layer=0, strides=(2048, 1024, 1024, 2048), **kw):
    a = dict(q=A, k=A, v=A, pos=A, slots=A, out=A)
    a.update(kw)
    return lib.trellis_qk_norm_rope_append(a["q"], strides[0], a["k"], strides[1], a["v"], strides[2], a["pos"], a["slots"], a["out"],
                                           strides[3], n, ctypes.byref(p or norm()), ctypes.byref(c or cache()), layer, None)


def test_norm_rope_errors_before_launch(lib):
    assert norm_rope(lib, n=0) == 0
    assert norm_rope(lib, n=-1) == EM
    assert norm_rope(lib, layer=2) == ESHAPE and norm_rope(lib, layer=-1) == ESHAPE
    for kw in (dict(kv_heads=4), dict(head_dim=64), dict(rotary_dim=136), dict(rotary_dim=24), dict(interleaved=2), dict(reserved=3),
               dict(q_heads=0), dict(max_pos=-1), dict(eps=float("nan")), dict(eps=-1.0), dict(weight_offset=float("inf"))):
        assert norm_rope(lib, p=norm(**kw)) == ESHAPE, kw
    for strides in ((2047, 1024, 1024, 2048), (2048, 1028, 1024, 2048), (2048, 1024, 512, 2048), (2048, 1024, 1024, 8)):
        assert norm_rope(lib, strides=strides) == ESHAPE
    for name in ("q", "k", "v", "pos", "slots", "out"):
        assert norm_rope(lib, **{name: None}) == ENULL
        assert norm_rope(lib, **{name: A + 2}) == EALIGN
    assert norm_rope(lib, p=norm(rope=None)) == ENULL and norm_rope(lib, p=norm(q_weight=None)) == ENULL
    assert norm_rope(lib, c=cache(page_size=20)) == ESHAPE


def attention(lib, c=None, d=None, layer=0, hq=16, scale=0.1, stride=2048, ws=A, ws_bytes=1 << 30, **kw):
    a = dict(q=A, out=A, lse=A)
    a.update(kw)
    return lib.trellis_tree_attention(a["q"], stride, ctypes.byref(c or cache()), layer, ctypes.byref(d or drafts()), hq, scale,
                                      a["out"], stride, a["lse"], ws, ws_bytes, None)


def test_tree_attention_errors_before_launch(lib):
    assert attention(lib, d=drafts(batch=0)) == 0 and attention(lib, d=drafts(n=0)) == 0
    for kw in (dict(batch=-1), dict(batch=1025), dict(n=-1), dict(max_tokens=0), dict(max_tokens=65)):
        assert attention(lib, d=drafts(**kw)) == EM, kw
    assert attention(lib, layer=5) == ESHAPE and attention(lib, hq=12) == ESHAPE and attention(lib, hq=0) == ESHAPE
    assert attention(lib, scale=float("nan")) == ESHAPE
    assert attention(lib, d=drafts(width=0)) == ESHAPE and attention(lib, d=drafts(width=1 << 27)) == ESHAPE
    assert attention(lib, d=drafts(batch=1024, width=1 << 22, max_tokens=64)) == ESHAPE  # steps past 32 bits
    assert attention(lib, stride=2040) == ESHAPE and attention(lib, stride=2052) == ESHAPE
    for kw in (dict(table=None), dict(prefix=None), dict(q_start=None)):
        assert attention(lib, d=drafts(**kw)) == ENULL
    assert attention(lib, q=None) == ENULL and attention(lib, out=A + 4) == EALIGN
    assert lib.trellis_tree_workspace_bytes(ctypes.byref(cache()), 2, 65, 16) == 0
    assert lib.trellis_tree_workspace_bytes(ctypes.byref(cache()), 2, 4, 12) == 0
    assert lib.trellis_tree_workspace_bytes(ctypes.byref(cache()), 2, 4, 16) > 0


def test_page_calls_errors_before_launch(lib):
    c, i = ctypes.byref(cache()), [A] * 6
    need = lib.trellis_cache_workspace_bytes(c, 4, 8)
    fork = lambda p=i, pairs=4, rows=5, width=8, room=0, w=A, n=need, cc=c: lib.trellis_cache_fork(cc, *p, pairs, rows, width, room, w, n, None)  # noqa: E731
    assert fork(pairs=0) == 0 and fork(pairs=-1) == EM and fork(pairs=1025) == EM
    assert fork(rows=0) == ESHAPE and fork(width=0) == ESHAPE and fork(room=-1) == ESHAPE
    assert fork(w=None) == EWS and fork(n=need - 4) == EWS and fork(w=A + 4) == EWS
    for k in range(6):
        assert fork(p=i[:k] + [None] + i[k + 1:]) == ENULL
        assert fork(p=i[:k] + [A + 4] + i[k + 1:]) == EALIGN
    assert fork(cc=ctypes.byref(cache(head_dim=32))) == ESHAPE
    assert lib.trellis_cache_compact(c, A, None, A, A, 4, 8, A, need, None) == ENULL
    assert lib.trellis_cache_compact(c, A, A, A, A, 0, 8, A, need, None) == ESHAPE
    assert lib.trellis_cache_compact(c, A, A, A, A, 4, 8, A, 16, None) == EWS
    assert lib.trellis_cache_commit(c, A, A, A, A, A, 0, 8, 4, None) == 0
    assert lib.trellis_cache_commit(c, A, A, A, A, A, 2, 8, 65, None) == EM
    assert lib.trellis_cache_commit(c, A, A, A, A, None, 2, 8, 4, None) == ENULL
    assert lib.trellis_cache_copy(c, A, A, 0, None) == 0 and lib.trellis_cache_copy(c, A, A, -1, None) == EM
    assert lib.trellis_cache_copy(c, None, A, 1, None) == ENULL
    assert lib.trellis_cache_workspace_bytes(c, 1025, 8) == 0


def test_logprobs_errors_before_launch(lib):
    need = lib.trellis_logprobs_workspace_bytes(3, 1000, 5)

    def call(logits=A, dtype=0, stride=1000, tokens=A, n=3, vocab=1000, cands=2, top=5, temp=1.0, outs=(A,) * 5, ws=A, size=need):
        return lib.trellis_token_logprobs(logits, dtype, stride, tokens, n, vocab, cands, top, temp, *outs, ws, size, None)

    assert call(n=0) == 0 and call(n=-1) == EM
    for kw in (dict(dtype=1), dict(vocab=0), dict(cands=65), dict(cands=-1), dict(top=33), dict(top=-1), dict(vocab=4, top=5),
               dict(temp=0.0), dict(temp=float("nan")), dict(temp=float("inf")), dict(temp=1e-39), dict(stride=999)):
        assert call(**kw) == ESHAPE, kw
    assert call(tokens=None) == ENULL and call(logits=None) == ENULL and call(outs=(A, A, A, None, A)) == ENULL
    assert call(logits=A + 2) == EALIGN and call(ws=None) == EWS and call(size=need - 16) == EWS
    assert lib.trellis_logprobs_workspace_bytes(3, 10, 11) == 0


def test_no_usable_device_without_gpu(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert norm_rope(lib) == -8 and attention(lib) == -8


def test_calls_refuse_host_tensors():
    with pytest.raises(ValueError, match="CUDA tensor"):
        tb.PagedCache(torch.zeros((1, 2, 2, 1, 16, 64), dtype=torch.bfloat16))
    w = torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tb.NormRope(w, w, None, 2, 1)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tb.DraftBatch(i.view(1, 3), i[:1], i[:2], 2, n=2)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tb.token_logprobs(torch.zeros((1, 8)), i.view(1, 3), 2, i)


# ---- the definitions themselves

def test_reference_attention_is_a_weighted_mean():
    q, k, v = np.array([[2.0, 0.0]]), np.array([[0.0, 1.0], [1.0, 0.0], [9.0, 9.0]]), np.array([[1.0], [3.0], [np.nan]])
    o, lse, mass, size = ref.attention(np.repeat(q, 2, 0), k, np.repeat(v, 2, 1), np.array([[1, 1, 0], [0, 0, 0]], bool), 0.5)
    assert np.allclose(o[0], (1 + 3 * np.e) / (1 + np.e)) and np.isclose(lse[0], np.log(1 + np.e))
    assert np.all(o[1] == 0) and lse[1] == -np.inf


def test_reference_norm_and_rotation():
    x = np.array([[[3.0, 4.0, 0.0, 5.0]]])
    y, _ = ref.norm_rope(x, np.ones(4), np.array([[0.0, 1.0, 1.0, 0.0]]), 4, False, 0.0, 0.0)
    r = np.sqrt(50 / 4)  # pair (0, 2) turned by a quarter, pair (1, 3) left
    assert np.allclose(y[0, 0], np.array([0.0, 4.0, 3.0, 5.0]) / r)
    y, _ = ref.norm_rope(x, np.ones(4), np.array([[0.0, 1.0]]), 2, True, 0.0, 1.0)
    assert np.allclose(y[0, 0], 2 * np.array([-4.0, 3.0, 0.0, 5.0]) / r)


def test_reference_fork_and_compact_keep_counts():
    rng = np.random.default_rng(0)
    table, lens, refs = np.full((6, 4), -1), np.zeros(6, int), np.zeros(40, int)
    table[0, :2], lens[0], refs[[3, 9]] = [3, 9], 20, 1
    for _ in range(30):
        child = rng.permutation(6)[:3]
        parent = np.array([rng.choice([-1, c, rng.integers(0, 6)]) for c in child])
        table, lens, refs, _, _ = ref.fork(table, lens, refs, parent, child, 16, int(rng.integers(0, 20)))
        held = np.bincount(table[table >= 0], minlength=40)
        assert np.array_equal(held, refs)
        if rng.random() < 0.3:
            table, refs, _ = ref.compact(table, refs)
            assert np.array_equal(np.bincount(table[table >= 0], minlength=40), refs)
            assert np.all(refs[:int((refs > 0).sum())] > 0)


def test_reference_logprobs_of_a_uniform_row():
    lp, lse, ent, ids, tlp = ref.logprobs(np.zeros((1, 8)), np.array([[3, 9]]), 3, 1.0)
    assert np.allclose([lp[0, 0], lse[0], ent[0]], [-np.log(8), np.log(8), np.log(8)]) and lp[0, 1] == -np.inf
    assert ids[0].tolist() == [0, 1, 2] and np.allclose(tlp, -np.log(8))


def test_reference_rounding_to_bf16():
    x = np.random.default_rng(1).standard_normal(20000) * np.exp(np.random.default_rng(2).standard_normal(20000) * 20)
    t = torch.tensor(x).float()
    assert np.array_equal(ref.bf16_round(t.double().numpy()), t.bfloat16().double().numpy())
