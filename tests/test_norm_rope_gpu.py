"""trellis_qk_norm_rope_append against the 64-bit definition.

Tolerance: the fp32 chain (sum of squares, reciprocal root, three products, the rotation) stays below 16 roundings of
2^-24 of the pair's size, allowed four times that (4e-6); then one rounding to bf16, checked as the parity tests do
(any bf16 number that a correctly rounded cast of a number inside the fp32 band gives), or to e4m3 (2^-4 of the number,
or 2^-10 below the smallest normal number)."""
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


def make(n, hq, hkv, d, rot, page, f8, seed=0, max_pos=300, pad=0, layers=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    qkv = rnd(n, (hq + 2 * hkv) * d + pad).bfloat16()
    q, k, v = (t.unflatten(1, (-1, d)) for t in (qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d],
                                                 qkv[:, (hq + hkv) * d:(hq + 2 * hkv) * d]))
    pages = -(-n // page) + 2
    pool = (rnd(layers, pages, 2, hkv, page, d) * 8).to(ref.F8 if f8 else torch.bfloat16)
    scales = torch.rand((layers, 2, hkv), generator=g, device="cuda") * 0.02 + 0.005 if f8 else None
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:n]
    pos = torch.randint(0, max_pos, (n,), generator=g, device="cuda").int()
    angle = torch.rand((max_pos, rot // 2), generator=g, device="cuda", dtype=torch.float64) * 6.3
    rope = torch.cat([angle.cos(), angle.sin()], 1).float() if rot else None
    wq, wk = (1 + 0.2 * rnd(d)).bfloat16(), (1 + 0.2 * rnd(d)).bfloat16()
    return q, k, v, pool, scales, slots, pos, rope, wq, wk


def check(q, k, v, before, cache, slots, pos, rope, wq, wk, out, layer, interleaved, eps, offset):
    page, f8 = cache.page_size, cache.scales is not None
    rot = 0 if rope is None else rope.shape[1]
    rows = ref.f64(rope)[pos.cpu().numpy()] if rot else np.zeros((q.shape[0], 0))
    y, size = ref.norm_rope(ref.f64(q), ref.f64(wq), rows, rot, interleaved, eps, offset)
    assert ref.in_bf16_band(ref.f64(out), y, 4e-6 * size)
    got = ref.f64(cache.pool[layer])
    want, written = ref.f64(before[layer]), np.zeros(got.shape, bool)
    tol = np.zeros(got.shape)  # of the numbers as stored (e4m3), or before their rounding to bf16
    ky, ksize = ref.norm_rope(ref.f64(k), ref.f64(wk), rows, rot, interleaved, eps, offset)
    vy = ref.f64(v)
    for i, s in enumerate(slots.tolist()):
        if not 0 <= s < cache.pages * page:
            continue
        for kv, (val, sz) in enumerate(((ky[i], ksize[i]), (vy[i], np.zeros_like(vy[i])))):
            at = (s // page, kv, slice(None), s % page)
            if f8:
                sc = ref.f64(cache.scales)[layer, kv][:, None]
                t = np.clip(val / sc, -448, 448)
                want[at], tol[at] = t, 2.0 ** -4 * np.abs(t) * (1 + 1e-5) + 2.0 ** -10 + 4e-6 * sz / sc
            else:
                want[at], tol[at] = val, 4e-6 * sz
            written[at] = True
    assert np.all(np.abs(got - want) <= tol) if f8 else ref.in_bf16_band(got, want, tol), "cache"
    same = torch.equal(cache.pool.view(torch.uint8)[1 - layer], before.view(torch.uint8)[1 - layer])
    assert same, "another layer was written"
    assert np.array_equal(got[~written], ref.f64(before[layer])[~written])


@pytest.mark.parametrize("n,hq,hkv,d,rot,page,f8,interleaved", [
    (1, 40, 8, 128, 128, 16, False, False), (1, 1, 1, 64, 0, 16, False, False), (3, 5, 1, 64, 16, 32, True, True),
    (7, 16, 2, 256, 64, 64, True, False), (33, 6, 3, 128, 48, 128, False, True), (130, 28, 4, 128, 96, 16, True, False),
    (1500, 4, 4, 64, 64, 32, False, False), (2, 9, 3, 256, 256, 16, False, True), (64, 17, 1, 256, 208, 128, True, True)])
def test_norms_rotation_and_append(n, hq, hkv, d, rot, page, f8, interleaved):
    q, k, v, pool, scales, slots, pos, rope, wq, wk = make(n, hq, hkv, d, rot, page, f8, seed=n + d, pad=8)
    before, cache = pool.clone(), tb.PagedCache(pool, scales)
    norm = tb.NormRope(wq, wk, rope, hq, hkv, interleaved=interleaved, eps=1e-5, weight_offset=0.5)
    out = tb.qk_norm_rope_append(q, k, v, pos, slots, norm, cache, 1)
    check(q, k, v, before, cache, slots, pos, rope, wq, wk, out, 1, interleaved, 1e-5, 0.5)


def test_in_place_padding_and_positions_out_of_range():
    q, k, v, pool, scales, slots, pos, rope, wq, wk = make(6, 4, 2, 128, 64, 16, False, seed=5)
    slots[1], slots[3] = -1, pool.shape[1] * 16  # one of padding, one past the pool
    pos[2], pos[4] = -1, rope.shape[0]
    before, cache, q0 = pool.clone(), tb.PagedCache(pool), q.clone()
    norm = tb.NormRope(wq, wk, rope, 4, 2)
    out = tb.qk_norm_rope_append(q, k, v, pos, slots, norm, cache, 0, out=q)
    assert out.data_ptr() == q.data_ptr()
    bad = torch.tensor([2, 4], device="cuda")
    assert out[bad].isnan().all()
    for i in bad.tolist():
        s = int(slots[i])
        assert cache.pool[0, s // 16, 0, :, s % 16].isnan().all()
        assert torch.equal(cache.pool[0, s // 16, 1, :, s % 16], v[i])
    good = torch.tensor([0, 1, 3, 5], device="cuda")
    before[0] = torch.where(cache.pool[0].isnan(), cache.pool[0], before[0])
    for i in bad.tolist():
        s = int(slots[i])
        before[0, s // 16, :, :, s % 16] = cache.pool[0, s // 16, :, :, s % 16]
    pool_view = torch.nan_to_num(cache.pool)
    cache2 = tb.PagedCache(pool_view.contiguous())
    check(q0[good], k[good], v[good], torch.nan_to_num(before), cache2, slots[good], pos[good], rope, wq, wk, out[good], 0,
          False, 1e-6, 0.0)


def test_large_numbers_saturate_and_nan_stays():
    q, k, v, pool, scales, slots, pos, rope, wq, wk = make(4, 2, 1, 64, 0, 16, True, seed=9)
    v = v.clone()
    v[0, 0, :4] = torch.tensor([1e30, -1e30, float("inf"), float("nan")], dtype=torch.bfloat16, device="cuda")
    cache = tb.PagedCache(pool, scales)
    tb.qk_norm_rope_append(q, k, v, pos, slots, tb.NormRope(wq, wk, None, 2, 1), cache, 0)
    s = int(slots[0])
    got = cache.pool[0, s // 16, 1, 0, s % 16, :4].float()
    assert got[:3].tolist() == [448.0, -448.0, 448.0] and got[3].isnan()


def test_another_stream_and_no_tokens():
    q, k, v, pool, scales, slots, pos, rope, wq, wk = make(9, 4, 2, 64, 64, 16, False, seed=3)
    before, cache = pool.clone(), tb.PagedCache(pool)
    norm = tb.NormRope(wq, wk, rope, 4, 2)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        out = tb.qk_norm_rope_append(q, k, v, pos, slots, norm, cache, 1)
    st.synchronize()
    check(q, k, v, before, cache, slots, pos, rope, wq, wk, out, 1, False, 1e-6, 0.0)
    kept = cache.pool.clone()
    tb.qk_norm_rope_append(q[:0], k[:0], v[:0], pos[:0], slots[:0], norm, cache, 1)
    torch.cuda.synchronize()
    assert torch.equal(cache.pool, kept)


def test_slots_past_32_bits_of_elements():
    # a layer of 2^25 rows of 128 numbers: the last page starts past element 2^32
    pages, page, d = (1 << 20) + 3, 16, 128
    pool = torch.zeros((1, pages, 2, 1, page, d), dtype=torch.bfloat16, device="cuda")
    cache = tb.PagedCache(pool)
    q, k, v, _, _, _, pos, rope, wq, wk = make(2, 1, 1, d, 0, page, False, seed=1)
    slots = torch.tensor([pages * page - 1, 5], device="cuda")
    tb.qk_norm_rope_append(q, k, v, pos, slots, tb.NormRope(wq, wk, None, 1, 1), cache, 0)
    assert torch.equal(pool[0, -1, 1, 0, page - 1], v[0, 0]) and torch.equal(pool[0, 0, 1, 0, 5], v[1, 0])
    assert int((pool[0, -1] != 0).any(-1).sum()) == 2


def test_refusals():
    q, k, v, pool, scales, slots, pos, rope, wq, wk = make(3, 4, 2, 64, 64, 16, False)
    cache, norm = tb.PagedCache(pool), tb.NormRope(wq, wk, rope, 4, 2)
    call = lambda *a, **kw: tb.qk_norm_rope_append(*a, **kw)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA tensor"):
        call(q.cpu(), k, v, pos, slots, norm, cache, 0)
    with pytest.raises(ValueError, match="dtype"):
        call(q.float(), k, v, pos, slots, norm, cache, 0)
    with pytest.raises(ValueError, match="shape"):
        call(q, k[:2], v, pos, slots, norm, cache, 0)
    with pytest.raises(ValueError, match="contiguous"):
        call(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, pos, slots, norm, cache, 0)
    with pytest.raises(ValueError, match="dtype"):
        call(q, k, v, pos.long(), slots, norm, cache, 0)
    for layer in (-1, 2):
        with pytest.raises(tb.TrellisError, match="ESHAPE"):
            call(q, k, v, pos, slots, norm, cache, layer)
    with pytest.raises(tb.TrellisError, match="ESHAPE"):  # another number of key/value heads than the cache's
        call(q[:, :2], k[:, :1], v[:, :1], pos, slots, tb.NormRope(wq, wk, rope, 2, 1), cache, 0)
    with pytest.raises(tb.TrellisError, match="ESHAPE"):
        call(q, k, v, pos, slots, tb.NormRope(wq, wk, rope[:, :24].contiguous(), 4, 2), cache, 0)
    with pytest.raises(tb.TrellisError, match="ESHAPE"):
        call(q, k, v, pos, slots, tb.NormRope(wq, wk, rope, 4, 2, eps=float("nan")), cache, 0)
    wide = torch.zeros((3, 4 * 64 + 4), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(tb.TrellisError, match="ESHAPE"):  # stride not a multiple of 8
        call(wide[:, :256].unflatten(1, (4, 64)), k, v, pos, slots, norm, cache, 0)
    flat = torch.zeros(3 * 256 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(tb.TrellisError, match="EALIGN"):
        call(flat[1:1 + 768].view(3, 4, 64), k, v, pos, slots, norm, cache, 0)
    with pytest.raises(ValueError, match="scales"):
        tb.PagedCache(pool, torch.ones((2, 2, 2), device="cuda"))
    with pytest.raises(tb.TrellisError, match="ESHAPE"):
        tb.PagedCache(torch.zeros((1, 2, 2, 1, 8, 64), dtype=torch.bfloat16, device="cuda"))
