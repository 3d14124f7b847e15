"""Pages of the cache: copy, fork, compact, commit.  Everything is whole numbers or moved bits and has to be equal to
the sequential definition."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from trellis_coded_weight_gb300 import binding as tb

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from trellis_coded_weight_gb300 import build
    build.build()
    tb.load()


def dev(a):
    return torch.as_tensor(np.asarray(a), dtype=I32).cuda()


def make_cache(layers, pages, heads, page, d, f8=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = ref.F8 if f8 else torch.bfloat16
    raw = torch.randint(0, 256, (layers, pages, 2, heads, page, d * (1 if f8 else 2)), generator=g, device="cuda").to(torch.uint8)
    return tb.PagedCache(raw.view(dtype))  # any bits, NaN among them: they are moved, not read as numbers


def bits(cache):
    return cache.pool.view(torch.uint8)


def run_fork(cache, table, lens, refs, parent, child, room):
    t, le, r = dev(table), dev(lens), dev(refs)
    status = torch.full((len(parent),), -7, dtype=I32, device="cuda")
    before = bits(cache).clone()
    tb.cache_fork(cache, t, le, r, dev(parent), dev(child), status, tb.new_cache_workspace(cache, t, len(parent)), room)
    want = ref.fork(table, lens, refs, parent, child, cache.page_size, room)
    for name, got, w in zip(("table", "lens", "refs", "status"), (t, le, r, status), want):
        assert np.array_equal(got.cpu().numpy(), w), name
    for src, dst in want[4]:
        before[:, dst] = before[:, src]
    assert torch.equal(bits(cache), before)
    return t.cpu().numpy(), le.cpu().numpy(), r.cpu().numpy(), status.cpu().numpy()


def random_rows(rng, rows, width, page, pages, used):
    """`used` rows of random lengths over distinct pages of a shuffled pool."""
    table, lens, refs = np.full((rows, width), -1), np.zeros(rows, int), np.zeros(pages, int)
    order, at = rng.permutation(pages), 0
    for r in range(used):
        lens[r] = rng.integers(0, width * page + 1)
        held = min(width, -(-lens[r] // page) + rng.integers(0, 2))  # some hold a page more than they fill
        if at + held > pages:
            held, lens[r] = 0, 0
        table[r, :held] = order[at:at + held]
        at += held
        refs[table[r, :held]] = 1
    return table, lens, refs


@pytest.mark.parametrize("seed", range(12))
def test_fork_of_random_rows(seed):
    rng = np.random.default_rng(seed)
    page = int(rng.choice([16, 32, 64, 128]))
    rows, width, pages = int(rng.integers(2, 60)), int(rng.integers(1, 40)), int(rng.integers(3, 1500))
    cache = make_cache(int(rng.integers(1, 4)), pages, int(rng.integers(1, 4)), page, int(rng.choice([64, 128])), bool(seed % 2), seed)
    state = random_rows(rng, rows, width, page, pages, rows // 2 + 1)
    for step in range(4):  # rows that share pages, and children that held some, from the second step on
        pairs = int(rng.integers(1, rows + 1))
        child = rng.permutation(rows)[:pairs]
        parent = np.array([rng.choice([-1, c, rng.integers(0, rows), rng.integers(0, rows)]) for c in child])
        state = run_fork(cache, *state[:3], parent, child, int(rng.integers(0, 3 * page)))
        assert np.all(state[2] >= 0)


def test_fork_reads_parents_as_they_were():
    cache = make_cache(2, 20, 2, 16, 64)
    table = np.full((4, 5), -1)
    table[0, :3], table[1, :2] = [7, 3, 11], [5, 2]
    refs = np.zeros(20, int)
    refs[[7, 3, 11, 5, 2]] = 1
    # two rows exchanged, a third copied from a row that is overwritten, a fourth freed and grown elsewhere
    run_fork(cache, table, np.array([41, 20, 0, 0]), refs, np.array([1, 0, 0]), np.array([0, 1, 2]), 9)


def test_fork_without_room_and_out_of_range():
    cache = make_cache(2, 6, 1, 16, 64)
    table = np.full((5, 3), -1)
    table[0, :3], table[1, :1] = [0, 1, 2], [3]
    refs = np.array([1, 1, 1, 1, 0, 0])
    lens = np.array([40, 10, 0, 0, 0])
    # two free pages: the first fork takes one, growth of row 1 by two pages finds one, a later fork none
    _, _, _, st = run_fork(cache, table, lens, refs, np.array([0, 1, 0, 9, 0, -2]), np.array([2, 1, 3, 4, 7, 4]), 7 + 16)
    assert set(st.tolist()) >= {1, 2}
    _, _, _, st = run_fork(cache, table, lens, refs, np.array([0, 1, 0]), np.array([2, 1, 3]), 0)
    assert st.tolist() == [0, 0, 0]
    bad = table.copy()
    bad[0, 1] = 6  # past the pool
    _, _, _, st = run_fork(cache, bad, lens, refs, np.array([0, 0]), np.array([2, 0]), 0)
    assert st.tolist() == [2, 2]
    run_fork(cache, table, np.array([-1, 10, 0, 0, 0]), refs, np.array([0]), np.array([2]), 0)
    run_fork(cache, table, np.array([0, 10, 0, 0, 0]), refs, np.array([0, 0]), np.array([2, 3]), 0)  # an empty parent


def test_fork_scans_large_pools_and_many_pairs():
    rng = np.random.default_rng(3)
    cache = make_cache(1, 70001, 1, 16, 64)
    table, lens, refs = random_rows(rng, 2000, 12, 16, 70001, 900)
    refs[table[table >= 0]] = 1
    refs[:69000] = np.maximum(refs[:69000], 1)  # free pages only at the end
    run_fork(cache, table, lens, refs, rng.integers(0, 900, 1024), np.arange(900, 1924), 20)


@pytest.mark.parametrize("seed", range(8))
def test_compact(seed):
    rng = np.random.default_rng(100 + seed)
    pages, rows, width = int(rng.integers(1, 3000)), int(rng.integers(1, 30)), int(rng.integers(1, 50))
    cache = make_cache(int(rng.integers(1, 4)), pages, 1 + seed % 3, 16 << seed % 4, 64, bool(seed % 2), seed)
    refs = np.where(rng.random(pages) < rng.choice([0, 0.2, 0.5, 0.9, 1]), rng.integers(1, 4, pages), 0)
    table = rng.integers(-2, pages + 2, (rows, width))
    before = bits(cache).clone()
    t, r = dev(table), dev(refs)
    ws = tb.new_cache_workspace(cache, t)
    in_place = seed % 2 == 0
    ot, orf = (None, None) if in_place else (torch.empty_like(t), torch.empty_like(r))
    got_t, got_r = tb.cache_compact(cache, t, r, ws, ot, orf)
    want_t, want_r, moves = ref.compact(table, refs)
    assert np.array_equal(got_t.cpu().numpy(), want_t) and np.array_equal(got_r.cpu().numpy(), want_r)
    if not in_place:
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), refs)
    for src, dst in moves:
        before[:, dst] = before[:, src]
    assert torch.equal(bits(cache), before)


@pytest.mark.parametrize("batch,tokens,page,layers,heads,d,f8,alias", [
    (1, 1, 16, 1, 1, 64, False, False), (5, 64, 16, 3, 2, 128, True, True), (9, 17, 32, 2, 8, 128, False, True),
    (3, 40, 128, 4, 3, 256, True, False), (70, 5, 64, 1, 16, 256, False, False)])
def test_commit(batch, tokens, page, layers, heads, d, f8, alias):
    rng = np.random.default_rng(batch * 100 + tokens)
    width = -(-(tokens + 3 * page) // page)
    cache = make_cache(layers, batch * width + 1, heads, page, d, f8, batch)
    table = rng.permutation(batch * width + 1)[:batch * width].reshape(batch, width)
    prefix = rng.integers(0, width * page - tokens + 1, batch)
    accepted = rng.integers(-1, tokens + 2, batch)  # clamped to the drafts
    path = np.full((batch, tokens), -1)
    for b in range(batch):
        n = min(max(accepted[b], 0), tokens)
        path[b, :n] = np.sort(rng.permutation(tokens)[:n])
    before = bits(cache).clone()
    pre = dev(prefix)
    lens = tb.cache_commit(cache, dev(table), pre, dev(path), dev(accepted), pre if alias else None)
    assert np.array_equal(lens.cpu().numpy(), prefix + np.clip(accepted, 0, tokens))
    want = before.clone()
    for b in range(batch):
        for i in range(min(max(accepted[b], 0), tokens)):
            a, z = prefix[b] + path[b, i], prefix[b] + i
            want[:, table[b, z // page], :, :, z % page] = before[:, table[b, a // page], :, :, a % page]
    assert torch.equal(bits(cache), want)


def test_commit_skips_entries_out_of_range():
    cache = make_cache(1, 4, 1, 16, 64)
    before = bits(cache).clone()
    table = dev([[0, 1], [2, 9], [3, -1]])
    path = dev([[1, 40, 63], [2, 17, 18], [3, 15, 16]])  # past the row's width, past the pool, an absent page
    lens = tb.cache_commit(cache, table, dev([0, 0, 0]), path, dev([3, 3, 3]))
    want = before.clone()
    want[:, 0, :, :, 0] = before[:, 0, :, :, 1]
    want[:, 2, :, :, 0] = before[:, 2, :, :, 2]
    want[:, 3, :, :, 0], want[:, 3, :, :, 1] = before[:, 3, :, :, 3], before[:, 3, :, :, 15]
    assert lens.tolist() == [3, 3, 3] and torch.equal(bits(cache), want)
    for pre in (-5, 100):  # prefixes out of range move nothing
        before = bits(cache).clone()
        tb.cache_commit(cache, table, dev([pre] * 3), path, dev([3, 3, 3]))
        assert torch.equal(bits(cache), before)


def test_copy_pages_and_empty_calls():
    cache = make_cache(3, 50, 3, 32, 128, True)
    before = bits(cache).clone()
    src, dst = [4, 9, 50, -1, 20, 11], [1, 40, 2, 3, 50, 12]
    tb.cache_copy(cache, dev(src), dev(dst))
    for s, d in ((4, 1), (9, 40), (11, 12)):
        before[:, d] = before[:, s]
    assert torch.equal(bits(cache), before)
    none = torch.zeros(0, dtype=I32, device="cuda")
    tb.cache_copy(cache, none, none)
    t, le, r = dev(np.full((2, 3), -1)), dev([0, 0]), dev(np.zeros(50))
    tb.cache_fork(cache, t, le, r, none, none, none, tb.new_cache_workspace(cache, t, 0))
    tb.cache_commit(cache, t[:0], le[:0], torch.zeros((0, 4), dtype=I32, device="cuda"), le[:0])
    assert torch.equal(bits(cache), before)


def test_layers_past_32_bits():
    # three layers of 1.6 GB: bytes past 2^32 from the third on
    cache = make_cache(3, 6200, 8, 64, 128)
    before = bits(cache)[:, [6199, 3]].clone()
    tb.cache_copy(cache, dev([6199]), dev([3]))
    assert torch.equal(bits(cache)[:, 3], before[:, 0]) and torch.equal(bits(cache)[:, 6199], before[:, 0])


def test_refusals():
    cache = make_cache(1, 8, 1, 16, 64)
    t, le, r = dev(np.full((4, 3), -1)), dev([0] * 4), dev([0] * 8)
    one = dev([0])
    ws = tb.new_cache_workspace(cache, t, 1)
    with pytest.raises(ValueError, match="shape"):
        tb.cache_fork(cache, t, le, r[:7].contiguous(), one, one, one.clone(), ws)
    with pytest.raises(ValueError, match="dtype"):
        tb.cache_fork(cache, t.long(), le, r, one, one, one.clone(), ws)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tb.cache_fork(cache, t, le, r, one.cpu(), one, one.clone(), ws)
    with pytest.raises(tb.TrellisError, match="EWORKSPACE"):
        tb.cache_fork(cache, t, le, r, one, one, one.clone(), ws[:4].contiguous())
    with pytest.raises(tb.TrellisError, match="ESHAPE"):
        tb.cache_fork(cache, t, le, r, one, one, one.clone(), ws, room=-1)
    many = torch.zeros(1025, dtype=I32, device="cuda")
    with pytest.raises(tb.TrellisError, match="EM"):
        tb.cache_fork(cache, t, le, r, many, many, many.clone(), torch.zeros(1 << 16, dtype=I32, device="cuda"))
    with pytest.raises(tb.TrellisError, match="EWORKSPACE"):
        tb.cache_compact(cache, t, r, ws[:4].contiguous())
    with pytest.raises(tb.TrellisError, match="EM"):
        tb.cache_commit(cache, t, le, torch.zeros((4, 65), dtype=I32, device="cuda"), le)
    with pytest.raises(ValueError, match="contiguous"):
        tb.cache_commit(cache, t.t().contiguous().t(), le, torch.zeros((4, 5), dtype=I32, device="cuda"), le)
