"""Page tables and slot maps from lengths against a pool kept as lists (needs a GB300). Whole
numbers: equal."""
from __future__ import annotations

import random

import pytest
import torch

import _layer_ref as R

pytestmark = pytest.mark.gpu

dt = pytest.importorskip("conditional_draft_tree_gb300")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conditional_draft_tree_gb300 import build
    build.build()


def make(pages, batch, width, page, seed=None):
    table = torch.zeros(batch, width, dtype=torch.int32, device="cuda")
    k = torch.zeros(pages, 1, page, 16, dtype=torch.bfloat16, device="cuda")
    cache = dt.PagedCache(k, k.clone(), table)
    pool = dt.PagePool.all_free(cache)
    model = R.Pool(pages, batch, width, page)
    if seed is not None:
        order = list(range(pages))
        random.Random(seed).shuffle(order)
        pool.free_pages.copy_(torch.tensor(order, dtype=torch.int32))
        model = R.Pool(pages, batch, width, page, order)
    return cache, pool, model


def reserve(cache, pool, model, lengths):
    cache.status.zero_()
    dt.cache_reserve(pool, torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    said = model.reserve(lengths)
    assert cache.table.tolist() == model.tables()
    assert pool.held.tolist() == [len(t) for t in model.table]
    assert pool.state.tolist() == [len(model.free), 0]
    assert pool.free_pages.tolist() == model.array
    code = {None: dt.OK, "over": dt.ERR_BAD_PAGE, "none": dt.ERR_NO_PAGES}
    assert cache.status.tolist() == [code[s] for s in said]


@pytest.mark.parametrize("pages,batch,width,page", [
    (7, 1, 9, 16), (40, 5, 9, 16), (64, 33, 4, 128), (700, 520, 3, 32), (5000, 70, 300, 64), (20000, 1100, 19, 16),
    (3000, 2, 9000, 16)])
def test_sequences(pages, batch, width, page):
    """Requests grow, shrink, end and begin in one call; pools that run out; lengths that are
    negative, on a page's border, or past the table."""
    cache, pool, model = make(pages, batch, width, page, seed=1)
    rng = random.Random(2)
    fair = max(1, pages // batch)
    for step in range(8):
        most = page * min(width, rng.choice((1, fair, fair, 2 * fair, 3 * fair)))
        lengths = [rng.choice((0, -3, rng.randint(0, most), rng.randint(0, most), page * rng.randint(0, width // 2),
                               most, page * width + rng.choice((0, 1)))) for _ in range(batch)]
        reserve(cache, pool, model, lengths)


def test_lengths_of_before_undo_a_call():
    cache, pool, model = make(400, 16, 40, 16, seed=3)
    rng = random.Random(4)
    before = [rng.randint(0, 300) for _ in range(16)]
    reserve(cache, pool, model, before)
    kept = [t.clone() for t in (cache.table, pool.held, pool.free_pages, pool.state)]
    reserve(cache, pool, model, [rng.randint(0, 380) for _ in range(16)])
    reserve(cache, pool, model, before)
    assert all(torch.equal(a, b) for a, b in zip(kept, (cache.table, pool.held, pool.free_pages, pool.state)))


def test_the_last_page_and_one_more():
    cache, pool, model = make(6, 3, 6, 16)
    reserve(cache, pool, model, [32, 32, 32])
    assert pool.state.tolist()[0] == 0
    reserve(cache, pool, model, [33, 32, 32])          # nothing left
    assert cache.status.tolist() == [dt.ERR_NO_PAGES, 0, 0]
    with pytest.raises(dt.DtError, match="too few free pages"):
        cache.check()
    reserve(cache, pool, model, [33, 32, 16])          # the last one gives back what the first one takes
    reserve(cache, pool, model, [64, 0, 48])           # the first fits, the third no more
    assert cache.status.tolist() == [0, 0, dt.ERR_NO_PAGES]
    reserve(cache, pool, model, [0, 0, 0])
    assert pool.state.tolist()[0] == 6


def test_the_largest_batch():
    cache, pool, model = make(40000, 16384, 3, 16)
    rng = random.Random(5)
    for _ in range(3):
        reserve(cache, pool, model, [rng.randint(0, 48) for _ in range(16384)])


def test_pages_that_the_pool_does_not_have():
    """A table entry that somebody overwrote: reported when it is given back, nothing outside is
    touched."""
    cache, pool, model = make(20, 2, 8, 16)
    reserve(cache, pool, model, [100, 50])
    cache.table[0, 6] = 20
    cache.table[1, 3] = -7
    dt.cache_reserve(pool, torch.tensor([0, 0], dtype=torch.int32, device="cuda"))
    assert cache.status.tolist() == [dt.ERR_BAD_PAGE, dt.ERR_BAD_PAGE]
    assert pool.state.tolist() == [20, 0] and bool((cache.table == -1).all())
    assert sorted(x for x in pool.free_pages.tolist() if 0 <= x < 20) == \
        sorted(set(range(20)) - {model.table[0][6], model.table[1][3]})


def test_a_stack_that_would_overflow():
    """Pages given back twice (the caller's mistake): the stack ends at the pool's size."""
    cache, pool, _ = make(4, 2, 4, 16)
    cache.table.copy_(torch.tensor([[0, 1, 2, 3], [0, 1, 2, 3]]))
    pool.held.fill_(4)
    pool.state[0] = 2
    guard = torch.full((8,), 77, dtype=torch.int32, device="cuda")
    guard[:4] = pool.free_pages
    pool = dt.PagePool(cache, pool.held, guard[:4], pool.state)
    dt.cache_reserve(pool, torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert guard.tolist()[4:] == [77] * 4 and pool.state.tolist() == [4, 0]


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("batch,n", [(1, 1), (3, 7), (5, 256), (4, 257), (130, 33), (2, 5003)])
def test_slots(page, batch, n):
    width = -(-(n + 100) // page)
    cache, pool, model = make(batch * width + 2, batch, width, page, seed=6)
    rng = random.Random(7)
    first = [rng.randint(0, 100) for _ in range(batch)]
    counts = [rng.choice((0, n, rng.randint(0, n))) for _ in range(batch)]
    reserve(cache, pool, model, [f + c for f, c in zip(first, counts)])
    t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    slots, positions = dt.cache_slots(cache, n, t(first), t(counts))
    for b in range(batch):
        at = list(range(first[b], first[b] + counts[b]))
        assert positions[b].tolist() == at + [-1] * (n - counts[b])
        assert slots[b].tolist() == [model.table[b][i // page] * page + i % page for i in at] + [-1] * (n - counts[b])
    cache.check()
    # without counts: rows that no page holds are reported, and have positions
    slots, positions = dt.cache_slots(cache, n, t(first))
    assert positions.tolist() == [[f + i for i in range(n)] for f in first]
    for b in range(batch):
        inside = [i // page < len(model.table[b]) for i in range(first[b], first[b] + n)]
        assert [s >= 0 for s in slots[b].tolist()] == inside
        assert (int(cache.status[b]) == dt.ERR_BAD_PAGE) == (not all(inside))


def test_slots_of_bad_rows_and_far_pools():
    """Rows before the first one; places past 2^31 (a table that names far pages: only numbers are made)."""
    cache, pool, _ = make(4, 2, 3, 16)
    cache.table.copy_(torch.tensor([[3, 4, -1], [2, 0, 1]]))
    slots, positions = dt.cache_slots(cache, 50, torch.tensor([-1, 3], dtype=torch.int32, device="cuda"))
    want = [-1] + [48 + i for i in range(16)] + [-1] * 33
    assert slots[0].tolist() == want and positions[0].tolist() == list(range(-1, 49))
    assert slots[1].tolist() == [32 + i for i in range(3, 16)] + list(range(16)) + [16 + i for i in range(16)] + [-1] * 5
    assert cache.status.tolist() == [dt.ERR_BAD_PAGE] * 2


def test_a_captured_round():
    """Reserve, slots and reserve again in a graph, replayed with other lengths."""
    cache, pool, model = make(300, 8, 30, 16, seed=8)
    lengths = torch.zeros(8, dtype=torch.int32, device="cuda")
    first = torch.zeros(8, dtype=torch.int32, device="cuda")
    slots = torch.empty(8, 9, dtype=torch.int64, device="cuda")
    positions = torch.empty(8, 9, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        dt.cache_reserve(pool, lengths)
        dt.cache_slots(cache, 9, first, slots=slots, positions=positions)
    rng = random.Random(9)
    for _ in range(4):
        at = [rng.randint(0, 400) for _ in range(8)]
        first.copy_(torch.tensor(at, dtype=torch.int32))
        lengths.copy_(first + 9)
        graph.replay()
        model.reserve([x + 9 for x in at])
        assert cache.table.tolist() == model.tables() and pool.free_pages.tolist() == model.array
        assert slots.tolist() == [[model.table[b][i // 16] * 16 + i % 16 for i in range(f, f + 9)] for b, f in enumerate(at)]
    cache.check()
