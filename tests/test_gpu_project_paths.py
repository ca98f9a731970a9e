"""Paths of the projection that sizes alone choose, and calls beside one another (needs a GB300): each
against the plain 64-bit form, as tests/test_gpu_project.py has it."""
from __future__ import annotations

import pytest
import torch

import _layer_ref as R
from test_gpu_project import BF, FP, Case, _built, dt, near  # noqa: F401  (_built is a fixture)

pytestmark = pytest.mark.gpu


def test_a_launch_before_with_room_beside_it():
    """Tiles of 80 rows in single blocks, and x A^T in blocks of one stage: their shared memory together is less
    than an SM has, so that nothing but registers keeps a block of each from the same SM. The second one
    takes all of TMEM and waits for the first launch, whose blocks must have their columns by then."""
    c = Case(1, 3996, 64, 1072, 64, 2, index=[1], seed=21)
    p, x, ad, index, _ = c.cuda()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [dt.project_workspace(p, 1, 3996, ad) for _ in streams]
    torch.cuda.synchronize()
    got = [dt.project(p, x, ad, index, workspace=spaces[k % 2], stream=streams[k % 2]) for k in range(20)]
    torch.cuda.synchronize()
    near(got[0].reshape(-1, 1072), c.y, c.slack)
    assert all(torch.equal(g, got[0]) for g in got)
    p.check()


@pytest.mark.parametrize("e8", [False, True])
def test_tiles_without_an_adapter_between_tiles_with_one(e8):
    """Many tiles a block, most of whose lists are empty: a list is given back where no product has
    read more than its length."""
    batch, n = 90, 200
    index = [b % 3 if b % 7 == 5 else -1 for b in range(batch)]
    Case(batch, n, 64, 1100, 16, 3, BF, e8, index=index, seed=22).check()
    Case(9000, 2, 64, 300, 16, 3, BF, e8, index=[2 if b % 1000 == 0 else -1 for b in range(9000)], seed=23).check()


def test_clusters_of_three_streams():
    """Launches in clusters of 2 to 8 blocks, x A^T's among them, and pairs, on three streams: a cluster has its
    SMs for itself, so that no block waits for columns that another launch's waiting block holds."""
    cases = [Case(80, 1, 2048, 300, seed=24), Case(400, 1, 1024, 700, 128, 2, seed=25), Case(77, 1, 4096, 1200, seed=26),
             Case(20, 65, 320, 2100, 16, 5, seed=27)]
    made = [c.cuda() for c in cases]
    wants = [dt.project(*m, dtype=BF) for m in made]
    streams = [torch.cuda.Stream() for _ in range(3)]
    spaces = [[dt.project_workspace(m[0], c.batch, c.n, m[2]) for c, m in zip(cases, made)] for _ in streams]
    torch.cuda.synchronize()
    got = []
    for k in range(40):
        for i, s in enumerate(streams):
            j = (k + i) % 4
            got.append((j, dt.project(*made[j], dtype=BF, workspace=spaces[i][j], stream=s)))
    torch.cuda.synchronize()
    assert all(torch.equal(y, wants[j]) for j, y in got)
    for c, w in zip(cases, wants):
        near(w.reshape(-1, c.O), c.y, c.slack)
    for m in made:
        m[0].check()


# single blocks, one tile and several; clusters that share K; pairs, one tile and several; x A^T a row a
# block, in single blocks and in clusters; 16 and 8 bits
WAITS = {"single": (40, 1, 128, 700), "cluster": (8, 1, 2048, 1040), "pairs": (20, 65, 640, 2100),
         "pairs e4m3": (20, 65, 640, 2100, 0, 0, BF, True), "pairs, many tiles": (3, 300, 64, 9000),
         "cluster, rows": (8, 1, 2048, 1040, 16, 5), "single, rows": (40, 1, 256, 5000, 32, 9, BF, True),
         "single, many tiles": (1, 3996, 64, 1072, 64, 2), "single, x A^T in clusters": (400, 1, 1024, 700, 128, 2),
         "pairs, adapters": (20, 65, 640, 2100, 16, 5), "pairs e4m3, adapters": (20, 65, 640, 2100, 16, 5, FP, True),
         "pairs, many tiles, adapters": (6, 300, 640, 9000, 64, 4, FP),
         "pairs e4m3, many tiles, adapters": (6, 300, 640, 9000, 48, 4, BF, True)}


@pytest.mark.parametrize("what", WAITS)
def test_waits_that_run_out(what):
    """Limits from one SM cycle on: a call ends by itself with DT_ERR_TIMEOUT (or, where no wait took as long, with its
    result), and the next one is right."""
    c = Case(*WAITS[what], seed=28)
    p, x, ad, index, x16 = c.cuda()
    run = lambda: dt.project(p, x, ad, index, x16, dtype=c.dtype)
    want = run()
    near(want.reshape(-1, c.O), c.y, c.slack)
    for limit in (1, 200, 500, 1000, 1500, 2000, 3000, 5000, 8000, 15000, 40000):
        p._struct.wait_cycles = limit
        got = run()
        said = int(p.status)
        assert said == dt.ERR_TIMEOUT or (limit > 1 and said == dt.OK and torch.equal(got, want)), limit
        p._struct.wait_cycles = 0
        p.status.zero_()
        assert torch.equal(run(), want), limit
        p.check()


@pytest.mark.parametrize("e8", [False, True])
def test_the_last_row_of_a_long_sequence(e8):
    """A single row whose tensor's strides are those of what it was cut from, and a row of results likewise."""
    c = Case(1, 1, 80, 37, 16, 2, BF, e8, index=[1], seed=29)
    p, x, ad, index, x16 = c.cuda()
    want = dt.project(p, x, ad, index, x16, dtype=BF)
    near(want.reshape(-1, 37), c.y, c.slack)
    last = lambda t, rows, more: torch.cat([torch.zeros(1, rows, t.shape[2] + more, dtype=t.dtype, device="cuda")], 1)[:, -1:, :t.shape[2]].copy_(t)
    if e8:
        y = dt.Rows8(last(x.codes.view(torch.uint8), 3, 5 * 16 + 48), x.exps)
        y16 = last(x16, 4, 8)
    else:
        y, y16 = last(x, 1, 16), None
    frame = torch.full((1, 40000, 1700), 7.0, dtype=BF, device="cuda")          # 40000 * 1700 > 2^26
    got = dt.project(p, y, ad, index, y16, dtype=BF, out=frame[:, -1:, 3:40])
    assert torch.equal(got, want)
    assert bool((frame[0, :-1] == 7).all()) and bool((frame[0, -1, :3] == 7).all()) and bool((frame[0, -1, 40:] == 7).all())


def test_check_waits_for_calls_on_every_stream():
    """What a call on a stream of its own has to report is there when check() returns."""
    c = Case(2, 3, 64, 40, 16, 2, index=[0, 5], seed=30)
    p, x, ad, index, _ = c.cuda()
    table = torch.tensor([[9, 0]], dtype=torch.int32, device="cuda")
    cache = dt.PagedCache.empty(4, 1, 16, 16, table)
    first = torch.zeros(1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(200_000_000)          # some 0.1 s
        dt.project(p, x, ad, index)
    with pytest.raises(dt.DtError, match="adapter index"):
        p.check()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(200_000_000)
        dt.cache_slots(cache, 3, first)
    with pytest.raises(dt.DtError, match="request 0"):
        cache.check()


@pytest.mark.parametrize("batch,n,K,O,rank,count,dtype,e8", [(2, 3, 65536, 200, 128, 2, BF, False), (9, 1, 65536, 40, 16, 3, FP, True),
                                                             (1, 300, 65536, 300, 16, 1, BF, True), (65535, 1, 16, 24, 16, 3, BF, False),
                                                             (5, 1, 32, 140000, 16, 4, FP, False)])
def test_the_largest_sizes(batch, n, K, O, rank, count, dtype, e8):
    Case(batch, n, K, O, rank, count, dtype, e8, seed=33).check()


def test_adapters_past_32_bits():
    """B of more than 4 GB, and values of A past 2^31: the last adapters' places."""
    count, rank, K, O, batch, n = 3000, 64, 16384, 20000, 5, 9
    g = torch.Generator().manual_seed(34)
    rnd = lambda *s: torch.randn(s, generator=g).to(BF)
    x, w = rnd(batch * n, K), rnd(O, K) * K ** -0.5
    used = [count - 1, 0, count - 2, -1, 2047]
    ad = dt.Adapters(torch.zeros(count, rank, K, dtype=BF, device="cuda"), torch.zeros(count, O, rank, dtype=BF, device="cuda"))
    small = {a: i for i, a in enumerate(sorted(set(used) - {-1}))}
    down, up = rnd(len(small), rank, K) * K ** -0.5, rnd(len(small), O, rank) * rank ** -0.5
    for a, i in small.items():
        ad.down[a], ad.up[a] = down[i].cuda(), up[i].cuda()
    index = torch.tensor([small.get(a, -1) for a in used], dtype=torch.int32)
    y = R.project(x.double(), w.double(), n, index, x, down, up)
    slack = R.project_slack(x.double(), w.double(), n, y, BF, index, x, down, up)
    p = dt.Projection(w.cuda())
    got = dt.project(p, x.cuda().view(batch, n, K), ad, torch.tensor(used, dtype=torch.int32, device="cuda"))
    near(got.reshape(-1, O), y, slack)
    p.check()


FIRST = """
import torch, conditional_draft_tree_gb300 as dt
g = torch.Generator().manual_seed(0)
rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()
x, w, down, up = rnd(20, 65, 640), rnd(2100, 640), rnd(3, 16, 640), rnd(3, 2100, 16)
index = torch.tensor([b % 4 - 1 for b in range(20)], dtype=torch.int32, device="cuda")
weight = rnd(640)
p, ad, norm = dt.Projection(w), dt.Adapters(down, up), dt.Norm(weight)
table = torch.full((20, 9), -1, dtype=torch.int32, device="cuda")
cache = dt.PagedCache.empty(180, 1, 16, 16, table)
pool = dt.PagePool.all_free(cache)
lengths, first = (torch.full((20,), v, dtype=torch.int32, device="cuda") for v in (100, 35))
def run():
    dt.cache_reserve(pool, lengths)
    places = dt.cache_slots(cache, 65, first)
    y, total = dt.rms_norm(norm, x, x)
    return (dt.project(p, y, ad, index), total) + places
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
want = run()
assert all(torch.equal(a, b) for a, b in zip(got, want)), "first"
p.check(); cache.check()
print("same")
"""


def test_the_first_calls_of_a_process_are_captured():
    """Kernels, limits and clusters that a process has not met yet, under a capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_threads_that_call_at_once():
    """Calls of four host threads, each on a stream of its own."""
    import threading
    cases = [Case(20, 65, 320, 2100, 16, 5, seed=35), Case(8, 1, 2048, 1040, 16, 5, seed=36), Case(40, 7, 128, 260, 112, 40, FP, True, seed=37),
             Case(3, 400, 512, 900, 64, 3, FP, seed=38)]
    made = [c.cuda() for c in cases]
    wants = [dt.project(*m, dtype=c.dtype) for c, m in zip(cases, made)]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        got = [dt.project(*made[(i + k) % 4], dtype=cases[(i + k) % 4].dtype, stream=stream) for k in range(40)]
        stream.synchronize()
        wrong.extend((i, k) for k, y in enumerate(got) if not torch.equal(y, wants[(i + k) % 4]))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    for m in made:
        m[0].check()
