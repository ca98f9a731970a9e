"""The shared projection with low-rank adapters of many requests against a plain 64-bit form (needs
a GB300). Tolerances count roundings: see tests/_layer_ref.py."""
from __future__ import annotations

import pytest
import torch

import _layer_ref as R

pytestmark = pytest.mark.gpu

dt = pytest.importorskip("conditional_draft_tree_gb300")

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conditional_draft_tree_gb300 import build
    build.build()


def near(got, ref, slack, what=""):
    got = got.double().cpu()
    assert bool(torch.isfinite(got).all()), what
    over = (got - ref).abs() - slack
    assert float(over.max()) <= 0, f"{what}: over by {float(over.max()):.3g}"


class Case:
    """Inputs of one projection on the host, its 64-bit answer and the slack."""

    def __init__(self, batch, n, K, O, rank=0, count=0, dtype=BF, e8=False, index=None, scaled=True, seed=0):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g)
        self.batch, self.n, self.K, self.O, self.dtype, self.e8 = batch, n, K, O, dtype, e8
        self.x = rnd(batch * n, K).to(dtype)
        self.w = (rnd(O, K) * K ** -0.5).to(dtype)
        self.index = self.down = self.up = self.scale = None
        if rank:
            self.down = (rnd(count, rank, K) * K ** -0.5).to(dtype)
            self.up = (rnd(count, O, rank) * rank ** -0.5).to(dtype)
            self.scale = torch.rand(count, generator=g) * 2 - 0.5 if scaled else None
            self.index = torch.randint(-1, count, (batch,), generator=g, dtype=torch.int32) if index is None \
                else torch.tensor(index, dtype=torch.int32)
        vx, vw = self.x.double(), self.w.double()
        if e8:
            import _cache_ref
            self.x8, self.w8 = _cache_ref.quantise(self.x), _cache_ref.quantise(self.w)
            vx, vw = R.from_rows8(*self.x8), R.from_rows8(*self.w8)
        low = (self.index, self.x, self.down, self.up, self.scale)
        self.y = R.project(vx, vw, n, *low)
        self.slack = R.project_slack(vx, vw, n, self.y, dtype, *low)

    def cuda(self, x=None):
        """projection, x, adapters, index, x16 on the device."""
        shape = (self.batch, self.n)
        dev = lambda t: None if t is None else t.cuda()
        if self.e8:
            rows = lambda c, s: dt.Rows8(c[0].cuda().view(*s, -1), c[1].cuda().view(*s))
            p = dt.Projection(rows(self.w8, (self.O,)))
            x = rows(self.x8, shape)
            x16 = self.x.cuda().view(*shape, -1) if self.index is not None else None
        else:
            p, x, x16 = dt.Projection(self.w.cuda()), self.x.cuda().view(*shape, -1), None
        ad = dt.Adapters(dev(self.down), dev(self.up), dev(self.scale)) if self.index is not None else None
        return p, x, ad, dev(self.index), x16

    def check(self, **kw):
        p, x, ad, index, x16 = self.cuda()
        ws = None
        if ad is not None:      # nothing that an earlier call left there plays a part
            ws = dt.project_workspace(p, self.batch, self.n, ad)
            ws.fill_(0xff)
        got = dt.project(p, x, ad, index, x16, dtype=self.dtype, workspace=ws, **kw)
        near(got.reshape(-1, self.O), self.y, self.slack)
        p.check()
        again = dt.project(p, x, ad, index, x16, dtype=self.dtype, workspace=ws, **kw)
        assert torch.equal(got, again)       # the same sums in the same order
        return got


KINDS = [(BF, False), (FP, False), (BF, True), (FP, True)]


@pytest.mark.parametrize("dtype,e8", KINDS)
@pytest.mark.parametrize("batch,n,K,O", [
    (1, 1, 16, 1), (1, 1, 64, 128), (3, 1, 48, 7), (1, 5, 4096, 33), (8, 1, 1040, 129), (1, 16, 128, 257),
    (17, 1, 208, 128), (1, 33, 4112, 640), (5, 13, 256, 300), (2, 128, 144, 1000), (1, 129, 512, 512),
    (256, 1, 64, 200), (1, 257, 96, 129), (3, 171, 640, 777), (4, 300, 272, 1537), (1, 2049, 64, 64)])
def test_shared(batch, n, K, O, dtype, e8):
    Case(batch, n, K, O, dtype=dtype, e8=e8).check()


@pytest.mark.parametrize("dtype,e8", KINDS)
@pytest.mark.parametrize("batch,n,K,O,rank,count", [
    (1, 1, 16, 1, 16, 1), (1, 1, 4096, 128, 16, 2), (8, 1, 1040, 129, 16, 5), (33, 1, 64, 250, 32, 40),
    (130, 1, 96, 140, 16, 130), (256, 1, 144, 64, 16, 256), (300, 1, 80, 36, 48, 7), (5, 13, 256, 300, 64, 3),
    (2, 128, 144, 513, 128, 2), (1, 300, 208, 200, 16, 3), (40, 7, 128, 260, 112, 40), (7, 100, 320, 640, 80, 4),
    (70, 9, 272, 129, 96, 64), (3, 700, 64, 128, 64, 2), (2, 33, 4112, 640, 32, 2)])
def test_adapters(batch, n, K, O, rank, count, dtype, e8):
    Case(batch, n, K, O, rank, count, dtype, e8).check()


@pytest.mark.parametrize("dtype,e8", [(BF, False), (FP, True)])
@pytest.mark.parametrize("index", [[-1] * 6, [0] * 6, [2, -1, 2, -5, 2, 2], [0, 1, 2, 0, 1, 2], [-1, -1, -1, -1, -1, 1]])
@pytest.mark.parametrize("n", [1, 45])
def test_who_has_an_adapter(index, n, dtype, e8):
    Case(6, n, 192, 200, 32, 3, dtype, e8, index=index, scaled=False).check()


def test_a_large_matrix_and_many_rows():
    """Several tiles a block in both directions, and offsets of rows far apart."""
    Case(2, 1500, 448, 2100, 64, 2).check()
    Case(1, 700, 2048, 4500, e8=True).check()


@pytest.mark.parametrize("e8", [False, True])
def test_strides(e8):
    c = Case(3, 5, 80, 37, 16, 2, BF, e8, seed=1)
    p, x, ad, index, x16 = c.cuda()
    want = dt.project(p, x, ad, index, x16, dtype=BF)
    spread = lambda t, k: torch.cat([t, torch.full_like(t[..., :k], float("nan") if t.dtype != torch.uint8 else 0x7f)], -1)[..., :t.shape[-1]]
    if e8:
        wide = dt.Rows8(spread(x.codes.view(torch.uint8), 16), x.exps)
        w = dt.Projection(dt.Rows8(spread(p.weight.codes.view(torch.uint8), 32), p.weight.exps))
        y16 = spread(x16, 8)
    else:
        wide, y16, w = spread(x, 8), None, dt.Projection(spread(p.weight, 24))
    frame = torch.full((3, 5, 41), 7.0, dtype=BF, device="cuda")
    got = dt.project(w, wide, ad, index, y16, dtype=BF, out=frame[..., 3:40])
    assert torch.equal(got, want) and got.data_ptr() == frame.data_ptr() + 6
    assert bool((frame[..., :3] == 7).all()) and bool((frame[..., 40:] == 7).all())


def test_an_index_that_no_adapter_has():
    c = Case(4, 3, 64, 40, 16, 2, index=[1, -1, 0, 0])
    p, x, ad, index, _ = c.cuda()
    want = dt.project(p, x, ad, index)
    plain = dt.project(p, x)
    index[2], index[3] = 2, 2147483647
    got = dt.project(p, x, ad, index)
    assert torch.equal(got[:2], want[:2]) and torch.equal(got[2:], plain[2:])
    with pytest.raises(dt.DtError, match="adapter index"):
        p.check()


@pytest.mark.parametrize("e8", [False, True])
def test_what_is_not_finite_stays_in_its_row(e8):
    """A row of x with a NaN, one with an infinity, a row of W with a NaN; an adapter that no row
    has, full of them, and x A^T past fp16's range."""
    c = Case(6, 3, 128, 150, 16, 3, FP, e8, index=[0, 1, -1, 1, 0, -1], seed=2)
    want = c.check()
    c.down[2] = float("nan")
    c.up[2] = float("inf")
    p, x, ad, index, x16 = c.cuda()
    assert torch.equal(dt.project(p, x, ad, index, x16, dtype=FP), want)
    if e8:
        x.exps[1, 1] = 255
        x.codes.view(torch.uint8)[1, 1] = 0x7f
        p.weight.exps[7] = 255
        p.weight.codes.view(torch.uint8)[7] = 0x7f
    else:
        x[1, 1, 5] = float("nan")
        p.weight[7, 3] = float("nan")
    rows16 = x16 if e8 else x
    if not e8:
        x[2, 0, 9] = float("inf")
    rows16[4, 2] = 60000.0
    ad.down[0] = 1.0             # sums of 60000 K: past 65504, an infinity in that row
    got = dt.project(p, x, ad, index, x16, dtype=FP)
    bad = torch.zeros(6, 3, 150, dtype=torch.bool, device="cuda")
    bad[..., 7] = True
    bad[1, 1] = bad[4, 2] = True
    bad[2, 0] |= not e8
    moved = torch.zeros_like(bad)
    moved[0] = moved[4] = True   # rows with the adapter that was changed
    assert not bool(torch.isfinite(got[bad]).any())
    assert bool(torch.isfinite(got[~bad]).all()) and torch.equal(got[~bad & ~moved], want[~bad & ~moved])


def test_streams_graphs_and_a_shared_workspace():
    c, d = Case(5, 9, 256, 300, 16, 4, seed=3), Case(3, 2, 256, 300, 16, 4, seed=4)
    p, x, ad, index, _ = c.cuda()
    q, z, ad2, index2, _ = d.cuda()
    ws = dt.project_workspace(p, 5, 9, ad)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = dt.project(p, x, ad, index, workspace=ws, stream=stream)
    small = dt.project(q, z, ad2, index2, workspace=ws, stream=stream)     # one after the other
    stream.synchronize()
    near(got.reshape(-1, 300), c.y, c.slack)
    near(small.reshape(-1, 300), d.y, d.slack)
    out, out2 = torch.empty_like(got), torch.empty_like(small)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        dt.project(p, x, ad, index, out=out, workspace=ws)
    with torch.cuda.graph(graphs[1]):
        dt.project(q, z, ad2, index2, out=out2, workspace=ws)
    for _ in range(3):           # both use the workspace, in turn
        out.zero_()
        out2.zero_()
        graphs[0].replay()
        graphs[1].replay()
        graphs[0].replay()
        assert torch.equal(out, got) and torch.equal(out2, small)
    x.copy_(x.flip(0))
    index.copy_(index.flip(0))
    graphs[0].replay()
    near(out.reshape(-1, 300), c.y.view(5, 9, -1).flip(0).reshape(-1, 300), c.slack.view(5, 9, -1).flip(0).reshape(-1, 300))


@pytest.mark.parametrize("e8", [False, True])
def test_after_the_norm(e8):
    """The norm's rows go straight into the projection, in 16 bits or 8."""
    batch, n, K, O, dtype = 3, 7, 512, 260, BF
    g = torch.Generator().manual_seed(5)
    x, res = (torch.randn(batch, n, K, generator=g).to(dtype).cuda() for _ in range(2))
    norm = dt.Norm((1 + 0.1 * torch.randn(K, generator=g)).to(dtype).cuda())
    c = Case(batch, n, K, O, 16, 3, dtype, e8, seed=6)
    p, _, ad, index, _ = c.cuda()
    (y, r8), _ = dt.rms_norm(norm, x, res, kind="both")
    got = dt.project(p, r8, ad, index, x16=y) if e8 else dt.project(p, y, ad, index)
    vx = R.from_rows8(r8.codes.cpu(), r8.exps.cpu()).view(-1, K) if e8 else y.cpu().double().view(-1, K)
    vw = R.from_rows8(*c.w8) if e8 else c.w.double()
    low = (c.index, y.cpu().view(-1, K), c.down, c.up, c.scale)
    ref = R.project(vx, vw, n, *low)
    near(got.reshape(-1, O), ref, R.project_slack(vx, vw, n, ref, dtype, *low))


@pytest.mark.parametrize("dtype,e8", KINDS)
@pytest.mark.parametrize("batch,n,K,O,rank,count", [
    (6, 1, 128, 150, 16, 3), (40, 1, 1040, 300, 32, 9), (130, 1, 96, 140, 48, 130), (5, 45, 256, 513, 64, 3),
    (2, 128, 144, 513, 128, 2), (33, 65, 320, 4100, 16, 5), (256, 1, 64, 90, 16, 256)])
def test_an_adapter_that_is_not_finite_stays_with_its_requests(batch, n, K, O, rank, count, dtype, e8):
    """B rows with infinities and NaN: those outputs are NaN for the rows with that adapter, and all others
    what they were. The same for A, whose adapter's rows are not finite as a whole."""
    c = Case(batch, n, K, O, rank, count, dtype, e8, seed=7)
    p, x, ad, index, x16 = c.cuda()
    want = dt.project(p, x, ad, index, x16, dtype=dtype)
    used = sorted(set(int(a) for a in c.index.tolist() if a >= 0))
    one, two = used[0], used[-1]
    g = torch.Generator().manual_seed(8)
    bad = torch.zeros(batch, n, O, dtype=torch.bool)
    for a, value in ((one, float("nan")), (two, float("inf")), (two, -float("inf"))):
        rows = torch.randperm(O, generator=g)[:max(1, O // 9)]
        for o in rows.tolist():
            ad.up[a, o, int(torch.randint(0, rank, (1,), generator=g))] = value
        bad[(c.index == a).nonzero()[:, 0][:, None], :, rows[None]] = True
    bad = bad.cuda()
    for _ in range(2):
        got = dt.project(p, x, ad, index, x16, dtype=dtype)
        assert bool(got[bad].isnan().all()) and torch.equal(got[~bad], want[~bad])
    ad.up.copy_(c.up)
    assert torch.equal(dt.project(p, x, ad, index, x16, dtype=dtype), want)      # nothing is left of it
    ad.down[one, rank // 2, K // 3] = float("nan")
    whole = (index == one)[:, None, None].expand(batch, n, O)
    got = dt.project(p, x, ad, index, x16, dtype=dtype)
    assert bool(got[whole].isnan().all()) and torch.equal(got[~whole], want[~whole])
    p.check()


@pytest.mark.parametrize("batch,n,O", [(3, 5, 40), (4, 300, 700)])
def test_8bit_rows_far_apart_in_size(batch, n, O):
    """Rows of x and of W whose powers of two are far from each other's: products in fp32's range come out
    right whatever the two are."""
    K, g = 144, torch.Generator().manual_seed(9)
    x = torch.randn(batch * n, K, generator=g) * torch.exp2(torch.randint(-110, 111, (batch * n, 1), generator=g).float())
    w = torch.randn(O, K, generator=g) * torch.exp2(torch.randint(-110, 111, (O, 1), generator=g).float())
    x, w = x.to(BF), w.to(BF)
    x8, w8 = dt.quantize_rows(x.cuda()), dt.quantize_rows(w.cuda())
    vx, vw = R.from_rows8(x8.codes.cpu(), x8.exps.cpu()), R.from_rows8(w8.codes.cpu(), w8.exps.cpu())
    rows = dt.Rows8(x8.codes.view(batch, n, K), x8.exps.view(batch, n))
    got = dt.project(dt.Projection(w8), rows).reshape(-1, O).double().cpu()
    ref = R.project(vx, vw, n)
    # sums of codes within 2^9 K: past fp32's largest number they are infinite, below its least lost
    inside = (ref.abs() < 2.0 ** 127) & (ref.abs() > 2.0 ** -100)
    slack = R.project_slack(vx, vw, n, ref, BF)
    assert bool(((got - ref).abs()[inside] <= slack[inside]).all())
    assert bool((got[ref.abs() > 2.0 ** 129].isinf()).all()) and bool((got.abs()[ref.abs() < 2.0 ** -140] < 2.0 ** -130).all())
    assert int(inside.sum()) > 0.5 * ref.numel()      # (of two uniform exponents' sum)


@pytest.mark.parametrize("rows,K,O,e8", [(60000, 16, 40000, False), (600000, 4096, 9, False), (1200000, 4096, 24, True)])
def test_offsets_past_32_bits(rows, K, O, e8):
    """Results, or rows of x, of more than 4 GB; a sample of the rows."""
    g = torch.Generator(device="cuda").manual_seed(10)
    x = torch.empty(rows, K, dtype=BF, device="cuda").normal_(generator=g)
    w = torch.randn(O, K, generator=g, device="cuda").to(BF)
    at = torch.cat([torch.arange(5), torch.randint(0, rows, (40,)), torch.arange(rows - 5, rows)])
    if e8:
        x8, w8 = dt.quantize_rows(x), dt.quantize_rows(w)
        del x
        vx = R.from_rows8(x8.codes.view(torch.uint8)[at.cuda()].cpu().view(torch.float8_e4m3fn), x8.exps.cpu()[at])
        vw = R.from_rows8(w8.codes.cpu(), w8.exps.cpu())
        got = dt.project(dt.Projection(w8), dt.Rows8(x8.codes.view(1, rows, K), x8.exps.view(1, rows)))
    else:
        vx, vw = x[at.cuda()].cpu().double(), w.cpu().double()
        got = dt.project(dt.Projection(w), x.view(1, rows, K))
    ref = R.project(vx, vw, len(at))
    near(got[0, at.cuda()], ref, R.project_slack(vx, vw, len(at), ref, BF))


def test_two_streams_at_once():
    """Calls of different forms (pairs, clusters, few rows, 8-bit) side by side on two streams, each with a
    workspace of its own, among norms: the results of one call after the other."""
    cases = [Case(32, 65, 640, 1100, 16, 5, BF, False, seed=11), Case(9, 1, 2048, 700, 32, 9, BF, True, seed=12),
             Case(3, 400, 512, 900, 64, 3, FP, False, seed=13), Case(130, 1, 1024, 300, 16, 60, FP, True, seed=14)]
    made = [c.cuda() for c in cases]
    norm = dt.Norm(None)
    run = lambda c, m, **kw: dt.project(*m, dtype=c.dtype, **kw)
    wants = [run(c, m) for c, m in zip(cases, made)]
    x = torch.randn(3000, 1032, generator=torch.Generator().manual_seed(15)).to(BF).cuda()
    want = dt.rms_norm(norm, x, kind="both")
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [[dt.project_workspace(m[0], c.batch, c.n, m[2]) for c, m in zip(cases, made)] for _ in streams]
    torch.cuda.synchronize()
    got = [[], []]
    for k in range(25):
        for i, s in enumerate(streams):
            order = list(range(4)) if i == 0 else [3, 1, 2, 0]
            for j in order:
                got[i].append((j, run(cases[j], made[j], workspace=spaces[i][j], stream=s)))
            got[i].append((-1, dt.rms_norm(norm, x, kind="both", stream=s)))
    torch.cuda.synchronize()
    for j, y in got[0] + got[1]:
        if j >= 0:
            assert torch.equal(y, wants[j]), j
        else:
            assert torch.equal(y[0], want[0]) and torch.equal(y[1].exps, want[1].exps)
            assert torch.equal(y[1].codes.view(torch.uint8), want[1].codes.view(torch.uint8))
    for m in made:
        m[0].check()
