"""Rotary positions, paged-cache write, read and commit, and attention over the cache
against plain 64-bit implementations (needs a GB300).

What is moved or quantised without a rotation has one right answer: bit-exact. A
rotation is off by the fp32 slack of `turn_slack` and one rounding. Attention is off by
`attention_slack`: the output's rounding, the weights' rounding to 16 bits and fp32
accumulation, each bounded from the 64-bit run's own weights and values.
"""
from __future__ import annotations

import math

import pytest
import torch

import _cache_ref as R

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
    odd = ~torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    assert torch.equal(got[odd & ~torch.isnan(ref)], ref[odd & ~torch.isnan(ref)]), what
    over = ((got - ref).abs() - slack)[~odd]
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: over by {float(over.max()):.3g}"


def strided_heads(batch, H, Hkv, n, dh, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(batch, n, H + 2 * Hkv, dh, generator=g).to(dtype).cuda().transpose(1, 2)
    return x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]


# ------------------------------------------------------------------- rotary

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dh,rot,interleaved,scaling,factor", [
    (128, 128, False, "none", 1.0), (128, 64, True, "parts", 16.0), (64, 64, True, "linear", 4.5),
    (80, 40, False, "base", 4.0), (96, 8, False, "none", 1.0), (256, 256, True, "none", 1.0),
    (256, 120, False, "parts", 40.0), (16, 16, False, "none", 1.0), (80, 72, True, "base", 2.0)])
def test_rotary(dtype, dh, rot, interleaved, scaling, factor):
    batch, H, Hkv, n = 2, 5, 2, 7
    q, k, _ = strided_heads(batch, H, Hkv, n, dh, dtype, 1)
    pos = torch.tensor([0, 1, -5, 4095, 131071, 1000003, 2147483647] * batch, dtype=torch.int32).view(batch, n)
    r = dt.Rotary(rot, interleaved, 10000.0, scaling, factor, trained=4096)
    f, mag = R.frequencies(rot, 10000.0, scaling, factor, 4096.0)
    for gradient in (False, True):
        got = dt.rotary(r, pos.cuda(), q, k, gradient=gradient)
        for x, y in zip((q, k), got):
            x = x.cpu()
            ref = R.turn(x, pos, f, mag, interleaved, gradient)
            # the 64-bit angle itself: positions to 2^31 times a rounding of 2^-52
            slack = R.HALF[dtype] * ref.abs() + R.TINY[dtype] + 2 * R.turn_slack(x, rot, mag, interleaved)
            near(y, ref, slack, f"gradient={gradient}")
            assert torch.equal(y[..., rot:].cpu(), x[..., rot:])
    alone = dt.rotary(r, pos.cuda(), q)
    assert torch.equal(alone, dt.rotary(r, pos.cuda(), q, k)[0])


def test_rotary_in_place_and_many_rows():
    batch, H, Hkv, n, dh = 3, 32, 8, 601, 128       # four tokens a block, the last block one
    q, k, _ = strided_heads(batch, H, Hkv, n, dh, BF, 2)
    pos = torch.arange(n, dtype=torch.int32)[None].repeat(batch, 1).contiguous().cuda()
    r = dt.Rotary(dh)
    want_q, want_k = dt.rotary(r, pos, q, k)
    f, mag = R.frequencies(dh)
    ref = R.turn(q.cpu(), pos.cpu(), f, mag, False)
    near(want_q, ref, R.HALF[BF] * ref.abs() + 2 * R.turn_slack(q.cpu(), dh, mag, False))
    got = dt.rotary(r, pos, q, k, q_out=q, k_out=k)
    assert torch.equal(got[0], want_q) and torch.equal(got[1], want_k)


def test_rotary_gradient_is_the_derivative():
    """Differences of the 64-bit sum(y w) along random directions against the kernel's
    gradient of it; fp16 inputs, the kernel's rounding bounded as above."""
    batch, H, n, dh = 1, 2, 3, 64
    x, _, w = strided_heads(batch, H, H, n, dh, FP, 3)
    pos = torch.tensor([[3, 77, 1234]], dtype=torch.int32)
    r = dt.Rotary(48, True, 10000.0, "parts", 8.0, trained=512)
    f, mag = R.frequencies(48, 10000.0, "parts", 8.0, 512.0)
    grad = dt.rotary(r, pos.cuda(), w, gradient=True).double().cpu()
    g = torch.Generator().manual_seed(4)
    loss = lambda z: (R.turn(z, pos, f, mag, True) * w.double().cpu()).sum()
    for _ in range(3):
        d = torch.randn(x.shape, generator=g, dtype=torch.float64)
        diff = (loss(x.double().cpu() + 1e-3 * d) - loss(x.double().cpu() - 1e-3 * d)) / 2e-3   # linear: exact
        slack = ((R.HALF[FP] * grad.abs() * 1.01 + R.TINY[FP] + 2 * R.turn_slack(w.cpu(), 48, mag, True)) * d.abs()).sum()
        assert abs(float((grad * d).sum() - diff)) <= float(slack) + 1e-9 * abs(float(diff))


def test_rotary_replays_in_a_graph_on_another_stream():
    q, k, _ = strided_heads(2, 4, 2, 9, 64, BF, 5)
    pos = torch.arange(18, dtype=torch.int32).view(2, 9).cuda()
    r = dt.Rotary(64)
    want = dt.rotary(r, pos, q, k)
    torch.cuda.synchronize()
    q2, k2 = torch.empty_like(want[0]), torch.empty_like(want[1])
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        dt.rotary(r, pos, q, k, q2, k2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])


# -------------------------------------------------------------- cache write

WRITES = [(BF, "16", 128, 64), (FP, "16", 64, 16), (BF, "e4m3", 128, 64), (FP, "e4m3", 80, 16),
          (BF, "e4m3", 256, 128), (BF, "16", 80, 32), (FP, "e4m3", 16, 32), (BF, "e4m3", 96, 16)]


@pytest.mark.parametrize("dtype,kind,dh,page", WRITES)
@pytest.mark.parametrize("n", [1, 37])
def test_write_and_read_bit_exact(dtype, kind, dh, page, n):
    batch, H, Hkv = 3, 4, 2
    _, k, v = strided_heads(batch, H, Hkv, n, dh, dtype, 10)
    # magnitudes over the types' whole range, zeros and the values at the codes' borders
    g = torch.Generator().manual_seed(11)
    lim = 14 if dtype == FP else 120
    amp = torch.exp2(torch.randint(-lim, lim, (batch, n, H + 2 * Hkv), generator=g).float()).cuda()
    base = k._base if k._base is not None else k
    base.view(batch, n, H + 2 * Hkv, dh).mul_(amp[..., None].to(torch.float32)).nan_to_num_(posinf=3e38 if dtype == BF else 65504.0, neginf=-3e38 if dtype == BF else -65504.0)
    k[0, 0, 0] = 0
    v[0, 0, 0, :4] = torch.tensor([448.0, 464.0, 0.0, -0.0], dtype=dtype)
    v[0, 0, 0, 4:] = 1.0
    first, counts = torch.tensor([0, 13, 70], dtype=torch.int32), torch.tensor([n, max(0, n - 5), 1], dtype=torch.int32)
    cache = R.make_cache(dt, kind, dtype, batch, 110, Hkv, page, dh, 12, fill=False)
    before = {w: getattr(cache, w).clone() for w in ("k", "v")}
    assert dt.cache_write(cache, k, v, first.cuda(), counts.cuda()) is None
    got_k, got_v = dt.cache_read(cache, n, first.cuda(), counts.cuda(), dtype=dtype)
    cache.check()
    for which, x, got in (("k", k, got_k), ("v", v, got_v)):
        want = before[which].cpu()
        wexp = torch.full(want.shape[:3], 127, dtype=torch.uint8)
        back = torch.zeros(batch, Hkv, n, dh, dtype=dtype)
        for b in range(batch):
            for i in range(int(counts[b])):
                j = int(first[b]) + i
                p, sl = int(cache.table[b, j // page]), j % page
                row = x[b, :, i].cpu()
                if kind == "e4m3":
                    code, e = R.quantise(row)
                    want.view(torch.uint8)[p, :, sl], wexp[p, :, sl] = code, e
                    val = R.dequantise(code, e)
                    back[b, :, i] = (val.clamp(-65504, 65504) if dtype == FP else val).to(dtype)
                else:
                    want[p, :, sl] = row
                    back[b, :, i] = row
        bits = torch.uint8 if kind == "e4m3" else torch.int16
        assert torch.equal(getattr(cache, which).cpu().view(bits), want.view(bits)), which
        if kind == "e4m3":
            assert torch.equal(getattr(cache, which + "_exp").cpu(), wexp), which
        assert torch.equal(got.cpu().view(torch.int16), back.view(torch.int16)), which


def test_8bit_rows_with_nan_infinity_and_the_largest_values():
    n, dh = 5, 32
    k = torch.ones(1, 1, n, dh, dtype=BF, device="cuda")
    k[0, 0, 0, 3] = math.nan
    k[0, 0, 1, 0] = math.inf
    k[0, 0, 2, 31] = torch.finfo(BF).max
    k[0, 0, 3] = 2.0 ** -133           # the least bf16 number: below every step of the least scale
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    cache = dt.PagedCache.empty(1, 1, 16, dh, table, torch.float8_e4m3fn)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    dt.cache_write(cache, k, -k, zero)
    gk, gv = dt.cache_read(cache, n, zero)
    assert torch.isnan(gk[0, 0, :2]).all() and torch.isnan(gv[0, 0, :2]).all()
    assert gk[0, 0, 2, 31] == 240.0 * 2.0 ** 120 and gv[0, 0, 2, 31] == -240.0 * 2.0 ** 120
    assert (gk[0, 0, 3] == 0).all() and (gk[0, 0, 4] == 1).all() and (gv[0, 0, 4] == -1).all()


@pytest.mark.parametrize("kind", ["16", "e4m3"])
@pytest.mark.parametrize("n,dh,rot", [(1, 128, 128), (33, 80, 40), (700, 128, 64)])
def test_write_turns_k_and_q(kind, n, dh, rot):
    batch, H, Hkv, page = 2, 6, 2, 32
    q, k, v = strided_heads(batch, H, Hkv, n, dh, BF, 20)
    first = torch.tensor([5, 64], dtype=torch.int32)
    pos = (first[:, None] + torch.arange(n)[None] % 16).to(torch.int32).contiguous()
    r = dt.Rotary(rot)
    cache = R.make_cache(dt, kind, BF, batch, 64 + n, Hkv, page, dh, 21, fill=False)
    q_out = dt.cache_write(cache, k, v, first.cuda(), rotary=r, positions=pos.cuda(), q=q)
    cache.check()
    assert torch.equal(q_out, dt.rotary(r, pos.cuda(), q))
    f, mag = R.frequencies(rot)
    turned = R.turn(k.cpu(), pos, f, mag, False)
    noise = 2 * R.turn_slack(k.cpu(), rot, mag, False)
    for b in range(batch):
        rows = range(int(first[b]), int(first[b]) + n)
        got_k, got_v = R.pool_rows(cache, "k", b, rows), R.pool_rows(cache, "v", b, rows)
        if kind == "16":
            near(got_k, turned[b], R.HALF[BF] * turned[b].abs() + noise[b])
            assert torch.equal(got_v, v[b].cpu().double())
        else:
            # half a step of 2^-4, or of the least step 2^-9 2^e, e one more where the
            # largest value sits at a border
            e = R.exponent(turned[b].abs().amax(-1)) + 1
            step = torch.pow(2.0, e.double() - 10)[..., None]
            near(got_k, turned[b], 2.0 ** -4 * turned[b].abs() + step + 2 * noise[b])
            code, ex = R.quantise(v[b].cpu())
            assert torch.equal(got_v, R.dequantise(code, ex))


def test_rows_outside_the_table_or_the_pool_are_reported_and_skipped():
    batch, Hkv, n, dh, page = 4, 2, 20, 64, 16
    _, k, v = strided_heads(batch, 2, Hkv, n, dh, BF, 30)
    cache = R.make_cache(dt, "16", BF, batch, 48, Hkv, page, dh, 31, fill=False)
    cache.table[1, 1] = cache.k.shape[0]        # past the pool
    cache.table[2, 0] = -1
    first = torch.tensor([40, 0, 0, -3], dtype=torch.int32).cuda()   # request 0 runs past its table
    before = cache.k.clone()
    dt.cache_write(cache, k, v, first)
    gk, _ = dt.cache_read(cache, n, first)
    assert cache.status.tolist() == [dt.ERR_BAD_PAGE] * 4
    with pytest.raises(dt.DtError, match="request 0"):
        cache.check()
    good = {0: range(0, 8), 1: range(0, 16), 2: range(16, 20), 3: range(3, 20)}
    for b in range(batch):
        for i in range(n):
            want = k[b, :, i] if i in good[b] else torch.zeros_like(k[b, :, i])
            assert torch.equal(gk[b, :, i], want), (b, i)
    untouched = torch.ones(cache.k.shape[0], page, dtype=torch.bool)
    for b in range(batch):
        for i in good[b]:
            j = int(first[b]) + i
            untouched[int(cache.table[b, j // page]), j % page] = False
    at = untouched.cuda()[:, None, :].expand(before.shape[:3])
    assert torch.equal(cache.k.view(torch.int16)[at], before.view(torch.int16)[at])
    q = torch.randn(batch, 4, n, dh).to(BF).cuda()
    cache.status.zero_()
    out = dt.cache_attention(cache, q, torch.tensor([28, 28, 28, -1], dtype=torch.int32).cuda())
    assert [c != 0 for c in cache.status.tolist()] == [False, True, True, True]


# ------------------------------------------------------------------- commit

@pytest.mark.parametrize("kind,dh,page", [("16", 128, 64), ("e4m3", 128, 16), ("16", 80, 32), ("e4m3", 256, 16)])
def test_commit_moves_the_path_and_nothing_else(kind, dh, page):
    batch, Hkv, n = 5, 2, 70
    cache = R.make_cache(dt, kind, BF, batch, 200, Hkv, page, dh, 40)
    first = torch.tensor([0, 15, 63, 100, 7], dtype=torch.int32)
    paths = [[0, 3, 9, 30, 69], [0, 1, 2, 3, 4], [0, 65], [0, 5, 4, 0, 2], []]      # one out of order
    width = 6
    path = torch.full((batch, width), 99, dtype=torch.int32)                        # unused entries
    for b, p in enumerate(paths):
        path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    lengths = torch.tensor([len(p) for p in paths], dtype=torch.int32)
    old = {w: getattr(cache, w).cpu().clone() for w in ("k", "v", "k_exp", "v_exp") if getattr(cache, w) is not None}
    dt.cache_commit(cache, first.cuda(), path.cuda(), lengths.cuda(), n)
    cache.check()
    table = cache.table.cpu()
    for w, x in old.items():
        want = x.clone()
        for b, p in enumerate(paths):
            for j, t in enumerate(p):
                a, z = int(first[b]) + t, int(first[b]) + j
                want[int(table[b, z // page]), :, z % page] = x[int(table[b, a // page]), :, a % page]
        bits = torch.uint8 if x.element_size() == 1 else torch.int16
        assert torch.equal(getattr(cache, w).cpu().view(bits), want.view(bits)), w


def test_commit_reports_rows_outside_the_tree():
    cache = R.make_cache(dt, "16", BF, 2, 64, 1, 16, 64, 41)
    old = cache.k.clone()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    dt.cache_commit(cache, i32([3, 3]), i32([[5, 20], [-1, 7]]), i32([2, 2]), 20)
    assert cache.status.tolist() == [dt.ERR_BAD_PAGE] * 2
    t = cache.table.cpu()
    want = old.clone()
    want[int(t[0, 0]), :, 3] = old[int(t[0, 0]), :, 8]       # 3 + 5 -> 3; 20 is no row of 20
    want[int(t[1, 0]), :, 4] = old[int(t[1, 0]), :, 10]      # 3 + 7 -> 4
    assert torch.equal(cache.k.view(torch.int16), want.view(torch.int16))


# ---------------------------------------------------------------- attention

def tree_mask(batch, n, seed, blank=()):
    g = torch.Generator().manual_seed(seed)
    m = torch.zeros(batch, n, n, dtype=torch.uint8)
    for b in range(batch):
        for i in range(n):
            if i:
                p = int(torch.randint(0, i, (1,), generator=g))
                m[b, i] = m[b, p]
            m[b, i, i] = 1
    for i in blank:
        if i < n:
            m[:, i] = 0
    return m


def run_attention(kind, dtype, n, G, Hkv, dh, page, prefix, counts=None, mask="tree", blank=(), seed=50,
                  scale=None, qamp=1.0, edit=None, qpos=False):
    batch = len(prefix)
    rows = max(prefix) + n
    cache = R.make_cache(dt, kind, dtype, batch, rows, Hkv, page, dh, seed)
    R.poison_behind(cache, [p + (counts[b] if counts else n) for b, p in enumerate(prefix)])
    if edit:
        edit(cache)
    g = torch.Generator().manual_seed(seed + 1)
    q = (qamp * torch.randn(batch, n, Hkv * G, dh, generator=g)).to(dtype).transpose(1, 2)
    if qpos:
        q = q.abs()
    m = tree_mask(batch, n, seed + 2, blank) if mask == "tree" else None
    pre = torch.tensor(prefix, dtype=torch.int32)
    cnt = torch.tensor(counts, dtype=torch.int32) if counts else None
    sc = dh ** -0.5 if scale is None else scale
    got = dt.cache_attention(cache, q.cuda(), pre.cuda(),
                             m.cuda() if m is not None else None, cnt.cuda() if cnt is not None else None, sc)
    cache.check()
    ref, mass, big = R.attention(cache, q, pre, m, cnt, sc)
    near(got, ref, R.attention_slack(ref, mass, big, dtype, dh, rows), f"{kind} {dtype} n={n} G={G} dh={dh}")
    return got


# (n, G): 1 to 1040 stacked rows, on and off the tiles' edges
@pytest.mark.parametrize("n,G", [(1, 1), (1, 4), (3, 5), (1, 16), (17, 1), (8, 4), (9, 4), (16, 4), (33, 2),
                                 (64, 2), (65, 4), (129, 1), (130, 8)])
@pytest.mark.parametrize("kind,dtype", [("16", BF), ("16", FP), ("e4m3", BF), ("e4m3", FP)])
def test_attention_rows_and_types(n, G, kind, dtype):
    run_attention(kind, dtype, n, G, 2, 128, 32, [0, 1, 63, 64, 200], [n, max(1, n - 3), n, 1, n])


@pytest.mark.parametrize("dh", [16, 64, 80, 96, 112, 192, 256])
@pytest.mark.parametrize("kind", ["16", "e4m3"])
@pytest.mark.parametrize("n", [1, 20, 70])
def test_attention_head_sizes(dh, kind, n):
    run_attention(kind, BF, n, 4, 1, dh, 16, [37, 130])


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [1, 12, 100])
def test_attention_pages_and_long_prefixes(page, n):
    """Lengths around the pages' and tiles' edges; 3000 keys are cut over many blocks."""
    run_attention("16", BF, n, 4, 1, 64, page, [page - 1, page, page + 1, 127, 128, 129, 3000])


@pytest.mark.parametrize("kind", ["16", "e4m3"])
@pytest.mark.parametrize("n", [1, 2, 31, 128, 300])
def test_attention_causal_chunks(kind, n):
    run_attention(kind, BF, n, 4, 2, 128, 64, [0, 5, 500], [n, max(1, n // 2), n], mask="causal")


@pytest.mark.parametrize("n", [6, 40])
def test_rows_that_see_nothing_are_zero(n):
    got = run_attention("16", BF, n, 4, 2, 64, 16, [0, 0, 9], [n, 0, 0], blank=(0, 3, 5))
    assert (got[0, :, [0, 3, 5]] == 0).all() and (got[1:] == 0).all()


@pytest.mark.parametrize("n", [7, 64])
@pytest.mark.parametrize("kind", ["16", "e4m3"])
def test_rows_not_seen_may_hold_anything(kind, n):
    """NaN and infinities in tree rows' keys and values reach the rows that see them and
    no other."""
    def edit(cache):
        page = cache.k.shape[2]
        for b, pre in enumerate((3, 130)):
            for t, val in ((1, math.nan), (4, math.inf)):
                j = pre + t
                p, s = int(cache.table[b, j // page]), j % page
                if kind == "e4m3":
                    cache.v_exp[p, 0, s] = 255
                    cache.v.view(torch.uint8)[p, 0, s] = 0x7f
                else:
                    cache.v[p, 0, s, 5] = val
                    cache.v[p, 1, s, :] = -val
            j = pre + 2
            p, s = int(cache.table[b, j // page]), j % page
            if kind == "16":
                cache.k[p, 0, s, 0] = math.nan
    run_attention(kind, BF, n, 2, 2, 64, 16, [3, 130], edit=edit)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("qamp", [1e-3, 30.0])
def test_attention_flat_and_peaked_scores(n, qamp):
    run_attention("16", FP, n, 4, 1, 128, 64, [700, 64], qamp=qamp)
    run_attention("16", BF, n, 4, 1, 128, 64, [700, 64], qamp=qamp, scale=-0.05)


def test_attention_many_requests():
    """More requests than threads of a block, ragged, most of them short."""
    prefix = [(37 * b) % 90 for b in range(300)]
    run_attention("16", BF, 2, 2, 1, 64, 16, prefix)


def test_attention_result_does_not_depend_on_the_run():
    cache = R.make_cache(dt, "e4m3", BF, 3, 5000, 2, 64, 128, 60)
    q = torch.randn(3, 8, 65, 128, generator=torch.Generator().manual_seed(61)).to(BF).cuda()
    pre = torch.tensor([4900, 11, 2500], dtype=torch.int32).cuda()
    mask = tree_mask(3, 65, 62).cuda()
    ws = dt.cache_attention_workspace(cache, 8, 65)
    a = dt.cache_attention(cache, q, pre, mask, workspace=ws)
    for _ in range(5):
        assert torch.equal(a, dt.cache_attention(cache, q, pre, mask, workspace=ws))


def test_attention_equals_the_dense_layer():
    """The framework's dense tree attention over the rows that the cache gives back."""
    batch, H, Hkv, n, P, dh = 2, 8, 2, 33, 96, 128
    cache = R.make_cache(dt, "e4m3", BF, batch, P + n, Hkv, 32, dh, 70)
    q = torch.randn(batch, H, n, dh, generator=torch.Generator().manual_seed(71)).to(BF).cuda()
    mask = tree_mask(batch, n, 72).cuda()
    pre = torch.tensor([P, P], dtype=torch.int32).cuda()
    got = dt.cache_attention(cache, q, pre, mask)
    k, v = dt.cache_read(cache, P + n, torch.zeros_like(pre))
    want = dt.tree_attention(q, k, v, mask, pre).double().cpu()
    ref, mass, big = R.attention(cache, q.cpu(), pre.cpu(), mask.cpu(), None, dh ** -0.5)
    near(got, want, R.attention_slack(ref, mass, big, BF, dh, P + n) + 2e-4)


def test_attention_replays_in_a_graph():
    cache = R.make_cache(dt, "16", BF, 2, 400, 2, 64, 64, 80)
    q = torch.randn(2, 4, 5, 64, generator=torch.Generator().manual_seed(81)).to(BF).cuda()
    pre = torch.tensor([390, 100], dtype=torch.int32).cuda()
    ws = dt.cache_attention_workspace(cache, 4, 5)
    out = torch.empty_like(q)
    dt.cache_attention(cache, q, pre, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dt.cache_attention(cache, q, pre, out=out, workspace=ws)
    pre.copy_(torch.tensor([7, 395], dtype=torch.int32))       # lengths are read on the device
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, dt.cache_attention(cache, q, pre))


def test_pool_past_32_bit_offsets():
    """A pool of more than 2^32 bytes and 2^31 elements; the rows used lie at its end."""
    page, Hkv, dh = 128, 8, 128
    pages = (1 << 31) // (page * Hkv * dh) + 40
    table = torch.arange(pages - 1, pages - 4, -1, dtype=torch.int32).view(1, 3).contiguous().cuda()
    cache = dt.PagedCache.empty(pages, Hkv, page, dh, table, BF)
    g = torch.Generator().manual_seed(90)
    k, v = (torch.randn(1, Hkv, 300, dh, generator=g).to(BF).cuda() for _ in range(2))
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    dt.cache_write(cache, k, v, zero)
    gk, gv = dt.cache_read(cache, 300, zero)
    assert torch.equal(gk, k) and torch.equal(gv, v)
    q = torch.randn(1, 16, 10, dh, generator=g).to(BF).cuda()
    small = dt.PagedCache.empty(3, Hkv, page, dh, torch.arange(3, dtype=torch.int32).view(1, 3).cuda(), BF)
    dt.cache_write(small, k, v, zero)
    pre = zero + 290
    assert torch.equal(dt.cache_attention(cache, q, pre), dt.cache_attention(small, q, pre))
    dt.cache_commit(cache, pre, torch.tensor([[2, 9]], dtype=torch.int32).cuda(), zero + 2, 10)
    gk, _ = dt.cache_read(cache, 2, pre)
    assert torch.equal(gk, k[:, :, [292, 299]])
    cache.check()


@pytest.mark.parametrize("kind", ["16", "e4m3"])
@pytest.mark.parametrize("dh", [64, 128])
def test_single_tokens_with_long_8bit_and_16bit_caches(kind, dh):
    """Many key tiles a block, the last of them cut by the length, poison behind it."""
    run_attention(kind, BF, 1, 4, 8, dh, 64, [8000, 7777, 4095, 513, 1, 6000], mask="tree")


@pytest.mark.parametrize("n,G", [(1, 4), (20, 2), (30, 5), (70, 4)])
@pytest.mark.parametrize("kind", ["16", "e4m3"])
def test_many_short_units_a_block(n, G, kind):
    """More units than blocks, of one to three key tiles each: a block passes from unit to
    unit many times, and holds most of them whole."""
    prefix = [(29 * b) % 300 for b in range(90)]
    run_attention(kind, BF, n, G, 8, 64, 16, prefix, [1 + (b * 7) % n for b in range(90)])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n", [1, 40])
def test_8bit_codes_of_every_size_count(dtype, n):
    """Rows whose codes are the least ones beside a single large one, and rows of very
    different scales: the values come out as they are."""
    def edit(cache):
        g = torch.Generator().manual_seed(7)
        code = torch.randint(0, 8, cache.v.shape, generator=g, dtype=torch.uint8)          # 0 to 7/512
        code |= torch.randint(0, 2, cache.v.shape, generator=g, dtype=torch.uint8) << 7     # signs
        code[..., 3] = 0x7e                                                                # 448
        cache.v.view(torch.uint8).copy_(code)
        cache.v_exp.copy_(torch.randint(100, 120, cache.v_exp.shape, generator=g, dtype=torch.uint8))
        code = torch.randint(0, 8, cache.k.shape, generator=g, dtype=torch.uint8)
        code[..., 5] = 0x70
        cache.k.view(torch.uint8).copy_(code)
        cache.k_exp.copy_(torch.randint(118, 124, cache.k_exp.shape, generator=g, dtype=torch.uint8))
    run_attention("e4m3", dtype, n, 2, 2, 128, 16, [3, 130], edit=edit)


@pytest.mark.parametrize("n", [1, 40])
def test_one_huge_value_that_hardly_counts(n):
    """A row of 2^60 whose weight is 2^-100 and less beside ordinary rows."""
    def edit(cache):
        for b in range(2):
            p = int(cache.table[b, 0])
            cache.v_exp[p, :, 2] = 127 + 60
            cache.k.view(torch.uint8)[p, :, 2] = 0xfe         # -448 2^-3 in every place
            cache.k_exp[p, :, 2] = 124
            cache.k.view(torch.uint8)[p, :, 5] = 0x78         # 256 2^-5: the row that is looked at
            cache.k_exp[p, :, 5] = 122
    run_attention("e4m3", BF, n, 2, 1, 64, 16, [20, 130], edit=edit, qpos=True)


@pytest.mark.parametrize("kind,n,G", [("e4m3", 129, 4), ("e4m3", 1, 4), ("e4m3", 70, 1), ("16", 65, 4), ("16", 3, 4)])
def test_repeated_runs_agree_bit_for_bit(kind, n, G):
    """Long enough for every ring to turn many times, with whole units, cut ones, and tiles
    of one and of two row tiles; no run may time out."""
    cache = R.make_cache(dt, kind, BF, 6, 9000, 4, 64, 128, 95)
    g = torch.Generator().manual_seed(96)
    q = torch.randn(6, 4 * G, n, 128, generator=g).to(BF).cuda()
    pre = torch.tensor([8800, 17, 300, 5000, 128, 2049], dtype=torch.int32).cuda()
    ws = dt.cache_attention_workspace(cache, 4 * G, n)
    want = dt.cache_attention(cache, q, pre, workspace=ws)
    differ = torch.zeros((), dtype=torch.int32, device="cuda")
    for _ in range(150):
        differ += (dt.cache_attention(cache, q, pre, workspace=ws).view(torch.int16) != want.view(torch.int16)).any()
    cache.check()
    assert int(differ) == 0
