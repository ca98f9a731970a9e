"""Paths of the paged-cache operators that need many rows, large heads or a stream of
their own (needs a GB300). Against 64-bit forms; what is moved or quantised bit for bit."""
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def normal(batch, heads, n, dh, dtype, seed, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    return (amp * torch.randn(batch, n, heads, dh, generator=g)).to(dtype).transpose(1, 2)


# 65536 head rows or more: a block takes several tokens, some of them of two requests, and the
# last one fewer than the others (7063 tokens: at 152 SMs 12 a block, 7 in the last)
@pytest.mark.parametrize("kind,dtype,dh,Hkv,H", [("16", BF, 64, 8, 8), ("e4m3", BF, 128, 8, 0), ("e4m3", FP, 80, 12, 8),
                                                 ("16", FP, 256, 10, 0), ("e4m3", BF, 256, 8, 8)])
@pytest.mark.parametrize("turned", [False, True])
def test_many_rows_written_and_read(kind, dtype, dh, Hkv, H, turned):
    batch, n, page = 7, 1009, 32         # 7063 tokens
    assert batch * n * (2 * Hkv + (H if turned else 0)) >= 65536
    k, v = normal(batch, Hkv, n, dh, dtype, 400).cuda(), normal(batch, Hkv, n, dh, dtype, 401).cuda()
    first = [0, 5, 31, 32, 100, 7, 64]
    counts = [n, n - 1, 17, 0, n, 500, n]
    cache = R.make_cache(dt, kind, dtype, batch, n + 100, Hkv, page, dh, 402, fill=False)
    kw = {}
    if turned:
        pos = (torch.tensor(first)[:, None] + torch.arange(n)).to(torch.int32).contiguous()
        r = dt.Rotary(dh // 2 // 8 * 8)
        kw = dict(rotary=r, positions=pos.cuda())
        if H:
            kw["q"] = q = normal(batch, H, n, dh, dtype, 403).cuda()
    q_out = dt.cache_write(cache, k, v, i32(first), i32(counts), **kw)
    cache.check()
    gk, gv = dt.cache_read(cache, n, i32(first), i32(counts), dtype=dtype)
    cache.check()
    for b in range(batch):
        c, rows = counts[b], range(first[b], first[b] + counts[b])
        assert bool((gk[b, :, c:] == 0).all()) and bool((gv[b, :, c:] == 0).all())
        if not c:
            continue
        got_k, got_v = R.pool_rows(cache, "k", b, rows), R.pool_rows(cache, "v", b, rows)
        for x, got, back in ((v, got_v, gv),) + (() if turned else ((k, got_k, gk),)):
            want = x[b, :, :c].cpu()
            want = R.dequantise(*R.quantise(want)) if kind == "e4m3" else want.double()
            assert torch.equal(got, want)
            assert torch.equal(back[b, :, :c].cpu(), want.clamp(-65504, 65504).to(dtype) if dtype == FP else want.to(dtype))
        if turned:
            f, mag = R.frequencies(r.rot)
            x = k[b:b + 1, :, :c].cpu()
            ref = R.turn(x, pos[b:b + 1, :c], f, mag, False)[0]
            noise = 2 * R.turn_slack(x, r.rot, mag, False)[0]
            if kind == "16":
                near(got_k, ref, R.HALF[dtype] * ref.abs() + R.TINY[dtype] + noise)
            else:
                step = torch.pow(2.0, (R.exponent(ref.abs().amax(-1)) + 1).double() - 10)[..., None]
                near(got_k, ref, 2.0 ** -4 * ref.abs() + step + 2 * noise)
    # nothing else was touched: exponents of other slots as they were
    if kind == "e4m3":
        other = torch.ones(cache.k.shape[0], page, dtype=torch.bool)
        for b in range(batch):
            for j in range(first[b], first[b] + counts[b]):
                other[int(cache.table[b, j // page]), j % page] = False
        assert bool((cache.v_exp.cpu()[other[:, None].expand(cache.v_exp.shape)] == 127).all())
    if turned and H:
        assert torch.equal(q_out, dt.rotary(r, pos.cuda(), q))


def test_calls_on_a_stream_of_their_own():
    """Each call behind a wait on another stream, with nothing allocated beforehand, while the
    current stream's memory is handed out and written over."""
    batch, H, Hkv, n, dh, rows = 3, 8, 2, 20, 128, 900
    q, k, v = (normal(batch, h, n, dh, BF, 410 + h).cuda() for h in (H, Hkv, Hkv + 1))
    v = v[:, :Hkv]
    r, first = dt.Rotary(dh), i32([880, 33, 400])
    pos = (first[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)).contiguous()
    path, lengths = i32([[0, 4, 9], [1, 2, 3], [0, 19, 5]]), i32([3, 2, 3])

    def everything(cache, stream):
        a = dt.cache_write(cache, k, v, first, rotary=r, positions=pos, q=q, stream=stream)
        b = dt.cache_attention(cache, a, first, stream=stream)
        dt.cache_commit(cache, first, path, lengths, n, stream=stream)
        return (a, b) + dt.cache_read(cache, n, first, stream=stream) + dt.rotary(r, pos, q, k, stream=stream)

    caches = [R.make_cache(dt, "16", BF, batch, rows, Hkv, 64, dh, 411) for _ in range(2)]
    want = everything(caches[0], None)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(50_000_000)
    got = everything(caches[1], stream)
    sizes = [t.numel() * 2 for t in got] + [dt.cache_attention_workspace(caches[0], H, n).numel()]
    junk = [torch.full((s,), 0xff, dtype=torch.uint8, device="cuda") for s in sizes * 2]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(caches[0].k, caches[1].k)
    caches[1].check()
    del junk


def attend(kind, dtype, n, G, Hkv, dh, prefix, counts=None, mask=None, edit=None, seed=420, page=16):
    batch, rows = len(prefix), max(prefix) + n
    cache = R.make_cache(dt, kind, dtype, batch, rows, Hkv, page, dh, seed)
    R.poison_behind(cache, [p + (counts[b] if counts else n) for b, p in enumerate(prefix)])
    if edit:
        edit(cache)
    q, scale = normal(batch, Hkv * G, n, dh, dtype, seed + 1), dh ** -0.5
    got = dt.cache_attention(cache, q.cuda(), i32(prefix), mask.cuda() if mask is not None else None,
                             i32(counts) if counts else None)
    cache.check()
    ref, mass, big = R.attention(cache, q, torch.tensor(prefix), mask, torch.tensor(counts) if counts else None, scale)
    near(got, ref, R.attention_slack(ref, mass, big, dtype, dh, rows), f"{kind} {dtype} n={n} dh={dh}")


def chains(batch, n):
    """Masks of trees of two interleaved chains under a root; row 0 sees nothing."""
    i, j = torch.arange(n)[:, None], torch.arange(n)[None]
    m = ((j <= i) & ((i - j) % 2 == 0)).to(torch.uint8)
    m[0] = 0
    return m[None].repeat(batch, 1, 1)


@pytest.mark.parametrize("kind,dtype", [("16", BF), ("16", FP), ("e4m3", BF), ("e4m3", FP)])
@pytest.mark.parametrize("dh", [144, 192, 256])
@pytest.mark.parametrize("n,G", [(1, 1), (2, 16), (3, 5), (17, 1), (16, 4), (33, 2), (130, 1), (200, 4)])
def test_large_heads_causal(kind, dtype, dh, n, G):
    attend(kind, dtype, n, G, 2, dh, [0, 1, 63, 64, 700], [n, max(1, n - 3), n, 1, n])


@pytest.mark.parametrize("kind,dtype", [("16", BF), ("16", FP), ("e4m3", BF), ("e4m3", FP)])
@pytest.mark.parametrize("dh", [192, 256])
@pytest.mark.parametrize("n", [7, 64])
def test_large_heads_with_values_that_are_not_finite(kind, dtype, dh, n):
    """In rows of the trees, reaching the rows that see them and no other; a row without keys."""
    def edit(cache):
        page = cache.k.shape[2]
        for b, pre in enumerate((3, 130, 0)):
            for t, val in ((1, math.nan), (4, math.inf)):
                p, s = int(cache.table[b, (pre + t) // page]), (pre + t) % page
                if kind == "e4m3":
                    cache.v_exp[p, 0, s] = 255
                    cache.v.view(torch.uint8)[p, 0, s] = 0x7f
                else:
                    cache.v[p, 0, s, 5] = val
                    cache.v[p, 1, s, :] = -val
    attend(kind, dtype, n, 2, 2, dh, [3, 130, 0], mask=chains(3, n), edit=edit)


@pytest.mark.parametrize("kind,dtype", [("16", BF), ("e4m3", FP)])
@pytest.mark.parametrize("n,G,dh", [(600, 4, 128), (257, 16, 64), (1000, 2, 256)])
def test_long_causal_chunks(kind, dtype, n, G, dh):
    """Units of many row tiles, each with keys of its own, behind prefixes of any length."""
    attend(kind, dtype, n, G, 1, dh, [0, 1000], [n, n - 130], page=64)


def test_large_heads_repeat_bit_for_bit():
    cache = R.make_cache(dt, "e4m3", FP, 4, 3000, 2, 64, 256, 430)
    q = normal(4, 8, 33, 256, FP, 431).cuda()
    pre = i32([2900, 17, 300, 1500])
    want = dt.cache_attention(cache, q, pre)
    for _ in range(30):
        assert torch.equal(dt.cache_attention(cache, q, pre), want)
    cache.check()


@pytest.mark.parametrize("kind,n,G,dh", [("16", 20, 2, 64), ("e4m3", 20, 2, 128), ("16", 3, 2, 192), ("e4m3", 20, 2, 256)])
def test_more_requests_than_a_warp_adds_up(kind, n, G, dh):
    """Above 128 requests a block finds its part of the work with all its threads."""
    attend(kind, BF, n, G, 1, dh, [(37 * b) % 90 for b in range(300)], [1 + (b * 7) % n for b in range(300)])
