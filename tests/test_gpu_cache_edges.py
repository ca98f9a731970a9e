"""Attention over the paged cache at the edges of what its kernels take: keys that are
not there, values that are not finite or far apart in size, workspaces and streams (needs
a GB300). Against 64-bit forms, with the tolerances of `_cache_ref.attention_slack`."""
from __future__ import annotations

import math
import types

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


def queries(batch, n, H, dh, dtype, seed, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    return (amp * torch.randn(batch, n, H, dh, generator=g)).to(dtype).transpose(1, 2)


def place(cache, b, j):
    """Page and slot of row j of request b."""
    page = cache.k.shape[2]
    return int(cache.table[b, j // page]), j % page


@pytest.mark.parametrize("entry", [-1, -2147483648, "pages", 2147483647])
@pytest.mark.parametrize("n,G,dh", [(1, 4, 128), (3, 4, 64), (20, 4, 128), (65, 4, 128), (1, 4, 256), (20, 2, 192), (70, 4, 256)])
@pytest.mark.parametrize("kind", ["16", "e4m3"])
def test_keys_on_bad_pages_are_left_out(kind, n, G, dh, entry):
    """A bad page inside the prefix, one that holds tree rows, and one that lets a unit begin
    with rows that are not there: reported, and the other keys attended to."""
    keys_on_bad_pages(kind, n, G, dh, entry)


def keys_on_bad_pages(kind, n, G, dh, entry):
    batch, Hkv, page = 4, 2, 16
    prefix = [200, 100, 40, 700]
    cache = R.make_cache(dt, kind, BF, batch, max(prefix) + n, Hkv, page, dh, 300)
    pages = cache.k.shape[0]
    good = types.SimpleNamespace(k=cache.k, v=cache.v, k_exp=cache.k_exp, v_exp=cache.v_exp, table=cache.table.clone())
    bad = [[5], [100 // page], [0], []]
    for b, at in enumerate(bad):
        for x in at:
            cache.table[b, x] = pages if entry == "pages" else entry
    q, scale = queries(batch, n, Hkv * G, dh, BF, 301), dh ** -0.5
    got = dt.cache_attention(cache, q.cuda(), i32(prefix))
    assert cache.status.tolist() == [dt.ERR_BAD_PAGE] * 3 + [dt.OK]
    for b in range(batch):
        keys = [j for j in range(prefix[b] + n) if j // page not in bad[b]]
        k, v = (R.pool_rows(good, w, b, keys) for w in "kv")
        see = torch.tensor(keys)[None] <= prefix[b] + torch.arange(n)[:, None]
        for h in range(Hkv * G):
            x = scale * q[b, h].double() @ k[h // G].T
            big = scale * float((q[b, h].double().abs() @ k[h // G].abs().T).max())
            p = torch.softmax(torch.where(see, x, -math.inf), -1)
            p = torch.where(see.any(-1, keepdim=True), p, 0.0)        # a row that sees nothing
            ref = p @ v[h // G]
            near(got[b, h], ref, R.attention_slack(ref, p @ v[h // G].abs(), big, BF, dh, prefix[b] + n), f"{b} {h}")


def dense(cache, prefix, counts, q, mask, scale):
    return R.attention(cache, q, torch.tensor(prefix), mask, torch.tensor(counts) if counts is not None else None, scale)


@pytest.mark.parametrize("n,G", [(1, 4), (20, 4), (70, 2)])
@pytest.mark.parametrize("dh", [64, 128, 192, 256])
@pytest.mark.parametrize("kind,dtype", [("16", BF), ("16", FP), ("e4m3", BF), ("e4m3", FP)])
def test_rows_past_the_count_are_zero_whatever_the_prefix_holds(kind, dtype, dh, n, G):
    """Values that are not finite in the prefix: rows that see them are NaN or infinite, rows
    past the count are zero, in units that a block holds whole (100 keys) and in cut ones."""
    prefix, counts = [100, 3000, 64, 700], [max(1, n - 13), max(1, n // 2), 0, n]
    cache = R.make_cache(dt, kind, dtype, 4, max(prefix) + n, 2, 16, dh, 310)
    for b, j, val in ((0, 10, math.nan), (1, 70, math.inf), (2, 3, -math.inf), (3, 5, math.nan)):
        p, s = place(cache, b, j)
        if kind == "e4m3":
            cache.v_exp[p, :, s] = 255
            cache.v.view(torch.uint8)[p, :, s] = 0x7f
        else:
            cache.v[p, 0, s, 7] = val
            cache.v[p, 1, s, :] = val
    q, scale = queries(4, n, 2 * G, dh, dtype, 311), dh ** -0.5
    got = dt.cache_attention(cache, q.cuda(), i32(prefix), counts=i32(counts))
    cache.check()
    for b, c in enumerate(counts):
        assert bool((got[b, :, c:] == 0).all()), b
    ref, mass, big = dense(cache, prefix, counts, q, None, scale)
    near(got, ref, R.attention_slack(ref, mass, big, dtype, dh, max(prefix) + n))


@pytest.mark.parametrize("n", [1, 20, 70])
@pytest.mark.parametrize("dh", [128, 192, 256])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_8bit_values_past_the_range_of_fp16_count_as_they_are(dtype, dh, n):
    """A row of 448 2^12 among rows of ordinary size, each with about the same weight: the
    result is a number of fp16, the row is not."""
    prefix = [700, 45]
    cache = R.make_cache(dt, "e4m3", dtype, 2, max(prefix) + n, 2, 16, dh, 320)
    for b in range(2):
        p, s = place(cache, b, 2)
        cache.v.view(torch.uint8)[p, :, s] = 0x7e
        cache.v_exp[p, :, s] = 127 + 12
    q, scale = queries(2, n, 8, dh, dtype, 321, amp=1e-3), dh ** -0.5
    got = dt.cache_attention(cache, q.cuda(), i32(prefix))
    cache.check()
    ref, mass, big = dense(cache, prefix, None, q, None, scale)
    near(got, ref, R.attention_slack(ref, mass, big, dtype, dh, max(prefix) + n))


@pytest.mark.parametrize("n", [1, 20, 70])
@pytest.mark.parametrize("dh", [192, 256])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_8bit_codes_of_every_size_count_at_large_heads(dtype, dh, n):
    """Rows whose codes are the least ones beside a single large one, of very different scales."""
    prefix = [3, 130]
    cache = R.make_cache(dt, "e4m3", dtype, 2, max(prefix) + n, 2, 16, dh, 330)
    g = torch.Generator().manual_seed(331)
    code = torch.randint(0, 8, cache.v.shape, generator=g, dtype=torch.uint8)
    code |= torch.randint(0, 2, cache.v.shape, generator=g, dtype=torch.uint8) << 7
    code[..., 3] = 0x7e
    cache.v.view(torch.uint8).copy_(code)
    cache.v_exp.copy_(torch.randint(100, 120, cache.v_exp.shape, generator=g, dtype=torch.uint8))
    q, scale = queries(2, n, 4, dh, dtype, 332), dh ** -0.5
    got = dt.cache_attention(cache, q.cuda(), i32(prefix))
    cache.check()
    ref, mass, big = dense(cache, prefix, None, q, None, scale)
    near(got, ref, R.attention_slack(ref, mass, big, dtype, dh, max(prefix) + n))


@pytest.mark.parametrize("n", [1, 3, 20])
@pytest.mark.parametrize("dh", [64, 128, 256])
@pytest.mark.parametrize("low,high,amp,scale", [(127 + 9, 127 + 11, 1e-4, 0.05), (92, 106, 30.0, 1024.0), (96, 142, 1e-3, 0.5)])
def test_fp16_scores_take_8bit_keys_as_they_are_read(low, high, amp, scale, dh, n, monkeypatch):
    """Keys past fp16's largest number, below its least step, and both: the scores are those of
    the keys that dt_cache_read gives in fp16, however many rows there are."""
    prefix = [300, 17]
    cache = R.make_cache(dt, "e4m3", FP, 2, max(prefix) + n, 2, 16, dh, 340)
    g = torch.Generator().manual_seed(341)
    cache.k_exp.copy_(torch.randint(low, high + 1, cache.k_exp.shape, generator=g, dtype=torch.uint8))
    q = queries(2, n, 8, dh, FP, 342, amp=amp)
    got = dt.cache_attention(cache, q.cuda(), i32(prefix), scale=scale)
    cache.check()
    rows = R.pool_rows
    monkeypatch.setattr(R, "pool_rows", lambda c, which, b, at: rows(c, which, b, at) if which == "v" else
                        rows(c, which, b, at).clamp(-65504, 65504).to(FP).double())
    ref, mass, big = dense(cache, prefix, None, q, None, scale)
    near(got, ref, R.attention_slack(ref, mass, big, FP, dh, max(prefix) + n))


@pytest.mark.parametrize("n,G,dh", [(1, 4, 128), (3, 4, 64), (20, 4, 128), (1, 4, 256)])
@pytest.mark.parametrize("kind", ["16", "e4m3"])
def test_a_table_entry_of_minus_two_is_a_bad_page_too(kind, n, G, dh):
    keys_on_bad_pages(kind, n, G, dh, -2)


@pytest.mark.parametrize("n", [1, 3, 20])
def test_a_score_of_zero_between_huge_vectors_is_zero(n):
    """q holds 2^60 in one place, a key 2^80 in another: their scales' product is no fp32 number,
    the score is zero."""
    dh = 128
    cache = R.make_cache(dt, "e4m3", BF, 2, 80, 2, 16, dh, 370)
    cache.k.view(torch.uint8)[..., 0] = 0
    p, s = place(cache, 0, 4)
    cache.k_exp[p, :, s] = 127 + 72
    cache.k.view(torch.uint8)[p, :, s, :] = 0
    cache.k.view(torch.uint8)[p, :, s, 1] = 0x7e
    q = torch.zeros(2, 8, n, dh, dtype=BF)
    q[..., 0] = 2.0 ** 60
    got = dt.cache_attention(cache, q.cuda(), i32([30, 40]))
    cache.check()
    ref, mass, _ = dense(cache, [30, 40], None, q, None, dh ** -0.5)
    near(got, ref, R.attention_slack(ref, mass, 0.0, BF, dh, 80))


@pytest.mark.parametrize("n,G", [(3, 2), (4, 4), (20, 2)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_a_huge_value_that_is_not_seen_changes_nothing(dtype, n, G):
    """Row 1 of a tree of siblings holds 2^100 and more; the others' results are as without it."""
    cache = R.make_cache(dt, "e4m3", dtype, 2, 60 + n, 2, 16, 128, 350)
    prefix = [5, 60]
    q, scale = queries(2, n, 2 * G, 128, dtype, 351), 128 ** -0.5
    mask = torch.eye(n, dtype=torch.uint8)[None].repeat(2, 1, 1)
    mask[:, :, 0] = 1
    results = []
    for e in (120, 127 + 100):
        for b in range(2):
            p, s = place(cache, b, prefix[b] + 1)
            cache.v_exp[p, :, s] = e
        results.append(dt.cache_attention(cache, q.cuda(), i32(prefix), mask=mask.cuda()))
    cache.check()
    ref, mass, big = dense(cache, prefix, None, q, mask, scale)
    others = [i for i in range(n) if i != 1]
    slack = R.attention_slack(ref, mass, big, dtype, 128, 60 + n)
    near(results[1][:, :, others], ref[:, :, others], slack[:, :, others])
    assert torch.equal(results[0][:, :, others], results[1][:, :, others])


@pytest.mark.parametrize("n,G", [(1, 4), (2, 8), (20, 1)])
@pytest.mark.parametrize("batch,length", [(2, 90), (24, 3000)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_huge_values_of_little_weight_beside_ordinary_ones(dtype, batch, length, n, G):
    """Scores of 0, -30 and -64 (powers of e), values of about e^0, e^30 and e^64 with them, in
    any order: each kind gives about as much of the result. A warp of the kernel for a few
    rows meets them in one step (90 keys) and over many (3000 keys of 24 requests)."""
    dh, Hkv = 64, 8
    cache = R.make_cache(dt, "e4m3", dtype, batch, length + n, Hkv, 64, dh, 360)
    g = torch.Generator().manual_seed(361)
    shape = cache.k_exp.shape
    what = torch.multinomial(torch.tensor([1.0, 5.0, 94.0]), shape.numel(), replacement=True, generator=g).view(shape)
    # q is 1 everywhere, scale 1/8: the score of a row of 64 values x is 8 x
    x = torch.tensor([0.0, -3.75, -8.0])[what]
    cache.k.view(torch.uint8).copy_(R.quantise(x[..., None].expand(cache.k.shape).contiguous().to(BF))[0])
    cache.k_exp.copy_(R.quantise(x[..., None].expand(cache.k.shape).contiguous().to(BF))[1])
    e = cache.v_exp.cpu().int() + torch.tensor([0, 43 - 3, 92 - 7])[what]
    cache.v_exp.copy_(e.to(torch.uint8))
    q = torch.ones(batch, Hkv * G, n, dh, dtype=dtype)
    prefix = [length - 7 * b for b in range(batch)]
    got = dt.cache_attention(cache, q.cuda(), i32(prefix), scale=0.125)
    cache.check()
    some = [0, batch - 1]
    for b in some:
        one = types.SimpleNamespace(k=cache.k, v=cache.v, k_exp=cache.k_exp, v_exp=cache.v_exp,
                                    table=cache.table[b:b + 1], Hkv=Hkv)
        ref, mass, big = dense(one, prefix[b:b + 1], None, q[b:b + 1], None, 0.125)
        if dtype == FP:         # a result past the type's largest number is rounded to infinity
            ref = torch.where(ref.abs() < 65520, ref, ref.sign() * math.inf)
        near(got[b:b + 1], ref, R.attention_slack(ref, mass, big, dtype, dh, length + n))


@pytest.mark.parametrize("H,Hkv,dh", [(32, 8, 128), (8, 8, 64), (40, 8, 128), (16, 4, 256), (64, 4, 96)])
@pytest.mark.parametrize("kind", ["16", "e4m3"])
def test_a_workspace_serves_any_smaller_call(kind, H, Hkv, dh):
    cache = R.make_cache(dt, kind, BF, 3, 600, Hkv, 32, dh, 380)
    L = dt.lib()
    sizes = [L.dt_cache_attention_workspace_bytes(cache._struct, H, n) for n in range(1, 300)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])) and sizes[0] > 0
    assert all(L.dt_cache_attention_workspace_bytes(cache._struct, h, 33) <= sizes[32] for h in range(Hkv, H + 1, Hkv))
    ws = dt.cache_attention_workspace(cache, H, 65)
    prefix = i32([500, 3, 130])
    for n in (65, 64, 33, 32, 17, 5, 1):
        q = queries(3, n, H, dh, BF, 381).cuda()
        assert torch.equal(dt.cache_attention(cache, q, prefix, workspace=ws), dt.cache_attention(cache, q, prefix))
    cache.check()
