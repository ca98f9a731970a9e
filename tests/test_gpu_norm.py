"""Root-mean-square norm with the residual's addition, and 8-bit rows, against plain 64-bit forms
(needs a GB300). Tolerances count roundings: see tests/_layer_ref.py."""
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
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    over = ((got - ref).abs() - slack)[torch.isfinite(ref)]
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: over by {float(over.max()):.3g}"


def rows(*shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * scale
    return (x * (1 + 8 * (torch.arange(shape[-1]) % 41 == 3))).to(dtype)


def check_rows8(r, y, slack):
    """Codes and exponents of the rows y (64 bits, off by at most `slack` in the kernel)."""
    codes, exps = r.codes.cpu(), r.exps.cpu()
    most = y.abs().amax(-1)
    want = R.exponent(most) + 127
    # a row whose largest value lies next to a border may have either exponent
    sure = R.exponent(most * (1 + 2.0 ** -17)) == R.exponent(most * (1 - 2.0 ** -17))
    assert torch.equal(exps.to(torch.int64)[sure], want.to(torch.int64)[sure])
    got = R.from_rows8(codes, exps)
    assert bool(((got - y).abs() <= R.rows8_slack(y, exps, slack)).all())
    assert torch.equal(r.values(torch.float32).cpu().double(), got)


# widths on every kernel shape and one past each border; odd ones go value by value
WIDTHS = [1, 7, 8, 64, 65, 72, 128, 136, 250, 256, 512, 520, 1000, 2048, 2056, 4096, 5001, 8192, 8200, 16384, 16392,
          32767, 32768]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", WIDTHS)
def test_norm(d, dtype):
    n = 5 if d > 4096 else 37
    x, res = rows(n, d, dtype=dtype, seed=d), rows(n, d, dtype=dtype, seed=d + 1)
    x[1] = 0
    res[1] = 0
    w = rows(d, dtype=dtype, seed=3)
    for offset, eps in ((0.0, 1e-6), (1.0, 1e-5)):
        y, t = R.norm(x, res, w, offset, eps)
        (out, r8), total = dt.rms_norm(dt.Norm(w.cuda(), eps, offset), x.cuda(), res.cuda(), kind="both")
        near(total, t, R.HALF[dtype] * t.abs() + R.TINY[dtype] + 2.0 ** -24 * t.abs(), "total")
        near(out, y, R.norm_slack(y, dtype), "out")
        check_rows8(r8, y, R.NORM_SLACK * y.abs())
        alone = dt.rms_norm(dt.Norm(w.cuda(), eps, offset), x.cuda(), res.cuda(), kind="e4m3")[0]
        assert torch.equal(alone.codes.view(torch.uint8), r8.codes.view(torch.uint8)) and torch.equal(alone.exps, r8.exps)
    y, _ = R.norm(x, None, None, 0.0, 1e-6)
    near(dt.rms_norm(dt.Norm(None), x.cuda()), y, R.norm_slack(y, dtype), "no weight")


@pytest.mark.parametrize("dtype", [BF, FP])
def test_norm_of_heads_in_a_projections_output(dtype):
    batch, n, H, all_heads, dh = 3, 5, 7, 11, 96
    x = rows(batch, n, all_heads, dh, dtype=dtype, seed=1)
    w = rows(dh, dtype=dtype, seed=2)
    y, _ = R.norm(x[:, :, 2:2 + H], None, w, 0.0, 1e-6)
    dev = x.cuda()
    keep = dev.clone()
    view = dev[:, :, 2:2 + H]
    near(dt.rms_norm(dt.Norm(w.cuda()), view), y, R.norm_slack(y, dtype))
    # in place, heads before the rows: [batch][heads][n][dh] views
    got = dt.rms_norm(dt.Norm(w.cuda()), view[0].transpose(0, 1), out=view[0].transpose(0, 1))
    near(got.transpose(0, 1), y[0], R.norm_slack(y[0], dtype))
    keep[0, :, 2:2 + H] = got.transpose(0, 1)
    assert torch.equal(dev, keep)          # nothing else was touched


@pytest.mark.parametrize("d,pad", [(40, 8), (40, 3), (33, 1), (4096, 8), (513, 0)])
def test_norm_in_place_over_strided_rows(d, pad):
    dtype, n = BF, 301
    x, res = rows(n, d + pad, dtype=dtype, seed=1).cuda(), rows(n, d + pad, dtype=dtype, seed=2).cuda()
    w = rows(d, dtype=dtype, seed=3).cuda()
    y, t = R.norm(x[:, :d].cpu(), res[:, :d].cpu(), w.cpu(), 0.0, 1e-6)
    edge = x[:, d:].clone(), res[:, d:].clone()
    norm = dt.Norm(w)
    want, want_t = dt.rms_norm(norm, x[:, :d].contiguous(), res[:, :d].contiguous())
    got, total = dt.rms_norm(norm, x[:, :d], res[:, :d], out=x[:, :d], total=res[:, :d])
    assert got.data_ptr() == x.data_ptr() and total.data_ptr() == res.data_ptr()
    near(got, y, R.norm_slack(y, dtype))
    near(total, t, (R.HALF[dtype] + 2.0 ** -24) * t.abs())
    assert torch.equal(got, want) and torch.equal(total, want_t)
    assert torch.equal(x[:, d:], edge[0]) and torch.equal(res[:, d:], edge[1])


def test_rows_far_from_one():
    """Squares that leave fp32 on either side; a row beside them is not touched by them."""
    d = 1000
    w = rows(d, dtype=BF, seed=3)
    x = torch.stack([rows(d, dtype=BF, seed=4, scale=s) for s in (1e37, 1e-30, 1e25, 1.0, 3e18, 1e-10)])
    x[2, 5] = 3e38
    y, _ = R.norm(x, None, w, 0.0, 1e-6)
    out, r8 = dt.rms_norm(dt.Norm(w.cuda()), x.cuda(), kind="both")
    near(out, y, R.norm_slack(y, BF))
    check_rows8(r8, y, R.NORM_SLACK * y.abs())
    big, _ = R.norm(x[:1, :40], None, w[:40], 0.0, 1e-6)        # the form of one warp
    near(dt.rms_norm(dt.Norm(w[:40].cuda()), x[:1, :40].cuda()), big, R.norm_slack(big, BF))


def test_rows_that_are_not_finite():
    d = 264
    x = rows(6, d, dtype=BF, seed=5)
    x[1, 7] = float("nan")
    x[3, 0] = float("inf")
    x[4, d - 1] = -float("inf")
    w = rows(d, dtype=BF, seed=6)
    y, _ = R.norm(x, None, w, 0.0, 1e-6)
    out, r8 = dt.rms_norm(dt.Norm(w.cuda()), x.cuda(), kind="both")
    fine = [0, 2, 5]
    near(out[fine], y[fine], R.norm_slack(y[fine], BF))
    assert bool(out[1].isnan().all())
    for b, at in ((3, 0), (4, d - 1)):      # infinity over infinity, and numbers over infinity
        assert bool(out[b, at].isnan()) and bool((out[b].cpu()[torch.arange(d) != at] == 0).all())
    assert r8.exps.tolist()[1] == 255 and r8.exps.tolist()[3] == 255 and r8.exps.tolist()[4] == 255
    assert bool((r8.codes.view(torch.uint8)[[1, 3, 4]] == 0x7f).all())
    assert bool(r8.values()[[1, 3, 4]].isnan().all())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [16, 100, 129, 4096, 9001])
def test_quantize_rows_is_exact(d, dtype):
    """x itself: one right answer for exponents and codes."""
    import _cache_ref
    x = rows(19, d, dtype=dtype, seed=7)
    x[0], x[2], x[3] = 0, 448.0, 449.0
    if dtype == BF:
        x[4] *= 1e30
        x[5, 0], x[6], x[7, 1] = 3.3e38, x[6] * 1e-38, float("nan")
    codes, exps = _cache_ref.quantise(x)
    r = dt.quantize_rows(x.cuda())
    assert torch.equal(r.exps.cpu(), exps) and torch.equal(r.codes.cpu().view(torch.uint8), codes)
    strided = rows(19, d + 5, dtype=dtype, seed=7)[:, :d]
    codes, exps = _cache_ref.quantise(strided)
    r = dt.quantize_rows(strided.cuda())
    assert torch.equal(r.exps.cpu(), exps) and torch.equal(r.codes.cpu().view(torch.uint8), codes)


def test_many_rows_and_a_stream():
    """More rows than the grid has room for at once; on a stream of its own, captured and replayed."""
    n, d = 20011, 128
    x = rows(n, d, dtype=FP, seed=8).cuda()
    w = rows(d, dtype=FP, seed=9).cuda()
    norm = dt.Norm(w)
    y, _ = R.norm(x.cpu(), None, w.cpu(), 0.0, 1e-6)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = dt.rms_norm(norm, x, stream=stream)
    stream.synchronize()
    near(got, y, R.norm_slack(y, FP))
    out, graph = torch.empty_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dt.rms_norm(norm, x, out=out)
    x.copy_(x.flip(0))
    graph.replay()
    assert torch.equal(out, got.flip(0))
