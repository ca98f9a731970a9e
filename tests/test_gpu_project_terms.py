"""x A^T in one 16-bit term or two before its product with B (needs a GB300): results whose adapters' values cancel, so that
the error of a term shows beside them. Tolerances count roundings: see tests/_layer_ref.py."""
from __future__ import annotations

import pytest
import torch

import _layer_ref as R
from test_gpu_project import BF, FP, KINDS, Case, _built, dt, near  # noqa: F401  (_built is a fixture)

pytestmark = pytest.mark.gpu


def slack(c, vx, vw, y, terms):
    """R.project_slack with what `terms` terms lose of x A^T: half a step of the first, 2^-8 or 2^-11 of a value, and of that
    half a step of the second; half the least step of the type where that is more."""
    half, dtype, u24 = R.HALF[c.dtype] ** terms, c.dtype, 2.0 ** -24
    over = c.K * u24 * (vx.abs() @ vw.abs().t())
    for b, a in enumerate(c.index.tolist()):
        if a >= 0:
            r, s = slice(b * c.n, (b + 1) * c.n), 1.0 if c.scale is None else float(c.scale[a])
            d, v, z = c.down[a].double(), c.up[a].double(), c.x[r].double()
            u = z @ d.t() * s
            off = half * u.abs() + (c.K + 2) * u24 * abs(s) * (z.abs() @ d.abs().t()) + R.TINY[dtype]
            over[r] += off @ v.abs().t() + (c.K + 2 * c.down.shape[1]) * u24 * (u.abs() @ v.abs().t())
    return R.HALF[dtype] * (y.abs() + over) + over + R.TINY[dtype]


def cancelling(*sizes, **kw):
    """A case whose ranks come in pairs: rows of A that differ by 2^-6 of their size in one place, columns of B of opposite
    sign; and a small W, so that y is that difference."""
    c = Case(*sizes, **kw)
    c.down[:, 1::2] = c.down[:, ::2]
    c.down[:, 1::2, 5] *= 1 + 2.0 ** -6
    c.up[..., 1::2] = -c.up[..., ::2]
    c.w *= 2.0 ** -9
    vx, vw = c.x.double(), c.w.double()
    if c.e8:
        import _cache_ref
        c.w8 = _cache_ref.quantise(c.w)
        vx, vw = R.from_rows8(*c.x8), R.from_rows8(*c.w8)
    c.y = R.project(vx, vw, c.n, c.index, c.x, c.down, c.up, c.scale)
    return c, slack(c, vx, vw, c.y, 2), slack(c, vx, vw, c.y, 1)


# rows' own blocks, stacked rows of A; single blocks, clusters and pairs; every rank's pieces
SIZES = [(1, 1, 64, 130, 16, 2), (8, 1, 2048, 1040, 16, 5), (130, 1, 96, 140, 48, 130), (256, 1, 144, 64, 16, 256),
         (5, 13, 256, 300, 64, 3), (40, 7, 128, 260, 112, 40), (1, 3996, 64, 1072, 64, 2), (400, 1, 1024, 700, 128, 2),
         (2, 128, 144, 513, 128, 2), (20, 65, 640, 2100, 16, 5), (6, 300, 256, 4100, 32, 4), (3, 700, 64, 2048, 96, 3),
         (4, 300, 320, 5000, 80, 4), (70, 9, 272, 129, 96, 64), (3, 1000, 128, 3001, 128, 3)]


@pytest.mark.parametrize("dtype,e8", KINDS)
@pytest.mark.parametrize("sizes", SIZES)
def test_two_terms(sizes, dtype, e8):
    c, close, far = cancelling(*sizes, dtype, e8, seed=31)
    p, x, ad, index, x16 = c.cuda()
    ws = dt.project_workspace(p, c.batch, c.n, ad)
    assert ws.numel() == 2 * dt.lib().dt_project_workspace_bytes(c.batch, c.n, ad.rank)
    ws.fill_(0xff)
    got = dt.project(p, x, ad, index, x16, dtype=dtype, workspace=ws)
    near(got.reshape(-1, c.O), c.y, close)
    assert torch.equal(dt.project(p, x, ad, index, x16, dtype=dtype, workspace=ws), got)
    # one term, in half the workspace
    one = dt.Adapters(ad.down, ad.up, ad.scale, terms=1)
    ws = torch.full((ws.numel() // 2 + 256,), 0xff, dtype=torch.uint8, device="cuda")
    guard = ws[-256:]
    got = dt.project(p, x, one, index, x16, dtype=dtype, workspace=ws[:-256])
    near(got.reshape(-1, c.O), c.y, far)
    assert bool((guard == 0xff).all())
    with pytest.raises(dt.DtError):
        dt.project(p, x, ad, index, x16, dtype=dtype, workspace=ws[:-256])
    p.check()


@pytest.mark.parametrize("e8", [False, True])
def test_past_the_types_range(e8):
    """x A^T past fp16's largest number is an infinity in either form, its second term nothing; small values keep what the
    second term can hold."""
    c = Case(3, 2, 64, 40, 16, 2, FP, e8, index=[0, 1, 0], scaled=False, seed=32)
    c.down[0] = 4.0
    c.x.view(3, 2, 64)[0, 1] = 400.0
    c.up[0] = 0.25
    c.down[1] *= 2.0 ** -11
    if e8:
        import _cache_ref
        c.x8 = _cache_ref.quantise(c.x)
    p, x, ad, index, x16 = c.cuda()
    for a in (ad, dt.Adapters(ad.down, ad.up, terms=1)):
        got = dt.project(p, x, a, index, x16, dtype=FP)
        assert bool((got[0, 1] == float("inf")).all()) and bool(torch.isfinite(got[0, 0]).all()) and \
            bool(torch.isfinite(got[1:]).all())
    vx, vw = (R.from_rows8(*c.x8), R.from_rows8(*c.w8)) if e8 else (c.x.double(), c.w.double())
    y = R.project(vx, vw, 2, c.index, c.x, c.down, c.up)
    got = dt.project(p, x, ad, index, x16, dtype=FP)
    near(got[1], y[2:4], slack(c, vx, vw, y, 2)[2:4])
