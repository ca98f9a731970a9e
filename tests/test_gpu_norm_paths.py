"""The norm's and the quantisation's forms over many rows and at every place (needs a GB300): each against plain 64-bit
forms, which run on the device here. Tolerances count roundings: see tests/_layer_ref.py."""
from __future__ import annotations

import pytest
import torch

import _layer_ref as R
from test_gpu_norm import BF, FP, _built, dt  # noqa: F401  (_built is a fixture)

pytestmark = pytest.mark.gpu


def rows(*shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda") * scale
    return (x * (1 + 8 * (torch.arange(shape[-1], device="cuda") % 41 == 3))).to(dtype)


def placed(t, lead, pad, fill):
    """t [n][d] in a frame of `fill`, `lead` values behind its beginning and rows d + pad apart: the frame, the view."""
    n, d = t.shape
    frame = torch.full((lead + n * (d + pad) + 8,), fill, dtype=t.dtype, device="cuda")
    view = frame[lead:lead + n * (d + pad)].view(n, d + pad)[:, :d]
    view.copy_(t)
    return frame, view


def untouched(frame, view, lead, fill):
    n, d = view.shape
    step = view.stride(0)
    rest = frame.clone()
    rest[lead:lead + n * step].view(n, step)[:, :d] = fill
    assert bool((rest == fill).all())


def near(got, ref, slack, what=""):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fine), what
    over = ((got - ref).abs() - slack)[fine]
    assert float(over.max()) <= 0, f"{what}: over by {float(over.max()):.3g}"


def check_rows8(r, y):
    """Codes and exponents of the rows y, off by R.NORM_SLACK of it; rows that are not finite are marked."""
    codes, exps = r.codes.view(torch.uint8), r.exps
    bad = ~torch.isfinite(y).all(-1)
    assert torch.equal(exps == 255, bad) and bool((codes[bad] == 0x7f).all())
    y, codes, exps = y[~bad], codes[~bad], exps[~bad]
    most = y.abs().amax(-1)
    sure = R.exponent(most * (1 + 2.0 ** -17)) == R.exponent(most * (1 - 2.0 ** -17))
    assert torch.equal(exps.long()[sure], (R.exponent(most) + 127).long()[sure])
    step = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), exps.long()[..., None] - 127)
    got = codes.view(torch.float8_e4m3fn).double() * step
    slack = torch.maximum(y.abs() * 2.0 ** -4, 2.0 ** -10 * step) + R.NORM_SLACK * y.abs()
    assert bool(((got - y).abs() <= slack).all())


def norm(x, res, w, eps):
    return R.norm(x, res, w, 0.0, eps)


# on boundaries: groups of 8, 16 and 32 threads, two chunks a thread, blocks whose size the compiler knows and
# others, four chunks, no row ahead. Off them: a warp a row of one and two chunks, blocks of two, four and five.
ALIGNED = [(64, 20000), (128, 12000), (256, 9000), (512, 5000), (520, 5500), (1000, 4000), (2048, 2500), (4096, 1500),
           (8200, 700), (16384, 500), (20000, 500)]
ODD = [(33, 15000), (250, 8000), (513, 5500), (2001, 3000), (5001, 1000), (7935, 700), (9001, 500), (15863, 460),
       (15871, 460), (20001, 460)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d,n", ALIGNED + ODD)
def test_many_rows_a_block(d, n, dtype):
    """Three times as many rows as run at once or more. Among them rows whose squares leave fp32, which are reduced
    twice, rows of zeros and rows that are not finite; sum and result in place of the inputs."""
    x, res, w = rows(n, d, dtype=dtype, seed=1), rows(n, d, dtype=dtype, seed=2), rows(d, dtype=dtype, seed=3)
    if dtype == BF:
        x[5::97] *= 1e36
        res[5::97] *= 1e36
    x[11::101], res[11::101] = 0, 0
    x[17::103, d // 2] = float("nan")
    y, t = norm(x, res, w, 1e-6)
    op = dt.Norm(w)
    (out, r8), total = dt.rms_norm(op, x, res, kind="both")
    slack = R.norm_slack(y, dtype)
    near(total, t, (R.HALF[dtype] + 2.0 ** -24) * t.abs() + R.TINY[dtype], "total")
    near(out, y, slack, "out")
    check_rows8(r8, y)
    alone = dt.rms_norm(op, x, res, kind="e4m3")[0]
    assert torch.equal(alone.codes.view(torch.uint8), r8.codes.view(torch.uint8)) and torch.equal(alone.exps, r8.exps)
    got, sums = dt.rms_norm(op, x, res, out=x, total=res)
    assert got.data_ptr() == x.data_ptr() and sums.data_ptr() == res.data_ptr()
    assert torch.equal(got.view(torch.int16), out.view(torch.int16)) and torch.equal(sums.view(torch.int16), total.view(torch.int16))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d,outer,inner,all_rows", [(96, 900, 7, 11), (1000, 1100, 3, 4), (4096, 300, 7, 8), (33, 3000, 7, 9),
                                                    (250, 1500, 3, 5), (513, 1500, 3, 4), (5001, 300, 3, 4)])
def test_rows_of_two_strides(d, outer, inner, all_rows, dtype):
    """Some of each outer row's rows, so that the next one of a block lies at another place and another distance."""
    x = rows(outer, all_rows, d, dtype=dtype, seed=4)
    w = rows(d, dtype=dtype, seed=5)
    y, _ = norm(x[:, 1:1 + inner], None, w, 1e-6)
    keep = x.clone()
    out, r8 = dt.rms_norm(dt.Norm(w), x[:, 1:1 + inner], kind="both")
    near(out, y, R.norm_slack(y, dtype))
    check_rows8(r8, y)
    got = dt.rms_norm(dt.Norm(w), x[:, 1:1 + inner], out=x[:, 1:1 + inner])
    keep[:, 1:1 + inner] = out
    assert torch.equal(x, keep) and torch.equal(got, out)
    # rows before the outer dimension
    z = keep.transpose(0, 1)[1:1 + inner]
    y, _ = norm(z, None, w, 1e-6)
    near(dt.rms_norm(dt.Norm(w), z), y, R.norm_slack(y, dtype))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d", [1, 7, 9, 33, 248, 250, 495, 513, 2001, 7929, 7935, 9001, 15863, 15871, 16001, 32767])
@pytest.mark.parametrize("places", [(1, 2, 3, 4), (7, 5, 0, 6), (0, 0, 1, 0), (4, 4, 4, 5), (6, 1, 7, 3)])
def test_a_place_of_its_own_for_each_tensor(places, d, dtype):
    """x, residual, sum and result at different distances from a 16-byte boundary, rows an odd distance apart; what lies
    beside them is not finite, and stays as it was."""
    n = 12
    x, res, w = rows(n, d, dtype=dtype, seed=6), rows(n, d, dtype=dtype, seed=7), rows(d, dtype=dtype, seed=8)
    y, t = norm(x, res, w, 1e-6)
    nan, pads = float("nan"), [(1 + 2 * k) % 8 for k in places]
    vx, vr = (placed(v, k, p, nan)[1] for v, k, p in ((x, places[0], pads[0]), (res, places[1], pads[1])))
    blank = torch.zeros(n, d, dtype=dtype, device="cuda")
    ft, vt = placed(blank, places[2], pads[2], 77.0)
    fo, vo = placed(blank, places[3], pads[3], 77.0)
    (out, r8), total = dt.rms_norm(dt.Norm(w), vx, vr, kind="both", out=vo, total=vt)
    near(total, t, (R.HALF[dtype] + 2.0 ** -24) * t.abs() + R.TINY[dtype], "total")
    near(out, y, R.norm_slack(y, dtype), "out")
    check_rows8(r8, y)
    untouched(ft, vt, places[2], 77.0)
    untouched(fo, vo, places[3], 77.0)
    near(dt.rms_norm(dt.Norm(w), vx), norm(x, None, w, 1e-6)[0], R.norm_slack(norm(x, None, w, 1e-6)[0], dtype), "alone")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("d,n", [(128, 12000), (4096, 1500), (20000, 500), (33, 15000), (250, 8000), (513, 5500), (5001, 1000),
                                 (9001, 500), (20001, 460)])
def test_quantisation_of_many_rows(d, n, dtype):
    """x itself in 8 bits: one right answer."""
    x = rows(n, d, dtype=dtype, seed=9) * torch.exp2(torch.randint(-8, 9, (n, 1), device="cuda")).to(dtype)
    x[3::31] = 0
    x[5::37, d // 3] = float("inf")
    r = dt.quantize_rows(x)
    y = x.double()
    bad = ~torch.isfinite(y).all(-1)
    e = R.exponent(y.abs().amax(-1))
    exps = torch.where(bad, 255, e.long() + 127)
    codes = torch.ldexp(torch.where(bad[:, None], 0.0, y), -e.long()[:, None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(r.exps.long(), exps)
    assert torch.equal(r.codes.view(torch.uint8), torch.where(bad[:, None], 0x7f, codes.long()).to(torch.uint8))
