"""The paged-cache entry points refuse bad arguments before any device work, the rotary
table is right, and cache rows are located without leaving the pool (CPU only)."""
from __future__ import annotations

import ctypes as C
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def dt():
    from conditional_draft_tree_gb300 import build
    build.build()
    import conditional_draft_tree_gb300 as dt
    return dt


def cache(dt, **over):
    a = dict(k=256, v=256, k_exp=None, v_exp=None, table=256, status=256, pages=10, page=64, Hkv=8,
             dh=128, dtype=dt.BF16, batch=4, table_width=3)
    a.update(over)
    return dt.DtCache(*a.values())


BAD_CACHES = [dict(k=None), dict(v=None), dict(table=None), dict(status=None), dict(k=264),
              dict(table=258), dict(status=257), dict(page=48), dict(page=8), dict(page=256),
              dict(pages=0), dict(Hkv=0), dict(dh=8), dict(dh=120), dict(dh=272), dict(batch=0),
              dict(batch=65536), dict(table_width=0), dict(dtype=0), dict(dtype=4),
              dict(dtype=3), dict(k_exp=256), dict(dtype=3, k_exp=256)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_bad_caches_are_refused_everywhere(dt, bad):
    L, c, h = dt.lib(), cache(dt, **bad), dt.DtHeads(256, 8, 1024, 128, 1024)
    ty = dt.BF16
    assert L.dt_cache_write(c, h, h, 1, ty, 256, None, None, None, None, None, None) == dt.ERR_INVALID_ARG
    assert L.dt_cache_read(c, 1, ty, 256, None, h, h, None) == dt.ERR_INVALID_ARG
    assert L.dt_cache_commit(c, 256, 256, 256, 4, 65, None) == dt.ERR_INVALID_ARG
    assert L.dt_cache_attention_workspace_bytes(c, 32, 1) == 0
    assert L.dt_cache_attention(c, h, 1, ty, 256, None, None, 1.0, h, 256, 1 << 30, None) == \
        dt.ERR_INVALID_ARG


def test_bad_arguments_are_refused(dt):
    L, c, inv = dt.lib(), cache(dt), dt.ERR_INVALID_ARG
    h, h32 = dt.DtHeads(256, 8, 1024, 128, 1024), dt.DtHeads(256, 32, 4096, 128, 4096)
    r = dt.DtRotation(256, 128, 0, 1.0)
    bad_heads = [dt.DtHeads(None, 8, 1024, 128, 1024), dt.DtHeads(264, 8, 1024, 128, 1024),
                 dt.DtHeads(256, 0, 1024, 128, 1024), dt.DtHeads(256, 8, 1020, 128, 1024),
                 dt.DtHeads(256, 8, 1024, 124, 1024), dt.DtHeads(256, 8, 1024, 128, 1025)]
    for b in bad_heads:
        assert L.dt_cache_write(c, b, h, 1, 1, 256, None, None, None, None, None, None) == inv
        assert L.dt_cache_write(c, h, b, 1, 1, 256, None, None, None, None, None, None) == inv
        assert L.dt_cache_read(c, 1, 1, 256, None, h, b, None) == inv
        assert L.dt_rotary(r, 256, 1, 1, 128, 1, b, h, None, None, 0, None) == inv
        assert L.dt_rotary(r, 256, 1, 1, 128, 1, h, h, b, h, 0, None) == inv
        assert L.dt_cache_attention(c, b, 1, 1, 256, None, None, 1.0, h, 256, 1 << 30, None) == inv
        assert L.dt_cache_attention(c, h, 1, 1, 256, None, None, 1.0, b, 256, 1 << 30, None) == inv
    # write: c k v n dtype first counts rot positions q q_out stream
    ok = [c, h, h, 4, 1, 256, None, r, 256, h32, h32, None]
    for at, bad in ((1, h32), (3, 0), (4, 0), (4, 2), (4, 3), (5, None), (5, 258), (6, 258), (7, None),
                    (8, None), (8, 258), (10, None), (9, None),
                    (7, dt.DtRotation(256, 136, 0, 1.0)), (7, dt.DtRotation(256, 12, 0, 1.0)),
                    (7, dt.DtRotation(None, 128, 0, 1.0)), (7, dt.DtRotation(260, 128, 0, 1.0)),
                    (7, dt.DtRotation(256, 0, 0, 1.0)), (7, dt.DtRotation(256, 128, 0, float("nan"))),
                    (3, 1 << 28)):
        a = list(ok)
        a[at] = bad
        assert L.dt_cache_write(*a) == inv, (at, bad)
    a = list(ok)
    a[7] = a[8] = None       # q without a rotation
    assert L.dt_cache_write(*a) == inv
    # rotary: rot positions batch n dh dtype x0 out0 x1 out1 gradient stream
    ok = [r, 256, 2, 4, 128, 1, h, h, h32, h32, 0, None]
    for at, bad in ((0, None), (1, None), (2, 0), (3, 0), (4, 120), (4, 272), (4, 64), (5, 3), (7, h32),
                    (8, None), (9, None), (9, h)):
        a = list(ok)
        a[at] = bad
        assert L.dt_rotary(*a) == inv, (at, bad)
    # commit: c first path lengths width n stream
    for over in ((None, 256, 256, 4, 65), (256, None, 256, 4, 65), (256, 256, None, 4, 65),
                 (256, 256, 256, 0, 65), (256, 256, 256, 66, 65), (256, 256, 256, 4, 0),
                 (256, 256, 256, 4, 1026), (258, 256, 256, 4, 65)):
        assert L.dt_cache_commit(c, *over, None) == inv, over
    # attention: c q n dtype prefix counts mask scale out workspace bytes stream
    ok = [c, h32, 65, 1, 256, None, 256, 0.1, h32, 256, 1 << 40, None]
    h30 = dt.DtHeads(256, 30, 4096, 128, 4096)
    for at, bad in ((1, h30), (8, h), (2, 0), (2, 1026), (3, 2), (3, 0), (4, None), (4, 258), (5, 258),
                    (7, float("inf")), (9, None), (9, 128)):
        a = list(ok)
        a[at] = bad
        assert L.dt_cache_attention(*a) == inv, (at, bad)
    a = list(ok)
    a[2], a[6] = 65537, None
    assert L.dt_cache_attention(*a) == inv
    for H, n in ((30, 1), (0, 1), (32, 0), (32, 65537)):
        assert L.dt_cache_attention_workspace_bytes(c, H, n) == 0


@pytest.mark.parametrize("kw", [dict(rot=4), dict(rot=60), dict(rot=264), dict(base=1.0), dict(base=float("nan")),
                                dict(factor=0.5), dict(factor=float("inf")), dict(scaling=4), dict(scaling=-1),
                                dict(scaling=3, trained=0.0), dict(scaling=3, beta_fast=1.0, beta_slow=1.0)])
def test_rotary_table_refusals(dt, kw):
    a = dict(rot=64, scaling=0, base=1e4, factor=1.0, trained=4096.0, beta_fast=32.0, beta_slow=1.0)
    a.update(kw)
    out, mag = (C.c_uint64 * 256)(), C.c_double()
    assert dt.lib().dt_rotary_table(C.byref(dt.DtRotaryParams(*a.values())), out, C.byref(mag)) == dt.ERR_INVALID_ARG


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 8.0), ("base", 4.0), ("parts", 16.0)])
@pytest.mark.parametrize("rot", [8, 64, 128, 256])
def test_rotary_table_values(dt, scaling, factor, rot):
    """Fractions of a turn against the formulas in numpy float64; pow and the division are
    each off by an ulp or two of 2^-53, so 1e-14 relative; the table holds whole 2^-64
    turns, half of which, 2^-65, is its rounding."""
    import _cache_ref as R
    code = {"none": 0, "linear": 1, "base": 2, "parts": 3}[scaling]
    out, mag = (C.c_uint64 * (rot // 2))(), C.c_double()
    p = dt.DtRotaryParams(rot, code, 1e4, factor, 4096.0, 32.0, 1.0)
    assert dt.lib().dt_rotary_table(C.byref(p), out, C.byref(mag)) == dt.OK
    f, m = R.frequencies(rot, 1e4, scaling, factor)
    np.testing.assert_allclose(np.array(out[:], dtype=np.float64) * 2.0 ** -64, f.numpy() / (2 * np.pi),
                               rtol=1e-14, atol=2.0 ** -65)
    assert mag.value == pytest.approx(m, rel=1e-15)


def test_cache_rows_are_located_inside_the_pool(tmp_path):
    """The kernels' own cache_row, run on the host: every index of tables with good and bad
    pages, far past the table and negative, against the layout's definition."""
    nvcc = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    exe = str(tmp_path / "cache_row_check")
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-I",
                    os.path.join(ROOT, "conditional_draft_tree_gb300", "csrc"), "-o", exe,
                    os.path.join(ROOT, "tests", "cuda", "cache_row_check.cu")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
