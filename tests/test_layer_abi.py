"""The entry points for page tables, norms and projections refuse bad arguments before any device
work (CPU only)."""
from __future__ import annotations

import pytest


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


def every(call, ok, bad, inv):
    for at, value in bad:
        a = list(ok)
        a[at] = value
        assert call(*a) == inv, (at, value)


def test_page_tables(dt):
    L, inv = dt.lib(), dt.ERR_INVALID_ARG
    c, pool = cache(dt), dt.DtPagePool(256, 256, 256)
    every(L.dt_cache_reserve, [c, pool, 256, None],
          [(0, cache(dt, page=48)), (0, cache(dt, table=None)), (0, cache(dt, batch=16385)), (0, None), (1, None),
           (1, dt.DtPagePool(None, 256, 256)), (1, dt.DtPagePool(256, None, 256)), (1, dt.DtPagePool(256, 256, None)),
           (1, dt.DtPagePool(258, 256, 256)), (1, dt.DtPagePool(256, 257, 256)), (1, dt.DtPagePool(256, 256, 259)),
           (2, None), (2, 258)], inv)
    every(L.dt_cache_slots, [c, 5, 256, 256, 256, 256, None],
          [(0, cache(dt, pages=0)), (1, 0), (1, -1), (2, None), (2, 258), (3, 257), (4, 260), (5, 258)], inv)
    assert L.dt_cache_slots(c, 5, 256, None, None, None, None) == inv
    assert L.dt_cache_slots(cache(dt, batch=65535), 1 << 30, 256, None, 256, 256, None) == inv


def test_norms(dt):
    L, inv, nan, inf = dt.lib(), dt.ERR_INVALID_ARG, float("nan"), float("inf")
    r = dt._pack_rows(256, 4096, 128)
    no, odd = dt._pack_rows(0, 4096, 128), dt._pack_rows(257, 4096, 128)
    # x residual total out codes exps weight offset eps outer inner d dtype stream
    ok = [r, r, r, r, 256, 256, 256, 0.0, 1e-6, 3, 4, 100, 1, None]
    every(L.dt_rms_norm, ok,
          [(0, None), (0, no), (0, odd), (1, None), (1, no), (1, odd), (2, None), (2, odd), (3, no), (3, odd), (4, None),
           (5, None), (6, 257), (7, nan), (7, inf), (8, 0.0), (8, 1e-31), (8, nan), (8, inf), (8, -1.0), (9, 0), (10, 0),
           (9, 1 << 30), (11, 0), (11, 32769), (12, 0), (12, 3), (12, 4)], inv)
    a = list(ok)
    a[3] = a[4] = a[5] = None          # no result
    assert L.dt_rms_norm(*a) == inv
    every(L.dt_quantize_rows, [r, 256, 256, 3, 4, 100, 1, None],
          [(0, None), (0, odd), (1, None), (2, None), (3, 0), (4, -1), (5, 0), (5, 32769), (6, 0), (6, 3)], inv)


def matrix(dt, **over):
    a = dict(data=256, exps=None, ld=128, O=100, K=128, dtype=dt.BF16)
    a.update(over)
    return dt.DtMatrix(*a.values())


def adapters(dt, **over):
    a = dict(down=256, up=256, scale=256, count=5, rank=32)
    a.update(over)
    return dt.DtAdapters(*a.values())


def test_projections(dt):
    L, inv, big = dt.lib(), dt.ERR_INVALID_ARG, 1 << 30
    # w x ldx x_exps batch n dtype adapters index x16 ldx16 y ldy status workspace bytes stream
    ok = [matrix(dt), 256, 128, None, 4, 3, dt.BF16, adapters(dt), 256, None, 0, 256, 100, 256, 256, big, None]
    w = lambda **over: (0, matrix(dt, **over))
    a = lambda **over: (7, adapters(dt, **over))
    every(L.dt_project, ok,
          [(0, None), w(data=None), w(data=264), w(exps=256), w(ld=120), w(ld=132), w(O=0), w(O=(1 << 24) + 1), w(K=0),
           w(K=120), w(K=65552), w(dtype=dt.F16), w(dtype=0), w(dtype=dt.E4M3), w(ld=(1 << 32) + 8),
           (1, None), (1, 264), (2, 120), (2, 132), (3, 256), (4, 0), (4, 65536), (5, 0), (5, 1 << 23), (6, 0), (6, 3),
           (7, None), a(down=None), a(down=264), a(up=None), a(up=264), a(scale=258), a(count=0), a(count=(1 << 20) + 1),
           a(rank=0), a(rank=8), a(rank=24), a(rank=144), (8, None), (8, 258), (9, 256), (11, None), (11, 257), (12, 99),
           (12, (1 << 26) + 1), (13, None), (13, 258), (14, None), (14, 264), (15, 100)], inv)
    # rows times outputs, and adapters times outputs, past what the kernels count
    every(L.dt_project, ok, [(0, matrix(dt, O=1 << 24)), ], inv)          # y's row is shorter
    far = list(ok)
    far[0], far[12], far[4], far[5] = matrix(dt, O=1 << 24), 1 << 24, 1 << 14, 2
    assert L.dt_project(*far) == inv
    far = list(ok)
    far[0], far[12], far[7] = matrix(dt, O=1 << 20), 1 << 20, adapters(dt, count=2048)
    assert L.dt_project(*far) == inv
    # 8-bit rows
    eight = dict(dtype=dt.E4M3, exps=256)
    ok = [matrix(dt, **eight), 256, 128, 256, 4, 3, dt.F16, adapters(dt), 256, 256, 128, 256, 100, 256, 256, big, None]
    every(L.dt_project, ok,
          [(0, matrix(dt, dtype=dt.E4M3)), (0, matrix(dt, ld=136, **eight)), (2, 136), (3, None), (9, None), (9, 264),
           (10, 120), (10, 132)], inv)
    plain = list(ok)
    plain[7] = plain[8] = None           # x16 without adapters
    assert L.dt_project(*plain) == inv


def test_workspace_sizes(dt):
    f = dt.lib().dt_project_workspace_bytes
    assert f(4, 3, 32) == 768 and f(1, 1, 16) == 256 and f(65535, 256, 128) == 65535 * 256 * 256
    for bad in ((0, 1, 16), (65536, 1, 16), (1, 0, 16), (65535, 257, 16), (1, 1, 8), (1, 1, 24), (1, 1, 144)):
        assert f(*bad) == 0


def test_status_strings(dt):
    assert "free pages" in dt.status_string(dt.ERR_NO_PAGES) and "adapter" in dt.status_string(dt.ERR_BAD_INDEX)


@pytest.mark.parametrize("size,strides,layout", [
    ((5, 8), (8, 1), (1, 0, 5, 8)), ((5, 8), (11, 1), (1, 0, 5, 11)), ((2, 3, 8), (24, 8, 1), (2, 24, 3, 8)),
    ((4, 2, 3, 8), (48, 24, 8, 1), (8, 24, 3, 8)), ((4, 1, 3, 8), (90, 7, 8, 1), (4, 90, 3, 8)),
    ((1, 1, 1, 8), (5, 5, 5, 1), (1, 0, 1, 5)), ((4, 2, 3, 8), (49, 24, 8, 1), None), ((5, 8), (16, 2), None),
    ((8,), (1,), None), ((3, 4, 8), (8, 24, 1), (3, 8, 4, 24))])
def test_row_layouts(dt, size, strides, layout):
    assert dt._row_layout(size, strides) == layout
