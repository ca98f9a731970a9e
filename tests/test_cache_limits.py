"""Sizes that the paged-cache entry points refuse before any device work (CPU only)."""
from __future__ import annotations

import pytest


@pytest.fixture(scope="module")
def dt():
    from conditional_draft_tree_gb300 import build
    build.build()
    import conditional_draft_tree_gb300 as dt
    return dt


@pytest.mark.parametrize("pages,Hkv", [(1 << 28, 8), (1 << 30, 2), (2147483647, 4096)])
@pytest.mark.parametrize("dh,dtype,exp", [(128, 1, None), (16, 3, 256), (256, 2, None)])
def test_pools_of_more_than_2_31_head_pages_are_refused(dt, pages, Hkv, dh, dtype, exp):
    """A tensor map's and the kernels' page numbers count pages times heads in 31 bits; such a
    pool would hold over 500 GB of keys."""
    c = dt.DtCache(256, 256, exp, exp, 256, 256, pages, 16, Hkv, dh, dtype, 4, 3)
    h, ty = dt.DtHeads(256, Hkv, 1024, 128, 1024), dt.F16 if dtype == 2 else dt.BF16
    L, inv = dt.lib(), dt.ERR_INVALID_ARG
    assert L.dt_cache_write(c, h, h, 1, ty, 256, None, None, None, None, None, None) == inv
    assert L.dt_cache_read(c, 1, ty, 256, None, h, h, None) == inv
    assert L.dt_cache_commit(c, 256, 256, 256, 4, 65, None) == inv
    assert L.dt_cache_attention_workspace_bytes(c, Hkv, 1) == 0
    assert L.dt_cache_attention(c, h, 1, ty, 256, None, None, 1.0, h, 256, 1 << 30, None) == inv
