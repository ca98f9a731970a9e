"""More of what the entry points for norms and projections refuse before any device work (CPU only)."""
from __future__ import annotations

import pytest

from test_layer_abi import adapters, dt, every, matrix  # noqa: F401  (dt is a fixture)


def test_limits_of_waits(dt):
    ok = [matrix(dt), 256, 128, None, 4, 3, dt.BF16, adapters(dt), 256, None, 0, 256, 100, 256, 256, 1 << 30, None]
    every(dt.lib().dt_project, ok, [(0, matrix(dt, wait_cycles=-1)), (0, matrix(dt, wait_cycles=-(1 << 31)))], dt.ERR_INVALID_ARG)


def test_terms_of_adapters(dt):
    ok = [matrix(dt), 256, 128, None, 4, 3, dt.BF16, adapters(dt, terms=2), 256, None, 0, 256, 100, 256, 256, 1 << 30, None]
    f = dt.lib().dt_project_workspace_bytes(4, 3, 32)
    every(dt.lib().dt_project, ok, [(7, adapters(dt, terms=3)), (7, adapters(dt, terms=-1)), (15, 2 * f - 1), (15, f)],
          dt.ERR_INVALID_ARG)


def test_results_of_a_norm_in_one_place(dt):
    L, inv = dt.lib(), dt.ERR_INVALID_ARG
    x, res, total, out = (dt._pack_rows(4096 * k, 4096, 128) for k in range(1, 5))
    # x residual total out codes exps weight offset eps outer inner d dtype stream
    ok = [x, res, total, out, 256, 256, 256, 0.0, 1e-6, 3, 4, 100, 1, None]
    every(L.dt_rms_norm, ok, [(2, out), (3, total), (2, dt._pack_rows(4096 * 4, 8192, 256))], inv)
    for same in (x, res):
        assert L.dt_rms_norm(x, res, same, same, None, None, 256, 0.0, 1e-6, 3, 4, 100, 1, None) == inv
    no, odd = dt._pack_rows(0, 4096, 128), dt._pack_rows(257, 4096, 128)
    every(L.dt_rms_norm, ok, [(k, bad) for k in range(4) for bad in (no, odd)] + [(1, None), (2, None), (8, 0.0), (11, 0)], inv)
