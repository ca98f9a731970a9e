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
