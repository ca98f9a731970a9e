"""More of what the entry points for norms and projections refuse before any device work (CPU only)."""
from __future__ import annotations

import pytest

from test_layer_abi import adapters, dt, every, matrix  # noqa: F401  (dt is a fixture)


def test_limits_of_waits(dt):
    ok = [matrix(dt), 256, 128, None, 4, 3, dt.BF16, adapters(dt), 256, None, 0, 256, 100, 256, 256, 1 << 30, None]
    every(dt.lib().dt_project, ok, [(0, matrix(dt, wait_cycles=-1)), (0, matrix(dt, wait_cycles=-(1 << 31)))], dt.ERR_INVALID_ARG)
