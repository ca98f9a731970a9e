"""More of what the Python calls for norms and projections decide before the library is entered (CPU only: stand-ins, as in
tests/test_layer_binding.py)."""
from __future__ import annotations

import pytest
import torch

import conditional_draft_tree_gb300 as dt
from test_layer_binding import BATCH, K, N, O, Tensor, adapters, ints, lib, more, projection, rows  # noqa: F401  (lib, more: fixtures)


def test_two_terms_take_twice_the_workspace(lib):
    one = dt.Adapters(Tensor(4, 16, K), Tensor(4, O, 16), terms=1)
    assert adapters().terms == 2 and adapters()._struct.terms == 2 and one._struct.terms == 1
    assert dt.project_workspace(projection(), BATCH, N, adapters()).numel() == 1024
    assert dt.project_workspace(projection(), BATCH, N, one).numel() == 512
    for terms in (0, 3):
        with pytest.raises(ValueError, match="terms"):
            dt.Adapters(Tensor(4, 16, K), Tensor(4, O, 16), terms=terms)
