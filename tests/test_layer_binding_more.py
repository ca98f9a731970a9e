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


class Strided(Tensor):
    def __init__(self, *shape, strides, **kw):
        super().__init__(*shape, **kw)
        self.strides = strides

    def stride(self, *d):
        return self.strides[d[0]] if d else self.strides


@pytest.mark.parametrize("strides", [(K, K, 1), (5 * K, K, 1), (7, 9, 1), (1 << 40, K + 3, 1)])
def test_the_stride_of_a_single_row_does_not_count(lib, strides):
    """The last row of a long sequence, or a row of a padded one: its distance to a next row may be past what a call
    takes, or no multiple of 16 bytes."""
    x = Strided(1, 1, K, strides=strides)
    out = Strided(1, 1, O, strides=strides)
    dt.project(projection(), x, out=out)
    args = lib.calls[-1][1]
    assert (args[2], args[12]) == (K, O)
    assert dt.Projection(Strided(1, K, strides=strides[1:]))._struct.ld == K
    one = Strided(2, 1, K, strides=(96, 7, 1))          # of several, the first stride does
    dt.project(projection(), one)
    assert lib.calls[-1][1][2] == 96


def test_check_waits_for_the_device(monkeypatch):
    """Not for the current stream alone: the status is read once all streams are done."""
    said = []
    monkeypatch.setattr(torch.cuda, "synchronize", lambda dev=None: said.append(dev))

    class Status(Tensor):
        def __int__(self):
            assert said == ["cuda:0"]
            return dt.ERR_BAD_INDEX

        def tolist(self):
            assert said == ["cuda:0"]
            return [0, dt.ERR_NO_PAGES]
    monkeypatch.setattr(dt, "status_string", str)
    p = projection()
    p.status = Status(1, dtype=torch.int32)
    with pytest.raises(dt.DtError, match="-9"):
        p.check()
    said.clear()
    cache = dt.PagedCache.__new__(dt.PagedCache)
    cache.device, cache.status = "cuda:0", Status(2, dtype=torch.int32)
    with pytest.raises(dt.DtError, match="request 1: -8"):
        cache.check()
