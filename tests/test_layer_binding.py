"""What the Python calls for page tables, norms and projections decide before the library is entered
(CPU only: tensors, streams and the library are stand-ins that record what is asked of them)."""
from __future__ import annotations

import types

import pytest
import torch

import conditional_draft_tree_gb300 as dt
from test_cache_binding import Library, Tensor, ints, lib, stream_of  # noqa: F401  (lib is a fixture)

BATCH, N, K, O = 2, 3, 64, 48
BF, E4 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def more(monkeypatch):
    """What these calls ask of a tensor beyond the cache's."""
    monkeypatch.setattr(Tensor, "dim", lambda t: len(t.shape), raising=False)
    monkeypatch.setattr(Tensor, "device", property(lambda t: "cuda:%d" % t.dev), raising=False)
    old = Tensor.stride
    monkeypatch.setattr(Tensor, "stride", lambda t, *d: old(t)[d[0]] if d else old(t))
    monkeypatch.setattr(torch, "zeros", lambda *s, **k: Tensor(*s, dtype=k.get("dtype")))


def norm(dev=0):
    return dt.Norm(Tensor(K, dev=dev))


def rows(dev=0, d=K):
    return Tensor(BATCH, N, d, dev=dev)


def rows8(dev=0, made=K):
    return dt.Rows8(Tensor(BATCH, N, made, dtype=E4, dev=dev), Tensor(BATCH, N, dtype=torch.uint8, dev=dev))


def projection(dev=0, eight=False):
    p = dt.Projection(dt.Rows8(Tensor(O, K, dtype=E4, dev=dev), Tensor(O, dtype=torch.uint8, dev=dev)) if eight
                      else Tensor(O, K, dev=dev))
    return p


def adapters(dev=0, dtype=BF, o=O, k=K):
    return dt.Adapters(Tensor(4, 16, k, dtype=dtype, dev=dev), Tensor(4, o, 16, dtype=dtype, dev=dev))


def cache(dev=0):
    return types.SimpleNamespace(batch=BATCH, _dev=dev, device="cuda:%d" % dev,
                                 _struct=types.SimpleNamespace(pages=7))


def pool(dev=0):
    return dt.PagePool(cache(dev), ints(BATCH, dev=dev), ints(7, dev=dev), ints(2, dev=dev))


# every call that makes tensors, and all that it returns
MAKERS = {
    "norm": lambda s: list(dt.rms_norm(norm(), rows(), rows(), stream=s)),
    "norm e4m3": lambda s: (lambda y: [y.codes, y.exps])(dt.rms_norm(norm(), rows(), kind="e4m3", stream=s)),
    "norm both": lambda s: (lambda y: [y[0], y[1].codes, y[1].exps])(dt.rms_norm(norm(), rows(), kind="both", stream=s)),
    "quantize": lambda s: (lambda y: [y.codes, y.exps])(dt.quantize_rows(rows(), stream=s)),
    "project": lambda s: [dt.project(projection(), rows(), stream=s)],
    "project with adapters": lambda s: [dt.project(projection(eight=True), rows8(), adapters(), ints(BATCH), rows(),
                                                   stream=s)],
    "slots": lambda s: list(dt.cache_slots(cache(), N, ints(BATCH), stream=s)),
}


@pytest.mark.parametrize("call", MAKERS)
def test_results_are_made_on_the_stream_that_writes_them(lib, call):
    stream = stream_of()
    made = MAKERS[call](stream)
    assert [t.made_on for t in made] == [stream] * len(made)
    assert [args[-1] for name, args in lib.calls if not name.endswith("_bytes")] == [77]
    assert all(t.made_on is None for t in MAKERS[call](None))


def test_a_workspace_of_a_call_is_made_on_the_stream_that_uses_it(lib, monkeypatch):
    made = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(empty(*a, **k)) or made[-1])
    stream = stream_of()
    dt.project(projection(), rows(), adapters(), ints(BATCH), out=rows(d=O), stream=stream)
    assert [t.made_on for t in made] == [stream]
    assert dt.project_workspace(projection(), BATCH, N, None) is None


ON = {
    "norm": lambda dev, s=None: dt.rms_norm(norm(dev), rows(dev), rows(dev), out=rows(dev), total=rows(dev), stream=s),
    "quantize": lambda dev, s=None: dt.quantize_rows(rows(dev), stream=s),
    "project": lambda dev, s=None: dt.project(projection(dev), rows(dev), adapters(dev), ints(BATCH, dev=dev),
                                              out=rows(dev, O), stream=s),
    "workspace": lambda dev, s=None: dt.project_workspace(projection(dev), BATCH, N, adapters(dev), stream=s),
    "slots": lambda dev, s=None: dt.cache_slots(cache(dev), N, ints(BATCH, dev=dev), stream=s),
    "reserve": lambda dev, s=None: dt.cache_reserve(pool(dev), ints(BATCH, dev=dev), stream=s),
}


@pytest.mark.parametrize("call", ON)
def test_tensors_off_the_current_device_are_refused(lib, call):
    with pytest.raises(ValueError, match="current device"):
        ON[call](1)
    assert not lib.calls
    with pytest.raises(ValueError, match="stream"):
        ON[call](0, stream_of(1))
    assert not lib.calls
    ON[call](0, stream_of(0))
    assert lib.calls


REFUSED = {
    "rows of a wrong type": lambda: dt.rms_norm(norm(), Tensor(BATCH, N, K, dtype=torch.float32)),
    "host rows": lambda: dt.rms_norm(norm(), rows(-1)),
    "a weight of another width": lambda: dt.rms_norm(norm(), rows(d=K + 8)),
    "a weight of another type": lambda: dt.rms_norm(norm(), Tensor(BATCH, N, K, dtype=torch.float16)),
    "a weight on another device": lambda: dt.rms_norm(norm(1), rows()),
    "a residual of another shape": lambda: dt.rms_norm(norm(), rows(), Tensor(BATCH, K)),
    "a residual on another device": lambda: dt.rms_norm(norm(), rows(), rows(1)),
    "total without residual": lambda: dt.rms_norm(norm(), rows(), total=rows()),
    "out for codes": lambda: dt.rms_norm(norm(), rows(), kind="e4m3", out=rows()),
    "an unknown kind": lambda: dt.rms_norm(norm(), rows(), kind="8"),
    "a norm weight of two dimensions": lambda: dt.Norm(Tensor(1, K)),
    "codes of a wrong type": lambda: dt.Rows8(Tensor(4, K), Tensor(4, dtype=torch.uint8)),
    "exponents of a wrong shape": lambda: dt.Rows8(Tensor(4, K, dtype=E4), Tensor(5, dtype=torch.uint8)),
    "a host weight": lambda: dt.Projection(Tensor(O, K, dev=-1)),
    "a weight of fp32": lambda: dt.Projection(Tensor(O, K, dtype=torch.float32)),
    "adapters of two types": lambda: dt.Adapters(Tensor(4, 16, K), Tensor(4, O, 16, dtype=torch.float16)),
    "adapters of two ranks": lambda: dt.Adapters(Tensor(4, 16, K), Tensor(4, O, 32)),
    "a scale of another length": lambda: dt.Adapters(Tensor(4, 16, K), Tensor(4, O, 16), Tensor(3, dtype=torch.float32)),
    "rows of another width": lambda: dt.project(projection(), rows(d=K + 16)),
    "rows of another type": lambda: dt.project(projection(), Tensor(BATCH, N, K, dtype=torch.float16)),
    "8-bit rows on 16-bit weights": lambda: dt.project(projection(), rows8()),
    "16-bit rows on 8-bit weights": lambda: dt.project(projection(eight=True), rows()),
    "adapters without an index": lambda: dt.project(projection(), rows(), adapters()),
    "an index without adapters": lambda: dt.project(projection(), rows(), index=ints(BATCH)),
    "an index of another length": lambda: dt.project(projection(), rows(), adapters(), ints(BATCH + 1)),
    "a host index": lambda: dt.project(projection(), rows(), adapters(), ints(BATCH, dev=-1)),
    "adapters of another projection": lambda: dt.project(projection(), rows(), adapters(o=O + 1), ints(BATCH)),
    "adapters of another type": lambda: dt.project(projection(), rows(), adapters(dtype=torch.float16), ints(BATCH)),
    "8-bit rows with adapters alone": lambda: dt.project(projection(eight=True), rows8(), adapters(), ints(BATCH)),
    "16-bit rows of another shape": lambda: dt.project(projection(eight=True), rows8(), adapters(), ints(BATCH),
                                                       rows(d=K + 16)),
    "an out of another type": lambda: dt.project(projection(), rows(), out=Tensor(BATCH, N, O, dtype=torch.float16)),
    "an out of another shape": lambda: dt.project(projection(), rows(), out=rows(d=O + 1)),
    "a host workspace": lambda: dt.project(projection(), rows(), adapters(), ints(BATCH),
                                           workspace=Tensor(4096, dtype=torch.uint8, dev=-1)),
    "held of another length": lambda: dt.PagePool(cache(), ints(BATCH + 1), ints(7), ints(2)),
    "free pages of another length": lambda: dt.PagePool(cache(), ints(BATCH), ints(6), ints(2)),
    "no state": lambda: dt.PagePool(cache(), ints(BATCH), ints(7), None),
    "lengths of another type": lambda: dt.cache_reserve(pool(), Tensor(BATCH, dtype=torch.int64)),
    "no lengths": lambda: dt.cache_reserve(pool(), None),
    "no first rows": lambda: dt.cache_slots(cache(), N, None),
    "slots of 32 bits": lambda: dt.cache_slots(cache(), N, ints(BATCH), slots=ints(BATCH, N)),
}


@pytest.mark.parametrize("what", REFUSED)
def test_refusals(lib, what):
    with pytest.raises(ValueError):
        REFUSED[what]()
    assert not lib.calls


def test_strided_rows_of_a_projection(lib):
    class Strided(Tensor):
        strides = None

        def stride(self, *d):
            return self.strides[d[0]] if d else self.strides

    def view(*strides):
        t = Strided(BATCH, N, K)
        t.strides = strides
        return t
    for strides in ((N * 80, 80, 1), (N * K, K, 1)):
        dt.project(projection(), view(*strides))
        assert lib.calls[-1][1][2] == strides[1]
    for strides in ((N * 80 + 8, 80, 1), (N * K, K, 2)):
        with pytest.raises(ValueError, match="stride"):
            dt.project(projection(), view(*strides))
