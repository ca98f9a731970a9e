"""What the paged-cache calls of the Python binding decide before the library is entered
(CPU only: tensors, streams and the library are stand-ins that record what is asked of them)."""
from __future__ import annotations

import contextlib
import types

import pytest
import torch

import conditional_draft_tree_gb300 as dt

BATCH, H, HKV, N, DH = 2, 4, 2, 3, 64


class Tensor:
    """As much of a dense CUDA tensor as the binding looks at."""

    def __init__(self, *shape, dtype=torch.bfloat16, dev=0, made_on=None):
        self.shape, self.dtype, self.dev, self.made_on = torch.Size(shape), dtype, dev, made_on

    def stride(self):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s)

    def get_device(self):
        return self.dev

    def data_ptr(self):
        return 4096

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 512 if name.endswith("_bytes") else dt.OK
        return call


@pytest.fixture
def lib(monkeypatch):
    """The library's stand-in; tensors that a call makes note the stream they are made on."""
    made_on = [None]

    @contextlib.contextmanager
    def on(stream):
        made_on.append(stream)
        yield
        made_on.pop()

    def empty(*shape, dtype=None, device=None):
        shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
        return Tensor(*shape, dtype=dtype, made_on=made_on[-1])

    library = Library()
    monkeypatch.setattr(dt, "lib", lambda: library)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda t, **_: Tensor(*t.shape, dtype=t.dtype, made_on=made_on[-1]))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 1, raising=False)
    return library


def stream_of(dev=0):
    return types.SimpleNamespace(cuda_stream=77, device_index=dev)


def cache_of(dev=0):
    return types.SimpleNamespace(batch=BATCH, Hkv=HKV, dh=DH, _dev=dev, device="cuda:%d" % dev, _struct=None,
                                 k=Tensor(8, HKV, 16, DH, dev=dev))


def ints(*shape, dev=0):
    return Tensor(*shape, dtype=torch.int32, dev=dev)


def rotation(dev=0):
    return types.SimpleNamespace(_struct=None, _dev=dev)


def heads(n=H, dev=0):
    return Tensor(BATCH, n, N, DH, dev=dev)


# every call that makes tensors, and all that it returns
MAKERS = {
    "rotary": lambda s: dt.rotary(rotation(), ints(BATCH, N), heads(), heads(HKV), stream=s),
    "write": lambda s: [dt.cache_write(cache_of(), heads(HKV), heads(HKV), ints(BATCH), rotary=rotation(),
                                       positions=ints(BATCH, N), q=heads(), stream=s)],
    "read": lambda s: dt.cache_read(cache_of(), N, ints(BATCH), stream=s),
    "attention": lambda s: [dt.cache_attention(cache_of(), heads(), ints(BATCH), stream=s)],
}


@pytest.mark.parametrize("call", MAKERS)
def test_results_are_made_on_the_stream_that_writes_them(lib, call):
    stream = stream_of()
    assert [t.made_on for t in MAKERS[call](stream)] == [stream] * (2 if call in ("rotary", "read") else 1)
    assert [args[-1] for name, args in lib.calls if not name.endswith("_bytes")] == [77]
    assert all(t.made_on is None for t in MAKERS[call](None))


def test_a_workspace_of_a_call_is_made_on_the_stream_that_uses_it(lib, monkeypatch):
    made = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(empty(*a, **k)) or made[-1])
    stream = stream_of()
    dt.cache_attention(cache_of(), heads(), ints(BATCH), out=heads(), stream=stream)
    assert [t.made_on for t in made] == [stream]


# every entry point, on tensors of device `dev`
ON = {
    "rotary": lambda dev, s=None: dt.rotary(rotation(dev), ints(BATCH, N, dev=dev), heads(dev=dev), stream=s),
    "write": lambda dev, s=None: dt.cache_write(cache_of(dev), heads(HKV, dev), heads(HKV, dev), ints(BATCH, dev=dev),
                                                stream=s),
    "read": lambda dev, s=None: dt.cache_read(cache_of(dev), N, ints(BATCH, dev=dev), k_out=heads(HKV, dev),
                                              v_out=heads(HKV, dev), stream=s),
    "commit": lambda dev, s=None: dt.cache_commit(cache_of(dev), ints(BATCH, dev=dev), ints(BATCH, 4, dev=dev),
                                                  ints(BATCH, dev=dev), N, stream=s),
    "attention": lambda dev, s=None: dt.cache_attention(cache_of(dev), heads(dev=dev), ints(BATCH, dev=dev), stream=s),
    "workspace": lambda dev, s=None: dt.cache_attention_workspace(cache_of(dev), H, N, stream=s),
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


@pytest.mark.parametrize("dev", [-1, 1])
def test_a_rotary_table_on_another_device_is_refused(lib, dev):
    """-1: a table left on the host, whose address a kernel cannot read."""
    with pytest.raises(ValueError, match="rotary table"):
        dt.rotary(rotation(dev), ints(BATCH, N), heads())
    with pytest.raises(ValueError, match="rotary table"):
        dt.cache_write(cache_of(), heads(HKV), heads(HKV), ints(BATCH), rotary=rotation(dev), positions=ints(BATCH, N))
    assert not lib.calls


def test_a_rotary_table_knows_its_device():
    from conditional_draft_tree_gb300 import build
    build.build()
    r = dt.Rotary(64, device="cpu")
    assert r._dev == r.turns.get_device() == -1
