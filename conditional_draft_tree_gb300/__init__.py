"""Python binding of ``libdt.so``, the GB300 conditional draft-tree builder.

Argument marshalling only: every step of a round runs in the library's CUDA
kernels. PyTorch provides device memory and streams. The functions mirror the
C ABI of ``include/dt.h`` (same names without the ``dt_`` prefix) and take
torch tensors where the C ABI takes pointers. When ``libdt.so`` is missing,
every call raises: there is no fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import functools
import os
import struct
from dataclasses import dataclass

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdt.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA = 0, -1, -2, -3
ERR_NONFINITE, ERR_TIMEOUT, ERR_BAD_TEMPERATURE, ERR_BAD_PAGE = -4, -5, -6, -7
ERR_NO_PAGES, ERR_BAD_INDEX = -8, -9
F32, BF16, F16, E4M3 = 0, 1, 2, 3
NUM_PHASE_EVENTS = 4
OPT_TEST_BARRIER_TIMEOUT = 2  # dt_options.flags: failure-detection test hook
OPT_MARGINAL = 8             # dt_options.flags: marginal (path-independent) scores
OPT_STAGE_HOST_LOGITS = 16   # dt_options.flags: copy mapped host logits instead of reading in place
MAX_SPEC = 16

# every symbol include/dt.h declares
EXPORTS = ("dt_abi_version", "dt_status_string", "dt_prepared_bytes", "dt_prepare_weights",
           "dt_workspace_bytes", "dt_build_trees", "dt_host_workspace_bytes",
           "dt_build_trees_host", "dt_select_topm_noalloc", "dt_kernel_launches",
           "dt_chain_prepared_bytes", "dt_prepare_chain", "dt_chain_workspace_bytes",
           "dt_chain_kernel_launches", "dt_decode_chains", "dt_tree_positions",
           "dt_tree_attention", "dt_adaptive_budget", "dt_mapped_host_pointer",
           "dt_rotary_table", "dt_rotary", "dt_cache_write", "dt_cache_read", "dt_cache_commit",
           "dt_cache_attention_workspace_bytes", "dt_cache_attention", "dt_cache_reserve",
           "dt_cache_slots", "dt_rms_norm", "dt_quantize_rows", "dt_project_workspace_bytes",
           "dt_project")
NOALLOC_SCRATCH_BYTES = 8 << 20


class DtDims(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("V", "d", "d_s", "r", "D", "M", "k", "N", "batch")]


class DtWeights(C.Structure):
    _fields_ = [("E", C.c_void_p), ("W_ih", C.c_void_p), ("W_hh", C.c_void_p),
                ("b_ih", C.c_void_p), ("b_hh", C.c_void_p), ("W1", C.c_void_p),
                ("W2", C.c_void_p), ("wdtype", C.c_int)]


class DtTreeOut(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("tokens", "parents", "depths", "scores", "mask",
                                           "topm", "status")]


class DtOptions(C.Structure):
    _fields_ = [("spec_width", C.c_int), ("phase_events", C.POINTER(C.c_void_p)),
                ("flags", C.c_int)]


class DtRotaryParams(C.Structure):
    _fields_ = [("rot", C.c_int), ("scaling", C.c_int)] + \
        [(n, C.c_double) for n in ("base", "factor", "trained", "beta_fast", "beta_slow")]


class DtRotation(C.Structure):
    _fields_ = [("turns", C.c_void_p), ("rot", C.c_int), ("interleaved", C.c_int),
                ("magnitude", C.c_float)]


class DtHeads(C.Structure):
    _fields_ = [("data", C.c_void_p), ("heads", C.c_int), ("stride_batch", C.c_int64),
                ("stride_head", C.c_int64), ("stride_row", C.c_int64)]


class DtCache(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("k", "v", "k_exp", "v_exp", "table", "status")] + \
        [(n, C.c_int) for n in ("pages", "page", "Hkv", "dh", "dtype", "batch", "table_width")]


class DtPagePool(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("held", "free_pages", "state")]


class DtRows(C.Structure):
    _fields_ = [("data", C.c_void_p), ("stride_outer", C.c_int64), ("stride_inner", C.c_int64)]


_pack_rows = struct.Struct("@Pqq").pack     # a dt_rows as bytes: half the time of a DtRows


class DtMatrix(C.Structure):
    _fields_ = [("data", C.c_void_p), ("exps", C.c_void_p), ("ld", C.c_int64)] + \
        [(n, C.c_int) for n in ("O", "K", "dtype", "wait_cycles")]


class DtAdapters(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("down", "up", "scale")] + \
        [(n, C.c_int) for n in ("count", "rank", "terms")]


class DtError(RuntimeError):
    pass


_lib = None


def lib():
    """Load libdt.so (built by ``build.build()``); raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise DtError(f"{LIB_PATH} is not built; run conditional_draft_tree_gb300.build.build()")
        L = C.CDLL(LIB_PATH)
        L.dt_abi_version.restype = C.c_int
        L.dt_status_string.restype = C.c_char_p
        L.dt_status_string.argtypes = [C.c_int]
        L.dt_prepared_bytes.restype = C.c_size_t
        L.dt_prepared_bytes.argtypes = [C.POINTER(DtDims)]
        L.dt_prepare_weights.argtypes = [C.POINTER(DtDims), C.POINTER(DtWeights), C.c_void_p,
                                         C.c_size_t, C.c_void_p]
        L.dt_workspace_bytes.restype = C.c_size_t
        L.dt_workspace_bytes.argtypes = [C.POINTER(DtDims), C.POINTER(DtOptions)]
        L.dt_host_workspace_bytes.restype = C.c_size_t
        L.dt_host_workspace_bytes.argtypes = [C.POINTER(DtDims), C.POINTER(DtOptions)]
        L.dt_kernel_launches.restype = C.c_int
        L.dt_kernel_launches.argtypes = [C.POINTER(DtDims), C.c_int, C.POINTER(DtOptions)]
        sig = [C.POINTER(DtDims), C.POINTER(DtWeights), C.c_void_p, C.c_void_p, C.c_void_p,
               C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t,
               C.POINTER(DtTreeOut), C.POINTER(DtOptions), C.c_void_p]
        L.dt_build_trees.argtypes = sig
        L.dt_build_trees_host.argtypes = sig
        L.dt_mapped_host_pointer.restype = C.c_void_p
        L.dt_mapped_host_pointer.argtypes = [C.c_void_p, C.c_size_t]
        L.dt_select_topm_noalloc.argtypes = [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int,
                                             C.c_void_p, C.c_void_p, C.c_void_p]
        L.dt_chain_prepared_bytes.restype = C.c_size_t
        L.dt_chain_prepared_bytes.argtypes = [C.POINTER(DtDims)]
        L.dt_prepare_chain.argtypes = [C.POINTER(DtDims), C.POINTER(DtWeights), C.c_void_p,
                                       C.c_size_t, C.c_void_p]
        L.dt_chain_workspace_bytes.restype = C.c_size_t
        L.dt_chain_workspace_bytes.argtypes = [C.POINTER(DtDims)]
        L.dt_chain_kernel_launches.restype = C.c_int
        L.dt_chain_kernel_launches.argtypes = [C.POINTER(DtDims)]
        L.dt_decode_chains.argtypes = [C.POINTER(DtDims), C.POINTER(DtWeights)] + \
            [C.c_void_p] * 9 + [C.c_size_t] + [C.c_void_p] * 4
        L.dt_adaptive_budget.argtypes = [C.POINTER(DtTreeOut), C.c_int, C.c_int, C.c_double,
                                         C.c_double, C.c_void_p, C.c_void_p]
        L.dt_tree_positions.argtypes = [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_void_p,
                                        C.c_void_p]
        L.dt_tree_attention.argtypes = [C.c_void_p] * 5 + [C.c_int] * 6 + [C.c_float, C.c_void_p,
                                                                          C.c_void_p]
        heads, cache, rot = C.POINTER(DtHeads), C.POINTER(DtCache), C.POINTER(DtRotation)
        L.dt_rotary_table.argtypes = [C.POINTER(DtRotaryParams), C.c_void_p,
                                      C.POINTER(C.c_double)]
        L.dt_rotary.argtypes = [rot, C.c_void_p] + [C.c_int] * 4 + [heads] * 4 + [C.c_int,
                                                                                  C.c_void_p]
        L.dt_cache_write.argtypes = [cache, heads, heads, C.c_int, C.c_int, C.c_void_p, C.c_void_p,
                                     rot, C.c_void_p, heads, heads, C.c_void_p]
        L.dt_cache_read.argtypes = [cache, C.c_int, C.c_int, C.c_void_p, C.c_void_p, heads, heads,
                                    C.c_void_p]
        L.dt_cache_commit.argtypes = [cache] + [C.c_void_p] * 3 + [C.c_int, C.c_int, C.c_void_p]
        L.dt_cache_attention_workspace_bytes.restype = C.c_size_t
        L.dt_cache_attention_workspace_bytes.argtypes = [cache, C.c_int, C.c_int]
        L.dt_cache_attention.argtypes = [cache, heads, C.c_int, C.c_int] + [C.c_void_p] * 3 + \
            [C.c_float, heads, C.c_void_p, C.c_size_t, C.c_void_p]
        # the dt_rows of a norm are packed bytes or the address of a DtRows
        rows, v, i, n64 = C.c_char_p, C.c_void_p, C.c_int, C.c_int64
        L.dt_cache_reserve.argtypes = [cache, C.POINTER(DtPagePool), v, v]
        L.dt_cache_slots.argtypes = [cache, i, v, v, v, v, v]
        L.dt_rms_norm.argtypes = [rows] * 4 + [v] * 3 + [C.c_float] * 2 + [i] * 4 + [v]
        L.dt_quantize_rows.argtypes = [rows, v, v] + [i] * 4 + [v]
        L.dt_project_workspace_bytes.restype = C.c_size_t
        L.dt_project_workspace_bytes.argtypes = [i] * 3
        L.dt_project.argtypes = [C.POINTER(DtMatrix), v, n64, v, i, i, i, C.POINTER(DtAdapters), v, v,
                                 n64, v, n64, v, v, C.c_size_t, v]
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().dt_status_string(int(code)).decode()


def abi_version() -> int:
    return lib().dt_abi_version()


def _check(rc: int, what: str):
    if rc != OK:
        raise DtError(f"{what}: {status_string(rc)} ({rc})")


def dims_of(V, d, d_s, r, D, M, k, N, batch) -> DtDims:
    return DtDims(V, d, d_s, r, D, M, k, N, batch)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def options(spec_width: int = 0, events=None, flags: int = 0) -> DtOptions:
    """Build a dt_options; ``events``: DT_NUM_PHASE_EVENTS torch.cuda.Event or None;
    ``flags``: OPT_* bits."""
    o = DtOptions(spec_width, None, flags)
    if events is not None:
        arr = (C.c_void_p * NUM_PHASE_EVENTS)(*[e.cuda_event for e in events])
        o.phase_events = C.cast(arr, C.POINTER(C.c_void_p))
        o._keep = arr
    return o


@dataclass
class DeviceWeights:
    """Domino head weights on the device (see dt_weights in include/dt.h)."""
    E: torch.Tensor
    W_ih: torch.Tensor
    W_hh: torch.Tensor
    W1: torch.Tensor
    W2: torch.Tensor
    b_ih: torch.Tensor | None = None
    b_hh: torch.Tensor | None = None

    @property
    def wdtype(self) -> int:
        return BF16 if self.E.dtype in (torch.int16, torch.uint16, torch.bfloat16) else F32

    def struct(self) -> DtWeights:
        return DtWeights(_ptr(self.E), _ptr(self.W_ih), _ptr(self.W_hh), _ptr(self.b_ih),
                         _ptr(self.b_hh), _ptr(self.W1), _ptr(self.W2), self.wdtype)


def prepared_bytes(dims: DtDims) -> int:
    return lib().dt_prepared_bytes(C.byref(dims))


def prepare_weights(dims: DtDims, w: DeviceWeights, prepared: torch.Tensor, stream=None):
    ws = w.struct()
    _check(lib().dt_prepare_weights(C.byref(dims), C.byref(ws), prepared.data_ptr(),
                                    prepared.numel() * prepared.element_size(), _stream(stream)),
           "dt_prepare_weights")


def workspace_bytes(dims: DtDims, opt: DtOptions | None = None) -> int:
    return lib().dt_workspace_bytes(C.byref(dims), C.byref(opt) if opt else None)


def kernel_launches(dims: DtDims, wdtype: int, opt: DtOptions | None = None) -> int:
    """Kernels one build_trees call launches (see dt_kernel_launches)."""
    return lib().dt_kernel_launches(C.byref(dims), int(wdtype), C.byref(opt) if opt else None)


def host_workspace_bytes(dims: DtDims, opt: DtOptions | None = None) -> int:
    return lib().dt_host_workspace_bytes(C.byref(dims), C.byref(opt) if opt else None)


def alloc_outputs(dims: DtDims, device, mask=True, topm=True, pin=False):
    """Output tensors of dt_tree_out (device, or pinned host with device='cpu', pin=True)."""
    n1 = dims.N + 1
    kw = dict(device=device, pin_memory=pin) if pin else dict(device=device)
    out = dict(tokens=torch.empty((dims.batch, n1), dtype=torch.int32, **kw),
               parents=torch.empty((dims.batch, n1), dtype=torch.int32, **kw),
               depths=torch.empty((dims.batch, n1), dtype=torch.int32, **kw),
               scores=torch.empty((dims.batch, n1), dtype=torch.float32, **kw),
               status=torch.empty((dims.batch,), dtype=torch.int32, **kw))
    out["mask"] = torch.empty((dims.batch, n1, n1), dtype=torch.uint8, **kw) if mask else None
    out["topm"] = (torch.empty((dims.batch, dims.D, dims.M), dtype=torch.int32, **kw)
                   if topm else None)
    return out


def _out_struct(out) -> DtTreeOut:
    return DtTreeOut(*[_ptr(out.get(n)) for n in ("tokens", "parents", "depths", "scores",
                                                  "mask", "topm", "status")])


def build_trees(dims: DtDims, w: DeviceWeights, prepared, base_logits, H, state0, anchor_tok,
                temperature, workspace, out, opt: DtOptions | None = None, stream=None):
    """Enqueue one round on device tensors (dt_build_trees). With OPT_MARGINAL in
    ``opt.flags``, ``w``, ``prepared``, ``H`` and ``state0`` may be None."""
    ws = w.struct() if w is not None else None
    o = _out_struct(out)
    _check(lib().dt_build_trees(C.byref(dims), C.byref(ws) if ws else None, _ptr(prepared),
                                _ptr(base_logits),
                                _ptr(H), _ptr(state0), _ptr(anchor_tok), _ptr(temperature),
                                _ptr(workspace), workspace.numel() * workspace.element_size(),
                                C.byref(o), C.byref(opt) if opt else None, _stream(stream)),
           "dt_build_trees")


def build_trees_host(dims: DtDims, w: DeviceWeights, prepared, base_logits, H, state0,
                     anchor_tok, temperature, workspace, host_out, opt: DtOptions | None = None,
                     stream=None):
    """Enqueue one round on HOST input/output tensors (dt_build_trees_host). Synchronise
    the stream before reading ``host_out``."""
    ws = w.struct() if w is not None else None
    o = _out_struct(host_out)
    _check(lib().dt_build_trees_host(C.byref(dims), C.byref(ws) if ws else None, _ptr(prepared),
                                     _ptr(base_logits), _ptr(H), _ptr(state0), _ptr(anchor_tok),
                                     _ptr(temperature), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), C.byref(o),
                                     C.byref(opt) if opt else None, _stream(stream)),
           "dt_build_trees_host")


def mapped_host_pointer(t) -> int | None:
    """dt_mapped_host_pointer for a host tensor's whole storage extent: the
    device address kernels can read it through in place, or None."""
    return lib().dt_mapped_host_pointer(_ptr(t), t.numel() * t.element_size()) or None


def select_topm_noalloc(base_logits, M: int, topm, status, stream=None) -> int:
    """dt_select_topm_noalloc on device tensors: base_logits [batch][D][V] fp32,
    topm [batch][D][M] int32 and status [batch] int32 outputs. Allocates no
    device memory (the library's static scratch is used; see include/dt.h).
    Returns the C status code."""
    if base_logits.dim() != 3 or base_logits.dtype != torch.float32 or \
            not base_logits.is_contiguous() or not base_logits.is_cuda:
        raise ValueError("base_logits must be a contiguous [batch][D][V] float32 CUDA tensor")
    batch, D, V = base_logits.shape
    dev = base_logits.device
    if topm.shape != (batch, D, int(M)) or topm.dtype != torch.int32 or \
            not topm.is_contiguous() or topm.device != dev:
        raise ValueError("topm must be a contiguous [batch][D][M] int32 tensor on base_logits' device")
    if status.shape != (batch,) or status.dtype != torch.int32 or \
            not status.is_contiguous() or status.device != dev:
        raise ValueError("status must be a contiguous [batch] int32 tensor on base_logits' device")
    with torch.cuda.device(dev):
        return lib().dt_select_topm_noalloc(_ptr(base_logits), batch, D, V, int(M), _ptr(topm),
                                            _ptr(status), _stream(stream))


class TreeBuilder:
    """Holds device weights, the prepared table and a workspace for one shape.

    ``TreeBuilder.from_numpy(workload)`` copies a host workload's weights to the
    device and prepares them; ``run(...)`` builds one round on device tensors."""

    def __init__(self, dims: DtDims, weights: DeviceWeights, spec_width: int = 0,
                 device="cuda", flags: int = 0):
        self.dims = dims
        self.w = weights
        self.device = torch.device(device)
        self.opt = options(spec_width, flags=flags)
        nbytes = prepared_bytes(dims)
        if nbytes == 0:
            raise DtError("invalid dims")
        self.prepared = torch.empty(nbytes // 4, dtype=torch.float32, device=self.device)
        prepare_weights(dims, weights, self.prepared)
        wsb = workspace_bytes(dims, self.opt)
        if wsb == 0:
            raise DtError("dt_workspace_bytes failed (invalid dims or unsupported device)")
        self.workspace = torch.empty(wsb, dtype=torch.uint8, device=self.device)

    @staticmethod
    def weights_from_numpy(wl, device="cuda") -> DeviceWeights:
        import numpy as np

        def t(a):
            if a is None:
                return None
            a = np.ascontiguousarray(a)
            if a.dtype == np.uint16:
                a = a.view(np.int16)
            return torch.from_numpy(a).to(device)
        return DeviceWeights(E=t(wl.E), W_ih=t(wl.W_ih), W_hh=t(wl.W_hh), W1=t(wl.W1),
                             W2=t(wl.W2), b_ih=t(wl.b_ih), b_hh=t(wl.b_hh))

    @classmethod
    def from_numpy(cls, wl, spec_width: int = 0, device="cuda", batch=None, flags: int = 0):
        dims = dims_of(wl.V, wl.d, wl.d_s, wl.r, wl.D, wl.M, wl.k, wl.N,
                       wl.batch if batch is None else batch)
        return cls(dims, cls.weights_from_numpy(wl, device), spec_width, device, flags)

    def run(self, base_logits, H, state0, anchor_tok, temperature=None, out=None, stream=None,
            opt=None):
        if out is None:
            out = alloc_outputs(self.dims, self.device)
        build_trees(self.dims, self.w, self.prepared, base_logits, H, state0, anchor_tok,
                    temperature, self.workspace, out, opt or self.opt, stream)
        return out

    def inputs_to_device(self, wl):
        import numpy as np
        f = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a, dtype=dt)).to(self.device)
        return dict(base_logits=f(wl.base_logits, np.float32), H=f(wl.H, np.float32),
                    state0=f(wl.state0, np.float32), anchor_tok=f(wl.anchor, np.int32),
                    temperature=f(wl.temperature, np.float32))


class MarginalTreeBuilder:
    """Workspace for marginal-score trees (OPT_MARGINAL) of one shape: no
    weights, no GRU state; ``run(base_logits, anchor_tok, temperature)`` builds
    one round on device tensors. ``dims`` keeps d, d_s and r only for the
    shape checks of the C ABI (any valid values)."""

    def __init__(self, dims: DtDims, device="cuda", spec_width: int = 0):
        self.dims = dims
        self.device = torch.device(device)
        self.opt = options(spec_width, flags=OPT_MARGINAL)
        wsb = workspace_bytes(dims, self.opt)
        if wsb == 0:
            raise DtError("dt_workspace_bytes failed (invalid dims or unsupported device)")
        self.workspace = torch.empty(wsb, dtype=torch.uint8, device=self.device)

    @classmethod
    def from_workload(cls, wl, device="cuda", batch=None):
        return cls(dims_of(wl.V, wl.d, wl.d_s, wl.r, wl.D, wl.M, wl.k, wl.N,
                           wl.batch if batch is None else batch), device)

    def run(self, base_logits, anchor_tok, temperature=None, out=None, stream=None, opt=None):
        if out is None:
            out = alloc_outputs(self.dims, self.device)
        build_trees(self.dims, None, None, base_logits, None, None, anchor_tok, temperature,
                    self.workspace, out, opt or self.opt, stream)
        return out

    def inputs_to_device(self, wl):
        import numpy as np
        f = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a, dtype=dt)).to(self.device)
        return dict(base_logits=f(wl.base_logits, np.float32), anchor_tok=f(wl.anchor, np.int32),
                    temperature=f(wl.temperature, np.float32))



# ------------------------------------------------------------ chain decoding

def chain_prepared_bytes(dims: DtDims) -> int:
    return lib().dt_chain_prepared_bytes(C.byref(dims))


def prepare_chain(dims: DtDims, w: DeviceWeights, chain_prepared: torch.Tensor, stream=None):
    """dt_prepare_chain: the weight tiles of the chain decoder's tensor-core products."""
    ws = w.struct()
    _check(lib().dt_prepare_chain(C.byref(dims), C.byref(ws), chain_prepared.data_ptr(),
                                  chain_prepared.numel() * chain_prepared.element_size(),
                                  _stream(stream)), "dt_prepare_chain")


def chain_workspace_bytes(dims: DtDims) -> int:
    return lib().dt_chain_workspace_bytes(C.byref(dims))


def chain_kernel_launches(dims: DtDims) -> int:
    return lib().dt_chain_kernel_launches(C.byref(dims))


def decode_chains(dims: DtDims, w: DeviceWeights, prepared, chain_prepared, base_logits, H,
                  state0, anchor_tok, temperature, uniforms, workspace, tokens, logprobs, status,
                  stream=None):
    """Enqueue one chain-decoding round on device tensors (dt_decode_chains)."""
    ws = w.struct()
    _check(lib().dt_decode_chains(C.byref(dims), C.byref(ws), _ptr(prepared), _ptr(chain_prepared),
                                  _ptr(base_logits), _ptr(H), _ptr(state0), _ptr(anchor_tok),
                                  _ptr(temperature), _ptr(uniforms), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _ptr(tokens),
                                  _ptr(logprobs), _ptr(status), _stream(stream)),
           "dt_decode_chains")


class ChainDecoder:
    """Device weights, both prepared tables and a workspace for Domino chain
    decoding of one shape (bf16 weights). ``run(...)`` decodes one round:
    D draft tokens and their log-probabilities per request."""

    def __init__(self, dims: DtDims, weights: DeviceWeights, device="cuda"):
        self.dims = dims
        self.w = weights
        self.device = torch.device(device)
        nbytes = prepared_bytes(dims)
        cbytes = chain_prepared_bytes(dims)
        if nbytes == 0 or cbytes == 0:
            raise DtError("invalid dims")
        self.prepared = torch.empty(nbytes // 4, dtype=torch.float32, device=self.device)
        prepare_weights(dims, weights, self.prepared)
        self.chain_prepared = torch.empty(cbytes, dtype=torch.uint8, device=self.device)
        prepare_chain(dims, weights, self.chain_prepared)
        wsb = chain_workspace_bytes(dims)
        if wsb == 0:
            raise DtError("dt_chain_workspace_bytes failed (invalid dims or unsupported device)")
        self.workspace = torch.empty(wsb, dtype=torch.uint8, device=self.device)

    @classmethod
    def from_numpy(cls, wl, device="cuda", batch=None):
        dims = dims_of(wl.V, wl.d, wl.d_s, wl.r, wl.D, wl.M, wl.k, wl.N,
                       wl.batch if batch is None else batch)
        return cls(dims, TreeBuilder.weights_from_numpy(wl, device), device)

    def alloc_outputs(self):
        B, D = self.dims.batch, self.dims.D
        return dict(tokens=torch.empty((B, D), dtype=torch.int32, device=self.device),
                    logprobs=torch.empty((B, D), dtype=torch.float32, device=self.device),
                    status=torch.empty((B,), dtype=torch.int32, device=self.device))

    def run(self, base_logits, H, state0, anchor_tok, temperature=None, uniforms=None, out=None,
            stream=None):
        if out is None:
            out = self.alloc_outputs()
        decode_chains(self.dims, self.w, self.prepared, self.chain_prepared, base_logits, H,
                      state0, anchor_tok, temperature, uniforms, self.workspace, out["tokens"],
                      out["logprobs"], out["status"], stream)
        return out

    def inputs_to_device(self, wl, uniforms=None):
        import numpy as np
        f = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a, dtype=dt)).to(self.device)
        d = dict(base_logits=f(wl.base_logits, np.float32), H=f(wl.H, np.float32),
                 state0=f(wl.state0, np.float32), anchor_tok=f(wl.anchor, np.int32),
                 temperature=f(wl.temperature, np.float32))
        if uniforms is not None:
            d["uniforms"] = f(uniforms, np.float32)
        return d



# ------------------------------------------------ verify-side consumption

def tree_positions(depths, prefix_len, out=None, stream=None):
    """dt_tree_positions on device tensors: depths [batch][n1] int32, prefix_len
    [batch] int32 -> position ids [batch][n1] int32."""
    batch, n1 = depths.shape
    if out is None:
        out = torch.empty_like(depths)
    _check(lib().dt_tree_positions(_ptr(depths), _ptr(prefix_len), batch, n1, _ptr(out),
                                   _stream(stream)), "dt_tree_positions")
    return out


def tree_attention(q, k, v, mask, prefix_len, scale=None, out=None, stream=None):
    """dt_tree_attention on device tensors: q [batch][H][n1][dh], k and v
    [batch][Hkv][P + n1][dh] (bf16, or int16/uint16 holding bf16 bits), mask
    [batch][n1][n1] uint8, prefix_len [batch] int32 -> fp32 [batch][H][n1][dh]."""
    batch, H, n1, dh = q.shape
    Hkv, L = k.shape[1], k.shape[2]
    if scale is None:
        scale = dh ** -0.5
    if out is None:
        out = torch.empty((batch, H, n1, dh), dtype=torch.float32, device=q.device)
    _check(lib().dt_tree_attention(_ptr(q), _ptr(k), _ptr(v), _ptr(mask), _ptr(prefix_len), batch,
                                   H, Hkv, n1, L - n1, dh, float(scale), _ptr(out),
                                   _stream(stream)), "dt_tree_attention")
    return out



def adaptive_budget(out: dict, N: int, c_fixed: float, c_node: float, counts=None, stream=None):
    """dt_adaptive_budget: cut the trees of ``out`` (alloc_outputs layout, on
    the device) in place by the cost-aware rule; returns counts [batch] int32."""
    batch = out["tokens"].shape[0]
    if counts is None:
        counts = torch.empty(batch, dtype=torch.int32, device=out["tokens"].device)
    o = _out_struct(out)
    _check(lib().dt_adaptive_budget(C.byref(o), batch, int(N), float(c_fixed), float(c_node),
                                    _ptr(counts), _stream(stream)), "dt_adaptive_budget")
    return counts


# --------------------------------- rotary positions and the paged key/value cache
#
# A call runs on ``stream`` (the current one when None), and the tensors that it makes belong
# to that stream, as under torch.cuda.stream(stream): use them on another stream after waiting
# for this one, and record_stream them there.

_TYPE16 = {torch.bfloat16: BF16, torch.float16: F16}


def _shape(t, what: str):
    """Shape of a [batch][heads][n][dh] tensor, its C type and device number. (These calls
    run once a layer, so their checks are few and plain: a launch takes 2 us.)"""
    shape, dtype, dev = t.shape, _TYPE16.get(t.dtype), t.get_device()
    if len(shape) != 4 or dtype is None or dev < 0:
        raise ValueError(f"{what} must be a [batch][heads][n][dh] bfloat16 or float16 CUDA tensor")
    return shape, dtype, dev


def _heads(t, what: str, shape, dtype, dev) -> DtHeads:
    """A view of that shape, C type and device (last dimension dense) as a dt_heads."""
    s = t.stride()
    if t.shape != shape or _TYPE16.get(t.dtype) != dtype or t.get_device() != dev or s[3] != 1:
        raise ValueError(f"{what} must be of shape {tuple(shape)} with a dense last dimension, and of "
                         "the other tensors' type and device")
    return DtHeads(t.data_ptr(), shape[1], s[0], s[1], s[2])


def _ints(t, what: str, shape, dev):
    if t is None:
        return None
    if t.shape != shape or t.dtype != torch.int32 or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{what} must be a contiguous int32 tensor of shape {tuple(shape)} on the "
                         "other tensors' device")
    return t.data_ptr()


_CURRENT = contextlib.nullcontext()


def _made_on(stream):
    """Where a call makes its tensors: on the stream that its kernels run on, whose part of the
    caching allocator they then belong to. Memory of another stream's part may still be in
    use there, and would be handed out again there while the kernels run."""
    return torch.cuda.stream(stream) if stream is not None else _CURRENT


def _dense_like(t, stream):
    if stream is None:
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    with _made_on(stream):
        return torch.empty_like(t, memory_format=torch.contiguous_format)


def _raw_stream(stream, dev):
    """The stream's handle: the current one of the tensors' device by default. The library
    launches on the thread's current device and sizes its grids for it, so that the tensors
    and the stream have to be of that one."""
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on device {dev}, which is not the current device "
                         "(torch.cuda.device makes it that)")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError("stream is not of the tensors' device")
    return stream.cuda_stream


class Rotary:
    """Rotary positions: the table of dt_rotary_table on the device, and how it is
    used (dt_rotation). ``scaling``: "none", "linear", "base" or "parts"."""

    SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}

    def __init__(self, rot: int, interleaved: bool = False, base: float = 10000.0,
                 scaling: str = "none", factor: float = 1.0, trained: float = 4096,
                 beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
        if scaling not in self.SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(self.SCALINGS)}")
        p = DtRotaryParams(int(rot), self.SCALINGS[scaling], base, factor, trained, beta_fast,
                           beta_slow)
        host = (C.c_uint64 * max(1, int(rot) // 2))()
        mag = C.c_double()
        _check(lib().dt_rotary_table(C.byref(p), host, C.byref(mag)), "dt_rotary_table")
        self.rot, self.interleaved, self.magnitude = int(rot), bool(interleaved), mag.value
        self.turns = torch.frombuffer(bytearray(host), dtype=torch.int64).to(device)
        self._dev = self.turns.get_device()
        self._struct = DtRotation(self.turns.data_ptr(), self.rot, int(self.interleaved),
                                  self.magnitude)


def _rotation(rot: Rotary | None, dev):
    if rot is None:
        return None
    if rot._dev != dev:
        raise ValueError("the rotary table must be on the tensors' device")
    return rot._struct


def rotary(rot: Rotary, positions, q, k=None, q_out=None, k_out=None, gradient=False, stream=None):
    """dt_rotary: q (and k, in the same launch) [batch][heads][n][dh] turned at
    positions [batch][n] int32. ``gradient``: the transposed rotation. Outputs
    default to new dense tensors and may be the inputs. Returns (q_out, k_out), or
    q_out alone without k."""
    shape, dtype, dev = _shape(q, "q")
    batch, _, n, dh = shape
    table, handle = _rotation(rot, dev), _raw_stream(stream, dev)
    x0 = _heads(q, "q", shape, dtype, dev)
    if q_out is None:
        q_out = _dense_like(q, stream)
    o0 = _heads(q_out, "q_out", shape, dtype, dev)
    x1 = o1 = None
    if k is not None:
        kshape = torch.Size((batch, k.shape[1], n, dh))
        x1 = _heads(k, "k", kshape, dtype, dev)
        if k_out is None:
            k_out = _dense_like(k, stream)
        o1 = _heads(k_out, "k_out", kshape, dtype, dev)
    _check(lib().dt_rotary(table, _ints(positions, "positions", (batch, n), dev), batch, n, dh,
                           dtype, x0, o0, x1, o1, int(gradient), handle), "dt_rotary")
    return q_out if k is None else (q_out, k_out)


class PagedCache:
    """A paged key/value cache (dt_cache): k and v [pages][Hkv][page][dh] (bfloat16,
    float16, or uint8 / float8_e4m3fn codes with k_exp and v_exp [pages][Hkv][page]
    uint8), table [batch][width] int32. ``status`` [batch] int32 collects the device's
    error codes; ``check()`` reads it and raises."""

    def __init__(self, k, v, table, k_exp=None, v_exp=None, status=None):
        kinds = {torch.bfloat16: BF16, torch.float16: F16, torch.uint8: E4M3,
                 torch.float8_e4m3fn: E4M3}
        if k.dim() != 4 or k.dtype not in kinds or v.shape != k.shape or v.dtype != k.dtype or \
                not (k.is_contiguous() and v.is_contiguous()) or not k.is_cuda or \
                v.device != k.device:
            raise ValueError("k and v must be contiguous [pages][Hkv][page][dh] CUDA tensors of "
                             "one cache type")
        for e in (k_exp, v_exp):
            if (kinds[k.dtype] == E4M3) != (e is not None):
                raise ValueError("k_exp and v_exp belong to 8-bit pages, and only to them")
            if e is not None and (e.shape != k.shape[:3] or e.dtype != torch.uint8 or
                                  not e.is_contiguous() or e.device != k.device):
                raise ValueError("k_exp and v_exp must be contiguous [pages][Hkv][page] uint8 "
                                 "tensors on the pages' device")
        if table.dim() != 2:
            raise ValueError("table must be [batch][width]")
        self.k, self.v, self.table, self.k_exp, self.v_exp = k, v, table, k_exp, v_exp
        self.device, self.batch = k.device, table.shape[0]
        self._dev = k.get_device()
        _ints(table, "table", table.shape, self._dev)
        self.status = torch.zeros(self.batch, dtype=torch.int32, device=k.device) \
            if status is None else status
        _ints(self.status, "status", (self.batch,), self._dev)
        pages, self.Hkv, page, self.dh = k.shape
        self._struct = DtCache(_ptr(k), _ptr(v), _ptr(k_exp), _ptr(v_exp), _ptr(table),
                               _ptr(self.status), pages, page, self.Hkv, self.dh, kinds[k.dtype],
                               self.batch, table.shape[1])

    @classmethod
    def empty(cls, pages: int, Hkv: int, page: int, dh: int, table, dtype=torch.bfloat16):
        """A cache of unwritten pages; dtype bfloat16, float16 or float8_e4m3fn."""
        kw = dict(device=table.device)
        k, v = (torch.empty((pages, Hkv, page, dh), dtype=dtype, **kw) for _ in range(2))
        ke = ve = None
        if dtype == torch.float8_e4m3fn:
            ke, ve = (torch.empty((pages, Hkv, page), dtype=torch.uint8, **kw) for _ in range(2))
        return cls(k, v, table, ke, ve)

    def check(self):
        """Wait for the device and raise if a call met a bad page or timed out."""
        torch.cuda.synchronize(self.device)     # calls may have run on any stream
        bad = [(b, c) for b, c in enumerate(self.status.tolist()) if c != OK]
        if bad:
            raise DtError("paged cache: " + ", ".join(f"request {b}: {status_string(c)}"
                                                      for b, c in bad))


def cache_write(cache: PagedCache, k, v, first, counts=None, rotary: Rotary | None = None,
                positions=None, q=None, q_out=None, stream=None):
    """dt_cache_write: rows of k and v [batch][Hkv][n][dh] to rows first[b].. of the
    cache, k turned by ``rotary`` at ``positions``; with q, returns its turned rows."""
    shape, dtype, dev = _shape(k, "k")
    n, b = shape[2], (cache.batch,)
    if shape != (cache.batch, cache.Hkv, n, cache.dh) or dev != cache._dev:
        raise ValueError("k does not match the cache's batch, heads, head size or device")
    table, handle = _rotation(rotary, dev), _raw_stream(stream, dev)
    hk, hv = _heads(k, "k", shape, dtype, dev), _heads(v, "v", shape, dtype, dev)
    hq = ho = None
    if q is not None:
        qshape = torch.Size((cache.batch, q.shape[1], n, cache.dh))
        hq = _heads(q, "q", qshape, dtype, dev)
        if q_out is None:
            q_out = _dense_like(q, stream)
        ho = _heads(q_out, "q_out", qshape, dtype, dev)
    _check(lib().dt_cache_write(cache._struct, hk, hv, n, dtype, _ints(first, "first", b, dev),
                                _ints(counts, "counts", b, dev), table,
                                _ints(positions, "positions", (cache.batch, n), dev),
                                hq, ho, handle), "dt_cache_write")
    return q_out


def cache_read(cache: PagedCache, n: int, first, counts=None, dtype=None, k_out=None, v_out=None,
               stream=None):
    """dt_cache_read: rows first[b] .. first[b] + counts[b] - 1 as dense k and v
    [batch][Hkv][n][dh] (zeros behind them). dtype defaults to the cache's 16-bit
    type, bfloat16 for an 8-bit cache."""
    if dtype is None:
        dtype = cache.k.dtype if cache.k.dtype in _TYPE16 else torch.bfloat16
    shape, dev = torch.Size((cache.batch, cache.Hkv, n, cache.dh)), cache._dev
    handle = _raw_stream(stream, dev)
    with _made_on(stream):
        if k_out is None:
            k_out = torch.empty(shape, dtype=dtype, device=cache.device)
        if v_out is None:
            v_out = torch.empty(shape, dtype=k_out.dtype, device=cache.device)
    ctype = _shape(k_out, "k_out")[1]
    hk, hv = _heads(k_out, "k_out", shape, ctype, dev), _heads(v_out, "v_out", shape, ctype, dev)
    b = (cache.batch,)
    _check(lib().dt_cache_read(cache._struct, n, ctype, _ints(first, "first", b, dev),
                               _ints(counts, "counts", b, dev), hk, hv, handle), "dt_cache_read")
    return k_out, v_out


def cache_commit(cache: PagedCache, first, path, lengths, n: int, stream=None):
    """dt_cache_commit: cache row first[b] + path[b][j] to row first[b] + j for
    j < lengths[b], in place; ``n`` is the trees' rows."""
    b, dev, width = (cache.batch,), cache._dev, path.shape[-1]
    _check(lib().dt_cache_commit(cache._struct, _ints(first, "first", b, dev),
                                 _ints(path, "path", (cache.batch, width), dev),
                                 _ints(lengths, "lengths", b, dev), width, int(n),
                                 _raw_stream(stream, dev)), "dt_cache_commit")


def cache_attention_workspace(cache: PagedCache, H: int, n: int, stream=None):
    """A workspace for cache_attention with up to H query heads and n rows, for calls on ``stream``."""
    _raw_stream(stream, cache._dev)      # the size follows the current device's SMs
    nbytes = lib().dt_cache_attention_workspace_bytes(cache._struct, int(H), int(n))
    if nbytes == 0:
        raise DtError("dt_cache_attention_workspace_bytes failed (invalid sizes or unsupported device)")
    with _made_on(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=cache.device)


def cache_attention(cache: PagedCache, q, prefix_len, mask=None, counts=None, scale=None, out=None,
                    workspace=None, stream=None):
    """dt_cache_attention: q [batch][H][n][dh] over the cache, with the trees' mask
    [batch][n][n] uint8 or causally (mask None). ``workspace`` (of
    cache_attention_workspace) is allocated for the call when None. Returns out,
    by default a new dense tensor of q's shape and type."""
    shape, dtype, dev = _shape(q, "q")
    batch, H, n, dh = shape
    if batch != cache.batch or dh != cache.dh or dev != cache._dev:
        raise ValueError("q does not match the cache's batch, head size or device")
    handle = _raw_stream(stream, dev)
    if mask is not None and (mask.shape != (batch, n, n) or not mask.is_contiguous() or
                             mask.dtype not in (torch.uint8, torch.bool) or
                             mask.get_device() != dev):
        raise ValueError(f"mask must be a contiguous uint8 tensor of shape {(batch, n, n)}")
    hq = _heads(q, "q", shape, dtype, dev)
    if out is None:
        out = _dense_like(q, stream)
    ho = _heads(out, "out", shape, dtype, dev)
    if workspace is None:
        workspace = cache_attention_workspace(cache, H, n, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    _check(lib().dt_cache_attention(cache._struct, hq, n, dtype,
                                    _ints(prefix_len, "prefix_len", (batch,), dev),
                                    _ints(counts, "counts", (batch,), dev), _ptr(mask),
                                    dh ** -0.5 if scale is None else scale, ho, workspace.data_ptr(),
                                    workspace.numel() * workspace.element_size(), handle),
           "dt_cache_attention")
    return out


# --------------------------- page tables, norms and projections around the cache's layers

class PagePool:
    """The free pages of ``cache`` and how many entries of its table row each request holds
    (dt_page_pool): held [batch] int32, free_pages [pages] int32 (the first state[0] are free),
    state [2] int32. ``PagePool.all_free(cache)`` begins with every page free and empty tables.
    Requests' pages are their own: a page that two rows of the table name is not for this class."""

    def __init__(self, cache: PagedCache, held, free_pages, state):
        dev = cache._dev
        self.cache, self.held, self.free_pages, self.state = cache, held, free_pages, state
        pages = cache._struct.pages
        for t in (held, free_pages, state):
            if t is None:
                raise ValueError("held, free_pages and state are needed")
        self._struct = DtPagePool(_ints(held, "held", (cache.batch,), dev),
                                  _ints(free_pages, "free_pages", (pages,), dev),
                                  _ints(state, "state", (2,), dev))

    @classmethod
    def all_free(cls, cache: PagedCache):
        """A pool of nothing but free pages (taken in rising order); the cache's table is set to -1."""
        pages = cache._struct.pages
        cache.table.fill_(-1)
        free = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=cache.device)
        held = torch.zeros(cache.batch, dtype=torch.int32, device=cache.device)
        return cls(cache, held, free, torch.tensor([pages, 0], dtype=torch.int32, device=cache.device))


def cache_reserve(pool: PagePool, lengths, stream=None):
    """dt_cache_reserve: the pages for lengths[b] rows of every request ([batch] int32), taken
    from the pool or given back to it; the cache's table, ``pool.held`` and the free pages change.
    A request that the pool has too few pages for gets none, which ``cache.check()`` reports."""
    cache = pool.cache
    handle = _raw_stream(stream, cache._dev)
    if lengths is None:
        raise ValueError("lengths are needed")
    _check(lib().dt_cache_reserve(cache._struct, pool._struct,
                                  _ints(lengths, "lengths", (cache.batch,), cache._dev), handle),
           "dt_cache_reserve")


def cache_slots(cache: PagedCache, n: int, first, counts=None, slots=None, positions=None, stream=None):
    """dt_cache_slots: for rows first[b] .. first[b] + counts[b] - 1 their places in the pool
    (page * page size + row in the page, [batch][n] int64) and their positions ([batch][n] int32);
    -1 behind them. Returns (slots, positions)."""
    dev, b = cache._dev, (cache.batch,)
    handle = _raw_stream(stream, dev)
    shape = torch.Size((cache.batch, n))
    with _made_on(stream):
        if slots is None:
            slots = torch.empty(shape, dtype=torch.int64, device=cache.device)
        if positions is None:
            positions = torch.empty(shape, dtype=torch.int32, device=cache.device)
    if slots.shape != shape or slots.dtype != torch.int64 or not slots.is_contiguous() or \
            slots.get_device() != dev:
        raise ValueError(f"slots must be a contiguous int64 tensor of shape {tuple(shape)} on the cache's device")
    if first is None:
        raise ValueError("first is needed")
    _check(lib().dt_cache_slots(cache._struct, int(n), _ints(first, "first", b, dev),
                                _ints(counts, "counts", b, dev), slots.data_ptr(),
                                _ints(positions, "positions", shape, dev), handle), "dt_cache_slots")
    return slots, positions


class Rows8:
    """8-bit rows: e4m3 codes [...][d] (float8_e4m3fn or uint8, dense rows) and the exponent byte of
    each row, exps [...] uint8; a row's values are code * 2^(exps - 127), all NaN for exps 255."""

    def __init__(self, codes, exps):
        if codes.dtype not in (torch.float8_e4m3fn, torch.uint8) or codes.dim() < 2 or \
                codes.get_device() < 0 or codes.stride(-1) != 1:
            raise ValueError("codes must be a [...][d] float8_e4m3fn or uint8 CUDA tensor with a dense last "
                             "dimension")
        if exps.shape != codes.shape[:-1] or exps.dtype != torch.uint8 or not exps.is_contiguous() or \
                exps.get_device() != codes.get_device():
            raise ValueError("exps must be a contiguous uint8 tensor, one a row, on the codes' device")
        self.codes, self.exps, self.shape = codes, exps, codes.shape

    @classmethod
    def _made(cls, codes, exps):
        """Of tensors that need no check."""
        self = cls.__new__(cls)
        self.codes, self.exps, self.shape = codes, exps, codes.shape
        return self

    def values(self, dtype=torch.float32):
        """The rows' values (plain torch operations, for looking at them)."""
        e = self.exps.to(torch.int32)
        scale = torch.ldexp(torch.ones((), device=e.device), e - 127)
        x = self.codes.view(torch.float8_e4m3fn).float() * scale[..., None]
        return torch.where((e == 255)[..., None], float("nan"), x).to(dtype)


@functools.lru_cache(maxsize=4096)
def _row_layout(size, strides):
    """A [...][d] shape as rows in two outer dimensions: rows lie at one stride within the
    second-last dimension and at one across those before it. (outer, its stride, inner, its
    stride), or None."""
    if len(size) < 2 or strides[-1] != 1:
        return None
    outer, step = 1, 0
    for n, s in zip(reversed(size[:-2]), reversed(strides[:-2])):
        if n == 1:
            continue
        if outer == 1:
            step = s
        elif s != step * outer:
            return None
        outer *= n
    return outer, step, size[-2], strides[-2]


def _rows(t, what: str):
    """A 16-bit tensor of rows: its packed dt_rows, its layout."""
    layout = _row_layout(t.shape, t.stride())
    if layout is None:
        raise ValueError(f"{what} must be [...][d] with a dense last dimension and rows at two strides: one within "
                         "the second-last dimension, one across those before it")
    return _pack_rows(t.data_ptr(), layout[1], layout[3]), layout


def _same_rows(t, what: str, like, dev):
    if t.shape != like.shape or t.dtype != like.dtype or t.get_device() != dev:
        raise ValueError(f"{what} must be of x's shape, type and device")
    return _rows(t, what)[0]


def _new_rows(like, inner, d, stream):
    """A dense tensor of like's shape and type, and its packed dt_rows."""
    t = _dense_like(like, stream)
    return t, _pack_rows(t.data_ptr(), inner * d, d)


class Norm:
    """A root-mean-square norm: weight [d] (bfloat16 or float16, or None), eps, and ``offset``
    added to the weight (1 where a model stores it that way)."""

    def __init__(self, weight, eps: float = 1e-6, offset: float = 0.0):
        if weight is not None and (weight.dim() != 1 or weight.dtype not in _TYPE16 or
                                   not weight.is_contiguous() or weight.get_device() < 0):
            raise ValueError("weight must be a contiguous [d] bfloat16 or float16 CUDA tensor")
        self.weight, self.eps, self.offset = weight, float(eps), float(offset)
        self._ptr = _ptr(weight)
        if weight is not None:
            self._d, self._type, self._dev = weight.shape[0], _TYPE16[weight.dtype], weight.get_device()


def _codes_like(x, stream):
    with _made_on(stream):
        return (torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device),
                torch.empty(x.shape[:-1], dtype=torch.uint8, device=x.device))


def rms_norm(norm: Norm, x, residual=None, kind: str = "16", out=None, total=None, stream=None):
    """dt_rms_norm of the rows x [...][d], of x + residual where that is given. ``kind``: "16" (a
    tensor of x's type), "e4m3" (a Rows8), or "both" ((tensor, Rows8), from the same fp32 values).
    Returns that, and with ``residual`` also the sum: (y, total). ``total`` and ``out`` may be
    x and residual, in either order, but not the same."""
    if kind not in ("16", "e4m3", "both"):
        raise ValueError('kind must be "16", "e4m3" or "both"')
    dtype, dev, w = _TYPE16.get(x.dtype), x.get_device(), norm.weight
    if dtype is None or dev < 0:
        raise ValueError("x must be a bfloat16 or float16 CUDA tensor")
    handle = _raw_stream(stream, dev)
    vx, (outer, _, inner, _) = _rows(x, "x")
    d = x.shape[-1]
    if w is not None and (norm._d != d or norm._type != dtype or norm._dev != dev):
        raise ValueError("the norm's weight must have one value a column, of the rows' type and device")
    vr = vt = vo = codes = exps = None
    if residual is not None:
        vr = _same_rows(residual, "residual", x, dev)
        if total is None:
            total, vt = _new_rows(x, inner, d, stream)
        else:
            vt = _same_rows(total, "total", x, dev)
    elif total is not None:
        raise ValueError("total is the sum of x and residual: residual is needed")
    if kind != "e4m3":
        if out is None:
            out, vo = _new_rows(x, inner, d, stream)
        else:
            vo = _same_rows(out, "out", x, dev)
    elif out is not None:
        raise ValueError('out is for kind "16" or "both"')
    if kind != "16":
        codes, exps = _codes_like(x, stream)
    _check(lib().dt_rms_norm(vx, vr, vt, vo, _ptr(codes), _ptr(exps), norm._ptr, norm.offset, norm.eps,
                             outer, inner, d, dtype, handle), "dt_rms_norm")
    if kind == "16":
        y = out
    else:
        y = Rows8._made(codes, exps)
        if kind == "both":
            y = out, y
    return y if residual is None else (y, total)


def quantize_rows(x, stream=None):
    """dt_quantize_rows: the rows x [...][d] as a Rows8 (a weight matrix, or a projection's input
    that comes from no norm)."""
    dtype, dev = _TYPE16.get(x.dtype), x.get_device()
    if dtype is None or dev < 0:
        raise ValueError("x must be a bfloat16 or float16 CUDA tensor")
    handle = _raw_stream(stream, dev)
    vx, (outer, _, inner, _) = _rows(x, "x")
    codes, exps = _codes_like(x, stream)
    _check(lib().dt_quantize_rows(vx, codes.data_ptr(), exps.data_ptr(), outer, inner, x.shape[-1], dtype, handle),
           "dt_quantize_rows")
    return Rows8._made(codes, exps)


class Projection:
    """A shared weight matrix W [O][K]: a bfloat16 or float16 tensor, or a Rows8 for 8-bit
    projections. ``status`` collects the device's error codes of its calls; ``check()`` reads it
    and raises."""

    def __init__(self, weight):
        t, exps = (weight.codes, weight.exps) if isinstance(weight, Rows8) else (weight, None)
        if t.dim() != 2 or t.get_device() < 0 or t.stride(1) != 1 or (exps is None and t.dtype not in _TYPE16):
            raise ValueError("weight must be a [O][K] bfloat16 or float16 CUDA tensor with dense rows, or a Rows8")
        self.weight, self.O, self.K, self.device = weight, t.shape[0], t.shape[1], t.device
        self._dev, self._type = t.get_device(), E4M3 if exps is not None else _TYPE16[t.dtype]
        self.status = torch.zeros(1, dtype=torch.int32, device=t.device)
        self._struct = DtMatrix(t.data_ptr(), _ptr(exps), self.K if self.O == 1 else t.stride(0), self.O, self.K,
                                self._type)

    def check(self):
        """Wait for the device and raise if a call met a bad adapter index or timed out."""
        torch.cuda.synchronize(self.device)     # calls may have run on any stream
        code = int(self.status)
        if code != OK:
            raise DtError(f"projection: {status_string(code)}")


class Adapters:
    """Low-rank adapters of one projection: down [count][rank][K], up [count][O][rank] (bfloat16 or
    float16, dense) and scale [count] fp32 (ones when None). Adapters of lower ranks are padded
    with zeros. ``terms``: how many 16-bit terms hold scale x A^T before its product with B (dt_project);
    1 takes half the workspace and rounds it as a 16-bit tensor would be."""

    def __init__(self, down, up, scale=None, terms: int = 2):
        dev = down.get_device()
        if down.dim() != 3 or up.dim() != 3 or down.dtype not in _TYPE16 or up.dtype != down.dtype or dev < 0 or \
                up.get_device() != dev or not (down.is_contiguous() and up.is_contiguous()) or \
                up.shape[0] != down.shape[0] or up.shape[2] != down.shape[1]:
            raise ValueError("down [count][rank][K] and up [count][O][rank] must be contiguous CUDA tensors of one "
                             "16-bit type")
        if scale is not None and (scale.shape != down.shape[:1] or scale.dtype != torch.float32 or
                                  not scale.is_contiguous() or scale.get_device() != dev):
            raise ValueError("scale must be a contiguous [count] float32 tensor on the adapters' device")
        if terms not in (1, 2):
            raise ValueError("terms must be 1 or 2")
        self.down, self.up, self.scale, self.terms = down, up, scale, terms
        self.count, self.rank, self.K, self.O = down.shape[0], down.shape[1], down.shape[2], up.shape[1]
        self._dev, self._type = dev, _TYPE16[down.dtype]
        self._struct = DtAdapters(down.data_ptr(), up.data_ptr(), _ptr(scale), self.count, self.rank, terms)


def project_workspace(projection: Projection, batch: int, n: int, adapters: Adapters | None, stream=None):
    """A workspace for project with up to ``batch`` requests of n rows, for calls on ``stream`` (None
    without adapters)."""
    _raw_stream(stream, projection._dev)
    if adapters is None:
        return None
    nbytes = adapters.terms * lib().dt_project_workspace_bytes(int(batch), int(n), adapters.rank)
    if nbytes == 0:
        raise DtError("dt_project_workspace_bytes failed (invalid sizes)")
    with _made_on(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=projection.device)


def _flat_rows(t, what: str, batch: int, n: int):
    """Stride of the rows of a [batch][n][d] tensor, which lie at one."""
    s = t.stride()
    if s[2] != 1 or (batch > 1 and n > 1 and s[0] != n * s[1]):
        raise ValueError(f"{what}'s rows must be dense and lie at one stride")
    return s[1] if n > 1 else s[0] if batch > 1 else t.shape[2]      # (of a single row: none that counts)


def project(projection: Projection, x, adapters: Adapters | None = None, index=None, x16=None, dtype=None,
            out=None, workspace=None, stream=None):
    """dt_project: y [batch][n][O] = x W^T, and for requests with an adapter (index [batch] int32,
    negative: none) scale (x A^T) B^T beside it. x: [batch][n][K] of the weight's type, or a Rows8 for
    an 8-bit weight; then ``x16``, the same rows in 16 bits, is what the adapters see, and
    ``dtype`` the result's type (that of out, x16 or the adapters, or bfloat16). ``workspace`` (of
    project_workspace) is allocated for the call when None and needed."""
    p, dev = projection, projection._dev
    t, exps = (x.codes, x.exps) if isinstance(x, Rows8) else (x, None)
    if t.dim() != 3 or t.shape[2] != p.K or t.get_device() != dev or (exps is not None) != (p._type == E4M3):
        raise ValueError("x must be [batch][n][K] rows on the weight's device, a Rows8 for an 8-bit weight only")
    batch, n, K = t.shape
    handle = _raw_stream(stream, dev)
    if exps is None:
        if _TYPE16.get(t.dtype) != p._type:
            raise ValueError("x must have the weight's type")
        dtype = t.dtype
    elif dtype is None:
        dtype = out.dtype if out is not None else x16.dtype if x16 is not None else torch.bfloat16
    kind = _TYPE16.get(dtype)
    if kind is None:
        raise ValueError("dtype must be bfloat16 or float16")
    ldx16, set_struct, indexes = 0, None, _ints(index, "index", (batch,), dev)
    if adapters is not None:
        if adapters._dev != dev or adapters._type != kind or adapters.K != K or adapters.O != p.O:
            raise ValueError("the adapters must match the weight's sizes and device and the result's type")
        if index is None:
            raise ValueError("adapters need an index of each request's")
        set_struct = adapters._struct
        if exps is not None:
            if x16 is None or x16.shape != t.shape or x16.dtype != dtype or x16.get_device() != dev:
                raise ValueError("adapters beside an 8-bit weight need x16, the rows in the result's type")
            ldx16 = _flat_rows(x16, "x16", batch, n)
        if workspace is None:
            workspace = project_workspace(p, batch, n, adapters, stream)
        elif workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the weight's device")
    elif index is not None:
        raise ValueError("an index needs adapters")
    if out is None:
        with _made_on(stream):
            out = torch.empty((batch, n, p.O), dtype=dtype, device=p.device)
    elif out.shape != (batch, n, p.O) or out.dtype != dtype or out.get_device() != dev:
        raise ValueError("out must be [batch][n][O] of the result's type, on the weight's device")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().dt_project(p._struct, t.data_ptr(), _flat_rows(t, "x", batch, n), _ptr(exps), batch, n, kind,
                            set_struct, indexes, x16.data_ptr() if ldx16 else None, ldx16, out.data_ptr(),
                            _flat_rows(out, "out", batch, n), p.status.data_ptr(), _ptr(workspace), ws_bytes,
                            handle), "dt_project")
    return out
