"""Thin Python binding of libe2f (include/e2f.h) through ctypes.

Argument marshalling only: tensors are passed as raw device pointers and
the current torch CUDA stream as a cudaStream_t; every step of the path runs
in the library's kernels.  PyTorch is used for device memory and streams.

The library must have been built (``python -m atomistic_mlip_b200.build``);
loading raises if it is missing -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import os
from typing import List, Optional, Sequence

import numpy as np

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libe2f.so")
MAX_L = 6
F32, BF16, I32, I64 = 0, 1, 2, 3

STATUS = {0: "ok", 1: "invalid argument", 2: "cutoff too large", 3: "capacity",
          4: "unsupported", 5: "CUDA error", 6: "timeout", 7: "domain", 8: "scratch limit"}


class E2FError(RuntimeError):
    def __init__(self, code: int, what: str, detail: str = ""):
        super().__init__(f"{what}: {STATUS.get(code, code)} ({code}) {detail}".rstrip())
        self.code = code


class Csr(ctypes.Structure):
    _fields_ = [("row_ptr", ctypes.c_void_p), ("col_idx", ctypes.c_void_p),
                ("n_nodes", ctypes.c_int64), ("n_edges", ctypes.c_int64),
                ("box", ctypes.c_float * 3), ("r_c", ctypes.c_float)]


_P7 = ctypes.c_void_p * (MAX_L + 1)


class Weights(ctypes.Structure):
    _fields_ = [("L_max", ctypes.c_int32), ("C", ctypes.c_int32), ("H", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("Wq", _P7), ("Wk", _P7), ("Wv", _P7),
                ("W0", ctypes.c_void_p), ("Wr", _P7), ("Wi", _P7),
                ("rad_W1", ctypes.c_void_p), ("rad_W2", ctypes.c_void_p)]


class BlockWeights(ctypes.Structure):
    _fields_ = [("attn", Weights), ("hidden", ctypes.c_int32), ("gamma1", ctypes.c_void_p),
                ("gamma2", ctypes.c_void_p), ("Wa", ctypes.c_void_p), ("Wb", _P7), ("Wd", _P7)]


class Linear(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("M", ctypes.c_int64), ("K", ctypes.c_int32),
                ("N", ctypes.c_int32), ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("W", ctypes.c_void_p),
                ("ldw", ctypes.c_int64), ("bias", ctypes.c_void_p)]


# name -> (restype, argtypes); must match include/e2f.h
SIGNATURES = {
    "e2f_status_string": (ctypes.c_char_p, [ctypes.c_int32]),
    "e2f_last_cuda_error": (ctypes.c_char_p, []),
    "e2f_build_neighbors": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float,
                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                             ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(Csr),
                                             ctypes.c_void_p]),
    "e2f_build_neighbors_noalloc": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                                     ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                                     ctypes.c_int64, ctypes.POINTER(ctypes.c_int64),
                                                     ctypes.POINTER(Csr), ctypes.c_void_p]),
    "e2f_attention_forward": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(Csr),
                                               ctypes.POINTER(Weights), ctypes.c_void_p, ctypes.c_void_p]),
    "e2f_attention_backward": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(Csr),
                                                ctypes.POINTER(Weights), ctypes.c_void_p, ctypes.c_void_p,
                                                ctypes.c_void_p, ctypes.c_void_p]),
    "e2f_block_forward": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(Csr),
                                           ctypes.POINTER(BlockWeights), ctypes.c_void_p, ctypes.c_void_p]),
    "e2f_attention_forward_multifocus": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(Csr),
                                                          ctypes.POINTER(Weights), ctypes.c_int32, ctypes.c_void_p,
                                                          ctypes.c_void_p, ctypes.c_void_p]),
    "e2f_cg_num_paths": (ctypes.c_int64, [ctypes.c_int32]),
    "e2f_cg_conv_forward": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.POINTER(Csr),
                                             ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_void_p]),
    "e2f_embed_forward": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p,
                                           ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, ctypes.c_float,
                                           ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]),
    "e2f_embed_backward": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p,
                                            ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, ctypes.c_float,
                                            ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]),
    "e2f_linear_forward": (ctypes.c_int32, [ctypes.POINTER(Linear), ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                            ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p]),
    "e2f_linear_backward": (ctypes.c_int32, [ctypes.POINTER(Linear), ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                                             ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                             ctypes.c_void_p, ctypes.c_void_p]),
    "e2f_stream_status": (ctypes.c_int32, [ctypes.c_void_p]),
    "e2f_wigner_d": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p,
                                      ctypes.c_void_p]),
    "e2f_project_qkv": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(Weights),
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "e2f_kernel_launches": (ctypes.c_int64, []),
    "e2f_profile_enable": (ctypes.c_int32, [ctypes.c_int32]),
    "e2f_profile_read": (ctypes.c_int32, [ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_double)]),
    "e2f_scratch_high_water": (ctypes.c_int32, [ctypes.POINTER(ctypes.c_int64), ctypes.c_int32]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Load libe2f.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"libe2f.so not found at {_LIB_PATH}; build it with "
                              "`python -m atomistic_mlip_b200.build`")
        L = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(code: int, what: str):
    if code != 0:
        detail = ""
        if code == 5:
            detail = lib().e2f_last_cuda_error().decode()
        raise E2FError(code, what, detail)


def _torch():
    import torch
    return torch


def _stream_ptr(stream=None) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


# ----------------------------------------------------------------------------
# neighbour list
# ----------------------------------------------------------------------------
@dataclasses.dataclass
class NeighborList:
    row_ptr: "object"       # torch.int32 [N+1] cuda
    col_idx: "object"       # torch.int32 [capacity] cuda (first n_edges valid)
    n_edges: int
    box: Optional[Sequence[float]]
    r_c: float

    @property
    def n_nodes(self) -> int:
        return int(self.row_ptr.numel()) - 1

    def csr(self) -> Csr:
        c = Csr()
        c.row_ptr = self.row_ptr.data_ptr()
        c.col_idx = self.col_idx.data_ptr() if self.col_idx.numel() else None
        c.n_nodes = self.n_nodes
        c.n_edges = self.n_edges
        for k in range(3):
            c.box[k] = float(self.box[k]) if self.box is not None else 0.0
        c.r_c = self.r_c
        return c


def build_neighbors(pos, box: Optional[Sequence[float]], r_c: float, capacity: Optional[int] = None,
                    stream=None, row_ptr=None, col_idx=None) -> NeighborList:
    """CSR radius graph of `pos` (torch float32 [N, 3] on a CUDA device).

    Allocates row_ptr / col_idx with torch unless given; if col_idx is too
    small the call is repeated once with the exact size the library reports."""
    torch = _torch()
    N = int(pos.shape[0])
    dev = pos.device
    if row_ptr is None:
        row_ptr = torch.empty(N + 1, dtype=torch.int32, device=dev)
    if col_idx is None:
        cap = capacity if capacity is not None else max(1024, 128 * N)
        col_idx = torch.empty(cap, dtype=torch.int32, device=dev)
    box_arr = None
    if box is not None:
        box_arr = (ctypes.c_float * 3)(*[float(b) for b in box])
    n_e = ctypes.c_int64(0)
    s = _stream_ptr(stream)
    code = lib().e2f_build_neighbors(_ptr(pos), N, box_arr, float(r_c), _ptr(row_ptr),
                                     _ptr(col_idx) if col_idx.numel() else None, int(col_idx.numel()),
                                     ctypes.byref(n_e), None, s)
    if code == 3:
        col_idx = torch.empty(max(1, n_e.value), dtype=torch.int32, device=dev)
        code = lib().e2f_build_neighbors(_ptr(pos), N, box_arr, float(r_c), _ptr(row_ptr), _ptr(col_idx),
                                         int(col_idx.numel()), ctypes.byref(n_e), None, s)
    _check(code, "e2f_build_neighbors")
    return NeighborList(row_ptr, col_idx, int(n_e.value), None if box is None else list(box), float(r_c))


# ----------------------------------------------------------------------------
# weights
# ----------------------------------------------------------------------------
class DeviceWeights:
    """Device copies of the attention weights plus the e2f_weights struct."""

    def __init__(self, L: int, C: int, H: int, dtype: int, Wq: List, Wk: List, Wv: List, W0, Wr: List,
                 Wi: List, rad_W1, rad_W2):
        self.L, self.C, self.H, self.dtype = L, C, H, dtype
        self.tensors = dict(Wq=Wq, Wk=Wk, Wv=Wv, W0=W0, Wr=Wr, Wi=Wi, rad_W1=rad_W1, rad_W2=rad_W2)
        w = Weights()
        w.L_max, w.C, w.H, w.dtype = L, C, H, dtype
        for l in range(L + 1):
            w.Wq[l], w.Wk[l], w.Wv[l] = Wq[l].data_ptr(), Wk[l].data_ptr(), Wv[l].data_ptr()
        w.W0 = W0.data_ptr()
        for m in range(1, L + 1):
            w.Wr[m], w.Wi[m] = Wr[m].data_ptr(), Wi[m].data_ptr()
        w.rad_W1, w.rad_W2 = rad_W1.data_ptr(), rad_W2.data_ptr()
        self.struct = w

    @classmethod
    def from_workload(cls, wl, device="cuda", dtype: Optional[str] = None) -> "DeviceWeights":
        torch = _torch()
        prec = dtype or wl.precision
        td = torch.float32 if prec == "fp32" else torch.bfloat16
        code = F32 if prec == "fp32" else BF16

        def up(a, t=td):
            return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(device=device, dtype=t)

        return cls(wl.L, wl.C, wl.H, code, [up(a) for a in wl.Wq], [up(a) for a in wl.Wk],
                   [up(a) for a in wl.Wv], up(wl.W0), [None] + [up(a) for a in wl.Wr[1:]],
                   [None] + [up(a) for a in wl.Wi[1:]], up(wl.rad_W1, torch.float32),
                   up(wl.rad_W2, torch.float32))

    @property
    def torch_dtype(self):
        torch = _torch()
        return torch.float32 if self.dtype == F32 else torch.bfloat16


# ----------------------------------------------------------------------------
# attention and unit entry points
# ----------------------------------------------------------------------------
def attention_forward(x, pos, nl: NeighborList, w: DeviceWeights, out=None, stream=None):
    """o = on-the-fly equivariant attention (float32 [N, Q, C])."""
    torch = _torch()
    N = int(pos.shape[0])
    Q = (w.L + 1) ** 2
    if out is None:
        out = torch.empty((N, Q, w.C), dtype=torch.float32, device=pos.device)
    csr = nl.csr()
    code = lib().e2f_attention_forward(_ptr(x), _ptr(pos), ctypes.byref(csr), ctypes.byref(w.struct),
                                       _ptr(out), _stream_ptr(stream))
    _check(code, "e2f_attention_forward")
    return out


def attention_forward_multifocus(x, pos, nl: NeighborList, w: DeviceWeights, F: int, focus_a, out=None,
                                 stream=None):
    """Multi-focus attention: F streams with their own SO(2) stacks,
    re-weighted per edge by a softmax over the streams (float32 [N, Q, C])."""
    torch = _torch()
    N = int(pos.shape[0])
    Q = (w.L + 1) ** 2
    if out is None:
        out = torch.empty((N, Q, w.C), dtype=torch.float32, device=pos.device)
    csr = nl.csr()
    code = lib().e2f_attention_forward_multifocus(_ptr(x), _ptr(pos), ctypes.byref(csr), ctypes.byref(w.struct),
                                                  int(F), _ptr(focus_a) if focus_a is not None else None,
                                                  _ptr(out), _stream_ptr(stream))
    _check(code, "e2f_attention_forward_multifocus")
    return out


def cg_num_paths(L: int) -> int:
    """Rows of the CG-convolution weights for degree L."""
    n = int(lib().e2f_cg_num_paths(int(L)))
    if n < 0:
        raise E2FError(1, "e2f_cg_num_paths", f"L = {L} out of range")
    return n


def cg_conv_forward(x, pos, nl: NeighborList, W, L: int, out=None, stream=None):
    """Re-indexed CG convolution of x (float32 or bfloat16 [N, (L+1)^2, C])
    with the harmonics of the edge directions; W float32 [cg_num_paths(L), C].
    Returns float32 [N, (L+1)^2, C]."""
    torch = _torch()
    N, Q, C = int(x.shape[0]), int(x.shape[1]), int(x.shape[2])
    if Q != (L + 1) ** 2:
        raise ValueError(f"x has {Q} components, L = {L} needs {(L + 1) ** 2}")
    dtype = F32 if x.dtype == torch.float32 else BF16
    if out is None:
        out = torch.empty((N, Q, C), dtype=torch.float32, device=pos.device)
    csr = nl.csr()
    code = lib().e2f_cg_conv_forward(_ptr(x), dtype, _ptr(pos), ctypes.byref(csr), int(L), C, _ptr(W), _ptr(out),
                                     _stream_ptr(stream))
    _check(code, "e2f_cg_conv_forward")
    return out


class DeviceBlockWeights:
    """Device copies of one block's weights (attention + merged norms + FFN)
    and the e2f_block_weights struct."""

    def __init__(self, attn: DeviceWeights, gamma1, gamma2, Wa, Wb: List, Wd: List):
        self.attn = attn
        self.tensors = dict(gamma1=gamma1, gamma2=gamma2, Wa=Wa, Wb=Wb, Wd=Wd)
        b = BlockWeights()
        b.attn = attn.struct
        b.hidden = int(Wa.shape[0])
        b.gamma1, b.gamma2, b.Wa = gamma1.data_ptr(), gamma2.data_ptr(), Wa.data_ptr()
        for l in range(attn.L + 1):
            b.Wb[l], b.Wd[l] = Wb[l].data_ptr(), Wd[l].data_ptr()
        self.struct = b

    @classmethod
    def from_layer(cls, lw: dict, device="cuda", dtype: Optional[str] = None) -> "DeviceBlockWeights":
        """From a layer-weights dict (atomistic_mlip_b200.workloads.make_layer_weights)."""
        torch = _torch()
        prec = dtype or lw["precision"]
        td = torch.float32 if prec == "fp32" else torch.bfloat16

        def up(a, t=td):
            return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(device=device, dtype=t)

        L = lw["L"]
        attn = DeviceWeights(L, lw["C"], lw["H"], F32 if prec == "fp32" else BF16,
                             [up(a) for a in lw["Wq"]], [up(a) for a in lw["Wk"]], [up(a) for a in lw["Wv"]],
                             up(lw["W0"]), [None] + [up(a) for a in lw["Wr"][1:]],
                             [None] + [up(a) for a in lw["Wi"][1:]], up(lw["rad_W1"], torch.float32),
                             up(lw["rad_W2"], torch.float32))
        return cls(attn, up(lw["gamma1"], torch.float32), up(lw["gamma2"], torch.float32), up(lw["Wa"]),
                   [up(a) for a in lw["Wb"]], [up(a) for a in lw["Wd"]])


def block_forward(x, pos, nl: NeighborList, bw: DeviceBlockWeights, out=None, stream=None):
    """One E2Former-V2 block on the fp32 residual stream x [N, Q, C]."""
    torch = _torch()
    if out is None:
        out = torch.empty_like(x)
    csr = nl.csr()
    code = lib().e2f_block_forward(_ptr(x), _ptr(pos), ctypes.byref(csr), ctypes.byref(bw.struct), _ptr(out),
                                   _stream_ptr(stream))
    _check(code, "e2f_block_forward")
    return out


def model_forward(x, pos, nl: NeighborList, layers: List[DeviceBlockWeights], stream=None):
    """Blocks in turn; two ping-pong buffers for the residual stream."""
    torch = _torch()
    a, b = x, torch.empty_like(x)
    for i, bw in enumerate(layers):
        block_forward(a, pos, nl, bw, out=b, stream=stream)
        a, b = b, (torch.empty_like(x) if i == 0 else a)
    return a


def attention_backward(x, pos, nl: NeighborList, w: DeviceWeights, grad_out, stream=None):
    """(dL/dx, dL/dpos) for L = sum(grad_out * attention_forward(x, pos, nl, w));
    the forces of an energy are -dL/dpos."""
    torch = _torch()
    N = int(pos.shape[0])
    gx = torch.empty(grad_out.shape, dtype=torch.float32, device=pos.device)
    gp = torch.empty((N, 3), dtype=torch.float32, device=pos.device)
    csr = nl.csr()
    code = lib().e2f_attention_backward(_ptr(x), _ptr(pos), ctypes.byref(csr), ctypes.byref(w.struct),
                                        _ptr(grad_out), _ptr(gx), _ptr(gp), _stream_ptr(stream))
    _check(code, "e2f_attention_backward")
    return gx, gp


# ----------------------------------------------------------------------------
# the two ends of a model
# ----------------------------------------------------------------------------
_FLOAT, _ID = {}, {}   # tensor type -> type code of the C ABI


def _types():
    torch = _torch()
    _FLOAT.update({torch.float32: F32, torch.bfloat16: BF16})
    _ID.update({torch.int32: I32, torch.int64: I64})


def _float_code(t, what: str) -> int:
    if not _FLOAT:
        _types()
    code = _FLOAT.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} has type {t.dtype}, expected float32 or bfloat16")
    return code


def _id_code(ids) -> int:
    if not _ID:
        _types()
    code = _ID.get(ids.dtype)
    if code is None:
        raise ValueError(f"ids have type {ids.dtype}, expected int32 or int64")
    return code


def _call(fn: str, stream, tensors, *args):
    """A library call on the one CUDA device that holds the tensors (made the
    current one while the call runs) and on `stream`, or that device's current
    stream."""
    torch = _torch()
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{fn}: tensors on several devices")
    if dev < 0:
        raise ValueError(f"{fn}: tensors are not on a CUDA device")
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device_index != dev:
        raise ValueError(f"{fn}: the stream is on device {stream.device_index}, the tensors on device {dev}")
    else:
        s = stream.cuda_stream
    f = getattr(_lib or lib(), fn)
    if torch.cuda.current_device() == dev:
        code = f(*args, s)
    else:
        with torch.cuda.device(dev):
            code = f(*args, s)
    if code:
        _check(code, fn)


def _on_stream(f):
    """f(..., stream=s) with s as the current stream, so that what f allocates
    comes from that stream's memory: neither work still pending elsewhere nor a
    later allocation elsewhere can meet the kernels of the call."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        with _torch().cuda.stream(stream):
            return f(*args, stream=stream, **kw)
    return call


@_on_stream
def embed_forward(ids, table, scale: float = 1.0, Q: int = 1, out_dtype=None, out=None, *, stream=None):
    """Features [N, Q, D] whose l = 0 row is scale * table[ids] and whose other
    rows are zero (Q = 1: an embedding lookup).  ids int32 or int64 [N], -1 for
    a padded row; table float32 or bfloat16 [V, D]; out_dtype float32 unless
    given.  An id outside the table gives zeros and is reported by
    stream_status()."""
    torch = _torch()
    if ids.dim() != 1 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous vector")
    if table.dim() != 2 or not table.is_contiguous():
        raise ValueError("table must be contiguous [V, D]")
    N, (V, D) = ids.shape[0], table.shape
    it, tt = _id_code(ids), _float_code(table, "table")
    if out is None:
        out = torch.empty(N, Q, D, dtype=out_dtype or torch.float32, device=table.device)
    elif out.shape != (N, Q, D) or not out.is_contiguous() or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError(f"out must be contiguous {(N, Q, D)}, of out_dtype if that is given")
    _call("e2f_embed_forward", stream, (ids, table, out), ids.data_ptr(), it, N, table.data_ptr(), tt, V, D, scale, Q,
          out.data_ptr(), _float_code(out, "out"))
    return out


@_on_stream
def embed_backward(ids, grad_out, V: int, scale: float = 1.0, grad_table=None, accumulate: bool = False, *, stream=None):
    """Gradient float32 [V, D] of embed_forward's table: scale * the sum of the
    l = 0 rows of grad_out (float32 or bfloat16 [N, Q, D] or [N, D]) over the
    rows of each id.  With accumulate the sums are added to grad_table.  Sums
    in a fixed order: the result repeats bit for bit."""
    torch = _torch()
    if ids.dim() != 1 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous vector")
    if grad_out.dim() not in (2, 3) or not grad_out.is_contiguous() or grad_out.shape[0] != ids.shape[0]:
        raise ValueError("grad_out must be contiguous [N, Q, D] or [N, D], N the number of ids")
    N, D = ids.shape[0], grad_out.shape[-1]
    Q = grad_out.shape[1] if grad_out.dim() == 3 else 1
    it, gt = _id_code(ids), _float_code(grad_out, "grad_out")
    if grad_table is None:
        if accumulate:
            raise ValueError("accumulate needs grad_table")
        grad_table = torch.empty(V, D, dtype=torch.float32, device=grad_out.device)
    elif grad_table.shape != (V, D) or not grad_table.is_contiguous() or grad_table.dtype != torch.float32:
        raise ValueError(f"grad_table must be contiguous float32 {(V, D)}")
    _call("e2f_embed_backward", stream, (ids, grad_out, grad_table), ids.data_ptr(), it, N, grad_out.data_ptr(), gt, V,
          D, scale, Q, grad_table.data_ptr(), 1 if accumulate else 0)
    return grad_table


ACT = {"none": 0, "silu": 1, "gelu": 2}


def _ld(t, rows: int, cols: int, what: str) -> int:
    """Row stride of a 2-D tensor whose rows are contiguous."""
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {(rows, cols)}")
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"the rows of {what} are not contiguous")
    if rows <= 1:
        return cols
    if s0 < cols:
        raise ValueError(f"the rows of {what} overlap")
    return s0


def _linear_struct(x, W, bias, act: str):
    if x.dim() != 2 or W.dim() != 2:
        raise ValueError("x and W must be [M, K] and [N, K]")
    M, (N, K) = x.shape[0], W.shape
    code = _float_code(x, "x")
    if W.dtype != x.dtype:
        raise ValueError(f"W has type {W.dtype}, x {x.dtype}")
    if act not in ACT:
        raise ValueError(f"act must be one of {sorted(ACT)}")
    bp = None
    if bias is not None:
        if bias.dtype != _torch().float32 or bias.shape != (N,) or not bias.is_contiguous():
            raise ValueError(f"bias must be contiguous float32 [{N}]")
        bp = bias.data_ptr()
    return Linear(code, ACT[act], M, K, N, x.data_ptr(), _ld(x, M, K, "x"), W.data_ptr(), _ld(W, N, K, "W"), bp), M, K, N


@_on_stream
def linear_forward(x, W, bias=None, residual=None, act: str = "none", out=None, out_dtype=None, *, stream=None):
    """act(x W^T + bias) + residual [M, N].  x [M, K] and W [N, K] float32 or
    bfloat16 with any row stride (x may be features[:, 0] of [M, Q, K]), bias
    float32 [N], act "none", "silu" or "gelu"; residual has the output's type
    (x's unless given by out_dtype or out) and may be out itself."""
    p, M, K, N = _linear_struct(x, W, bias, act)
    if out is None:
        out = x.new_empty(M, N) if out_dtype is None else _torch().empty(M, N, dtype=out_dtype, device=x.device)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out has another type than out_dtype")
    ldo, ldr = _ld(out, M, N, "out"), N
    if residual is not None:
        ldr = _ld(residual, M, N, "residual")
        if residual.dtype != out.dtype:
            raise ValueError(f"residual has type {residual.dtype}, the output {out.dtype}")
    _call("e2f_linear_forward", stream, (x, W, bias, residual, out), ctypes.byref(p), _ptr(residual), ldr,
          out.data_ptr(), ldo, _float_code(out, "out"))
    return out


@_on_stream
def linear_backward(x, W, grad_out, bias=None, act: str = "none", need_x: bool = True, need_W: bool = True,
                    need_bias: Optional[bool] = None, grad_x=None, grad_W=None, *, stream=None):
    """(grad_x, grad_W, grad_bias) of sum(grad_out * linear_forward(x, W, bias,
    act=act)): the first two in x's type, grad_bias float32; None where not
    needed (grad_bias: needed if there is a bias, unless told).  grad_x and
    grad_W may be given, with any row stride.  The residual's gradient is
    grad_out itself."""
    torch = _torch()
    p, M, K, N = _linear_struct(x, W, bias, act)
    ldg = _ld(grad_out, M, N, "grad_out")
    if need_bias is None:
        need_bias = bias is not None
    gb = torch.empty(N, dtype=torch.float32, device=x.device) if need_bias else None
    ldgx = ldgw = K
    if grad_x is not None:
        ldgx = _ld(grad_x, M, K, "grad_x")
        if grad_x.dtype != x.dtype:
            raise ValueError(f"grad_x has type {grad_x.dtype}, x {x.dtype}")
    elif need_x:
        grad_x = x.new_empty(M, K)
    if grad_W is not None:
        ldgw = _ld(grad_W, N, K, "grad_W")
        if grad_W.dtype != x.dtype:
            raise ValueError(f"grad_W has type {grad_W.dtype}, x {x.dtype}")
    elif need_W:
        grad_W = x.new_empty(N, K)
    _call("e2f_linear_backward", stream, (x, W, bias, grad_out, grad_x, grad_W), ctypes.byref(p), grad_out.data_ptr(),
          ldg, _float_code(grad_out, "grad_out"), _ptr(grad_x), ldgx, _ptr(grad_W), ldgw, _ptr(gb))
    return grad_x, grad_W, gb


class DeviceReadout:
    """Readout of per-atom energies from the invariant features, float32 on the
    device: e_n = W2 SiLU(W1 x[n, (0, 0)] + b1) + b2, W1 [Hr, C], b1 [Hr],
    W2 [1, Hr], b2 [1]."""

    def __init__(self, W1, b1, W2, b2):
        self.W1, self.b1, self.W2, self.b2 = W1, b1, W2, b2


@_on_stream
def readout_forward(x, head: DeviceReadout, *, stream=None):
    """(per-atom energies [N, 1], hidden features [N, Hr]) of the residual
    stream or attention output x (float32 [N, Q, C])."""
    h = linear_forward(x[:, 0], head.W1, bias=head.b1, act="silu", stream=stream)
    return linear_forward(h, head.W2, bias=head.b2, stream=stream), h


@_on_stream
def readout_backward(x, h, grad_e, head: DeviceReadout, *, stream=None):
    """Gradients of sum(grad_e * e): (dL/dx [N, Q, C], zero for l > 0, and a
    dict of those of W1, b1, W2, b2); h from readout_forward."""
    torch = _torch()
    gh, gW2, gb2 = linear_backward(h, head.W2, grad_e, bias=head.b2, stream=stream)
    gx = torch.zeros_like(x)
    _, gW1, gb1 = linear_backward(x[:, 0], head.W1, gh, bias=head.b1, act="silu", grad_x=gx[:, 0], stream=stream)
    return gx, dict(W1=gW1, b1=gb1, W2=gW2, b2=gb2)


@_on_stream
def structure_sum(values, structure, n_structures: int, *, stream=None):
    """Sums [n_structures] of per-atom values [N, 1] by the structure index of
    every atom (-1: the atom takes no part)."""
    return embed_backward(structure, values, n_structures, stream=stream)[:, 0]


@_on_stream
def model_energy(species, pos, nl: NeighborList, table, layers: List[DeviceBlockWeights], head: DeviceReadout, structure,
                 n_structures: int, scale: float = 1.0, *, stream=None):
    """Energies [n_structures] from species: scaled embedding -> blocks ->
    readout -> sum over the atoms of each structure.  table float32 [V, C]."""
    Q = (layers[0].attn.L + 1) ** 2
    x = embed_forward(species, table, scale=scale, Q=Q, stream=stream)
    e, _ = readout_forward(model_forward(x, pos, nl, layers, stream=stream), head, stream=stream)
    return structure_sum(e, structure, n_structures, stream=stream)


@_on_stream
def attention_energy_forces(species, pos, nl: NeighborList, table, w: DeviceWeights, head: DeviceReadout, structure,
                            n_structures: int, scale: float = 1.0, grad_energy=None, *, stream=None):
    """Energies, conservative forces and training gradients of the model
    species -> scaled embedding -> attention -> readout -> structure sums.

    Returns (energies [n_structures], forces [N, 3], gradients: "table", "W1",
    "b1", "W2", "b2"); the last two are those of sum(grad_energy * energies)
    (grad_energy float32 [n_structures], ones unless given)."""
    torch = _torch()
    x = embed_forward(species, table, scale=scale, Q=(w.L + 1) ** 2, out_dtype=w.torch_dtype, stream=stream)
    o = attention_forward(x, pos, nl, w, stream=stream)
    e, h = readout_forward(o, head, stream=stream)
    energies = structure_sum(e, structure, n_structures, stream=stream)
    gE = torch.ones_like(energies) if grad_energy is None else grad_energy
    ge = embed_forward(structure, gE.view(n_structures, 1), stream=stream)[:, :, 0]   # every atom its structure's
    go, grads = readout_backward(o, h, ge, head, stream=stream)
    gx, gp = attention_backward(x, pos, nl, w, go, stream=stream)
    grads["table"] = embed_backward(species, gx, table.shape[0], scale=scale, stream=stream)
    return energies, gp.neg_(), grads


def project_qkv(x, w: DeviceWeights, stream=None):
    torch = _torch()
    q, k, v = (torch.empty_like(x) for _ in range(3))
    code = lib().e2f_project_qkv(_ptr(x), int(x.shape[0]), ctypes.byref(w.struct), _ptr(q), _ptr(k), _ptr(v),
                                 _stream_ptr(stream))
    _check(code, "e2f_project_qkv")
    return q, k, v


def wigner_size(L: int) -> int:
    return sum((2 * l + 1) ** 2 for l in range(L + 1))


def wigner_d(R, L: int, stream=None):
    """Real Wigner-D blocks for rotations R (float32 [n, 3, 3] cuda) -> [n, S]."""
    torch = _torch()
    n = int(R.shape[0])
    D = torch.empty((n, wigner_size(L)), dtype=torch.float32, device=R.device)
    _check(lib().e2f_wigner_d(_ptr(R), n, L, _ptr(D), _stream_ptr(stream)), "e2f_wigner_d")
    return D


def stream_status(stream=None) -> int:
    return int(lib().e2f_stream_status(_stream_ptr(stream)))


def kernel_launches() -> int:
    return int(lib().e2f_kernel_launches())


def profile_enable(on: bool = True):
    _check(lib().e2f_profile_enable(1 if on else 0), "e2f_profile_enable")


def profile_read():
    n = ctypes.c_int64(0)
    ms = ctypes.c_double(0.0)
    _check(lib().e2f_profile_read(ctypes.byref(n), ctypes.byref(ms)), "e2f_profile_read")
    return int(n.value), float(ms.value)


def scratch_high_water(reset: bool = False) -> int:
    b = ctypes.c_int64(0)
    _check(lib().e2f_scratch_high_water(ctypes.byref(b), 1 if reset else 0), "e2f_scratch_high_water")
    return int(b.value)
