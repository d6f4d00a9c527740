"""Python binding of libdion: one Dion / Orth-Dion optimizer step on an
MI355X (gfx950), through the C ABI of include/dion.h.

This module only marshals arguments (ctypes): torch tensors supply device
memory and the current HIP stream, and every part of the step runs in
libdion's HIP kernels.  There is no CPU or PyTorch fallback: calls raise
when the built library is missing.

    import rank_orthonormalized_optimizer_dion_amd as dion
    ws = dion.step(X, G, R, V, eta=0.01, beta=0.95, variant="orth")
    dion.check_status(ws, 1)        # optional: waits, raises on breakdown

Work is enqueued on ``stream`` (a torch stream; default: the current one) and
is ordered behind that stream's earlier work only: tensors that another stream
writes have to be waited for there (``stream.wait_stream``).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import List, Optional, Sequence, Tuple

__all__ = [
    "DionError", "Breakdown", "Plan", "load", "library_path", "workspace_size",
    "workspace_size_batched", "step", "step_batched", "step_noalloc", "status",
    "check_status", "version", "VARIANTS", "NS_COEFFS", "orthogonalize", "orthogonalize_batched",
    "muon_step", "muon_step_batched", "linear_forward", "linear_backward", "ACTS",
]

OK = 0
ERR_INVALID_ARG = -1
ERR_WORKSPACE = -2
ERR_HIP = -3
ERR_BREAKDOWN = -4

VARIANTS = {"dion": 0, "orth": 1}
MATH = {"f32": 0x000, "bf16x3": 0x100}
SHARDED = 0x200
GRAM_F64 = 0x400   # OR into math: float64 MFMA Gram matrix instead of sliced int8
SCHED_GROUPED = 0x800   # OR into math: small matrices through the grouped schedule too
SHARD_GRAM, SHARD_W = 0, 1
BUF_W, BUF_P, BUF_U = 1, 2, 3   # dion_plan_buffer: intermediate factors of the last step
STATUS_ORTH_P, STATUS_ORTH_W, STATUS_COLNORM = 1, 2, 4
STATUS_NONFINITE = 8   # orthogonalize, muon_step: non-finite input
MATH_NS = {"f32": 0x0000, "f16": 0x1000}   # orthogonalize, muon_step
ACTS = {"none": 0, "relu": 1, "relu2": 2, "gelu": 3, "silu": 4}   # linear_forward / _backward
# the quintic Newton-Schulz coefficients in common use
NS_COEFFS = (3.4445, -4.7750, 2.0315)

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB: Optional[ctypes.CDLL] = None


def library_path() -> str:
    return os.environ.get("LIBDION_PATH", os.path.join(_HERE, "libdion.so"))


class DionError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libdion error {code}: {msg}")
        self.code = code


class Breakdown(DionError):
    """The step hit a numerical breakdown; X, R, V were left unchanged."""

    def __init__(self, code: int, msg: str, per_matrix: List[int]):
        super().__init__(code, msg)
        self.per_matrix = per_matrix


class dion_matrix(ctypes.Structure):
    _fields_ = [("X", ctypes.c_void_p), ("G", ctypes.c_void_p), ("R", ctypes.c_void_p),
                ("V", ctypes.c_void_p), ("m", ctypes.c_int64), ("n", ctypes.c_int64),
                ("r", ctypes.c_int64)]


class dion_ns_matrix(ctypes.Structure):
    _fields_ = [("G", ctypes.c_void_p), ("O", ctypes.c_void_p), ("m", ctypes.c_int64),
                ("n", ctypes.c_int64), ("ldg", ctypes.c_int64), ("ldo", ctypes.c_int64)]


class dion_muon_matrix(ctypes.Structure):
    _fields_ = [("X", ctypes.c_void_p), ("G", ctypes.c_void_p), ("M", ctypes.c_void_p),
                ("m", ctypes.c_int64), ("n", ctypes.c_int64), ("scale", ctypes.c_float)]


class dion_linear(ctypes.Structure):
    _fields_ = [("t", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("w", ctypes.c_void_p), ("ldw", ctypes.c_int64),
                ("bias", ctypes.c_void_p),
                ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
                ("z", ctypes.c_void_p), ("ldz", ctypes.c_int64),
                ("dy", ctypes.c_void_p), ("lddy", ctypes.c_int64),
                ("dx", ctypes.c_void_p), ("lddx", ctypes.c_int64),
                ("dw", ctypes.c_void_p), ("lddw", ctypes.c_int64),
                ("db", ctypes.c_void_p),
                ("act", ctypes.c_int), ("dtype", ctypes.c_int), ("accumulate", ctypes.c_int)]


def load() -> ctypes.CDLL:
    """Load libdion.so (built by ``build.py``); raises if it is missing."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(
            f"libdion is not built ({path} missing); run "
            "`python -m rank_orthonormalized_optimizer_dion_amd.build`")
    lib = ctypes.CDLL(path)
    c_size, c_int, c_i64, c_f, vp = (ctypes.c_size_t, ctypes.c_int, ctypes.c_int64,
                                     ctypes.c_float, ctypes.c_void_p)
    mats_p = ctypes.POINTER(dion_matrix)
    ns_p, muon_p, f_p = (ctypes.POINTER(dion_ns_matrix), ctypes.POINTER(dion_muon_matrix),
                         ctypes.POINTER(ctypes.c_float))
    lin_p = ctypes.POINTER(dion_linear)
    sig = {
        "dion_version": (c_int, []),
        "dion_error_string": (ctypes.c_char_p, [c_int]),
        "dion_workspace_size": (c_size, [c_i64, c_i64, c_i64, c_int, c_int]),
        "dion_step": (c_int, [vp, vp, vp, vp, c_i64, c_i64, c_i64, c_f, c_f, c_int, c_int,
                              vp, c_size, vp]),
        "dion_workspace_size_batched": (c_size, [mats_p, c_int, c_int, c_int]),
        "dion_step_batched": (c_int, [mats_p, c_int, c_f, c_f, c_int, c_int, vp, c_size, vp]),
        "dion_plan_create": (c_int, [mats_p, c_int, c_int, c_int, ctypes.POINTER(vp)]),
        "dion_plan_workspace_size": (c_size, [vp]),
        "dion_plan_count": (c_int, [vp]),
        "dion_plan_step": (c_int, [vp, c_f, c_f, vp, c_size, vp]),
        "dion_plan_destroy": (None, [vp]),
        "dion_status": (c_int, [vp, c_int, vp, ctypes.POINTER(c_int)]),
        "dion_plan_timing_enable": (c_int, [vp, c_int]),
        "dion_plan_timing_read": (c_int, [vp, ctypes.POINTER(ctypes.c_double),
                                          ctypes.POINTER(c_int)]),
        "dion_plan_shard_stage": (c_int, [vp, c_int, c_f, c_f, vp, c_size, vp]),
        "dion_plan_shard_buffer": (c_int, [vp, c_int, c_int, ctypes.POINTER(c_size),
                                           ctypes.POINTER(c_size)]),
        "dion_plan_buffer": (c_int, [vp, c_int, c_int, ctypes.POINTER(c_size),
                                     ctypes.POINTER(c_size)]),
        "dion_step_noalloc": (c_int, [vp, vp, vp, vp, c_i64, c_i64, c_i64, c_f, c_f, c_int,
                                      c_int, vp, vp]),
        "dion_orthogonalize_workspace_size": (c_size, [ns_p, c_int, c_int]),
        "dion_orthogonalize_batched": (c_int, [ns_p, c_int, f_p, c_int, c_int, c_int, c_int, vp,
                                               c_size, vp]),
        "dion_orthogonalize": (c_int, [vp, c_i64, vp, c_i64, c_i64, c_i64, f_p, c_int, c_int, c_int,
                                       c_int, vp, c_size, vp]),
        "dion_muon_workspace_size": (c_size, [muon_p, c_int, c_int]),
        "dion_muon_step_batched": (c_int, [muon_p, c_int, c_f, c_f, c_int, c_f, f_p, c_int, c_int,
                                           c_int, vp, c_size, vp]),
        "dion_muon_step": (c_int, [vp, vp, vp, c_i64, c_i64, c_f, c_f, c_f, c_int, c_f, f_p, c_int,
                                   c_int, c_int, vp, c_size, vp]),
        "dion_linear_forward_workspace_size": (c_size, [lin_p]),
        "dion_linear_forward": (c_int, [lin_p, vp, c_size, vp]),
        "dion_linear_backward_workspace_size": (c_size, [lin_p]),
        "dion_linear_backward": (c_int, [lin_p, vp, c_size, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = lib
    return lib


def version() -> int:
    return load().dion_version()


def _err(code: int) -> DionError:
    msg = load().dion_error_string(code).decode()
    return DionError(code, msg)


def _variant(v, math="f32") -> int:
    """Rule (``"dion"`` / ``"orth"`` or its code) OR-ed with the math mode
    (``"f32"``: float32 MFMA products; ``"bf16x3"``: split-bfloat16)."""
    if isinstance(v, str):
        if v not in VARIANTS:
            raise ValueError(f"variant must be one of {list(VARIANTS)}")
        v = VARIANTS[v]
    if isinstance(math, str):
        if math not in MATH:
            raise ValueError(f"math must be one of {list(MATH)}")
        math = MATH[math]
    return int(v) | int(math)


def _torch():
    import torch
    return torch


def _gdtype(G) -> int:
    torch = _torch()
    if G.dtype == torch.float32:
        return 0
    if G.dtype == torch.bfloat16:
        return 1
    raise TypeError("G must be float32 or bfloat16")


def _stream_handle(stream, device) -> int:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return int(stream.cuda_stream)


def _check(X, G, R, V):
    torch = _torch()
    for name, t in (("X", X), ("G", G), ("R", R), ("V", V)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous (row-major)")
        if t.dim() != 2:
            raise ValueError(f"{name} must be 2-D")
    for name, t in (("X", X), ("R", R), ("V", V)):
        if t.dtype != torch.float32:
            raise TypeError(f"{name} must be float32")
    m, n = X.shape
    if tuple(G.shape) != (m, n) or tuple(R.shape) != (m, n) or V.shape[0] != n:
        raise ValueError("shape mismatch: X, G, R are m x n and V is n x r")
    return m, n, V.shape[1]


def workspace_size(m: int, n: int, r: int, variant="orth", g_dtype=None, math="f32") -> int:
    torch = _torch()
    gd = 1 if g_dtype == torch.bfloat16 else 0
    size = load().dion_workspace_size(m, n, r, _variant(variant, math), gd)
    if size == 0:
        raise ValueError("invalid shape or rank")
    return int(size)


def _new_workspace(nbytes: int, device, stream):
    """nbytes from the memory of the stream that will use them: memory of
    another stream's pool may be in use by work that is still pending there,
    and nothing would order that before this use."""
    torch = _torch()
    with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _workspace(nbytes: int, device, workspace, stream=None):
    if workspace is None:
        return _new_workspace(nbytes, device, stream)
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"workspace too small: need {nbytes} bytes")
    return workspace


def step(X, G, R, V, eta: float, beta: float, variant="orth", workspace=None, stream=None,
         math="f32"):
    """One step on one matrix, enqueued on `stream` (default: current).

    X, R, V (float32) are updated in place; G (float32 or bfloat16) is read.
    Returns the workspace tensor (pass it back to reuse it, or to
    ``status``)."""
    m, n, r = _check(X, G, R, V)
    lib = load()
    gd, var = _gdtype(G), _variant(variant, math)
    nbytes = lib.dion_workspace_size(m, n, r, var, gd)
    if nbytes == 0:
        raise _err(ERR_INVALID_ARG)
    ws = _workspace(nbytes, X.device, workspace, stream)
    rc = lib.dion_step(X.data_ptr(), G.data_ptr(), R.data_ptr(), V.data_ptr(), m, n, r,
                       float(eta), float(beta), var, gd, ws.data_ptr(), nbytes,
                       _stream_handle(stream, X.device))
    if rc != OK:
        raise _err(rc)
    return ws


def step_noalloc(X, G, R, V, eta: float, beta: float, variant="orth", status_out=None,
                 stream=None, math="f32"):
    """One step on one matrix with the library's own scratch (no workspace
    argument; dion_step_noalloc).  status_out: optional int32 GPU tensor of
    one element that receives the matrix's status word."""
    m, n, r = _check(X, G, R, V)
    lib = load()
    if status_out is not None and (not status_out.is_cuda or status_out.numel() < 1 or
                                   status_out.dtype != _torch().int32):
        raise ValueError("status_out must be an int32 GPU tensor")
    rc = lib.dion_step_noalloc(X.data_ptr(), G.data_ptr(), R.data_ptr(), V.data_ptr(), m, n, r,
                               float(eta), float(beta), _variant(variant, math), _gdtype(G),
                               status_out.data_ptr() if status_out is not None else None,
                               _stream_handle(stream, X.device))
    if rc != OK:
        raise _err(rc)


def _mat_array(mats: Sequence[Tuple]) -> Tuple[ctypes.Array, int]:
    if len(mats) == 0:
        raise ValueError("empty matrix list")
    gd = None
    arr = (dion_matrix * len(mats))()
    for i, (X, G, R, V) in enumerate(mats):
        m, n, r = _check(X, G, R, V)
        g = _gdtype(G)
        if gd is None:
            gd = g
        elif g != gd:
            raise TypeError("every G of a grouped step must have the same dtype")
        arr[i] = dion_matrix(X.data_ptr(), G.data_ptr(), R.data_ptr(), V.data_ptr(), m, n, r)
    return arr, gd


def workspace_size_batched(mats: Sequence[Tuple], variant="orth", math="f32") -> int:
    arr, gd = _mat_array(mats)
    size = load().dion_workspace_size_batched(arr, len(mats), _variant(variant, math), gd)
    if size == 0:
        raise _err(ERR_INVALID_ARG)
    return int(size)


def step_batched(mats: Sequence[Tuple], eta: float, beta: float, variant="orth",
                 workspace=None, stream=None, math="f32"):
    """Grouped step over a list of (X, G, R, V) tuples; returns the workspace."""
    arr, gd = _mat_array(mats)
    lib = load()
    var = _variant(variant, math)
    nbytes = lib.dion_workspace_size_batched(arr, len(mats), var, gd)
    if nbytes == 0:
        raise _err(ERR_INVALID_ARG)
    dev = mats[0][0].device
    ws = _workspace(nbytes, dev, workspace, stream)
    rc = lib.dion_step_batched(arr, len(mats), float(eta), float(beta), var, gd,
                               ws.data_ptr(), nbytes, _stream_handle(stream, dev))
    if rc != OK:
        raise _err(rc)
    return ws


class Plan:
    """A grouped step over a fixed list of matrices (dion_plan_*)."""

    def __init__(self, mats: Sequence[Tuple], variant="orth", math="f32", sharded=False):
        """sharded: the matrices are row shards of global matrices, stepped
        with dion_plan_shard_stage / shard_buffer (see include/dion.h)."""
        arr, gd = _mat_array(mats)
        self._lib = load()
        self._mats = list(mats)          # keep the tensors alive
        self.count = len(mats)
        self.device = mats[0][0].device
        h = ctypes.c_void_p()
        var = _variant(variant, math) | (SHARDED if sharded else 0)
        rc = self._lib.dion_plan_create(arr, self.count, var, gd, ctypes.byref(h))
        if rc != OK:
            raise _err(rc)
        self._h = h
        self.workspace_bytes = int(self._lib.dion_plan_workspace_size(h))

    def new_workspace(self, stream=None):
        """stream: the one that will run the steps, where it is not the
        current one."""
        return _workspace(self.workspace_bytes, self.device, None, stream)

    def step(self, eta: float, beta: float, workspace, stream=None):
        if self._h is None:
            raise RuntimeError("plan is closed")
        if workspace.numel() * workspace.element_size() < self.workspace_bytes:
            raise ValueError("workspace too small")
        rc = self._lib.dion_plan_step(self._h, float(eta), float(beta), workspace.data_ptr(),
                                      self.workspace_bytes, _stream_handle(stream, self.device))
        if rc != OK:
            raise _err(rc)

    def shard_stage(self, stage: int, eta: float, beta: float, workspace, stream=None):
        """Stage 0, 1 or 2 of a sharded step (dion_plan_shard_stage)."""
        if self._h is None:
            raise RuntimeError("plan is closed")
        if workspace.numel() * workspace.element_size() < self.workspace_bytes:
            raise ValueError("workspace too small")
        rc = self._lib.dion_plan_shard_stage(self._h, int(stage), float(eta), float(beta),
                                             workspace.data_ptr(), self.workspace_bytes,
                                             _stream_handle(stream, self.device))
        if rc != OK:
            raise _err(rc)

    def shard_buffer(self, workspace, which: int, index: int):
        """The exchange buffer `which` (SHARD_GRAM: float64 rp x rp; SHARD_W:
        float32 n x r) of matrix `index`, as a view into `workspace`."""
        torch = _torch()
        off, nbytes = ctypes.c_size_t(), ctypes.c_size_t()
        rc = self._lib.dion_plan_shard_buffer(self._h, int(which), int(index), ctypes.byref(off),
                                              ctypes.byref(nbytes))
        if rc != OK:
            raise _err(rc)
        raw = workspace.view(torch.uint8)[off.value:off.value + nbytes.value]
        if which == SHARD_GRAM:
            rp = int(round((nbytes.value // 8) ** 0.5))
            return raw.view(torch.float64).view(rp, rp)
        n, r = self._mats[index][3].shape
        return raw.view(torch.float32).view(n, r)

    def buffer(self, workspace, which: int, index: int):
        """Intermediate factor `which` (BUF_P: P = M V, BUF_U: U = orth(P),
        both m x r; BUF_W: W = M^T U, n x r; float32) of matrix `index` after
        the last step on `workspace`, as a view into it
        (dion_plan_buffer)."""
        torch = _torch()
        off, nbytes = ctypes.c_size_t(), ctypes.c_size_t()
        rc = self._lib.dion_plan_buffer(self._h, int(which), int(index), ctypes.byref(off),
                                        ctypes.byref(nbytes))
        if rc != OK:
            raise _err(rc)
        raw = workspace.view(torch.uint8)[off.value:off.value + nbytes.value]
        X, V = self._mats[index][0], self._mats[index][3]
        rows = V.shape[0] if which == BUF_W else X.shape[0]
        return raw.view(torch.float32).view(rows, V.shape[1])

    PHASES = ("mv", "orth_p", "mtu", "right", "update")

    def timing_enable(self, max_steps: int) -> None:
        """Record per-phase HIP events on the next `max_steps` steps."""
        rc = self._lib.dion_plan_timing_enable(self._h, int(max_steps))
        if rc != OK:
            raise _err(rc)

    def timing_read(self):
        """Wait for the recorded steps; return ({phase: summed ms}, steps)."""
        ms = (ctypes.c_double * len(self.PHASES))()
        steps = ctypes.c_int()
        rc = self._lib.dion_plan_timing_read(self._h, ms, ctypes.byref(steps))
        if rc != OK:
            raise _err(rc)
        return dict(zip(self.PHASES, list(ms))), steps.value

    def close(self):
        if getattr(self, "_h", None) is not None:
            self._lib.dion_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def status(workspace, count: int, stream=None) -> Tuple[int, List[int]]:
    """Wait for `stream`; return (code, per-matrix DION_STATUS_* flags)."""
    lib = load()
    per = (ctypes.c_int * count)()
    rc = lib.dion_status(workspace.data_ptr(), count,
                         _stream_handle(stream, workspace.device), per)
    if rc not in (OK, ERR_BREAKDOWN):
        raise _err(rc)
    return rc, list(per)


def check_status(workspace, count: int, stream=None) -> None:
    """Raise Breakdown if the last step on `workspace` broke down."""
    rc, per = status(workspace, count, stream)
    if rc == ERR_BREAKDOWN:
        raise Breakdown(rc, load().dion_error_string(rc).decode(), per)



# --- Newton-Schulz orthogonalization and the Muon step ---------------------

def _ns_coeffs(coeffs, steps: int):
    """One (a, b, c) for every iteration, or a list of `steps` of them."""
    rows = list(coeffs)
    if len(rows) == 3 and all(isinstance(v, (int, float)) for v in rows):
        rows = [tuple(rows)] * int(steps)
    if len(rows) != int(steps) or any(len(r) != 3 for r in rows):
        raise ValueError("coeffs must be (a, b, c) or one (a, b, c) per iteration")
    flat = [float(v) for r in rows for v in r]
    return (ctypes.c_float * max(len(flat), 1))(*flat)


def _ns_math(math) -> int:
    if isinstance(math, str):
        if math not in MATH_NS:
            raise ValueError(f"math must be one of {list(MATH_NS)}")
        math = MATH_NS[math]
    return int(math)


def _check_rows(name, t, shape=None, dtypes=None, device=None):
    """A 2-D GPU tensor whose rows are contiguous; returns its row pitch."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    got = t.shape
    if len(got) != 2:
        raise ValueError(f"{name} must be 2-D")
    if shape is not None and got != shape:
        raise ValueError(f"shape mismatch: {name} is {tuple(got)}, expected {tuple(shape)}")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {[str(d) for d in dtypes]}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    m, n = got
    row, col = t.stride()
    if n > 1 and col != 1:
        raise ValueError(f"{name} must have contiguous rows")
    pitch = row if m > 1 else n
    if pitch < n:
        raise ValueError(f"{name} must have rows that do not overlap")
    return pitch


def _launch(size, run, device, workspace, stream):
    """run(pointer, bytes, stream) on `device` with the caller's workspace, or
    with a new one of size() bytes; returns the workspace."""
    torch = _torch()
    if workspace is None:
        nbytes = size()
        if nbytes == 0:
            raise _err(ERR_INVALID_ARG)
        workspace = _new_workspace(nbytes, device, stream)
    else:
        if workspace.device != device:
            raise ValueError(f"workspace is on {workspace.device}, expected {device}")
        nbytes = workspace.numel() * workspace.element_size()
    args = (workspace.data_ptr(), nbytes, _stream_handle(stream, device))
    if torch.cuda.current_device() == device.index:
        rc = run(*args)
    else:
        with torch.cuda.device(device):
            rc = run(*args)
    if rc == ERR_WORKSPACE:
        raise ValueError(f"workspace too small: need {size()} bytes, 16-byte aligned")
    if rc != OK:
        raise _err(rc)
    return workspace


def _same_dtype(tensors, name):
    first = tensors[0].dtype
    if any(t.dtype != first for t in tensors):
        raise TypeError(f"every {name} of a grouped call must have the same dtype")
    return 1 if first == _torch().bfloat16 else 0


def orthogonalize_batched(mats: Sequence[Tuple], coeffs=NS_COEFFS, steps: int = 5, math="f32",
                          workspace=None, stream=None):
    """Newton-Schulz orthogonalization of a list of (G, O) tensor pairs: O
    (float32 or bfloat16) receives the orthogonalized G (float32 or
    bfloat16).  math: "f32" (float32 accuracy) or "f16" (one float16 matrix
    product per product).  Returns the workspace (for reuse and ``status``)."""
    torch = _torch()
    if len(mats) == 0:
        raise ValueError("empty matrix list")
    types = (torch.float32, torch.bfloat16)
    dev = mats[0][0].device
    arr = (dion_ns_matrix * len(mats))()
    for i, (G, O) in enumerate(mats):
        ldg = _check_rows("G", G, None, types, dev)
        ldo = _check_rows("O", O, G.shape, types, dev)
        arr[i] = dion_ns_matrix(G.data_ptr(), O.data_ptr(), G.shape[0], G.shape[1], ldg, ldo)
    gd, od = _same_dtype([g for g, _ in mats], "G"), _same_dtype([o for _, o in mats], "O")
    mode, cf = _ns_math(math), _ns_coeffs(coeffs, steps)
    lib, count = load(), len(mats)
    return _launch(
        lambda: lib.dion_orthogonalize_workspace_size(arr, count, mode),
        lambda ws, nbytes, st: lib.dion_orthogonalize_batched(arr, count, cf, int(steps), mode, gd, od,
                                                              ws, nbytes, st),
        dev, workspace, stream)


def orthogonalize(G, O, coeffs=NS_COEFFS, steps: int = 5, math="f32", workspace=None, stream=None):
    """``orthogonalize_batched`` of one matrix."""
    return orthogonalize_batched([(G, O)], coeffs, steps, math, workspace, stream)


def _muon_scale(scale, m: int, n: int) -> float:
    if scale == "none":
        return 1.0
    if scale == "spectral":
        return max(1.0, m / n) ** 0.5
    if scale == "rms":
        return 0.2 * max(m, n) ** 0.5
    if isinstance(scale, str):
        raise ValueError("scale must be 'none', 'spectral', 'rms' or a number")
    return float(scale)


def muon_step_batched(mats: Sequence[Tuple], lr: float, momentum: float = 0.95,
                      nesterov: bool = True, weight_decay: float = 0.0, scale="spectral",
                      coeffs=NS_COEFFS, steps: int = 5, math="f32", workspace=None, stream=None):
    """Muon step over a list of (X, G, M): M <- momentum M + G, D = G +
    momentum M (nesterov) or M, X <- (1 - lr weight_decay) X - lr s
    orthogonalize(D).  X, M float32, updated in place; G float32 or bfloat16.
    scale: s = 1 ("none"), sqrt(max(1, m / n)) ("spectral"), 0.2
    sqrt(max(m, n)) ("rms"), or a number.  Returns the workspace."""
    torch = _torch()
    if len(mats) == 0:
        raise ValueError("empty matrix list")
    dev = mats[0][0].device
    arr = (dion_muon_matrix * len(mats))()
    for i, (X, G, M) in enumerate(mats):
        for name, t, types in (("X", X, (torch.float32,)), ("M", M, (torch.float32,)),
                               ("G", G, (torch.float32, torch.bfloat16))):
            if _check_rows(name, t, X.shape, types, dev) != t.shape[1]:
                raise ValueError(f"{name} must be contiguous (row-major)")
        m, n = X.shape
        arr[i] = dion_muon_matrix(X.data_ptr(), G.data_ptr(), M.data_ptr(), m, n,
                                  _muon_scale(scale, m, n) if m and n else 0.0)
    gd = _same_dtype([g for _, g, _ in mats], "G")
    mode, cf = _ns_math(math), _ns_coeffs(coeffs, steps)
    lib, count = load(), len(mats)
    return _launch(
        lambda: lib.dion_muon_workspace_size(arr, count, mode),
        lambda ws, nbytes, st: lib.dion_muon_step_batched(
            arr, count, float(lr), float(momentum), 1 if nesterov else 0, float(weight_decay), cf,
            int(steps), mode, gd, ws, nbytes, st),
        dev, workspace, stream)


def muon_step(X, G, M, lr: float, momentum: float = 0.95, nesterov: bool = True,
              weight_decay: float = 0.0, scale="spectral", coeffs=NS_COEFFS, steps: int = 5,
              math="f32", workspace=None, stream=None):
    """``muon_step_batched`` of one matrix."""
    return muon_step_batched([(X, G, M)], lr, momentum, nesterov, weight_decay, scale, coeffs,
                             steps, math, workspace, stream)


# --- linear layer -----------------------------------------------------------

def _act(act) -> int:
    if isinstance(act, str):
        if act not in ACTS:
            raise ValueError(f"act must be one of {list(ACTS)}")
        act = ACTS[act]
    return int(act)


def _put(s, name, ld, tensor, shape, dtype, device):
    if tensor is None:
        return
    pitch = _check_rows(name, tensor, shape, (dtype,), device)
    setattr(s, name, tensor.data_ptr())
    setattr(s, ld, pitch)


def _put_vector(s, name, tensor, n, device):
    if tensor is None:
        return
    if not tensor.is_cuda or tensor.device != device or tensor.dtype != _torch().float32:
        raise TypeError(f"{name} must be a float32 GPU tensor on the same device")
    if tuple(tensor.shape) != (n,) or not tensor.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {n} elements")
    setattr(s, name, tensor.data_ptr())


def _linear(name, s, device, workspace, stream):
    lib, ref = load(), ctypes.byref(s)
    size = getattr(lib, f"dion_linear_{name}_workspace_size")
    run = getattr(lib, f"dion_linear_{name}")
    return _launch(lambda: size(ref), lambda ws, nbytes, st: run(ref, ws, nbytes, st), device,
                   workspace, stream)


def _linear_dtype(t, name) -> int:
    torch = _torch()
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"{name} must be float32 or bfloat16")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    return 1 if t.dtype == torch.bfloat16 else 0


def linear_forward(x, weight, y, bias=None, act="none", residual=None, preact=None,
                   workspace=None, stream=None):
    """y = act(x weight^T + bias) + residual (dion_linear_forward).

    x (t x k), weight (n x k), y, residual, preact (t x n): float32 or
    bfloat16, one type; bias (n) float32.  act: one of ACTS.  preact receives
    x weight^T + bias, which the backward of an activation needs.  residual
    may be y itself.  Returns the workspace."""
    s = dion_linear(dtype=_linear_dtype(x, "x"), act=_act(act))
    if weight.dim() != 2:
        raise ValueError("weight must be 2-D")
    t, k = x.shape
    n = weight.shape[0]
    s.t, s.n, s.k = t, n, k
    dev = x.device
    _put(s, "x", "ldx", x, (t, k), x.dtype, dev)
    _put(s, "w", "ldw", weight, (n, k), x.dtype, dev)
    _put(s, "y", "ldy", y, (t, n), x.dtype, dev)
    _put(s, "residual", "ldr", residual, (t, n), x.dtype, dev)
    _put(s, "z", "ldz", preact, (t, n), x.dtype, dev)
    _put_vector(s, "bias", bias, n, dev)
    return _linear("forward", s, dev, workspace, stream)


def linear_backward(dy, x=None, weight=None, dx=None, dw=None, db=None, act="none", preact=None,
                    accumulate: bool = False, workspace=None, stream=None):
    """Gradients of linear_forward (dion_linear_backward): dz = dy act'(preact),
    dx = dz weight, dw = dz^T x, db = the sum of dz over tokens, those of the
    three that are given.  accumulate: add to dw and db.  The residual's
    gradient is dy.  Returns the workspace."""
    s = dion_linear(dtype=_linear_dtype(dy, "dy"), act=_act(act), accumulate=int(bool(accumulate)))
    t, n = dy.shape
    given = [v.shape[1] for v in (x, weight, dx, dw) if v is not None and v.dim() == 2]
    k = given[0] if given else 1
    s.t, s.n, s.k = t, n, k
    dev = dy.device
    if s.act and preact is None:
        raise ValueError("the backward of an activation needs preact")
    if dx is not None and weight is None or dw is not None and x is None:
        raise ValueError("dx needs weight, dw needs x")
    _put(s, "dy", "lddy", dy, (t, n), dy.dtype, dev)
    _put(s, "z", "ldz", preact if s.act else None, (t, n), dy.dtype, dev)
    _put(s, "x", "ldx", x, (t, k), dy.dtype, dev)
    _put(s, "w", "ldw", weight, (n, k), dy.dtype, dev)
    _put(s, "dx", "lddx", dx, (t, k), dy.dtype, dev)
    _put(s, "dw", "lddw", dw, (n, k), dy.dtype, dev)
    _put_vector(s, "db", db, n, dev)
    return _linear("backward", s, dev, workspace, stream)
