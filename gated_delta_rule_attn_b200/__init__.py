"""Causal linear attention (ELU+1 / GLA / gated delta rule) for B200, the gated
linear recurrence with a vector state, and the norms around them.

Thin Python binding over the C ABI in ``include/la.h``: it only checks tensor
properties, allocates outputs with PyTorch and passes pointers, sizes and the
current CUDA stream to ``libla_b200.so``.  Every step of the computation runs in
the library's CUDA kernels; there is no CPU path.  If the library is missing
the import of the binding raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libla_b200.so")
ABI_VERSION = 3   # LA_ABI_VERSION of include/la.h that these struct layouts follow

GATES = {"value": 0, "logit": 1}
NORMS = {"layer": 0, "rms": 1}
RULES = {"elu": 0, "gla": 1, "gdn": 2, "kda": 3}
DTYPES = {torch.float32: 0, torch.bfloat16: 1}
STATUS = {0: "LA_OK", 1: "LA_ERR_INVALID_ARG", 2: "LA_ERR_UNSUPPORTED", 3: "LA_ERR_ALIGNMENT",
          4: "LA_ERR_CUDA", 5: "LA_ERR_TIMEOUT", 6: "LA_ERR_RANGE", 7: "LA_ERR_INTERNAL",
          8: "LA_ERR_WORKSPACE"}

# Symbols include/la.h and include/la_testing.h declare (checked by the CPU test suite).
EXPORTS = ("la_fwd", "la_fwd_workspace_size", "la_step", "la_fwd_host_staging_size",
           "la_fwd_host", "la_check_device", "la_status_string", "la_last_error_message",
           "la_abi_version", "la_fwd_noalloc", "la_testing_set_wait_limit",
           "la_scan_fwd", "la_scan_bwd", "la_scan_step", "la_scan_fwd_workspace_size", "la_scan_bwd_workspace_size",
           "la_norm_fwd", "la_norm_bwd", "la_norm_bwd_workspace_size")


class LAError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class FwdArgs(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("rule", ctypes.c_int), ("dtype", ctypes.c_int),
                ("B", ctypes.c_int64), ("T", ctypes.c_int64), ("H", ctypes.c_int64),
                ("dk", ctypes.c_int64), ("dv", ctypes.c_int64),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("g", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("S0", ctypes.c_void_p),
                ("z0", ctypes.c_void_p), ("eps", ctypes.c_float), ("o", ctypes.c_void_p),
                ("S_out", ctypes.c_void_p), ("z_out", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("cu_seqlens", ctypes.c_void_p), ("max_seqlen", ctypes.c_int64),
                ("out_norm", ctypes.c_int32), ("norm_eps", ctypes.c_float), ("norm_w", ctypes.c_void_p)]


class StepArgs(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("rule", ctypes.c_int), ("dtype", ctypes.c_int),
                ("N", ctypes.c_int64), ("H", ctypes.c_int64), ("dk", ctypes.c_int64),
                ("dv", ctypes.c_int64),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("g", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("S", ctypes.c_void_p),
                ("z", ctypes.c_void_p), ("eps", ctypes.c_float), ("o", ctypes.c_void_p),
                ("out_norm", ctypes.c_int32), ("norm_eps", ctypes.c_float), ("norm_w", ctypes.c_void_p)]


_U, _I, _L, _V, _F = ctypes.c_uint32, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class ScanFwdArgs(ctypes.Structure):
    _fields_ = [("struct_size", _U), ("dtype", _I), ("gate_dtype", _I), ("gate", _I), ("tied", ctypes.c_int32),
                ("B", _L), ("T", _L), ("D", _L), ("x", _V), ("x_row", _L), ("g", _V), ("g_row", _L),
                ("h0", _V), ("h", _V), ("h_row", _L), ("h_last", _V), ("cu_seqlens", _V), ("max_seqlen", _L),
                ("workspace", _V), ("workspace_bytes", ctypes.c_size_t)]


class ScanBwdArgs(ctypes.Structure):
    _fields_ = [("struct_size", _U), ("dtype", _I), ("gate_dtype", _I), ("gate", _I), ("tied", ctypes.c_int32),
                ("B", _L), ("T", _L), ("D", _L), ("x", _V), ("x_row", _L), ("g", _V), ("g_row", _L),
                ("h", _V), ("h_row", _L), ("dh", _V), ("dh_row", _L), ("h0", _V), ("dh_last", _V),
                ("dx", _V), ("dx_row", _L), ("dg", _V), ("dg_row", _L), ("dh0", _V),
                ("cu_seqlens", _V), ("max_seqlen", _L), ("workspace", _V), ("workspace_bytes", ctypes.c_size_t)]


class ScanStepArgs(ctypes.Structure):
    _fields_ = [("struct_size", _U), ("dtype", _I), ("gate_dtype", _I), ("gate", _I), ("tied", ctypes.c_int32),
                ("N", _L), ("D", _L), ("x", _V), ("x_row", _L), ("g", _V), ("g_row", _L), ("state", _V),
                ("h", _V), ("h_row", _L)]


class NormFwdArgs(ctypes.Structure):
    _fields_ = [("struct_size", _U), ("dtype", _I), ("kind", _I), ("R", _L), ("D", _L), ("x", _V), ("x_row", _L),
                ("w", _V), ("b", _V), ("eps", _F), ("y", _V), ("y_row", _L), ("mean", _V), ("rstd", _V)]


class NormBwdArgs(ctypes.Structure):
    _fields_ = [("struct_size", _U), ("dtype", _I), ("kind", _I), ("R", _L), ("D", _L), ("x", _V), ("x_row", _L),
                ("dy", _V), ("dy_row", _L), ("w", _V), ("mean", _V), ("rstd", _V), ("dx", _V), ("dx_row", _L),
                ("dw", _V), ("db", _V), ("workspace", _V), ("workspace_bytes", ctypes.c_size_t)]


_lib = None


def lib():
    """Load ``libla_b200.so`` (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python gated_delta_rule_attn_b200/build.py` (no CPU fallback exists)")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        L.la_fwd.argtypes = [ctypes.POINTER(FwdArgs), P]
        L.la_fwd_workspace_size.argtypes = [ctypes.POINTER(FwdArgs), ctypes.POINTER(ctypes.c_size_t)]
        L.la_step.argtypes = [ctypes.POINTER(StepArgs), P]
        L.la_fwd_host_staging_size.argtypes = [ctypes.POINTER(FwdArgs), ctypes.POINTER(ctypes.c_size_t)]
        L.la_fwd_host.argtypes = [ctypes.POINTER(FwdArgs), P, ctypes.c_size_t, P]
        L.la_check_device.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
        L.la_fwd_noalloc.argtypes = [ctypes.POINTER(FwdArgs), P]
        L.la_testing_set_wait_limit.argtypes = [ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)]
        L.la_testing_set_wait_limit.restype = ctypes.c_int
        L.la_status_string.argtypes = [ctypes.c_int]
        L.la_status_string.restype = ctypes.c_char_p
        L.la_last_error_message.restype = ctypes.c_char_p
        for f, args in ((L.la_scan_fwd, ScanFwdArgs), (L.la_scan_bwd, ScanBwdArgs), (L.la_scan_step, ScanStepArgs),
                        (L.la_norm_fwd, NormFwdArgs), (L.la_norm_bwd, NormBwdArgs)):
            f.argtypes = [ctypes.POINTER(args), P]
        for f, args in ((L.la_scan_fwd_workspace_size, ScanFwdArgs), (L.la_scan_bwd_workspace_size, ScanBwdArgs),
                        (L.la_norm_bwd_workspace_size, NormBwdArgs)):
            f.argtypes = [ctypes.POINTER(args), ctypes.POINTER(ctypes.c_size_t)]
        for f in (L.la_fwd, L.la_fwd_workspace_size, L.la_step, L.la_fwd_host_staging_size,
                  L.la_fwd_host, L.la_check_device, L.la_fwd_noalloc, L.la_scan_fwd, L.la_scan_bwd,
                  L.la_scan_step, L.la_scan_fwd_workspace_size, L.la_scan_bwd_workspace_size,
                  L.la_norm_fwd, L.la_norm_bwd, L.la_norm_bwd_workspace_size):
            f.restype = ctypes.c_int
        L.la_abi_version.restype = ctypes.c_int
        if L.la_abi_version() != ABI_VERSION:
            raise ImportError(f"{LIB_PATH} has ABI version {L.la_abi_version()}, the binding expects "
                              f"{ABI_VERSION}: rebuild it")
        _lib = L
    return _lib


def _check(status: int):
    if status != 0:
        raise LAError(status, lib().la_last_error_message().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, name, device=True):
    if t is None:
        return
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _set_norm(a, out_norm, norm_w, norm_eps):
    """Output normalisation fields (la.h, ABI version 3)."""
    a.out_norm = 1 if out_norm else 0
    a.norm_eps = norm_eps
    a.norm_w = norm_w.data_ptr() if norm_w is not None else None


def make_fwd_args(rule, q, k, v, g=None, beta=None, S0=None, z0=None, eps=1e-6,
                  o=None, S_out=None, z_out=None, cu_seqlens=None, max_seqlen=None,
                  out_norm=False, norm_w=None, norm_eps=1e-6) -> FwdArgs:
    """Marshal tensors into la_fwd_args.  With ``cu_seqlens`` (int64 [B+1] on the
    device) the token tensors are one packed axis [1, T, H, d] and B is the
    number of sequences; ``max_seqlen`` bounds their lengths.  ``out_norm``:
    each (token, head) row of o is RMS-normalised over dv (weight ``norm_w``
    fp32 [dv] or None, ``norm_eps`` > 0)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if cu_seqlens is not None:
        if B != 1:
            raise ValueError("packed sequences take q, k, v as [1, T, H, d]")
        if cu_seqlens.dtype != torch.int64 or cu_seqlens.dim() != 1:
            raise ValueError("cu_seqlens must be a 1-D int64 tensor")
        B = cu_seqlens.numel() - 1
        if max_seqlen is None:
            raise ValueError("packed sequences need max_seqlen")
    a = FwdArgs()
    a.struct_size = ctypes.sizeof(FwdArgs)
    a.rule = RULES[rule]
    a.dtype = DTYPES[q.dtype]
    a.B, a.T, a.H, a.dk, a.dv = B, T, H, dk, dv
    a.q, a.k, a.v, a.g, a.beta = (t.data_ptr() if t is not None else None for t in (q, k, v, g, beta))
    a.S0 = S0.data_ptr() if S0 is not None else None
    a.z0 = z0.data_ptr() if z0 is not None else None
    a.eps = eps
    a.o = o.data_ptr() if o is not None else None
    a.S_out = S_out.data_ptr() if S_out is not None else None
    a.z_out = z_out.data_ptr() if z_out is not None else None
    if cu_seqlens is not None:
        a.cu_seqlens = cu_seqlens.data_ptr()
        a.max_seqlen = int(max_seqlen)
    _set_norm(a, out_norm, norm_w, norm_eps)
    return a


_WORKSPACES = {}


def _workspace(device, stream, nbytes: int):
    """Scratch for la_fwd, cached per (device, stream): calls on one stream are
    ordered, so they can share it.  It is allocated with that stream current, so
    that when a larger one replaces it, the allocator reuses the old block only
    for work ordered after the kernels that used it."""
    key = (device.index, stream.cuda_stream)
    ws = _WORKSPACES.get(key)
    if ws is None or ws.numel() < nbytes:
        with torch.cuda.stream(stream):
            ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _WORKSPACES[key] = ws
    return ws


def fwd(rule: str, q, k, v, g=None, beta=None, S0=None, z0=None, eps: float = 1e-6,
        o=None, S_out=None, z_out=None, stream=None, want_state: bool = True, workspace=None,
        cu_seqlens=None, max_seqlen=None, out_norm: bool = False, norm_w=None, norm_eps: float = 1e-6):
    """Chunked prefill: returns (o, S_out, z_out-or-None). Enqueued on the current stream.

    ``workspace`` (a CUDA uint8 tensor of at least ``fwd_workspace_size`` bytes)
    is allocated and cached per stream when not given.  ``cu_seqlens`` /
    ``max_seqlen``: packed variable-length sequences (see ``make_fwd_args``);
    the states are then [number of sequences, H, dk, dv].  ``out_norm``,
    ``norm_w``, ``norm_eps``: head-wise RMS normalisation of o (see
    ``make_fwd_args``)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (g, "g"), (beta, "beta"), (S0, "S0"), (z0, "z0"),
                 (cu_seqlens, "cu_seqlens"), (norm_w, "norm_w")):
        _need(t, n)
    NS = B if cu_seqlens is None else cu_seqlens.numel() - 1   # sequences (state rows)
    if q.dtype != k.dtype or q.dtype != v.dtype:
        raise ValueError("q, k, v must share a dtype")
    if o is None:
        o = torch.empty(B, T, H, dv, dtype=q.dtype, device=q.device)
    if S_out is None and want_state:
        S_out = torch.empty(NS, H, dk, dv, dtype=torch.float32, device=q.device)
    if rule == "elu" and z_out is None and want_state:
        z_out = torch.empty(NS, H, dk, dtype=torch.float32, device=q.device)
    a = make_fwd_args(rule, q, k, v, g, beta, S0, z0, eps, o, S_out, z_out, cu_seqlens, max_seqlen,
                      out_norm, norm_w, norm_eps)
    st = stream if stream is not None else torch.cuda.current_stream(q.device)
    sh = _stream_handle(st)
    n = ctypes.c_size_t()
    _check(lib().la_fwd_workspace_size(ctypes.byref(a), ctypes.byref(n)))
    if n.value:
        ws = workspace if workspace is not None else _workspace(q.device, st, n.value)
        a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel()
    _check(lib().la_fwd(ctypes.byref(a), sh))
    return o, S_out, z_out


def fwd_workspace_size(rule, q, k, v, g=None, beta=None, S0=None, z0=None) -> int:
    """Bytes of workspace ``fwd`` needs for these inputs (shapes only are read)."""
    a = make_fwd_args(rule, q, k, v, g, beta, S0, z0)
    # the query validates the arguments as la_fwd does, which needs a non-NULL o;
    # no data is touched, so q's address stands in for it
    a.o = a.q
    n = ctypes.c_size_t()
    _check(lib().la_fwd_workspace_size(ctypes.byref(a), ctypes.byref(n)))
    return n.value


def step(rule: str, q, k, v, S, z=None, g=None, beta=None, eps: float = 1e-6, o=None,
         stream=None, out_norm: bool = False, norm_w=None, norm_eps: float = 1e-6):
    """Decode step: updates S (and z) in place, returns o [N,H,dv] (RMS-normalised
    per (sequence, head) over dv with ``out_norm``)."""
    N, H, dk = q.shape
    dv = v.shape[-1]
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (g, "g"), (beta, "beta"), (S, "S"), (z, "z"),
                 (norm_w, "norm_w")):
        _need(t, n)
    if o is None:
        o = torch.empty(N, H, dv, dtype=q.dtype, device=q.device)
    a = StepArgs()
    a.struct_size = ctypes.sizeof(StepArgs)
    a.rule = RULES[rule]
    a.dtype = DTYPES[q.dtype]
    a.N, a.H, a.dk, a.dv = N, H, dk, dv
    a.q, a.k, a.v, a.g, a.beta, a.S, a.z = (t.data_ptr() if t is not None else None
                                            for t in (q, k, v, g, beta, S, z))
    a.eps = eps
    a.o = o.data_ptr()
    _set_norm(a, out_norm, norm_w, norm_eps)
    _check(lib().la_step(ctypes.byref(a), _stream_handle(stream)))
    return o


def host_staging_size(rule, q, k, v, g=None, beta=None, S0=None, z0=None, want_state=True,
                      out_norm=False, norm_w=None, norm_eps=1e-6) -> int:
    """Bytes of device staging ``fwd_host`` needs for these host tensors."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    a = make_fwd_args(rule, q, k, v, g, beta, S0, z0, out_norm=out_norm, norm_w=norm_w, norm_eps=norm_eps)
    # output pointers only mark presence for the size computation
    a.o = 1
    a.S_out = 1 if want_state else None
    a.z_out = 1 if (want_state and rule == "elu") else None
    n = ctypes.c_size_t()
    _check(lib().la_fwd_host_staging_size(ctypes.byref(a), ctypes.byref(n)))
    return n.value


def fwd_host(rule: str, q, k, v, g=None, beta=None, S0=None, z0=None, eps: float = 1e-6,
             o=None, S_out=None, z_out=None, staging=None, stream=None,
             out_norm: bool = False, norm_w=None, norm_eps: float = 1e-6):
    """la_fwd on host (CPU, ideally pinned) tensors through the C ABI: the library
    copies inputs into ``staging`` (a CUDA uint8 tensor), runs, copies outputs back
    and synchronises the stream.  Returns (o, S_out, z_out)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (g, "g"), (beta, "beta"), (S0, "S0"), (z0, "z0"),
                 (o, "o"), (S_out, "S_out"), (z_out, "z_out"), (norm_w, "norm_w")):
        _need(t, n, device=False)
    a = make_fwd_args(rule, q, k, v, g, beta, S0, z0, eps, o, S_out, z_out,
                      out_norm=out_norm, norm_w=norm_w, norm_eps=norm_eps)
    _check(lib().la_fwd_host(ctypes.byref(a), ctypes.c_void_p(staging.data_ptr()),
                             staging.numel(), _stream_handle(stream)))
    return o, S_out, z_out


# ---------------------------------------------------------------------------
# Gated linear recurrence and row norms.
# ---------------------------------------------------------------------------
def _tokens(t, name, lead, tail, dtype, device):
    """The distance in elements between the rows of ``t``, a tensor of shape
    ``lead + tail`` whose trailing dims are dense and whose leading dims are one
    axis of equally spaced rows (0 when the whole tensor is dense)."""
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor on the device of the other tensors")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != lead + tail:
        raise ValueError(f"{name} must have shape {tuple(lead + tail)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return 0
    size, stride = t.shape, t.stride()
    n, D = len(lead), 1
    for i in range(len(size) - 1, n - 1, -1):
        if size[i] != 1 and stride[i] != D:
            raise ValueError(f"{name}: the elements of a row must be contiguous")
        D *= size[i]
    row, step = 0, 0
    for i in range(n - 1, -1, -1):
        if size[i] == 1:
            continue
        if not row:
            row = step = stride[i]
            if row < D:
                raise ValueError(f"{name}: rows overlap (a broadcast tensor has to be made contiguous)")
        elif stride[i] != step:
            raise ValueError(f"{name}: the leading dims must be one axis of equally spaced rows")
        step *= size[i]
    return row


def _dense(t, name, shape, device, dtype=torch.float32):
    """Address of a dense fp32 tensor of that shape, or None."""
    if t is None:
        return None
    if t.device != device or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a dense {dtype} tensor of shape {tuple(shape)} on {device}")
    return t.data_ptr()


class _On:
    """The device and the stream of a call: the current stream of the tensors'
    device, or ``stream``.  Inside, new tensors belong to that stream; the memory
    of ``tensors`` is kept until the work queued on a given ``stream`` is done."""

    def __init__(self, device, stream, *tensors):
        if device.type != "cuda":
            raise ValueError("the tensors must be on a CUDA device")
        self.ctx = None
        if stream is not None:
            if stream.device != device:
                raise ValueError("stream belongs to another device than the tensors")
            self.ctx = torch.cuda.stream(stream)
        elif torch._C._cuda_getDevice() != device.index:
            self.ctx = torch.cuda.device(device)
        self.device, self.stream, self.tensors = device, stream, tensors

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        if self.stream is not None:
            return self.stream.cuda_stream
        return torch._C._cuda_getCurrentRawStream(self.device.index)

    def __exit__(self, *exc):
        try:
            if self.stream is not None:
                for t in self.tensors:
                    if isinstance(t, torch.Tensor) and t.device == self.device:   # (a refused one may be elsewhere)
                        t.record_stream(self.stream)
        finally:                           # whatever was refused, the caller's stream is current again
            if self.ctx is not None:
                self.ctx.__exit__(*exc)
        return False


def _call_scratch(size_of, a, device):
    """The scratch that ``size_of`` asks for, allocated for this call and set in ``a``
    (calls on different streams and captured graphs share none)."""
    n = ctypes.c_size_t()
    _check(size_of(ctypes.byref(a), ctypes.byref(n)))
    if not n.value:
        return None
    ws = torch.empty(n.value, dtype=torch.uint8, device=device)
    a.workspace, a.workspace_bytes = ws.data_ptr(), n.value
    return ws


def _choice(table, key, name):
    try:
        return table[key]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be one of {', '.join(map(str, table))}, got {key!r}") from None


def _scan_shape(g, cu_seqlens, max_seqlen):
    """(lead, tail, sequences, D, address of cu_seqlens, max_seqlen) of token tensors like g."""
    if g.dim() < 3:
        raise ValueError("token tensors are [B, T, D] or [B, T, H, d]")
    lead, tail = g.shape[:2], g.shape[2:]
    D = 1
    for n in tail:
        D *= n
    if cu_seqlens is None:
        if max_seqlen is not None:
            raise ValueError("max_seqlen goes with cu_seqlens")
        return lead, tail, lead[0], D, None, 0
    if lead[0] != 1:
        raise ValueError("packed sequences take token tensors as [1, T, ...]")
    if cu_seqlens.dtype is not torch.int64 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a 1-D int64 tensor of at least 2 offsets")
    if max_seqlen is None:
        raise ValueError("packed sequences need max_seqlen")
    return (lead, tail, cu_seqlens.numel() - 1, D,
            _dense(cu_seqlens, "cu_seqlens", cu_seqlens.shape, g.device, torch.int64), int(max_seqlen))


def scan_fwd(x, g, h0=None, gate: str = "value", tied: bool = False, h=None, h_last=None,
             want_state: bool = True, cu_seqlens=None, max_seqlen=None, stream=None):
    """Gated linear recurrence ``h_t = a_t h_{t-1} + u_t`` per channel (la_scan_fwd
    in la.h): returns (h, h_last), on the current stream of the tensors' device.

    ``x``, ``g`` [B, T, D] or [B, T, H, d], fp32 or bf16 each; their rows may be
    slices of wider ones.  ``gate``: ``"value"`` (a = g) or ``"logit"``
    (a = sigmoid(g)).  ``tied``: u = (1 - a) x instead of x.  ``h0``, ``h_last``
    fp32 [B, D] ([B, H, d]); ``h_last`` may be ``h0``.  ``cu_seqlens`` /
    ``max_seqlen``: packed sequences as for ``fwd`` (states [sequences, ...])."""
    dev = x.device
    lead, tail, N, D, cu, ms = _scan_shape(g, cu_seqlens, max_seqlen)
    gt, dt = _choice(GATES, gate, "gate"), _choice(DTYPES, x.dtype, "x.dtype")
    gd = _choice(DTYPES, g.dtype, "g.dtype")
    xr, gr = _tokens(x, "x", lead, tail, x.dtype, dev), _tokens(g, "g", lead, tail, g.dtype, dev)
    state = (N,) + tuple(tail)
    with _On(dev, stream, x, g, h0, h, h_last, cu_seqlens) as st:
        if h is None:
            h = torch.empty(lead + tail, dtype=x.dtype, device=dev)
        if h_last is None and want_state:
            h_last = torch.empty(state, dtype=torch.float32, device=dev)
        a = ScanFwdArgs(ctypes.sizeof(ScanFwdArgs), dt, gd, gt, 1 if tied else 0, N, lead[1], D,
                        x.data_ptr(), xr, g.data_ptr(), gr, _dense(h0, "h0", state, dev), h.data_ptr(),
                        _tokens(h, "h", lead, tail, x.dtype, dev), _dense(h_last, "h_last", state, dev), cu, ms)
        ws = _call_scratch(lib().la_scan_fwd_workspace_size, a, dev)  # noqa: F841 (kept until the call is queued)
        _check(lib().la_scan_fwd(ctypes.byref(a), st))
    return h, h_last


def scan_bwd(g, h, dh, x=None, h0=None, dh_last=None, gate: str = "value", tied: bool = False,
             dx=None, dg=None, dh0=None, want_state: bool = True, cu_seqlens=None, max_seqlen=None, stream=None):
    """Gradients of ``scan_fwd`` (la_scan_bwd in la.h): returns (dx, dg, dh0).

    ``h`` is what ``scan_fwd`` returned, ``dh`` the gradient of h, ``dh_last`` that
    of h_last (fp32, or None for zero).  ``x`` is needed for a tied input only.
    dx has the type of dh, dg that of g, dh0 is fp32."""
    dev = g.device
    lead, tail, N, D, cu, ms = _scan_shape(g, cu_seqlens, max_seqlen)
    gt, dt = _choice(GATES, gate, "gate"), _choice(DTYPES, dh.dtype, "dh.dtype")
    gd = _choice(DTYPES, g.dtype, "g.dtype")
    if tied and x is None:
        raise ValueError("a tied input's gradient needs x")
    xr = _tokens(x, "x", lead, tail, dh.dtype, dev) if tied else 0
    gr, hr = _tokens(g, "g", lead, tail, g.dtype, dev), _tokens(h, "h", lead, tail, dh.dtype, dev)
    dhr = _tokens(dh, "dh", lead, tail, dh.dtype, dev)
    state = (N,) + tuple(tail)
    with _On(dev, stream, x, g, h, dh, h0, dh_last, dx, dg, dh0, cu_seqlens) as st:
        if dx is None:
            dx = torch.empty(lead + tail, dtype=dh.dtype, device=dev)
        if dg is None:
            dg = torch.empty(lead + tail, dtype=g.dtype, device=dev)
        if dh0 is None and want_state:
            dh0 = torch.empty(state, dtype=torch.float32, device=dev)
        a = ScanBwdArgs(ctypes.sizeof(ScanBwdArgs), dt, gd, gt, 1 if tied else 0, N, lead[1], D,
                        x.data_ptr() if tied else None, xr, g.data_ptr(), gr, h.data_ptr(), hr,
                        dh.data_ptr(), dhr, _dense(h0, "h0", state, dev), _dense(dh_last, "dh_last", state, dev),
                        dx.data_ptr(), _tokens(dx, "dx", lead, tail, dh.dtype, dev),
                        dg.data_ptr(), _tokens(dg, "dg", lead, tail, g.dtype, dev),
                        _dense(dh0, "dh0", state, dev), cu, ms)
        ws = _call_scratch(lib().la_scan_bwd_workspace_size, a, dev)  # noqa: F841
        _check(lib().la_scan_bwd(ctypes.byref(a), st))
    return dx, dg, dh0


def scan_step(x, g, state, gate: str = "value", tied: bool = False, h=None, stream=None):
    """One token of the recurrence per sequence: ``state`` (fp32 [N, D] or
    [N, H, d]) is updated in place, the new state rounded to x's type is returned."""
    dev = x.device
    if x.dim() < 2:
        raise ValueError("x and g are [N, D] or [N, H, d]")
    lead, tail = x.shape[:1], x.shape[1:]
    D = 1
    for n in tail:
        D *= n
    gt, dt = _choice(GATES, gate, "gate"), _choice(DTYPES, x.dtype, "x.dtype")
    gd = _choice(DTYPES, g.dtype, "g.dtype")
    xr, gr = _tokens(x, "x", lead, tail, x.dtype, dev), _tokens(g, "g", lead, tail, g.dtype, dev)
    if state is None:
        raise ValueError("state is needed")
    with _On(dev, stream, x, g, state, h) as st:
        if h is None:
            h = torch.empty(x.shape, dtype=x.dtype, device=dev)
        a = ScanStepArgs(ctypes.sizeof(ScanStepArgs), dt, gd, gt, 1 if tied else 0, lead[0], D, x.data_ptr(), xr,
                         g.data_ptr(), gr, _dense(state, "state", x.shape, dev), h.data_ptr(),
                         _tokens(h, "h", lead, tail, x.dtype, dev))
        _check(lib().la_scan_step(ctypes.byref(a), st))
    return h


def norm_fwd(x, w=None, b=None, kind: str = "layer", eps: float = 1e-6, y=None, want_stats: bool = True, stream=None):
    """Layer norm (``kind="layer"``) or RMS norm (``"rms"``) over the last dim of
    ``x`` (la_norm_fwd in la.h): returns (y, mean, rstd), the statistics fp32 of
    the leading shape (mean is None for an RMS norm; both are None without
    ``want_stats``).  ``w``, ``b`` fp32 [D] or None.  The leading dims must be one
    axis of equally spaced rows."""
    dev = x.device
    if x.dim() < 1:
        raise ValueError("x needs at least one dim")
    lead, tail = x.shape[:-1], x.shape[-1:]
    kd, dt = _choice(NORMS, kind, "kind"), _choice(DTYPES, x.dtype, "x.dtype")
    xr = _tokens(x, "x", lead, tail, x.dtype, dev)
    with _On(dev, stream, x, w, b, y) as st:
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=dev)
        mean = rstd = None
        if want_stats:
            if kd == 0:
                mean, rstd = torch.empty((2,) + lead, dtype=torch.float32, device=dev).unbind(0)
            else:
                rstd = torch.empty(lead, dtype=torch.float32, device=dev)
        a = NormFwdArgs(ctypes.sizeof(NormFwdArgs), dt, kd, lead.numel(), tail[0], x.data_ptr(), xr,
                        _dense(w, "w", tail, dev), _dense(b, "b", tail, dev), eps, y.data_ptr(),
                        _tokens(y, "y", lead, tail, x.dtype, dev),
                        mean.data_ptr() if mean is not None else None, rstd.data_ptr() if want_stats else None)
        _check(lib().la_norm_fwd(ctypes.byref(a), st))
    return y, mean, rstd


def norm_bwd(dy, x, rstd, mean=None, w=None, kind: str = "layer", dx=None, want_dw: bool = True,
             want_db: bool = True, stream=None):
    """Gradients of ``norm_fwd`` (la_norm_bwd in la.h): returns (dx, dw, db), dw and
    db fp32 [D] (None where not wanted).  ``rstd`` and ``mean`` (layer only) are
    what ``norm_fwd`` returned.  The partial sums' scratch is allocated for the
    call, so calls on different streams and captured graphs share none."""
    dev = x.device
    if x.dim() < 1:
        raise ValueError("x needs at least one dim")
    lead, tail = x.shape[:-1], x.shape[-1:]
    kd, dt = _choice(NORMS, kind, "kind"), _choice(DTYPES, x.dtype, "x.dtype")
    xr, dyr = _tokens(x, "x", lead, tail, x.dtype, dev), _tokens(dy, "dy", lead, tail, x.dtype, dev)
    if rstd is None or (kd == 0) != (mean is not None):
        raise ValueError("rstd is needed, and mean for a layer norm only")
    with _On(dev, stream, dy, x, rstd, mean, w, dx) as st:
        if dx is None:
            dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
        dw = torch.empty(tail, dtype=torch.float32, device=dev) if want_dw else None
        db = torch.empty(tail, dtype=torch.float32, device=dev) if want_db else None
        a = NormBwdArgs(ctypes.sizeof(NormBwdArgs), dt, kd, lead.numel(), tail[0], x.data_ptr(), xr,
                        dy.data_ptr(), dyr, _dense(w, "w", tail, dev), _dense(mean, "mean", lead, dev),
                        _dense(rstd, "rstd", lead, dev), dx.data_ptr(),
                        _tokens(dx, "dx", lead, tail, x.dtype, dev),
                        dw.data_ptr() if want_dw else None, db.data_ptr() if want_db else None, None, 0)
        if want_dw or want_db:
            ws = _call_scratch(lib().la_norm_bwd_workspace_size, a, dev)  # noqa: F841
        _check(lib().la_norm_bwd(ctypes.byref(a), st))
    return dx, dw, db


def check_device(stream=None) -> int:
    """Synchronise and read/clear the device error word; raises on a recorded error."""
    flags = ctypes.c_uint32()
    _check(lib().la_check_device(_stream_handle(stream), ctypes.byref(flags)))
    return flags.value


def abi_version() -> int:
    return lib().la_abi_version()
