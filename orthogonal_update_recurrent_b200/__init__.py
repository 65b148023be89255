"""Python binding of liblattice (B200, sm_100a): the Lattice compression-layer
state recurrence ("Lattice: Learning to Efficiently Compress the Memory",
arXiv 2504.05646, §3).

This module only marshals arguments: it checks tensor placement, dtypes and
shapes, and passes raw device pointers and the current CUDA stream to the C
ABI declared in include/lattice.h. Every step of the computation runs in the
library's CUDA kernels. There is no CPU or PyTorch fallback: without the built
library every call raises.

Tensors (row-major, contiguous, on one CUDA device):
    x   [B, T, H, d]  float32 or bfloat16      c   [B, T, H, m] float32
    q   [B, T, H, m]  float32 or bfloat16      mu  [B, T, H]    float32
    eta [B, T, H]     float32 or None (=1)     S0  [B, H, m, d] float32
Decode calls drop the T axis.

Beside the state recurrence: the gated linear recurrence (gated_scan_fwd,
gated_scan_bwd, gated_step) and the norms after and before a block (block_norm_fwd,
block_norm_bwd). These also take float16, and rows that are slices of wider ones (their
last axes contiguous).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

__all__ = ["LatticeError", "lib", "scan_fwd", "scan_bwd", "scan_bwd_workspace_bytes", "step",
           "readout", "chunk_impl", "device_status", "selftest_bounded_wait", "LIB_PATH",
           "gated_scan_fwd", "gated_scan_bwd", "gated_scan_marks", "gated_step", "block_norm_fwd",
           "block_norm_bwd"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblattice.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT = range(5)
_F32, _BF16 = 0, 1
_IMPL = {"auto": 0, "simt": 1, "tcgen05": 2, "tcgen05_split": 3, "split_reg": 4, "split_reg8": 5}
_MODE = {"sim": 0, "dec": 1}
_lib = None


class LatticeError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        msg = _lib.lattice_status_string(code).decode() if _lib is not None else str(code)
        if code == ERR_CUDA and _lib is not None:
            msg += " [" + _lib.lattice_last_cuda_error().decode() + "]"
        super().__init__(f"{what}: {msg} (status {code})")


def lib() -> ctypes.CDLL:
    """Load liblattice.so (built in-tree by orthogonal_update_recurrent_b200.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"liblattice.so not found at {LIB_PATH}; build it with "
                "`python -m orthogonal_update_recurrent_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, fp = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p
        L.lattice_scan_fwd.argtypes = [vp, i, fp, vp, i, fp, fp, fp, fp, fp, i, i, i, i, i, i, i, vp]
        L.lattice_scan_fwd_impl.argtypes = [vp, i, fp, vp, i, fp, fp, fp, fp, fp, i, i, i, i, i,
                                            i, i, i, vp]
        L.lattice_scan_fwd_ex.argtypes = [vp, i, fp, vp, i, fp, fp, fp, fp, fp, i, i, i, i, i,
                                          i, i, i, i, vp]
        L.lattice_scan_bwd.argtypes = [vp, i, fp, vp, i, fp, fp, fp, fp, fp, fp, fp, fp, fp, fp,
                                       fp, vp, ctypes.c_size_t, i, i, i, i, i, i, i, vp]
        L.lattice_scan_bwd_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
        L.lattice_scan_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.lattice_step.argtypes = [fp, vp, i, fp, vp, i, fp, fp, fp, i, i, i, i, i, vp]
        L.lattice_readout.argtypes = [fp, vp, i, fp, i, i, i, i, vp]
        L.lattice_get_device_status.argtypes = [vp]
        L.lattice_selftest_bounded_wait.argtypes = [ctypes.c_ulonglong, vp]
        L.lattice_status_string.argtypes = [i]
        L.lattice_status_string.restype = ctypes.c_char_p
        L.lattice_version.argtypes = []
        L.lattice_chunk_impl.argtypes = [i, i, i, i, i, i, i]
        L.lattice_last_cuda_error.argtypes = []
        L.lattice_last_cuda_error.restype = ctypes.c_char_p
        ll, f32 = ctypes.c_longlong, ctypes.c_float
        L.lattice_gated_scan_fwd.argtypes = [vp, i, ll, ll, vp, i, ll, ll, i, fp, fp, vp, fp, vp, i, i, i, i, i, i,
                                             f32, vp]
        L.lattice_gated_scan_bwd.argtypes = [vp, i, ll, ll, vp, i, ll, ll, i, vp, ll, ll, fp, fp, vp, vp, fp, vp,
                                             i, i, i, i, i, i, f32, vp]
        L.lattice_gated_scan_marks_bytes.argtypes = [i, i, i, i]
        L.lattice_gated_scan_marks_bytes.restype = ctypes.c_size_t
        L.lattice_gated_step.argtypes = [fp, fp, vp, i, ll, vp, i, ll, i, vp, i, i, i, i, i, f32, vp]
        L.lattice_block_norm_fwd.argtypes = [vp, i, ll, vp, ll, vp, i, ll, vp, vp, i, vp, vp, i, ll, i, i, i, i, f32,
                                             f32, vp]
        L.lattice_block_norm_bwd.argtypes = [vp, i, ll, vp, ll, vp, i, ll, vp, vp, i, vp, i, ll, vp, ll, vp, vp, vp, fp,
                                             fp, vp, ctypes.c_size_t, i, ll, i, i, i, i, f32, f32, vp]
        L.lattice_block_norm_bwd_workspace_bytes.argtypes = [ll, i]
        L.lattice_block_norm_bwd_workspace_bytes.restype = ctypes.c_size_t
        for f in ("lattice_gated_scan_fwd", "lattice_gated_scan_bwd", "lattice_gated_step", "lattice_block_norm_fwd",
                  "lattice_block_norm_bwd"):
            getattr(L, f).restype = ctypes.c_int
        for f in ("lattice_scan_fwd", "lattice_scan_fwd_impl", "lattice_scan_fwd_ex", "lattice_scan_bwd",
                  "lattice_step", "lattice_readout", "lattice_selftest_bounded_wait",
                  "lattice_get_device_status", "lattice_version", "lattice_chunk_impl"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _adr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return _F32
    if t.dtype == torch.bfloat16:
        return _BF16
    raise TypeError(f"expected float32 or bfloat16, got {t.dtype}")


def _chk(t: torch.Tensor, name: str, shape, dtypes=(torch.float32,)):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _raise(code: int, what: str):
    if code != OK:
        raise LatticeError(code, what)


_XQ = (torch.float32, torch.bfloat16)


def scan_fwd(x: torch.Tensor, c: torch.Tensor, q: torch.Tensor, mu: torch.Tensor,
             S0: torch.Tensor, eta: Optional[torch.Tensor] = None, chunk: int = 1,
             S_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
             impl: str = "auto", stream=None, mode: str = "sim",
             lin: int = 2, norm: str = "token") -> Tuple[torch.Tensor, torch.Tensor]:
    """Whole-sequence forward (the paper's lattice_compress, Appendix D).
    chunk == 1: exact recurrence; chunk > 1: the chunked form, Eq. 17 (lin=2) or
    eq. recurrence_linear1 (lin=1); norm "chunk" drops the per-token normaliser and
    projects the slots onto the unit sphere after each chunk. mode "sim": similarity
    objective; "dec": reconstruction objective.
    Returns (y [B,T,H,d] float32, S_T [B,H,m,d] float32). S_out may be S0."""
    B, T, H, d = x.shape
    m = c.shape[-1]
    _chk(x, "x", (B, T, H, d), _XQ)
    _chk(c, "c", (B, T, H, m))
    _chk(q, "q", (B, T, H, m), _XQ)
    _chk(mu, "mu", (B, T, H))
    _chk(S0, "S0", (B, H, m, d))
    if eta is not None:
        _chk(eta, "eta", (B, T, H))
    if S_out is None:
        S_out = torch.empty_like(S0)
    _chk(S_out, "S_out", (B, H, m, d))
    if y is None:
        y = torch.empty((B, T, H, d), dtype=torch.float32, device=x.device)
    _chk(y, "y", (B, T, H, d))
    L = lib()
    code = L.lattice_scan_fwd_ex(_ptr(x), _dt(x), _ptr(c), _ptr(q), _dt(q), _ptr(mu), _ptr(eta),
                                 _ptr(S0), _ptr(S_out), _ptr(y), B, T, H, m, d, int(chunk),
                                 _MODE[mode], {2: 0, 1: 1}[lin] | {"token": 0, "chunk": 2}[norm],
                                 _IMPL[impl], _stream(stream))
    _raise(code, "lattice_scan_fwd")
    return y, S_out


def scan_bwd_workspace_bytes(B: int, T: int, H: int, m: int, d: int, chunk: int = 1,
                             seg: int = 0) -> int:
    """Device workspace bytes scan_bwd needs (0: the shape is not supported)."""
    return int(lib().lattice_scan_bwd_workspace_bytes(B, T, H, m, d, int(chunk), int(seg)))


def scan_bwd(x: torch.Tensor, c: torch.Tensor, q: torch.Tensor, mu: torch.Tensor,
             S0: torch.Tensor, dy: torch.Tensor, dS_T: Optional[torch.Tensor] = None,
             eta: Optional[torch.Tensor] = None, chunk: int = 1, seg: int = 0,
             workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Backward pass of scan_fwd (similarity objective; exact for chunk 1, Eq. 17
    otherwise): gradients of L = sum_t dy_t . y_t + dS_T . S_T. Returns a dict with
    dx, dc, dq, dmu, deta (None when eta is None) and dS0, all float32. seg: tokens
    between state checkpoints (0: default). workspace: optional uint8 device tensor of
    at least scan_bwd_workspace_bytes(...) bytes; allocated when None."""
    B, T, H, d = x.shape
    m = c.shape[-1]
    _chk(x, "x", (B, T, H, d), _XQ)
    _chk(c, "c", (B, T, H, m))
    _chk(q, "q", (B, T, H, m), _XQ)
    _chk(mu, "mu", (B, T, H))
    _chk(S0, "S0", (B, H, m, d))
    _chk(dy, "dy", (B, T, H, d))
    if dS_T is not None:
        _chk(dS_T, "dS_T", (B, H, m, d))
    if eta is not None:
        _chk(eta, "eta", (B, T, H))
    L = lib()
    need = L.lattice_scan_bwd_workspace_bytes(B, T, H, m, d, int(chunk), int(seg))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous CUDA tensor")
    f32 = dict(dtype=torch.float32, device=x.device)
    out = {"dx": torch.empty((B, T, H, d), **f32), "dc": torch.empty((B, T, H, m), **f32),
           "dq": torch.empty((B, T, H, m), **f32), "dmu": torch.empty((B, T, H), **f32),
           "deta": None if eta is None else torch.empty((B, T, H), **f32),
           "dS0": torch.empty((B, H, m, d), **f32)}
    code = L.lattice_scan_bwd(_ptr(x), _dt(x), _ptr(c), _ptr(q), _dt(q), _ptr(mu), _ptr(eta),
                              _ptr(S0), _ptr(dy), _ptr(dS_T), _ptr(out["dx"]), _ptr(out["dc"]),
                              _ptr(out["dq"]), _ptr(out["dmu"]), _ptr(out["deta"]), _ptr(out["dS0"]),
                              _ptr(workspace), workspace.numel() * workspace.element_size(),
                              B, T, H, m, d, int(chunk), int(seg), _stream(stream))
    _raise(code, "lattice_scan_bwd")
    return out


def step(S: torch.Tensor, x: torch.Tensor, c: torch.Tensor, q: torch.Tensor, mu: torch.Tensor,
         eta: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
         stream=None, mode: str = "sim") -> torch.Tensor:
    """One decode step, state updated in place. S [B,H,m,d], x [B,H,d], c/q [B,H,m],
    mu/eta [B,H]. Returns y [B,H,d]."""
    B, H, m, d = S.shape
    _chk(S, "S", (B, H, m, d))
    _chk(x, "x", (B, H, d), _XQ)
    _chk(c, "c", (B, H, m))
    _chk(q, "q", (B, H, m), _XQ)
    _chk(mu, "mu", (B, H))
    if eta is not None:
        _chk(eta, "eta", (B, H))
    if y is None:
        y = torch.empty((B, H, d), dtype=torch.float32, device=S.device)
    _chk(y, "y", (B, H, d))
    code = lib().lattice_step(_ptr(S), _ptr(x), _dt(x), _ptr(c), _ptr(q), _dt(q), _ptr(mu),
                              _ptr(eta), _ptr(y), B, H, m, d, _MODE[mode], _stream(stream))
    _raise(code, "lattice_step")
    return y


def readout(S: torch.Tensor, q: torch.Tensor, y: Optional[torch.Tensor] = None,
            stream=None) -> torch.Tensor:
    """y[b,h,:] = sum_i q[b,h,i] S[b,h,i,:]."""
    B, H, m, d = S.shape
    _chk(S, "S", (B, H, m, d))
    _chk(q, "q", (B, H, m), _XQ)
    if y is None:
        y = torch.empty((B, H, d), dtype=torch.float32, device=S.device)
    _chk(y, "y", (B, H, d))
    code = lib().lattice_readout(_ptr(S), _ptr(q), _dt(q), _ptr(y), B, H, m, d, _stream(stream))
    _raise(code, "lattice_readout")
    return y


def chunk_impl(B: int, H: int, m: int, d: int, chunk: int, x_dtype=torch.bfloat16,
               q_dtype=torch.bfloat16) -> str:
    """Name of the kernel the automatic choice runs for a chunked scan of B x H sequences:
    "split_reg", "tcgen05_split", "tcgen05" or "simt"."""
    dt = lambda t: _BF16 if t == torch.bfloat16 else _F32
    code = lib().lattice_chunk_impl(B, H, m, d, chunk, dt(x_dtype), dt(q_dtype))
    return {1: "simt", 2: "tcgen05", 3: "tcgen05_split", 4: "split_reg", 5: "split_reg8"}[code]


def device_status(stream=None) -> int:
    """Synchronise the stream; raise LatticeError if a kernel gave up a bounded wait."""
    code = lib().lattice_get_device_status(_stream(stream))
    _raise(code, "lattice_get_device_status")
    return code


def selftest_bounded_wait(limit_ns: int = 1_000_000, stream=None) -> None:
    """Launch the library's bounded-wait self-test: one warp waits on a barrier that
    nothing completes and gives up after limit_ns. The next device_status() on the
    same stream then raises LatticeError with code ERR_TIMEOUT."""
    _raise(lib().lattice_selftest_bounded_wait(int(limit_ns), _stream(stream)),
           "lattice_selftest_bounded_wait")


# ---------------------------------------------------------------- gated recurrence

_DT = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_FLOATS = (torch.float32, torch.bfloat16, torch.float16)
_MARK = 16  # tokens between the states kept for the backward pass
_GATE = {"value": 0, "logit": 1}
_WRITE = {"plain": 0, "leaky": 1, "unit": 2}


def _rows(t, name: str, shape, lead: int, dtypes, device):
    """Checks a tensor whose first `lead` axes may be strided and whose other axes are
    contiguous; returns its strides (the first `lead` are the ones that matter)."""
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype in dtypes and t.device == device:
        strides = t.stride()
        if t.is_contiguous():
            return strides
        want = 1
        for k in range(len(shape) - 1, lead - 1, -1):
            if shape[k] != 1 and strides[k] != want:
                raise ValueError(f"{name} must be contiguous in its last {len(shape) - lead} axes")
            want *= shape[k]
        return strides
    return _like(t, name, shape, dtypes, device)


def _like(t, name: str, shape, dtypes, device):
    """Checks a tensor's place, type and shape."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _whole(t, name: str, shape, dtypes, device):
    """Checks a contiguous tensor; None passes."""
    if t is not None and not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype in dtypes
                              and t.device == device and t.is_contiguous()):
        _rows(t, name, shape, 0, dtypes, device)


# the current stream's handle without a Stream object (a few microseconds less per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _enter(device, stream):
    """(context, stream handle) of a call: on the tensors' device, its buffers allocated on the
    stream that the kernels use, so that memory freed after the call is reused in that
    stream's order. The context (or None) is entered; the caller leaves it."""
    if stream is None:
        if device.index == torch.cuda.current_device():
            return None, _raw_stream(device.index)
        ctx = torch.cuda.device(device)
        ctx.__enter__()
        return ctx, _raw_stream(device.index)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    ctx = torch.cuda.stream(stream)
    ctx.__enter__()
    return ctx, stream.cuda_stream


def _leave(ctx):
    if ctx is not None:
        ctx.__exit__(None, None, None)


def _new(t, dtype=None):
    """An empty contiguous tensor like t."""
    if t.is_contiguous() and (dtype is None or dtype == t.dtype):
        return torch.empty_like(t)
    return torch.empty(t.shape, dtype=dtype or t.dtype, device=t.device)


_F32_ONLY = (torch.float32,)
_XZ = {t: (t, torch.float32) for t in (torch.float32, torch.bfloat16, torch.float16)}


_INT_MAX = 0x7fffffff


def _fits(what: str, *sizes):
    """Refuses sizes that are no C int: ctypes would cut them off."""
    if max(sizes) > _INT_MAX:
        raise LatticeError(ERR_UNSUPPORTED, what)


def _gated_args(x, z, lead: int, lengths, gate: str, write: str):
    if not isinstance(x, torch.Tensor) or x.dim() != lead + 2:
        raise ValueError("x must be a tensor [B, T, H, d] (one token: [B, H, d])")
    shape, device = x.shape, x.device
    if x.numel() > _INT_MAX:
        _fits("the gated recurrence's sizes", *shape)
    xs = _rows(x, "x", shape, lead, _FLOATS, device) if x.is_cuda else _like(x, "x", shape, _FLOATS, device)
    per_head = isinstance(z, torch.Tensor) and z.dim() == lead + 1
    zs = _rows(z, "z", shape[:-1] if per_head else shape, lead, _XZ[x.dtype], device)
    if lengths is not None:
        _whole(lengths, "lengths", shape[:1], (torch.int32,), device)
    if gate not in _GATE or write not in _WRITE:
        raise ValueError(f"gate is one of {tuple(_GATE)}, write one of {tuple(_WRITE)}")
    return xs, zs, per_head


def gated_scan_marks(x: torch.Tensor) -> torch.Tensor:
    """An empty buffer for the states that gated_scan_fwd leaves for gated_scan_bwd: the
    state before every 16th token, [B, ceil(T/16), H, d] float32."""
    B, T, H, d = x.shape
    return torch.empty((B, (T + _MARK - 1) // _MARK, H, d), dtype=torch.float32, device=x.device)


def gated_scan_fwd(x: torch.Tensor, z: torch.Tensor, h0: Optional[torch.Tensor] = None, *, gate: str = "logit",
                   write: str = "leaky", tau: float = 1.0, lengths: Optional[torch.Tensor] = None,
                   marks: Optional[torch.Tensor] = None, h_out: Optional[torch.Tensor] = None,
                   y: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Gated linear recurrence h_t = a_t h_{t-1} + s(a_t) x_t over whole sequences, y_t = h_t.
    x [B,T,H,d]; z [B,T,H,d], or [B,T,H] for one gate per head (d 16, 32, 64 or 128); both may
    be slices of wider rows. z has x's dtype or float32. h0 [B,H,d] float32 or None (0).
    gate "logit": a = sigmoid(z)**tau; "value": a = z, |a| <= 1. write "plain": s = 1;
    "leaky": s = 1 - a; "unit": s = sqrt(1 - a*a). lengths int32 [B] or None (T): tokens behind
    a sequence's length are not read and their y is 0. marks: a buffer of gated_scan_marks to
    fill for gated_scan_bwd. h_out may be h0.
    Returns (y [B,T,H,d] in x's dtype, h_T [B,H,d] float32, the state at each length)."""
    xs, zs, per_head = _gated_args(x, z, 2, lengths, gate, write)
    shape, dev = x.shape, x.device
    B, T, H, d = shape
    state = (B, H, d)
    _whole(h0, "h0", state, _F32_ONLY, dev)
    _whole(marks, "marks", (B, (T + _MARK - 1) // _MARK, H, d), _F32_ONLY, dev)
    _whole(h_out, "h_out", state, _F32_ONLY, dev)
    _whole(y, "y", shape, (x.dtype,), dev)
    ctx, st = _enter(dev, stream)
    try:
        if h_out is None:
            h_out = torch.empty(state, dtype=torch.float32, device=dev) if h0 is None else torch.empty_like(h0)
        if y is None:
            y = _new(x)
        code = lib().lattice_gated_scan_fwd(
            x.data_ptr(), _DT[x.dtype], xs[0], xs[1], z.data_ptr(), _DT[z.dtype], zs[0], zs[1], per_head, _adr(h0),
            h_out.data_ptr(), y.data_ptr(), _adr(marks), _adr(lengths), B, T, H, d, _GATE[gate], _WRITE[write], tau, st)
    finally:
        _leave(ctx)
    if code:
        _raise(code, "lattice_gated_scan_fwd")
    return y, h_out


def gated_scan_bwd(x: torch.Tensor, z: torch.Tensor, dy: torch.Tensor, marks: torch.Tensor, *,
                   dh_T: Optional[torch.Tensor] = None, gate: str = "logit", write: str = "leaky", tau: float = 1.0,
                   lengths: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Backward pass of gated_scan_fwd: gradients of L = sum_t dy_t . y_t + dh_T . h_T. x, z,
    the forms, lengths and the filled marks are those of the forward call; dy has x's dtype
    and may be strided as x. Returns a dict with dx (x's dtype), dz (z's dtype and shape) and
    dh0 (float32); gradients of tokens behind a sequence's length are 0."""
    xs, zs, per_head = _gated_args(x, z, 2, lengths, gate, write)
    shape, dev = x.shape, x.device
    B, T, H, d = shape
    dys = _rows(dy, "dy", shape, 2, (x.dtype,), dev)
    _rows(marks, "marks", (B, (T + _MARK - 1) // _MARK, H, d), 0, _F32_ONLY, dev)
    _whole(dh_T, "dh_T", (B, H, d), _F32_ONLY, dev)
    ctx, st = _enter(dev, stream)
    try:
        dx, dz = _new(x), _new(z)
        dh0 = torch.empty((B, H, d), dtype=torch.float32, device=dev)
        code = lib().lattice_gated_scan_bwd(
            x.data_ptr(), _DT[x.dtype], xs[0], xs[1], z.data_ptr(), _DT[z.dtype], zs[0], zs[1], per_head, dy.data_ptr(),
            dys[0], dys[1], marks.data_ptr(), _adr(dh_T), dx.data_ptr(), dz.data_ptr(), dh0.data_ptr(), _adr(lengths),
            B, T, H, d, _GATE[gate], _WRITE[write], tau, st)
    finally:
        _leave(ctx)
    if code:
        _raise(code, "lattice_gated_scan_bwd")
    return {"dx": dx, "dz": dz, "dh0": dh0}


def gated_step(h: torch.Tensor, x: torch.Tensor, z: torch.Tensor, *, gate: str = "logit", write: str = "leaky",
               tau: float = 1.0, h_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """One token of the gated recurrence: h [B,H,d] float32, x [B,H,d], z [B,H,d] or [B,H].
    The state is updated in place, or written to h_out. Returns y [B,H,d] in x's dtype."""
    xs, zs, per_head = _gated_args(x, z, 1, None, gate, write)
    shape, dev = x.shape, x.device
    B, H, d = shape
    if h_out is None:
        h_out = h
    else:
        _whole(h_out, "h_out", shape, _F32_ONLY, dev)
    _rows(h, "h", shape, 0, _F32_ONLY, dev)
    _whole(y, "y", shape, (x.dtype,), dev)
    ctx, st = _enter(dev, stream)
    try:
        if y is None:
            y = _new(x)
        code = lib().lattice_gated_step(
            h.data_ptr(), h_out.data_ptr(), x.data_ptr(), _DT[x.dtype], xs[0], z.data_ptr(), _DT[z.dtype], zs[0], per_head,
            y.data_ptr(), B, H, d, _GATE[gate], _WRITE[write], tau, st)
    finally:
        _leave(ctx)
    if code:
        _raise(code, "lattice_gated_step")
    return y


# ---------------------------------------------------------------- block norms

_ACT = {"none": 0, "sigmoid": 1, "silu": 2, "gelu": 3}


def _groups(tensors, shape):
    """(G, strides): rows in groups of G, contiguous within a group, for every (name, tensor)
    of `shape` (None: stride 0), with the stride between groups."""
    D, lead = shape[-1], shape[:-1]
    for _, t in tensors:
        if t is not None and not t.is_contiguous():
            break
    else:
        return 1, (D,) * len(tensors)
    for G, outer in ((1, lead), (lead[-1] if lead else 1, lead[:-1])):
        strides = []
        for _, t in tensors:
            if t is None:
                strides.append(0)
                continue
            st = t.stride()
            ok = D == 1 or st[-1] == 1
            if G > 1:
                ok = ok and st[-2] == D
            s, width = None, 1  # the outer axes collapse into one, of stride s
            for n, k in zip(reversed(outer), reversed(st[:len(outer)])):
                if n != 1:
                    if s is None:
                        s = k
                    ok = ok and k == s * width
                    width *= n
            strides.append(G * D if s is None else s)
            if not ok:
                break
        else:
            return G, strides
    names = ", ".join(k for k, t in tensors if t is not None)
    raise ValueError(f"the rows of {names} must be contiguous, with one stride between rows, or between the groups of rows "
                     "that the last axis but one makes")


def _norm_args(y, w_post, gate, residual, w_pre, act, dtype):
    if not isinstance(y, torch.Tensor) or not y.is_cuda or y.dim() < 1:
        raise TypeError("y must be a CUDA tensor [..., D]")
    shape, dev = y.shape, y.device
    if y.numel() > _INT_MAX:
        _fits("the norm's sizes", *shape[-2:])
    if dtype is None:
        dtype = gate.dtype if isinstance(gate, torch.Tensor) else y.dtype
    both = _XZ.get(dtype)
    if both is None:
        raise TypeError(f"the output dtype must be one of {_FLOATS}, got {dtype}")
    if y.dtype not in both:
        _like(y, "y", shape, both, dev)
    if gate is not None:
        _like(gate, "gate", shape, (dtype,), dev)
    if residual is not None:
        _like(residual, "residual", shape, both, dev)
    w_dtype = torch.float32
    if w_post is not None:
        _whole(w_post, "w_post", shape[-1:], both, dev)
        w_dtype = w_post.dtype
    if w_pre is not None:
        _whole(w_pre, "w_pre", shape[-1:], both, dev)
        if w_post is not None and w_dtype != w_pre.dtype:
            raise TypeError("w_post and w_pre must have the same dtype")
        w_dtype = w_pre.dtype
    if act not in _ACT:
        raise ValueError(f"act is one of {tuple(_ACT)}")
    return shape, dev, dtype, w_dtype


def block_norm_fwd(y: torch.Tensor, w_post: Optional[torch.Tensor] = None, *, gate: Optional[torch.Tensor] = None,
                   act: str = "gelu", residual: Optional[torch.Tensor] = None, w_pre: Optional[torch.Tensor] = None,
                   pre_norm: Optional[bool] = None, post_norm: bool = True, scale: float = 1.0, eps: float = 1e-6,
                   out_dtype: Optional[torch.dtype] = None, r_out: Optional[torch.Tensor] = None,
                   n_out: Optional[torch.Tensor] = None, stream=None):
    """The norm after a block with its gate and residual scale, and the norm before the next:
    per row of the last axis u = y / sqrt(mean(y^2) + eps) (u = y without post_norm),
    r = residual + scale * u * w_post * act(gate), n = r / sqrt(mean(r^2) + eps) * w_pre.
    y [..., D]; gate, residual of y's shape or None; weights [D] or None (1). n is formed with
    w_pre, or with pre_norm=True. act: "sigmoid", "silu" or "gelu". Dtypes: out_dtype (default:
    the gate's, else y's) is that of the gate, of n, and of r without a residual; y, the
    residual, whose dtype r then has, and the weights are of it or float32. Inputs may be
    slices of wider rows. r_out may be the residual. Returns (r, n), n None if not formed."""
    shape, dev, dtype, w_dtype = _norm_args(y, w_post, gate, residual, w_pre, act, out_dtype)
    if pre_norm is None:
        pre_norm = w_pre is not None or n_out is not None
    elif not pre_norm and (w_pre is not None or n_out is not None):
        raise ValueError("w_pre and n_out need pre_norm")
    r_dtype = dtype if residual is None else residual.dtype
    _whole(r_out, "r_out", shape, (r_dtype,), dev)
    _whole(n_out, "n_out", shape, (dtype,), dev)
    D = shape[-1]
    N = y.numel() // D if D else 0
    G, gs = _groups((("y", y), ("gate", gate), ("residual", residual)), shape)
    ctx, st = _enter(dev, stream)
    try:
        if r_out is None:
            r_out = _new(y if residual is None else residual, r_dtype)
        if n_out is None and pre_norm:
            n_out = _new(y, dtype)
        code = lib().lattice_block_norm_fwd(
            y.data_ptr(), _DT[y.dtype], gs[0], _adr(gate), gs[1], _adr(residual), _DT[r_dtype], gs[2], _adr(w_post),
            _adr(w_pre), _DT[w_dtype], r_out.data_ptr(), _adr(n_out), _DT[dtype], N, G, D, _ACT[act], post_norm, scale,
            eps, st)
    finally:
        _leave(ctx)
    if code:
        _raise(code, "lattice_block_norm_fwd")
    return r_out, n_out


def block_norm_bwd(y: torch.Tensor, w_post: Optional[torch.Tensor] = None, *, dr: Optional[torch.Tensor] = None,
                   dn: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, act: str = "gelu",
                   residual: Optional[torch.Tensor] = None, w_pre: Optional[torch.Tensor] = None, post_norm: bool = True,
                   scale: float = 1.0, eps: float = 1e-6, workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Backward pass of block_norm_fwd from its inputs: gradients of L = sum(dr * r) + sum(dn * n).
    dr: cotangent of r (with a residual in its dtype, else in the call's or float32) or None
    (0); dn: cotangent of n or None (n was not formed). The call's dtype is dn's, else the
    gate's, else dr's. Returns a dict with dy, dgate, dresidual (their input's dtype, None
    without one) and dw_post, dw_pre (float32, None without the weight). workspace: optional
    contiguous uint8 tensor for the weights' gradients; allocated when None. The gradient of a
    learned scale is (dw_post * w_post).sum() / scale."""
    dtype = next((t.dtype for t in (dn, gate, dr) if isinstance(t, torch.Tensor)), None)
    if dtype is None:
        raise ValueError("one of dr and dn is needed")
    if dn is None and gate is None and dtype == torch.float32:  # r in float32 says nothing about the call's dtype
        dtype = next((t.dtype for t in (y, residual, w_post) if isinstance(t, torch.Tensor) and t.dtype != dtype), dtype)
    shape, dev, dtype, w_dtype = _norm_args(y, w_post, gate, residual, w_pre, act, dtype)
    if w_pre is not None and dn is None:
        raise ValueError("w_pre needs dn")
    if dr is not None:
        _like(dr, "dr", shape, (residual.dtype,) if residual is not None else (dtype, torch.float32), dev)
    if dn is not None:
        _like(dn, "dn", shape, (dtype,), dev)
    D = shape[-1]
    N = y.numel() // D if D else 0
    G, gs = _groups((("y", y), ("gate", gate), ("residual", residual), ("dr", dr), ("dn", dn)), shape)
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous() or workspace.device != dev:
            raise TypeError("workspace must be a contiguous tensor on the inputs' device")
    L = lib()
    ctx, st = _enter(dev, stream)
    try:
        dy = _new(y)
        dgate = None if gate is None else _new(gate)
        dresidual = None if residual is None else _new(residual)
        dw_post = None if w_post is None else _new(w_post, torch.float32)
        dw_pre = None if w_pre is None else _new(w_pre, torch.float32)
        bytes_ = 0
        if w_post is not None or w_pre is not None:
            if workspace is None:
                workspace = torch.empty(L.lattice_block_norm_bwd_workspace_bytes(N, D), dtype=torch.uint8, device=dev)
            bytes_ = workspace.numel() * workspace.element_size()
        code = L.lattice_block_norm_bwd(
            y.data_ptr(), _DT[y.dtype], gs[0], _adr(gate), gs[1], _adr(residual),
            0 if residual is None else _DT[residual.dtype], gs[2], _adr(w_post), _adr(w_pre), _DT[w_dtype], _adr(dr),
            0 if dr is None else _DT[dr.dtype], gs[3], _adr(dn), gs[4], dy.data_ptr(), _adr(dgate), _adr(dresidual),
            _adr(dw_post), _adr(dw_pre), _adr(workspace), bytes_, _DT[dtype], N, G, D, _ACT[act], post_norm, scale, eps, st)
    finally:
        _leave(ctx)
    if code:
        _raise(code, "lattice_block_norm_bwd")
    return {"dy": dy, "dgate": dgate, "dresidual": dresidual, "dw_post": dw_post, "dw_pre": dw_pre}
