"""Thin ctypes binding of libgdn.so (argument marshalling only).

Every step of the computation runs in the library's CUDA kernels; this module
only turns torch tensors into pointers, allocates outputs and the workspace on
the caller's behalf (torch owns that memory), and raises on a non-OK status.
The library must have been built (``build.py``); there is no fallback.

The function names follow the C ABI in include/gdn.h, gdn_conv.h and gdn_layer.h.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

GDN_OK = 0
GDN_DTYPE_F32 = 0
GDN_DTYPE_BF16 = 1

_STATUS = {0: "GDN_OK", 1: "GDN_ERR_INVALID_ARG", 2: "GDN_ERR_UNSUPPORTED",
           3: "GDN_ERR_WORKSPACE", 4: "GDN_ERR_CUDA", 5: "GDN_ERR_TIMEOUT"}

EXPORTS = ["gdn_chunk_workspace_bytes", "gdn_chunk_fwd", "gdn_chunk_bwd",
           "gdn_varlen_workspace_bytes", "gdn_varlen_fwd", "gdn_varlen_bwd",
           "gdn_status_str", "gdn_workspace_status", "gdn_path", "gdn_version",
           "gdn_chunk_fwd_noalloc", "gdn_chunk_saved_bytes", "gdn_chunk_fwd_save",
           "gdn_chunk_bwd_saved", "gdn_noalloc_status"]
GDN_WS_SAVED = 2
# include/gdn_conv.h
CONV_EXPORTS = ["gdn_conv_workspace_bytes", "gdn_conv_fwd", "gdn_conv_bwd"]
CONV_ACT = {"none": 0, "silu": 1}
# include/gdn_layer.h
LAYER_EXPORTS = ["gdn_step", "gdn_conv_step", "gdn_prep_fwd", "gdn_prep_bwd",
                 "gdn_prep_workspace_bytes", "gdn_gate_norm_fwd", "gdn_gate_norm_bwd",
                 "gdn_gate_norm_workspace_bytes", "gdn_res_norm_fwd", "gdn_res_norm_bwd",
                 "gdn_res_norm_workspace_bytes"]
GATE_ACT = {"silu": 1, "sigmoid": 2}


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {_STATUS.get(status, status)}")
        self.status = status


class gdn_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("dtype", ctypes.c_int)]


class gdn_conv_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("C", ctypes.c_int),
                ("W", ctypes.c_int), ("dtype", ctypes.c_int), ("act", ctypes.c_int)]


_I, _L, _F = ctypes.c_int, ctypes.c_longlong, ctypes.c_float


class gdn_step_shape(ctypes.Structure):
    _fields_ = [("N", _I), ("n_tok", _I), ("n_slots", _I), ("H", _I), ("Hk", _I), ("dk", _I),
                ("dv", _I), ("dtype", _I), ("ldq", _L), ("ldk", _L), ("ldv", _L), ("ldg", _L),
                ("ldb", _L), ("q_scale", _F), ("eps", _F)]


class gdn_conv_step_shape(ctypes.Structure):
    _fields_ = [("N", _I), ("n_tok", _I), ("n_slots", _I), ("C", _I), ("W", _I), ("dtype", _I),
                ("act", _I), ("ldx", _L)]


class gdn_prep_shape(ctypes.Structure):
    _fields_ = [("rows", _I), ("H", _I), ("Hk", _I), ("dk", _I), ("dtype", _I), ("ldq", _L),
                ("ldk", _L), ("ldg", _L), ("ldb", _L), ("q_scale", _F), ("eps", _F)]


class gdn_gate_norm_shape(ctypes.Structure):
    _fields_ = [("rows", _I), ("H", _I), ("d", _I), ("dtype", _I), ("act", _I), ("ldz", _L),
                ("eps", _F)]


class gdn_res_norm_shape(ctypes.Structure):
    _fields_ = [("rows", _I), ("C", _I), ("dtype", _I), ("res_dtype", _I), ("eps", _F)]


_lib = None


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False):
    """Load libgdn.so. Raises if it is missing (no CPU fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB
    if not os.path.exists(path):
        if not build_if_missing:
            raise RuntimeError(f"libgdn.so not built ({path}); run "
                               "`python -m chunked_linear_recurrence_gated_gb300.build`")
        _build.build()
    lib = ctypes.CDLL(path)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    SP = ctypes.POINTER(gdn_shape)
    lib.gdn_chunk_workspace_bytes.argtypes = [SP, I]
    lib.gdn_chunk_workspace_bytes.restype = Z
    lib.gdn_varlen_workspace_bytes.argtypes = [SP, I, I]
    lib.gdn_varlen_workspace_bytes.restype = Z
    lib.gdn_chunk_fwd.argtypes = [SP] + [P] * 8 + [P, Z, P]
    lib.gdn_chunk_bwd.argtypes = [SP] + [P] * 14 + [P, Z, P]
    lib.gdn_varlen_fwd.argtypes = [SP, P, I] + [P] * 8 + [P, Z, P]
    lib.gdn_varlen_bwd.argtypes = [SP, P, I] + [P] * 14 + [P, Z, P]
    for f in (lib.gdn_chunk_fwd, lib.gdn_chunk_bwd, lib.gdn_varlen_fwd, lib.gdn_varlen_bwd):
        f.restype = I
    lib.gdn_status_str.argtypes = [I]
    lib.gdn_status_str.restype = ctypes.c_char_p
    lib.gdn_workspace_status.argtypes = [P, P]
    lib.gdn_workspace_status.restype = I
    lib.gdn_path.argtypes = [SP]
    lib.gdn_path.restype = I
    lib.gdn_version.argtypes = []
    lib.gdn_version.restype = I
    lib.gdn_chunk_fwd_noalloc.argtypes = [SP] + [P] * 8 + [P]
    lib.gdn_chunk_fwd_noalloc.restype = I
    lib.gdn_noalloc_status.argtypes = [P]
    lib.gdn_noalloc_status.restype = I
    lib.gdn_diag_wait_timeout_noalloc.argtypes = [I, P]
    lib.gdn_diag_wait_timeout_noalloc.restype = I
    lib.gdn_diag_set_fwd_split.argtypes = [I, I, I]
    lib.gdn_diag_set_fwd_split.restype = None
    lib.gdn_chunk_saved_bytes.argtypes = [SP]
    lib.gdn_chunk_saved_bytes.restype = Z
    lib.gdn_chunk_fwd_save.argtypes = [SP] + [P] * 8 + [P, Z, P, Z, P]
    lib.gdn_chunk_fwd_save.restype = I
    lib.gdn_chunk_bwd_saved.argtypes = [SP] + [P] * 14 + [P, Z, P, Z, P]
    lib.gdn_chunk_bwd_saved.restype = I
    CP = ctypes.POINTER(gdn_conv_shape)
    lib.gdn_conv_workspace_bytes.argtypes = [CP]
    lib.gdn_conv_workspace_bytes.restype = Z
    lib.gdn_conv_fwd.argtypes = [CP] + [P] * 6 + [P]
    lib.gdn_conv_fwd.restype = I
    lib.gdn_conv_bwd.argtypes = [CP] + [P] * 10 + [P, Z, P]
    lib.gdn_conv_bwd.restype = I
    for name, shape, nptr, ws in (("gdn_step", gdn_step_shape, 13, False),
                                  ("gdn_conv_step", gdn_conv_step_shape, 9, False),
                                  ("gdn_prep_fwd", gdn_prep_shape, 10, False),
                                  ("gdn_prep_bwd", gdn_prep_shape, 16, True),
                                  ("gdn_gate_norm_fwd", gdn_gate_norm_shape, 4, False),
                                  ("gdn_gate_norm_bwd", gdn_gate_norm_shape, 7, True),
                                  ("gdn_res_norm_fwd", gdn_res_norm_shape, 7, False),
                                  ("gdn_res_norm_bwd", gdn_res_norm_shape, 12, True)):
        f = getattr(lib, name)
        f.argtypes = [ctypes.POINTER(shape)] + [P] * nptr + ([P, Z, P] if ws else [P])
        f.restype = I
    for name, shape in (("prep", gdn_prep_shape), ("gate_norm", gdn_gate_norm_shape),
                        ("res_norm", gdn_res_norm_shape)):
        f = getattr(lib, f"gdn_{name}_workspace_bytes")
        f.argtypes = [ctypes.POINTER(shape)]
        f.restype = Z
    lib.gdn_profile_arm.argtypes = [P, I]
    lib.gdn_profile_arm.restype = None
    lib.gdn_profile_count.argtypes = []
    lib.gdn_profile_count.restype = I
    lib.gdn_diag_wait_timeout.argtypes = [P, I, P]
    lib.gdn_diag_wait_timeout.restype = I
    lib.gdn_profile_name.argtypes = [I]
    lib.gdn_profile_name.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return GDN_DTYPE_F32
    if t.dtype == torch.bfloat16:
        return GDN_DTYPE_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _p(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def shape_of(q: torch.Tensor, v: torch.Tensor) -> gdn_shape:
    B, T, H, dk = q.shape
    return gdn_shape(B, T, H, dk, v.shape[-1], _dtype_code(q))


def path(q, v) -> int:
    s = shape_of(q, v)
    return load().gdn_path(ctypes.byref(s))


def chunk_workspace_bytes(shape: gdn_shape, is_bwd: bool) -> int:
    return load().gdn_chunk_workspace_bytes(ctypes.byref(shape), int(is_bwd))


def varlen_workspace_bytes(shape: gdn_shape, nseq: int, is_bwd: bool) -> int:
    return load().gdn_varlen_workspace_bytes(ctypes.byref(shape), nseq, int(is_bwd))


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _check(rc: int, where: str):
    if rc != GDN_OK:
        raise GdnError(rc, where)


def gdn_chunk_fwd(q, k, v, g, beta, S_in=None, o=None, S_out=None, workspace=None,
                  stream=None, want_state=True):
    """Forward of one chunk. Returns (o, S_out)."""
    lib = load()
    s = shape_of(q, v)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty(B, T, H, dv, dtype=q.dtype, device=q.device)
    if S_out is None and want_state:
        S_out = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    need = lib.gdn_chunk_workspace_bytes(ctypes.byref(s), 0)
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    rc = lib.gdn_chunk_fwd(ctypes.byref(s), _p(q), _p(k), _p(v), _p(g), _p(beta), _p(S_in),
                           _p(o), _p(S_out), _p(workspace), workspace.numel(), _stream(stream))
    _check(rc, "gdn_chunk_fwd")
    return o, S_out


def gdn_chunk_bwd(q, k, v, g, beta, S_in, dout, dS_out=None, grads=None, dS_in=None,
                  workspace=None, stream=None, want_state=True):
    """Backward of one chunk. Returns (dq, dk, dv, dg, dbeta, dS_in)."""
    lib = load()
    s = shape_of(q, v)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if grads is None:
        grads = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v),
                 torch.empty_like(g), torch.empty_like(beta))
    if dS_in is None and want_state:
        dS_in = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    need = lib.gdn_chunk_workspace_bytes(ctypes.byref(s), 1)
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    rc = lib.gdn_chunk_bwd(ctypes.byref(s), _p(q), _p(k), _p(v), _p(g), _p(beta), _p(S_in),
                           _p(dout), _p(dS_out), *[_p(t) for t in grads], _p(dS_in),
                           _p(workspace), workspace.numel(), _stream(stream))
    _check(rc, "gdn_chunk_bwd")
    return (*grads, dS_in)


def chunk_saved_bytes(shape: gdn_shape) -> int:
    return load().gdn_chunk_saved_bytes(ctypes.byref(shape))


def gdn_chunk_fwd_save(q, k, v, g, beta, S_in=None, saved=None, o=None, S_out=None,
                       workspace=None, stream=None, want_state=True):
    """Forward of one chunk that keeps its per-block products for
    gdn_chunk_bwd_saved. Returns (o, S_out, saved)."""
    lib = load()
    s = shape_of(q, v)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty(B, T, H, dv, dtype=q.dtype, device=q.device)
    if S_out is None and want_state:
        S_out = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    if saved is None:
        saved = alloc_workspace(lib.gdn_chunk_saved_bytes(ctypes.byref(s)), q.device)
    if workspace is None:
        workspace = alloc_workspace(lib.gdn_chunk_workspace_bytes(ctypes.byref(s), GDN_WS_SAVED),
                                    q.device)
    rc = lib.gdn_chunk_fwd_save(ctypes.byref(s), _p(q), _p(k), _p(v), _p(g), _p(beta), _p(S_in),
                                _p(o), _p(S_out), _p(saved), saved.numel(), _p(workspace),
                                workspace.numel(), _stream(stream))
    _check(rc, "gdn_chunk_fwd_save")
    return o, S_out, saved


def gdn_chunk_bwd_saved(q, k, v, g, beta, S_in, dout, saved, dS_out=None, grads=None,
                        dS_in=None, workspace=None, stream=None, want_state=True):
    """Backward of one chunk from the products gdn_chunk_fwd_save kept.
    Returns (dq, dk, dv, dg, dbeta, dS_in)."""
    lib = load()
    s = shape_of(q, v)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if grads is None:
        grads = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v),
                 torch.empty_like(g), torch.empty_like(beta))
    if dS_in is None and want_state:
        dS_in = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(lib.gdn_chunk_workspace_bytes(ctypes.byref(s), GDN_WS_SAVED),
                                    q.device)
    rc = lib.gdn_chunk_bwd_saved(ctypes.byref(s), _p(q), _p(k), _p(v), _p(g), _p(beta),
                                 _p(S_in), _p(dout), _p(dS_out), *[_p(t) for t in grads],
                                 _p(dS_in), _p(saved), saved.numel(), _p(workspace),
                                 workspace.numel(), _stream(stream))
    _check(rc, "gdn_chunk_bwd_saved")
    return (*grads, dS_in)


def gdn_varlen_fwd(cu_seqlens, q, k, v, g, beta, S0=None, o=None, S_final=None,
                   workspace=None, stream=None):
    """Packed varlen forward (q: [1, T, H, dk]). Returns (o, S_final [nseq, H, dk, dv])."""
    lib = load()
    s = shape_of(q, v)
    _, T, H, dk = q.shape
    dv = v.shape[-1]
    nseq = cu_seqlens.numel() - 1
    if o is None:
        o = torch.empty(1, T, H, dv, dtype=q.dtype, device=q.device)
    if S_final is None:
        S_final = torch.empty(nseq, H, dk, dv, dtype=torch.float32, device=q.device)
    need = lib.gdn_varlen_workspace_bytes(ctypes.byref(s), nseq, 0)
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    rc = lib.gdn_varlen_fwd(ctypes.byref(s), _p(cu_seqlens), nseq, _p(q), _p(k), _p(v), _p(g),
                            _p(beta), _p(S0), _p(o), _p(S_final), _p(workspace),
                            workspace.numel(), _stream(stream))
    _check(rc, "gdn_varlen_fwd")
    return o, S_final


def gdn_varlen_bwd(cu_seqlens, q, k, v, g, beta, S0, dout, dS_final=None, grads=None,
                   dS0=None, workspace=None, stream=None):
    """Packed varlen backward. Returns (dq, dk, dv, dg, dbeta, dS0)."""
    lib = load()
    s = shape_of(q, v)
    _, T, H, dk = q.shape
    dv = v.shape[-1]
    nseq = cu_seqlens.numel() - 1
    if grads is None:
        grads = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v),
                 torch.empty_like(g), torch.empty_like(beta))
    if dS0 is None:
        dS0 = torch.empty(nseq, H, dk, dv, dtype=torch.float32, device=q.device)
    need = lib.gdn_varlen_workspace_bytes(ctypes.byref(s), nseq, 1)
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    rc = lib.gdn_varlen_bwd(ctypes.byref(s), _p(cu_seqlens), nseq, _p(q), _p(k), _p(v), _p(g),
                            _p(beta), _p(S0), _p(dout), _p(dS_final), *[_p(t) for t in grads],
                            _p(dS0), _p(workspace), workspace.numel(), _stream(stream))
    _check(rc, "gdn_varlen_bwd")
    return (*grads, dS0)


def conv_shape_of(x: torch.Tensor, w: torch.Tensor, act: str) -> gdn_conv_shape:
    B, T, C = x.shape
    return gdn_conv_shape(B, T, C, w.shape[1], _dtype_code(x), CONV_ACT[act])


def gdn_conv_fwd(x, w, b=None, state_in=None, act="silu", y=None, state_out=None,
                 want_state=True, stream=None):
    """Causal short convolution of one chunk, x [B, T, C]. Returns (y, state_out [B, W-1, C])."""
    lib = load()
    s = conv_shape_of(x, w, act)
    B, T, C = x.shape
    if y is None:
        y = torch.empty_like(x)
    if state_out is None and want_state:
        state_out = torch.empty(B, w.shape[1] - 1, C, dtype=x.dtype, device=x.device)
    rc = lib.gdn_conv_fwd(ctypes.byref(s), _p(x), _p(w), _p(b), _p(state_in), _p(y),
                          _p(state_out), _stream(stream))
    _check(rc, "gdn_conv_fwd")
    return y, state_out


def gdn_conv_bwd(x, w, b, state_in, dy, dstate_out=None, act="silu", dx=None, dw=None,
                 db=None, dstate_in=None, workspace=None, stream=None, want_state=True):
    """Backward of one chunk. Returns (dx, dw, db, dstate_in)."""
    lib = load()
    s = conv_shape_of(x, w, act)
    B, T, C = x.shape
    if dx is None:
        dx = torch.empty_like(x)
    if dw is None:
        dw = torch.empty_like(w)
    if db is None and b is not None:
        db = torch.empty_like(b)
    if dstate_in is None and want_state:
        dstate_in = torch.empty(B, w.shape[1] - 1, C, dtype=x.dtype, device=x.device)
    if workspace is None:
        workspace = alloc_workspace(lib.gdn_conv_workspace_bytes(ctypes.byref(s)), x.device)
    rc = lib.gdn_conv_bwd(ctypes.byref(s), _p(x), _p(w), _p(b), _p(state_in), _p(dy),
                          _p(dstate_out), _p(dx), _p(dw), _p(db), _p(dstate_in), _p(workspace),
                          workspace.numel(), _stream(stream))
    _check(rc, "gdn_conv_bwd")
    return dx, dw, db, dstate_in


# ------------------------------------------------- layer operators (include/gdn_layer.h)
# A generation step makes these calls once per layer and token, so what they do
# on the host is kept short: one condition over all arguments that holds for
# every well-formed call (plain attribute reads, no calls of our own), and the
# checks that name the offending argument only where it does not.
def _on_stream(fn, stream, *args, **kw):
    """fn with `stream` current, so that what it allocates (outputs, workspace)
    belongs to the stream its kernels run on."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def _raw_stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):  # the same value without a Stream object
    _raw_stream = torch._C._cuda_getCurrentRawStream  # noqa: F811

_f32, _i32 = torch.float32, torch.int32
_codes = {torch.float32: GDN_DTYPE_F32, torch.bfloat16: GDN_DTYPE_BF16}


def _code(dtype):
    code = _codes.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def _on_gpu(name, t, ndim):
    """Index of the GPU that holds t."""
    dev = t.get_device()
    if dev < 0 or t.dim() < ndim:
        raise ValueError(f"{name}: a CUDA tensor with {ndim} dimensions is expected, got "
                         f"{tuple(t.shape)} on {t.device}")
    return dev


def _want(name, t, shape, dtype, dev):
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype} on cuda:{dev}, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")


def _ptr(name, t, shape, dtype, dev):
    """Pointer of a contiguous tensor (None for an absent one)."""
    if t is None:
        return None
    if (t.shape != shape or t.dtype is not dtype or t.get_device() != dev
            or not t.is_contiguous()):
        _want(name, t, shape, dtype, dev)
        raise ValueError(f"{name}: must be contiguous, got strides {t.stride()}")
    return t.data_ptr()


def _rows(name, t, ndim):
    """Stride of the rows of t [..., n1, .., nk] (k = ndim trailing dimensions that
    have to be dense) when its leading dimensions flatten to one."""
    st, sh = t.stride(), t.shape
    inner = 1
    for i in range(1, ndim + 1):
        if sh[-i] != 1 and st[-i] != inner:
            raise ValueError(f"{name}: the last {ndim} dimensions must be dense")
        inner *= sh[-i]
    ld, n = inner, 1
    for i in range(len(sh) - ndim - 1, -1, -1):
        if sh[i] == 1:
            continue
        if n == 1:
            ld = st[i]
        elif st[i] != ld * n:
            raise ValueError(f"{name}: the rows must have one stride")
        n *= sh[i]
    return ld


def _cache_ptrs(N, dev, slot_in, slot_out, cu_seqlens, n_commit):
    """Pointers of the index arrays of gdn_step and gdn_conv_step."""
    return (None if slot_in is None else _ptr("slot_in", slot_in, (N,), _i32, dev),
            None if slot_out is None else _ptr("slot_out", slot_out, (N,), _i32, dev),
            None if cu_seqlens is None else _ptr("cu_seqlens", cu_seqlens, (N + 1,), _i32, dev),
            None if n_commit is None else _ptr("n_commit", n_commit, (N,), _i32, dev))


def _scratch(t, dev):
    """Pointer and bytes of a workspace."""
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on cuda:{dev}")
    return t.data_ptr(), t.nbytes


def gdn_step(q, k, v, g, beta, S, slot_in=None, slot_out=None, cu_seqlens=None, n_commit=None,
             gate=None, q_scale=1.0, eps=1e-6, o=None, stream=None):
    """The gated delta rule token by token over the states S [n_slots, H, dk, dv]
    (fp32, updated in place) of N sequences whose new tokens are packed:
    q, k [n_tok, Hk, dk], v [n_tok, H, dv], g, beta [n_tok, H], rows strided.

    cu_seqlens [N + 1]: the sequences' rows (None: one token each). slot_in /
    slot_out [N]: the slot a sequence's state is read from (-1: zero state) and
    written to (-1: nowhere); None: slot s for sequence s. n_commit [N]: the state
    after that many of its tokens is written (None: all). All int32 on the device.
    gate = (rate, bias) [H] fp32: g and beta are the inputs of gdn_prep_fwd's maps
    and q, k are normalised. Returns o [n_tok, H, dv]."""
    if stream is not None:
        return _on_stream(gdn_step, stream, q, k, v, g, beta, S, slot_in, slot_out, cu_seqlens,
                          n_commit, gate, q_scale, eps, o)
    dt, dev = q.dtype, q.get_device()
    n, Hk, dk = shape = q.shape
    _, H, dv = v.shape
    n_slots = S.shape[0]
    gates = (n, H)
    sq, sk, sv, sg, sb = q.stride(), k.stride(), v.stride(), g.stride(), beta.stride()
    if (dev >= 0 and k.shape == shape and v.shape[0] == n and g.shape == gates
            and beta.shape == gates and k.dtype is dt and v.dtype is dt and g.dtype is dt
            and beta.dtype is dt and k.get_device() == dev and v.get_device() == dev
            and g.get_device() == dev and beta.get_device() == dev
            and sq[2] == sk[2] == sv[2] == sg[1] == sb[1] == 1 and sq[1] == sk[1] == dk
            and sv[1] == dv):
        ldq, ldk, ldv, ldg, ldb = sq[0], sk[0], sv[0], sg[0], sb[0]
    else:
        _on_gpu("q", q, 3)
        for name, t, sh in (("k", k, shape), ("v", v, (n, H, dv)), ("g", g, gates),
                            ("beta", beta, gates)):
            _want(name, t, sh, dt, dev)
        ldq, ldk, ldv = _rows("q", q, 2), _rows("k", k, 2), _rows("v", v, 2)
        ldg, ldb = _rows("g", g, 1), _rows("beta", beta, 1)
    if o is None:
        o = torch.empty((n, H, dv), dtype=dt, device=q.device)
        po = o.data_ptr()
    else:
        po = _ptr("o", o, (n, H, dv), dt, dev)
    if gate is None:
        rate = bias = None
    else:
        rate, bias = _ptr("rate", gate[0], (H,), _f32, dev), _ptr("bias", gate[1], (H,), _f32, dev)
    N = n if cu_seqlens is None else cu_seqlens.shape[0] - 1
    rc = load().gdn_step(
        gdn_step_shape(N, n, n_slots, H, Hk, dk, dv, _code(dt), ldq, ldk, ldv, ldg, ldb, q_scale,
                       eps),
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), rate, bias,
        _ptr("S", S, (n_slots, H, dk, dv), _f32, dev),
        *_cache_ptrs(N, dev, slot_in, slot_out, cu_seqlens, n_commit), po, _raw_stream(dev))
    if rc:
        raise GdnError(rc, "gdn_step")
    return o


def gdn_conv_step(x, w, b, state, slot_in=None, slot_out=None, cu_seqlens=None, n_commit=None,
                  act="silu", y=None, stream=None):
    """The short convolution of packed new tokens x [n_tok, C] (rows strided) over
    the cached last inputs state [n_slots, W - 1, C] (updated in place), for the
    sequences of gdn_step. Returns y [n_tok, C]."""
    if stream is not None:
        return _on_stream(gdn_conv_step, stream, x, w, b, state, slot_in, slot_out, cu_seqlens,
                          n_commit, act, y)
    dt, dev = x.dtype, _on_gpu("x", x, 2)
    n, C = shape = x.shape
    W, n_slots = w.shape[1], state.shape[0]
    sx = x.stride()
    if y is None:
        y = torch.empty(shape, dtype=dt, device=x.device)
        py = y.data_ptr()
    else:
        py = _ptr("y", y, shape, dt, dev)
    N = n if cu_seqlens is None else cu_seqlens.shape[0] - 1
    rc = load().gdn_conv_step(
        gdn_conv_step_shape(N, n, n_slots, C, W, _code(dt), CONV_ACT[act],
                            sx[0] if sx[1] == 1 else _rows("x", x, 1)),
        x.data_ptr(), _ptr("w", w, (C, W), _f32, dev), _ptr("b", b, (C,), _f32, dev),
        _ptr("state", state, (n_slots, W - 1, C), dt, dev),
        *_cache_ptrs(N, dev, slot_in, slot_out, cu_seqlens, n_commit), py, _raw_stream(dev))
    if rc:
        raise GdnError(rc, "gdn_conv_step")
    return y


def _prep_shape_of(q, k, xg, xb, rate, bias, q_scale, eps):
    """(shape, GPU, pointers of the inputs) of gdn_prep_fwd and gdn_prep_bwd."""
    dt, dev = q.dtype, q.get_device()
    B, T, Hk, dk = shape = q.shape
    H = xg.shape[-1]
    gates = (B, T, H)
    sq, sk, sg, sb = q.stride(), k.stride(), xg.stride(), xb.stride()
    if (dev >= 0 and B == 1 and k.shape == shape and xg.shape == gates and xb.shape == gates
            and k.dtype is dt and xg.dtype is dt and xb.dtype is dt and k.get_device() == dev
            and xg.get_device() == dev and xb.get_device() == dev
            and sq[3] == sk[3] == sg[2] == sb[2] == 1 and sq[2] == sk[2] == dk):
        ldq, ldk, ldg, ldb = sq[1], sk[1], sg[1], sb[1]
    else:
        _on_gpu("q", q, 4)
        _want("k", k, shape, dt, dev)
        _want("xg", xg, gates, dt, dev)
        _want("xb", xb, gates, dt, dev)
        ldq, ldk, ldg, ldb = (_rows("q", q, 2), _rows("k", k, 2), _rows("xg", xg, 1),
                              _rows("xb", xb, 1))
    return (gdn_prep_shape(B * T, H, Hk, dk, _code(dt), ldq, ldk, ldg, ldb, q_scale, eps), dev,
            (q.data_ptr(), k.data_ptr(), xg.data_ptr(), xb.data_ptr(),
             _ptr("rate", rate, (H,), _f32, dev), _ptr("bias", bias, (H,), _f32, dev)))


def gdn_prep_fwd(q, k, xg, xb, rate, bias, q_scale=1.0, eps=1e-6, stream=None):
    """The maps before the recurrence. q, k [B, T, Hk, dk] and xg, xb [B, T, H] (rows
    strided), rate, bias [H] fp32. Returns (q, k [B, T, H, dk], g, beta [B, T, H]) as
    gdn_chunk_fwd takes them: q and k of unit norm (q times q_scale), each key
    head repeated for its H / Hk value heads, g = -exp(rate) softplus(xg + bias),
    beta = sigmoid(xb)."""
    if stream is not None:
        return _on_stream(gdn_prep_fwd, stream, q, k, xg, xb, rate, bias, q_scale, eps)
    s, dev, ins = _prep_shape_of(q, k, xg, xb, rate, bias, q_scale, eps)
    B, T, _, dk = q.shape
    dt, at = q.dtype, q.device
    heads, gates = (B, T, s.H, dk), (B, T, s.H)
    qn = torch.empty(heads, dtype=dt, device=at)
    kn = torch.empty(heads, dtype=dt, device=at)
    g = torch.empty(gates, dtype=dt, device=at)
    beta = torch.empty(gates, dtype=dt, device=at)
    rc = load().gdn_prep_fwd(s, *ins, qn.data_ptr(), kn.data_ptr(), g.data_ptr(),
                             beta.data_ptr(), _raw_stream(dev))
    if rc:
        raise GdnError(rc, "gdn_prep_fwd")
    return qn, kn, g, beta


def gdn_prep_bwd(q, k, xg, xb, rate, bias, dq, dk, dg, dbeta, q_scale=1.0, eps=1e-6,
                 workspace=None, stream=None):
    """Gradients of gdn_prep_fwd from those of its outputs, as gdn_chunk_bwd
    returns them. Returns (dq, dk [B, T, Hk, dk], dxg, dxb [B, T, H], drate, dbias [H])."""
    if stream is not None:
        return _on_stream(gdn_prep_bwd, stream, q, k, xg, xb, rate, bias, dq, dk, dg, dbeta,
                          q_scale, eps, workspace)
    lib = load()
    s, dev, ins = _prep_shape_of(q, k, xg, xb, rate, bias, q_scale, eps)
    B, T, _, D = shape = q.shape
    H, dt, at = s.H, q.dtype, q.device
    heads, gates = (B, T, H, D), (B, T, H)
    if workspace is None:
        workspace = alloc_workspace(lib.gdn_prep_workspace_bytes(s), at)
    oq = torch.empty(shape, dtype=dt, device=at)
    ok = torch.empty(shape, dtype=dt, device=at)
    og = torch.empty(gates, dtype=dt, device=at)
    ob = torch.empty(gates, dtype=dt, device=at)
    drate = torch.empty(H, dtype=_f32, device=at)
    dbias = torch.empty(H, dtype=_f32, device=at)
    rc = lib.gdn_prep_bwd(s, *ins, _ptr("dq", dq, heads, dt, dev), _ptr("dk", dk, heads, dt, dev),
                          _ptr("dg", dg, gates, dt, dev), _ptr("dbeta", dbeta, gates, dt, dev),
                          oq.data_ptr(), ok.data_ptr(), og.data_ptr(), ob.data_ptr(),
                          drate.data_ptr(), dbias.data_ptr(), *_scratch(workspace, dev),
                          _raw_stream(dev))
    if rc:
        raise GdnError(rc, "gdn_prep_bwd")
    return oq, ok, og, ob, drate, dbias


def _gate_norm_shape_of(o, z, w, act, eps):
    """(shape, GPU, pointers of the inputs) of gdn_gate_norm_fwd and gdn_gate_norm_bwd."""
    dt, dev = o.dtype, _on_gpu("o", o, 4)
    B, T, H, d = shape = o.shape
    sz = z.stride()
    if (B == 1 and z.shape == shape and z.dtype is dt and z.get_device() == dev and sz[3] == 1
            and sz[2] == d):
        ldz = sz[1]
    else:
        _want("z", z, shape, dt, dev)
        ldz = _rows("z", z, 2)
    return (gdn_gate_norm_shape(B * T, H, d, _code(dt), GATE_ACT[act], ldz, eps), dev,
            (_ptr("o", o, shape, dt, dev), z.data_ptr(), _ptr("w", w, (d,), _f32, dev)))


def gdn_gate_norm_fwd(o, z, w, act="silu", eps=1e-6, y=None, stream=None):
    """y = rms_norm(o) * w * act(z) over the last dimension of o [B, T, H, d]; z [B, T, H, d]
    with strided token rows, w [d] fp32, act "silu" or "sigmoid"."""
    if stream is not None:
        return _on_stream(gdn_gate_norm_fwd, stream, o, z, w, act, eps, y)
    s, dev, ins = _gate_norm_shape_of(o, z, w, act, eps)
    if y is None:
        y = torch.empty_like(o)
    rc = load().gdn_gate_norm_fwd(s, *ins, _ptr("y", y, o.shape, o.dtype, dev), _raw_stream(dev))
    if rc:
        raise GdnError(rc, "gdn_gate_norm_fwd")
    return y


def gdn_gate_norm_bwd(o, z, w, dy, act="silu", eps=1e-6, workspace=None, stream=None):
    """Backward of gdn_gate_norm_fwd. Returns (do, dz, dw)."""
    if stream is not None:
        return _on_stream(gdn_gate_norm_bwd, stream, o, z, w, dy, act, eps, workspace)
    lib = load()
    s, dev, ins = _gate_norm_shape_of(o, z, w, act, eps)
    if workspace is None:
        workspace = alloc_workspace(lib.gdn_gate_norm_workspace_bytes(s), o.device)
    do, dz, dw = torch.empty_like(o), torch.empty_like(o), torch.empty_like(w)
    rc = lib.gdn_gate_norm_bwd(s, *ins, _ptr("dy", dy, o.shape, o.dtype, dev), do.data_ptr(),
                               dz.data_ptr(), dw.data_ptr(), *_scratch(workspace, dev),
                               _raw_stream(dev))
    if rc:
        raise GdnError(rc, "gdn_gate_norm_bwd")
    return do, dz, dw


def gdn_res_norm_fwd(h, x, w, w_post=None, scale=None, eps=1e-6, h_out=None, y=None, dtype=None,
                     stream=None):
    """Block boundary: h_out = h + scale * (rms_norm(x) * w_post), y = rms_norm(h_out) * w.

    h [..., C] is the residual stream (fp32, or x's dtype), x [..., C] the block's
    output; w, w_post, scale [C] fp32. w_post None: x as it is; scale None: 1; x None
    (before the first block): y is the norm of h, in `dtype` (default h's).
    h_out may be h. Returns (h_out, y); h_out is None where x is."""
    if stream is not None:
        return _on_stream(gdn_res_norm_fwd, stream, h, x, w, w_post, scale, eps, h_out, y, dtype)
    rt, dev, shape = h.dtype, _on_gpu("h", h, 1), h.shape
    C = shape[-1]
    row = (C,)
    dt = x.dtype if x is not None else dtype or rt
    if y is None:
        y = torch.empty(shape, dtype=dt, device=h.device)
    if h_out is None and x is not None:
        h_out = torch.empty_like(h)
    rc = load().gdn_res_norm_fwd(
        gdn_res_norm_shape(h.numel() // max(C, 1), C, _code(dt), _code(rt), eps),
        _ptr("h", h, shape, rt, dev), _ptr("x", x, shape, dt, dev), _ptr("w", w, row, _f32, dev),
        _ptr("w_post", w_post, row, _f32, dev), _ptr("scale", scale, row, _f32, dev),
        _ptr("h_out", h_out, shape, rt, dev), _ptr("y", y, shape, dt, dev), _raw_stream(dev))
    if rc:
        raise GdnError(rc, "gdn_res_norm_fwd")
    return h_out, y


def gdn_res_norm_bwd(h_out, x, w, dy, dh_out=None, w_post=None, scale=None, eps=1e-6, dh=None,
                     workspace=None, stream=None):
    """Backward of gdn_res_norm_fwd at the residual it returned (for x None: at h).
    dh may be dh_out. Returns (dh, dx, dw, dw_post, dscale); dx is dh itself where
    they are equal (no w_post, no scale, one dtype)."""
    if stream is not None:
        return _on_stream(gdn_res_norm_bwd, stream, h_out, x, w, dy, dh_out, w_post, scale, eps,
                          dh, workspace)
    lib = load()
    rt, dt, dev, shape = h_out.dtype, dy.dtype, _on_gpu("h_out", h_out, 1), h_out.shape
    C = shape[-1]
    row = (C,)
    s = gdn_res_norm_shape(h_out.numel() // max(C, 1), C, _code(dt), _code(rt), eps)
    if workspace is None:
        workspace = alloc_workspace(lib.gdn_res_norm_workspace_bytes(s), h_out.device)
    if dh is None:
        dh = torch.empty_like(h_out)
    same = w_post is None and scale is None and (dt is rt or x is None)
    dx = None if same else torch.empty_like(dy)
    dw = torch.empty_like(w)
    dpost = None if w_post is None else torch.empty_like(w_post)
    dscale = None if scale is None else torch.empty_like(scale)
    rc = lib.gdn_res_norm_bwd(
        s, _ptr("h_out", h_out, shape, rt, dev), _ptr("x", x, shape, dt, dev),
        _ptr("w", w, row, _f32, dev), _ptr("w_post", w_post, row, _f32, dev),
        _ptr("scale", scale, row, _f32, dev), _ptr("dy", dy, shape, dt, dev),
        _ptr("dh_out", dh_out, shape, rt, dev), _ptr("dh", dh, shape, rt, dev),
        None if dx is None else dx.data_ptr(), dw.data_ptr(),
        None if dpost is None else dpost.data_ptr(),
        None if dscale is None else dscale.data_ptr(), *_scratch(workspace, dev),
        _raw_stream(dev))
    if rc:
        raise GdnError(rc, "gdn_res_norm_bwd")
    return dh, (dh if same else dx), dw, dpost, dscale


def gdn_workspace_status(workspace, stream=None) -> int:
    return load().gdn_workspace_status(_p(workspace), _stream(stream))


def diag_wait_timeout(workspace, limit_log2=20, stream=None) -> int:
    """Runs the bounded-wait self-check (include/gdn_profile.h); read the
    outcome with gdn_workspace_status."""
    return load().gdn_diag_wait_timeout(_p(workspace), limit_log2, _stream(stream))


def gdn_noalloc_status(stream=None) -> int:
    return load().gdn_noalloc_status(_stream(stream))


def diag_wait_timeout_noalloc(limit_log2=20, stream=None) -> int:
    """The bounded-wait self-check on the no-allocation forward's scratch;
    read the outcome with gdn_noalloc_status."""
    return load().gdn_diag_wait_timeout_noalloc(limit_log2, _stream(stream))


def set_fwd_split(segments=0, first_permille=0, chain_rg=0):
    """Measurement override of the split forward (include/gdn_profile.h):
    segments 1 = no split, 0 = the library's default."""
    load().gdn_diag_set_fwd_split(segments, first_permille, chain_rg)


def gdn_status_str(code: int) -> str:
    return load().gdn_status_str(code).decode()


class KernelTimer:
    """Per-kernel CUDA-event timing through the library's diagnostic hook
    (include/gdn_profile.h). Events are recorded on the stream each kernel is
    launched on, around every launch of the calls made while armed."""

    def __init__(self, capacity: int = 4096):
        self.capacity = capacity
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(capacity)]
        self.n = 0
        self.names = []

    def __enter__(self):
        for e in self.events:  # materialise the lazily-created events
            e.record()
        torch.cuda.synchronize()
        self._handles = (ctypes.c_void_p * self.capacity)(
            *[e.cuda_event for e in self.events])
        load().gdn_profile_arm(ctypes.cast(self._handles, ctypes.c_void_p), self.capacity)
        return self

    def __exit__(self, *exc):
        lib = load()
        self.n = lib.gdn_profile_count()
        self.names = [lib.gdn_profile_name(i) for i in range(self.n)]
        lib.gdn_profile_arm(None, 0)
        return False

    def per_kernel(self):
        """{kernel name: [durations in ms]} (call after synchronising)."""
        out = {}
        for i in range(self.n - 1):
            name = self.names[i]
            if name is None:
                continue
            out.setdefault(name.decode(), []).append(self.events[i].elapsed_time(self.events[i + 1]))
        return out
