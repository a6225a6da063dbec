"""Python binding of libefla.so, the B200 Exact Flow Linear Attention forward.

Argument checks and marshalling only: every step of the computation runs in the library's CUDA
kernels.  PyTorch provides device memory and streams.  The names mirror the C ABI of
include/efla.h.  Importing this package loads the in-tree libefla.so and fails loudly if
it has not been built (python delta_rule_linear_02_b200/build.py); without _efla_native.so it warns.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import warnings
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libefla.so")
# the same entry points built with EFLA_CHECKED=1: the tensor-core forward's kernels test
# every direct global access against its buffer and report EFLA_ERR_BOUNDS through the
# workspace status instead of touching memory out of range (build.py --checked)
LIB_CHECKED_PATH = os.path.join(_PKG, "libefla_checked.so")

EFLA_OK, EFLA_ERR_INVALID_ARG, EFLA_ERR_UNSUPPORTED, EFLA_ERR_CUDA, EFLA_ERR_TIMEOUT, EFLA_ERR_BOUNDS = range(6)
EFLA_ERR_SLOT, EFLA_ERR_FULL = 6, 7
EFLA_DTYPE_F32, EFLA_DTYPE_BF16 = 0, 1
EFLA_RULE_EXACT, EFLA_RULE_EULER = 0, 1     # exact-flow gate, or alpha = beta (the delta rule)
CHUNK = 64

_DTYPES = {torch.float32: EFLA_DTYPE_F32, torch.bfloat16: EFLA_DTYPE_BF16}


class EflaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {efla_status_string(status)} ({status})")


class _PythonWay:
    """In the place of a native module that cannot be used: no call is ordinary, the layer below makes them all."""

    def __getattr__(self, name):
        return lambda *args: None


def _load_native():
    """The short way of the calls whose time is the call itself (csrc/efla_native.cpp).  Without it, or with one that was
    built for another torch, the same calls take 5 to 10 us more."""
    try:
        from . import _efla_native as native
        built_for = getattr(native, "torch_version", "unknown")
        if built_for != torch.__version__:
            raise ImportError(f"it was built for torch {built_for}, this is {torch.__version__}")
        return native
    except ImportError as e:
        warnings.warn(f"_efla_native.so is not used, calls take longer ({e}); run "
                      "`python delta_rule_linear_02_b200/build.py`", RuntimeWarning, stacklevel=3)
        return _PythonWay()


_native = _load_native()


def _load(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{os.path.basename(path)} is not built at {path}; run "
                          "`python delta_rule_linear_02_b200/build.py` (nvcc, sm_100a)")
    lib = ctypes.CDLL(path)
    vp, I, L, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_long, ctypes.c_size_t
    lib.efla_status_string.argtypes = [I]
    lib.efla_status_string.restype = ctypes.c_char_p
    lib.efla_gate.argtypes = [vp, vp, vp, L, I, I, vp]
    lib.efla_gate.restype = I
    lib.efla_chunk_fwd_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
    lib.efla_chunk_fwd_workspace_bytes.restype = Z
    lib.efla_chunk_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, I, I, I, I, I, I, I, vp, Z, vp]
    lib.efla_chunk_fwd.restype = I
    lib.efla_chunk_fwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, I, I, I, I, I, I, I, I, vp, Z, vp]
    lib.efla_chunk_fwd_ex.restype = I
    lib.efla_chunk_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, I, I, I, I, I, I, I, vp]
    lib.efla_chunk_fwd_noalloc.restype = I
    lib.efla_workspace_status.argtypes = [vp, I, vp]
    lib.efla_workspace_status.restype = I
    lib.efla_noalloc_status.argtypes = [I, vp]
    lib.efla_noalloc_status.restype = I
    lib.efla_chunk_fwd_gated_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
    lib.efla_chunk_fwd_gated_workspace_bytes.restype = Z
    lib.efla_chunk_fwd_gated.argtypes = [vp] * 8 + [I, I, I, I, I, I, I, I, vp, Z, vp]
    lib.efla_chunk_fwd_gated.restype = I
    lib.efla_recurrent_step_gated.argtypes = [vp] * 7 + [I, I, I, I, I, I, vp]
    lib.efla_recurrent_step_gated.restype = I
    lib.efla_chunk_fwd_segmented_workspace_bytes.argtypes = [I, I, I, I, I, I, I, I, I]
    lib.efla_chunk_fwd_segmented_workspace_bytes.restype = Z
    lib.efla_chunk_fwd_segmented.argtypes = [vp] * 8 + [I] * 9 + [vp, Z, vp]
    lib.efla_chunk_fwd_segmented.restype = I
    lib.efla_chunk_fwd_varlen_workspace_bytes.argtypes = [vp, I, I, I, I, I, I, I]
    lib.efla_chunk_fwd_varlen_workspace_bytes.restype = Z
    lib.efla_chunk_fwd_varlen.argtypes = [vp] * 9 + [I, I, I, I, I, I, I, vp, Z, vp]
    lib.efla_chunk_fwd_varlen.restype = I
    lib.efla_selftest_wait_timeout.argtypes = [vp, ctypes.c_longlong, vp]
    lib.efla_selftest_wait_timeout.restype = I
    lib.efla_recurrent_step.argtypes = [vp, vp, vp, vp, vp, vp, I, I, I, I, I, vp]
    lib.efla_recurrent_step.restype = I
    lib.efla_recurrent_step_ex.argtypes = [vp, vp, vp, vp, vp, vp, I, I, I, I, I, I, vp]
    lib.efla_recurrent_step_ex.restype = I
    lib.efla_backward_workspace_bytes.argtypes = [I, I, I, I, I, I]
    lib.efla_backward_workspace_bytes.restype = Z
    lib.efla_backward.argtypes = [vp] * 12 + [I, I, I, I, I, I, vp, Z, vp]
    lib.efla_backward.restype = I
    lib.efla_backward_ex.argtypes = [vp] * 12 + [I, I, I, I, I, I, I, vp, Z, vp]
    lib.efla_backward_ex.restype = I
    lib.efla_train_saved_bytes.argtypes = [I, I, I, I, I, I, I]
    lib.efla_train_saved_bytes.restype = Z
    lib.efla_chunk_fwd_save.argtypes = [vp] * 7 + [I] * 8 + [vp, Z, vp]
    lib.efla_chunk_fwd_save.restype = I
    lib.efla_backward_saved_workspace_bytes.argtypes = [I, I, I, I, I, I]
    lib.efla_backward_saved_workspace_bytes.restype = Z
    lib.efla_backward_saved.argtypes = [vp] * 11 + [I] * 7 + [vp, Z, vp, Z, vp]
    lib.efla_backward_saved.restype = I
    lib.efla_scan_workspace_bytes.argtypes = [I] * 7
    lib.efla_scan_workspace_bytes.restype = Z
    lib.efla_scan_fwd.argtypes = [vp] * 6 + [I] * 7 + [vp, Z, vp]
    lib.efla_scan_fwd.restype = I
    lib.efla_scan_backward_workspace_bytes.argtypes = [I] * 8
    lib.efla_scan_backward_workspace_bytes.restype = Z
    lib.efla_scan_backward.argtypes = [vp] * 9 + [I] * 7 + [vp, Z, vp, Z, vp]
    lib.efla_scan_backward.restype = I
    lib.efla_scan_step.argtypes = [vp] * 4 + [I] * 6 + [vp]
    lib.efla_scan_step.restype = I
    lib.efla_scan_step_paged.argtypes = [vp, vp, vp, I, I, vp, Z, vp, vp, vp] + [I] * 6 + [vp]
    lib.efla_scan_step_paged.restype = I
    lib.efla_recurrent_step_paged.argtypes = [vp] * 6 + [I, I, vp, Z, vp, vp, vp] + [I] * 6 + [vp]
    lib.efla_recurrent_step_paged.restype = I
    lib.efla_pages_bytes.argtypes = [I, I]
    lib.efla_pages_bytes.restype = Z
    lib.efla_pages_init.argtypes = [vp, Z, I, I, vp]
    lib.efla_pages_free.argtypes = [vp, I, I, vp, I, vp]
    lib.efla_pages_compact.argtypes = [vp, I, I, vp, Z, Z, vp]
    lib.efla_pages_status.argtypes = [vp, I, vp]
    for f in (lib.efla_pages_fork, lib.efla_pages_copy):
        f.argtypes = [vp, I, I, vp, Z, Z, vp, vp, I, vp]
    for f in (lib.efla_pages_write, lib.efla_pages_read):
        f.argtypes = [vp, I, I, vp, Z, vp, Z, vp, I, vp]
    for f in (lib.efla_pages_init, lib.efla_pages_free, lib.efla_pages_compact, lib.efla_pages_status,
              lib.efla_pages_fork, lib.efla_pages_copy, lib.efla_pages_write, lib.efla_pages_read):
        f.restype = I
    # their order is that of Entries in csrc/efla_native.cpp
    lib.entries = _native.bind(*(ctypes.cast(f, vp).value for f in (
        lib.efla_scan_workspace_bytes, lib.efla_scan_fwd, lib.efla_scan_backward_workspace_bytes, lib.efla_scan_backward,
        lib.efla_scan_step, lib.efla_scan_step_paged, lib.efla_recurrent_step_paged, lib.efla_pages_fork,
        lib.efla_pages_copy, lib.efla_pages_free, lib.efla_pages_compact)))
    return lib


lib = _load()


def load_checked() -> ctypes.CDLL:
    """The checked build (libefla_checked.so) with the same argument types as `lib`; the
    wrappers below call whichever library the module attribute `lib` holds."""
    return _load(LIB_CHECKED_PATH)


def efla_status_string(status: int) -> str:
    return lib.efla_status_string(int(status)).decode()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _raise(status: int, where: str):
    if status != EFLA_OK:
        raise EflaError(status, where)


def efla_gate(k: torch.Tensor, beta: torch.Tensor, out: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """alpha [...] float32 from keys k [..., d_k] and gates beta [...] (same dtype)."""
    _check(k, "k"); _check(beta, "beta", k.dtype)
    n = beta.numel()
    if out is None:
        out = torch.empty(beta.shape, device=k.device, dtype=torch.float32)
    _check(out, "out", torch.float32)
    _raise(lib.efla_gate(_ptr(k), _ptr(beta), _ptr(out), n, k.shape[-1], _DTYPES[k.dtype],
                         _stream(stream)), "efla_gate")
    return out


def efla_chunk_fwd_workspace_bytes(B, H, T, d_k, d_v, chunk=CHUNK, dtype=torch.bfloat16) -> int:
    return int(lib.efla_chunk_fwd_workspace_bytes(B, H, T, d_k, d_v, chunk, _DTYPES[dtype]))


def new_workspace(B, H, T, d_k, d_v, chunk=CHUNK, dtype=torch.bfloat16, device="cuda"):
    """A zeroed workspace tensor (uint8) sized for efla_chunk_fwd."""
    n = efla_chunk_fwd_workspace_bytes(B, H, T, d_k, d_v, chunk, dtype)
    if n == 0:
        raise EflaError(EFLA_ERR_UNSUPPORTED, "efla_chunk_fwd_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def efla_chunk_fwd(q, k, v, beta, S0=None, chunk: int = CHUNK, o=None, S_T=None,
                   workspace=None, want_state: bool = True, stream=None, rule: int = EFLA_RULE_EXACT
                   ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Chunked EFLA forward. q, k [B,H,T,d_k], v [B,H,T,d_v], beta [B,H,T] (one dtype),
    S0 [B,H,d_k,d_v] float32 or None.  Returns (o [B,H,T,d_v], S_T or None).
    rule: EFLA_RULE_EXACT (the method) or EFLA_RULE_EULER (the delta rule, alpha = beta)."""
    dt = k.dtype
    for t, nme in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta")):
        _check(t, nme, dt)
    B, H, T, d_k = k.shape
    d_v = v.shape[-1]
    if S0 is not None:
        _check(S0, "S0", torch.float32)
    if o is None:
        o = torch.empty((B, H, T, d_v), device=k.device, dtype=dt)
    _check(o, "o", dt)
    if S_T is None and want_state:
        S_T = torch.empty((B, H, d_k, d_v), device=k.device, dtype=torch.float32)
    if S_T is not None:
        _check(S_T, "S_T", torch.float32)
    if workspace is None:
        workspace = new_workspace(B, H, T, d_k, d_v, chunk, dt, k.device)
    st = lib.efla_chunk_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(S0), _ptr(o), _ptr(S_T),
                               B, H, T, d_k, d_v, chunk, _DTYPES.get(dt, -1), int(rule), _ptr(workspace),
                               workspace.numel(), _stream(stream))
    _raise(st, "efla_chunk_fwd")
    return o, S_T


def efla_chunk_fwd_gated(q, k, v, beta, g, S0=None, chunk: int = CHUNK, o=None, S_T=None,
                         workspace=None, want_state: bool = True, stream=None, rule: int = EFLA_RULE_EXACT
                         ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gated EFLA forward: efla_chunk_fwd plus g [B,H,T] float32, the per-token log-decay."""
    dt = k.dtype
    for t, nme in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta")):
        _check(t, nme, dt)
    _check(g, "g", torch.float32)
    B, H, T, d_k = k.shape
    d_v = v.shape[-1]
    if S0 is not None:
        _check(S0, "S0", torch.float32)
    if o is None:
        o = torch.empty((B, H, T, d_v), device=k.device, dtype=dt)
    _check(o, "o", dt)
    if S_T is None and want_state:
        S_T = torch.empty((B, H, d_k, d_v), device=k.device, dtype=torch.float32)
    if S_T is not None:
        _check(S_T, "S_T", torch.float32)
    if workspace is None:
        n = int(lib.efla_chunk_fwd_gated_workspace_bytes(B, H, T, d_k, d_v, chunk, _DTYPES.get(dt, -1)))
        if n == 0:
            raise EflaError(EFLA_ERR_UNSUPPORTED, "efla_chunk_fwd_gated_workspace_bytes")
        workspace = torch.zeros(n, dtype=torch.uint8, device=k.device)
    st = lib.efla_chunk_fwd_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(S0), _ptr(o), _ptr(S_T),
                                  B, H, T, d_k, d_v, chunk, _DTYPES.get(dt, -1), int(rule), _ptr(workspace),
                                  workspace.numel(), _stream(stream))
    _raise(st, "efla_chunk_fwd_gated")
    return o, S_T


def efla_recurrent_step_gated(q, k, v, beta, g, S, o=None, stream=None, rule: int = EFLA_RULE_EXACT):
    """One gated decode token: efla_recurrent_step plus g [N,H] float32, the log-decay."""
    dt = k.dtype
    for t, nme in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta")):
        _check(t, nme, dt)
    _check(g, "g", torch.float32)
    _check(S, "S", torch.float32)
    N, H, d_k = k.shape
    d_v = v.shape[-1]
    if o is None:
        o = torch.empty((N, H, d_v), device=k.device, dtype=dt)
    _check(o, "o", dt)
    _raise(lib.efla_recurrent_step_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(S), _ptr(o),
                                         N, H, d_k, d_v, _DTYPES.get(dt, -1), int(rule), _stream(stream)),
           "efla_recurrent_step_gated")
    return o


def efla_chunk_fwd_segmented(q, k, v, beta, S0=None, g=None, segments: int = 0, chunk: int = CHUNK, o=None,
                             S_T=None, workspace=None, want_state: bool = True, stream=None,
                             rule: int = EFLA_RULE_EXACT) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """efla_chunk_fwd (or, with g, efla_chunk_fwd_gated) as a segmented scan of `segments`
    segments per stream (0: the library's choice)."""
    dt = k.dtype
    for t, nme in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta")):
        _check(t, nme, dt)
    if g is not None:
        _check(g, "g", torch.float32)
    B, H, T, d_k = k.shape
    d_v = v.shape[-1]
    if S0 is not None:
        _check(S0, "S0", torch.float32)
    if o is None:
        o = torch.empty((B, H, T, d_v), device=k.device, dtype=dt)
    _check(o, "o", dt)
    if S_T is None and want_state:
        S_T = torch.empty((B, H, d_k, d_v), device=k.device, dtype=torch.float32)
    if S_T is not None:
        _check(S_T, "S_T", torch.float32)
    if workspace is None:
        n = int(lib.efla_chunk_fwd_segmented_workspace_bytes(B, H, T, d_k, d_v, chunk, _DTYPES.get(dt, -1),
                                                             int(g is not None), int(segments)))
        if n == 0:
            raise EflaError(EFLA_ERR_UNSUPPORTED, "efla_chunk_fwd_segmented_workspace_bytes")
        workspace = torch.zeros(n, dtype=torch.uint8, device=k.device)
    st = lib.efla_chunk_fwd_segmented(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(S0), _ptr(o), _ptr(S_T),
                                      B, H, T, d_k, d_v, chunk, _DTYPES.get(dt, -1), int(rule), int(segments),
                                      _ptr(workspace), workspace.numel(), _stream(stream))
    _raise(st, "efla_chunk_fwd_segmented")
    return o, S_T


def efla_chunk_fwd_varlen(q, k, v, beta, cu_seqlens, S0=None, g=None, chunk: int = CHUNK, o=None, S_T=None,
                          workspace=None, want_state: bool = True, stream=None, rule: int = EFLA_RULE_EXACT
                          ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Packed variable-length forward: q, k [H,total_T,d_k], v [H,total_T,d_v], beta [H,total_T];
    cu_seqlens: N+1 offsets (a sequence of ints or a CPU int32 tensor); S0 [N,H,d_k,d_v] or None;
    g [H,total_T] float32 (gated flow) or None.  Returns (o, S_T [N,H,d_k,d_v] or None)."""
    dt = k.dtype
    for t, nme in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta")):
        _check(t, nme, dt)
    if g is not None:
        _check(g, "g", torch.float32)
    cu = torch.as_tensor(cu_seqlens, dtype=torch.int32, device="cpu").contiguous()
    N = cu.numel() - 1
    H, total_T, d_k = k.shape
    d_v = v.shape[-1]
    if S0 is not None:
        _check(S0, "S0", torch.float32)
    if o is None:
        o = torch.empty((H, total_T, d_v), device=k.device, dtype=dt)
    _check(o, "o", dt)
    if S_T is None and want_state:
        S_T = torch.empty((N, H, d_k, d_v), device=k.device, dtype=torch.float32)
    if S_T is not None:
        _check(S_T, "S_T", torch.float32)
    cup = ctypes.c_void_p(cu.data_ptr())
    if workspace is None:
        n = int(lib.efla_chunk_fwd_varlen_workspace_bytes(cup, N, H, d_k, d_v, chunk, _DTYPES.get(dt, -1),
                                                          int(g is not None)))
        if n == 0:
            raise EflaError(EFLA_ERR_INVALID_ARG, "efla_chunk_fwd_varlen_workspace_bytes")
        workspace = torch.zeros(n, dtype=torch.uint8, device=k.device)
    st = lib.efla_chunk_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), cup, _ptr(S0), _ptr(o),
                                   _ptr(S_T), N, H, d_k, d_v, chunk, _DTYPES.get(dt, -1), int(rule),
                                   _ptr(workspace), workspace.numel(), _stream(stream))
    _raise(st, "efla_chunk_fwd_varlen")
    return o, S_T


def efla_train_saved_bytes(B, H, T, d_k, d_v, chunk=CHUNK, dtype=torch.bfloat16) -> int:
    return int(lib.efla_train_saved_bytes(B, H, T, d_k, d_v, chunk, _DTYPES.get(dtype, -1)))


def efla_chunk_fwd_save(q, k, v, beta, S0=None, saved=None, o=None, S_T=None, want_state: bool = True,
                        stream=None, rule: int = EFLA_RULE_EXACT):
    """efla_chunk_fwd that also keeps the residuals efla_backward_saved needs (bf16, d = 128).
    Returns (o, S_T or None, saved); `saved` is a uint8 tensor of efla_train_saved_bytes."""
    dt = k.dtype
    for t, nme in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta")):
        _check(t, nme, dt)
    B, H, T, d_k = k.shape
    d_v = v.shape[-1]
    if S0 is not None:
        _check(S0, "S0", torch.float32)
    if o is None:
        o = torch.empty((B, H, T, d_v), device=k.device, dtype=dt)
    _check(o, "o", dt)
    if S_T is None and want_state:
        S_T = torch.empty((B, H, d_k, d_v), device=k.device, dtype=torch.float32)
    if S_T is not None:
        _check(S_T, "S_T", torch.float32)
    if saved is None:
        n = efla_train_saved_bytes(B, H, T, d_k, d_v, CHUNK, dt)
        if n == 0:
            raise EflaError(EFLA_ERR_UNSUPPORTED, "efla_train_saved_bytes")
        saved = torch.zeros(n, dtype=torch.uint8, device=k.device)
    st = lib.efla_chunk_fwd_save(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(S0), _ptr(o), _ptr(S_T),
                                 B, H, T, d_k, d_v, CHUNK, _DTYPES.get(dt, -1), int(rule), _ptr(saved),
                                 saved.numel(), _stream(stream))
    _raise(st, "efla_chunk_fwd_save")
    return o, S_T, saved


def efla_backward_saved(q, k, v, beta, dO, saved, dS_T=None, want_dS0: bool = True, grads=None,
                        workspace=None, stream=None, rule: int = EFLA_RULE_EXACT):
    """efla_backward from the residuals efla_chunk_fwd_save kept (no forward recompute).
    Returns (dq, dk, dv, dbeta, dS0 or None), all float32."""
    dt = k.dtype
    for t, nme in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta"), (dO, "dO")):
        _check(t, nme, dt)
    B, H, T, d_k = k.shape
    d_v = v.shape[-1]
    if dS_T is not None:
        _check(dS_T, "dS_T", torch.float32)
    f32 = dict(device=k.device, dtype=torch.float32)
    if grads is None:
        grads = (torch.empty((B, H, T, d_k), **f32), torch.empty((B, H, T, d_k), **f32),
                 torch.empty((B, H, T, d_v), **f32), torch.empty((B, H, T), **f32),
                 torch.empty((B, H, d_k, d_v), **f32) if want_dS0 else None)
    for t, nme in zip(grads, ("dq", "dk", "dv", "dbeta", "dS0")):
        if t is not None:
            _check(t, nme, torch.float32)
    if workspace is None:
        n = int(lib.efla_backward_saved_workspace_bytes(B, H, T, d_k, d_v, _DTYPES.get(dt, -1)))
        if n == 0:
            raise EflaError(EFLA_ERR_UNSUPPORTED, "efla_backward_saved_workspace_bytes")
        workspace = torch.zeros(n, dtype=torch.uint8, device=k.device)
    st = lib.efla_backward_saved(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(dO), _ptr(dS_T),
                                 *(_ptr(g) for g in grads), B, H, T, d_k, d_v, _DTYPES.get(dt, -1), int(rule),
                                 _ptr(saved), saved.numel(), _ptr(workspace), workspace.numel(), _stream(stream))
    _raise(st, "efla_backward_saved")
    return grads


def efla_chunk_fwd_noalloc(q, k, v, beta, S0=None, chunk: int = CHUNK, o=None, S_T=None,
                           want_state: bool = True, stream=None
                           ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """efla_chunk_fwd using the library's internal static scratch instead of a workspace.
    o and S_T are allocated here when not given (pass them in to allocate nothing)."""
    dt = k.dtype
    for t, nme in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta")):
        _check(t, nme, dt)
    B, H, T, d_k = k.shape
    d_v = v.shape[-1]
    if S0 is not None:
        _check(S0, "S0", torch.float32)
    if o is None:
        o = torch.empty((B, H, T, d_v), device=k.device, dtype=dt)
    _check(o, "o", dt)
    if S_T is None and want_state:
        S_T = torch.empty((B, H, d_k, d_v), device=k.device, dtype=torch.float32)
    if S_T is not None:
        _check(S_T, "S_T", torch.float32)
    st = lib.efla_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(S0), _ptr(o),
                                    _ptr(S_T), B, H, T, d_k, d_v, chunk, _DTYPES.get(dt, -1),
                                    _stream(stream))
    _raise(st, "efla_chunk_fwd_noalloc")
    return o, S_T


def efla_workspace_status(workspace: torch.Tensor, clear: bool = False, stream=None) -> int:
    return int(lib.efla_workspace_status(_ptr(workspace), int(clear), _stream(stream)))


def efla_noalloc_status(clear: bool = False, stream=None) -> int:
    """Device error word of efla_chunk_fwd_noalloc's static scratch (current device)."""
    return int(lib.efla_noalloc_status(int(clear), _stream(stream)))


def efla_selftest_wait_timeout(workspace: torch.Tensor, limit_ns: int = 1_000_000, stream=None) -> None:
    _raise(lib.efla_selftest_wait_timeout(_ptr(workspace), int(limit_ns), _stream(stream)),
           "efla_selftest_wait_timeout")


def efla_recurrent_step(q, k, v, beta, S, o=None, stream=None, rule: int = EFLA_RULE_EXACT) -> torch.Tensor:
    """One decode token: q, k [N,H,d_k], v [N,H,d_v], beta [N,H]; S [N,H,d_k,d_v] float32
    updated in place.  Returns o [N,H,d_v].  rule as in efla_chunk_fwd."""
    dt = k.dtype
    for t, nme in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta")):
        _check(t, nme, dt)
    _check(S, "S", torch.float32)
    N, H, d_k = k.shape
    d_v = v.shape[-1]
    if o is None:
        o = torch.empty((N, H, d_v), device=k.device, dtype=dt)
    _check(o, "o", dt)
    _raise(lib.efla_recurrent_step_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(S), _ptr(o),
                                      N, H, d_k, d_v, _DTYPES.get(dt, -1), int(rule), _stream(stream)),
           "efla_recurrent_step")
    return o


def efla_backward_workspace_bytes(B, H, T, d_k, d_v, dtype=torch.bfloat16) -> int:
    return int(lib.efla_backward_workspace_bytes(B, H, T, d_k, d_v, _DTYPES[dtype]))


def efla_backward(q, k, v, beta, dO, S0=None, dS_T=None, want_dS0: bool = True, grads=None,
                  workspace=None, stream=None, rule: int = EFLA_RULE_EXACT):
    """Gradients of efla_chunk_fwd for the loss sum(dO * o) + sum(dS_T * S_T).

    q, k [B,H,T,d_k], v, dO [B,H,T,d_v], beta [B,H,T] (one dtype); S0, dS_T [B,H,d_k,d_v]
    float32 or None.  Returns (dq, dk, dv, dbeta, dS0 or None), all float32.  `grads` may
    supply those five tensors preallocated (dS0 may be None)."""
    dt = k.dtype
    for t, nme in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta"), (dO, "dO")):
        _check(t, nme, dt)
    B, H, T, d_k = k.shape
    d_v = v.shape[-1]
    for t, nme in ((S0, "S0"), (dS_T, "dS_T")):
        if t is not None:
            _check(t, nme, torch.float32)
    f32 = dict(device=k.device, dtype=torch.float32)
    if grads is None:
        grads = (torch.empty((B, H, T, d_k), **f32), torch.empty((B, H, T, d_k), **f32),
                 torch.empty((B, H, T, d_v), **f32), torch.empty((B, H, T), **f32),
                 torch.empty((B, H, d_k, d_v), **f32) if want_dS0 else None)
    for t, nme in zip(grads, ("dq", "dk", "dv", "dbeta", "dS0")):
        if t is not None:
            _check(t, nme, torch.float32)
    if workspace is None:
        n = efla_backward_workspace_bytes(B, H, T, d_k, d_v, dt)
        if n == 0 and B * H * T > 0:
            raise EflaError(EFLA_ERR_UNSUPPORTED, "efla_backward_workspace_bytes")
        workspace = torch.zeros(max(n, 16), dtype=torch.uint8, device=k.device)
    st = lib.efla_backward_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(S0), _ptr(dO), _ptr(dS_T),
                              *(_ptr(g) for g in grads), B, H, T, d_k, d_v, _DTYPES.get(dt, -1), int(rule),
                              _ptr(workspace), workspace.numel(), _stream(stream))
    _raise(st, "efla_backward")
    return grads


# ---------------------------------------------------------------- the per-channel gated recurrence
def _call(fn, where: str, device: torch.device, stream, *args):
    """fn(*args, stream) with the tensors' device current; `stream` None: that device's current one."""
    index = device.index
    if index is None:
        raise ValueError(f"{where}: tensors must be on a CUDA device, got {device}")
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)      # torch.cuda.current_stream costs 2 us of every call
    else:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if index == torch.cuda.current_device():
        status = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            status = fn(*args, raw)
    if status != EFLA_OK:
        raise EflaError(status, where)


def _made(out, where: str) -> bool:
    """Whether the native way has made the call (None: it is for the way below); raises what the library answered."""
    if out is None:
        return False
    if type(out) is int and out != EFLA_OK:
        raise EflaError(out, where)
    return True


def _made_on(stream, device: torch.device):
    """The context in which a call on `stream` makes its tensors: in that stream's memory, which no work queued on
    another one still uses (None: the current stream's)."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _handed_over(stream, device: torch.device, *tensors) -> None:
    """Results in another stream's memory: it is not given away before the current stream is done with them."""
    if stream is not None:
        current = torch.cuda.current_stream(device)
        for t in tensors:
            if t is not None:
                t.record_stream(current)


def _zeros(like: torch.Tensor, shape, stream) -> torch.Tensor:
    """Zeros made on `stream` (None: the current one), so that the call that fills them comes after."""
    with _made_on(stream, like.device):
        out = like.new_zeros(shape)
    _handed_over(stream, like.device, out)
    return out


def _tensor(t: Optional[torch.Tensor], name: str, dtype, device, shape) -> Optional[int]:
    """The address of a contiguous tensor of this type, device and shape (None: NULL)."""
    if t is None:
        return None
    if t.shape == shape and t.dtype is dtype and t.get_device() == device.index and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on {device if device.type == 'cuda' else 'a CUDA device'}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _offsets(cu_seqlens) -> torch.Tensor:
    """A packed batch's offsets as a contiguous int32 tensor in host memory (one that is that already: itself)."""
    cu = torch.as_tensor(cu_seqlens, device="cpu")
    if cu.dim() != 1 or cu.numel() < 2:
        raise ValueError("cu_seqlens must hold B + 1 offsets of at least one sequence")
    if cu.is_floating_point() or cu.is_complex() or cu.dtype == torch.bool:
        raise ValueError(f"cu_seqlens must hold whole numbers, got {cu.dtype}")
    if cu.dtype != torch.int32:
        if int(cu.min()) < 0 or int(cu.max()) >= 2 ** 31:
            raise ValueError("cu_seqlens must hold offsets of 32 bits")
        cu = cu.to(torch.int32)
    return cu.contiguous()


def _scan_shape(x: torch.Tensor, g: torch.Tensor, cu_seqlens):
    """(B, H, T, d, g_width, dtype, offsets or None) of a dense [B,H,T,d] or packed [H,T,d] batch."""
    if x.dtype not in _DTYPES:
        raise ValueError(f"x must be one of {list(_DTYPES)}, got {x.dtype}")
    if cu_seqlens is None:
        if x.dim() != 4:
            raise ValueError(f"x must be [B,H,T,d], got {tuple(x.shape)}")
        B, H, T, d = x.shape
        cu = None
    else:
        if x.dim() != 3:
            raise ValueError(f"x must be [H,T,d] with cu_seqlens, got {tuple(x.shape)}")
        H, T, d = x.shape
        cu = _offsets(cu_seqlens)
        B = cu.numel() - 1
    if g.shape != x.shape and g.shape != x.shape[:-1]:
        raise ValueError(f"g must be {tuple(x.shape)} or {tuple(x.shape[:-1])}, got {tuple(g.shape)}")
    return B, H, T, d, (d if g.dim() == x.dim() else 1), _DTYPES[x.dtype], cu


def efla_scan_workspace_bytes(B, H, T, d, g_width, dtype=torch.bfloat16, packed: bool = False) -> int:
    return int(lib.efla_scan_workspace_bytes(B, H, T, d, g_width, _DTYPES.get(dtype, -1), int(packed)))


def _scan_fwd(x, g, S0, cu_seqlens, o, S_T, workspace, want_state, stream, rule):
    if stream is None:
        out = _native.scan_fwd(lib.entries, x, g, S0, cu_seqlens, o, S_T, workspace, want_state, rule)
        if _made(out, "efla_scan_fwd"):
            return out
    B, H, T, d, gw, dt, cu = _scan_shape(x, g, cu_seqlens)
    dev, f32 = x.device, torch.float32
    if dev.index is None:
        raise ValueError(f"x must be on a CUDA device, got {dev}")
    px, pg = _tensor(x, "x", x.dtype, dev, x.shape), _tensor(g, "g", f32, dev, g.shape)
    pS0 = _tensor(S0, "S0", f32, dev, (B, H, d))
    made = []
    with _made_on(stream, dev):
        if o is None:
            o = torch.empty_like(x)
            made.append(o)
        if S_T is None and want_state:
            S_T = x.new_empty((B, H, d), dtype=f32)
            made.append(S_T)
        if workspace is None:
            n = lib.efla_scan_workspace_bytes(B, H, T, d, gw, dt, int(cu is not None))
            if n == 0:
                raise EflaError(EFLA_ERR_UNSUPPORTED, "efla_scan_workspace_bytes")
            # (a call without streams uses no workspace, so its status is that of zeros)
            workspace = x.new_empty(n, dtype=torch.uint8) if B * H else x.new_zeros(n, dtype=torch.uint8)
            made.append(workspace)
    _handed_over(stream, dev, *made)
    po, pS_T = _tensor(o, "o", x.dtype, dev, x.shape), _tensor(S_T, "S_T", f32, dev, (B, H, d))
    n = workspace.numel()
    pw = _tensor(workspace, "workspace", torch.uint8, dev, (n,))
    _call(lib.efla_scan_fwd, "efla_scan_fwd", dev, stream, px, pg, None if cu is None else cu.data_ptr(), pS0, po, pS_T,
          B, H, T, d, gw, dt, int(rule), pw, n)
    return o, S_T, workspace


def efla_scan_fwd(x, g, S0=None, cu_seqlens=None, o=None, S_T=None, workspace=None, want_state: bool = True,
                  stream=None, rule: int = EFLA_RULE_EXACT) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The per-channel gated recurrence h_t = e^g_t h_{t-1} + phi(g_t) x_t, o_t = h_t (EFLA_RULE_EULER: 1 for phi).
    x [B,H,T,d] float32 or bfloat16; g float32, x's shape or [B,H,T] (one decay per head); S0 [B,H,d] float32 or
    None.  Packed: cu_seqlens (B + 1 offsets, ints or a CPU int32 tensor) with x [H,T,d], g [H,T,d] or [H,T].
    (Up to 255 sequences the offsets travel with the launch.  Of more, a pinned tensor has to stay as it is until the
    call has run, and for every replay of a captured one; captured from other memory they are refused.)
    stream: a torch stream or a cudaStream_t as an int, None: the current one.  What the call makes itself is made there;
    the caller orders its inputs before and the use of the results behind it, as with every call that takes a stream.
    Returns (o like x, S_T [B,H,d] float32 or None)."""
    return _scan_fwd(x, g, S0, cu_seqlens, o, S_T, workspace, want_state, stream, rule)[:2]


def efla_scan_fwd_save(x, g, S0=None, cu_seqlens=None, saved=None, o=None, S_T=None, want_state: bool = True,
                       stream=None, rule: int = EFLA_RULE_EXACT):
    """efla_scan_fwd that also returns what efla_scan_backward starts from: (o, S_T or None, saved); `saved` is a
    uint8 tensor of efla_scan_workspace_bytes."""
    return _scan_fwd(x, g, S0, cu_seqlens, o, S_T, saved, want_state, stream, rule)


def efla_scan_backward(x, g, dO, S0=None, dS_T=None, saved=None, cu_seqlens=None, want_dS0: bool = True, grads=None,
                       workspace=None, stream=None, rule: int = EFLA_RULE_EXACT):
    """Gradients of efla_scan_fwd for the loss sum(dO * o) + sum(dS_T * S_T): (dx, dg, dS0 or None), all float32.
    dO like x, dS_T [B,H,d] float32 or None; saved: from efla_scan_fwd_save on the same x, g, S0, cu_seqlens and rule
    (None: computed again).  `grads` may supply the three tensors preallocated (dS0 may be None)."""
    if stream is None and grads is None and workspace is None:
        out = _native.scan_backward(lib.entries, x, g, dO, S0, dS_T, saved, cu_seqlens, want_dS0, rule)
        if _made(out, "efla_scan_backward"):
            return out
    B, H, T, d, gw, dt, cu = _scan_shape(x, g, cu_seqlens)
    dev, f32 = x.device, torch.float32
    px, pg = _tensor(x, "x", x.dtype, dev, x.shape), _tensor(g, "g", f32, dev, g.shape)
    pS0, pdO = _tensor(S0, "S0", f32, dev, (B, H, d)), _tensor(dO, "dO", x.dtype, dev, x.shape)
    pdS_T = _tensor(dS_T, "dS_T", f32, dev, (B, H, d))
    with _made_on(stream, dev):
        if grads is None:
            grads = (torch.empty_like(x, dtype=f32), torch.empty_like(g),
                     x.new_empty((B, H, d), dtype=f32) if want_dS0 else None)
            made = grads
        else:
            made = ()
        if workspace is None:
            n = lib.efla_scan_backward_workspace_bytes(B, H, T, d, gw, dt, int(cu is not None), int(saved is not None))
            if n == 0:
                raise EflaError(EFLA_ERR_UNSUPPORTED, "efla_scan_backward_workspace_bytes")
            workspace = x.new_empty(n, dtype=torch.uint8)
    _handed_over(stream, dev, *made)
    out = [_tensor(t, name, f32, dev, shape)
           for t, name, shape in zip(grads, ("dx", "dg", "dS0"), (x.shape, g.shape, (B, H, d)))]
    n = workspace.numel()
    ns = 0 if saved is None else saved.numel()
    _call(lib.efla_scan_backward, "efla_scan_backward", dev, stream, px, pg, None if cu is None else cu.data_ptr(), pS0,
          pdO, pdS_T, *out, B, H, T, d, gw, dt, int(rule), _tensor(saved, "saved", torch.uint8, dev, (ns,)), ns,
          _tensor(workspace, "workspace", torch.uint8, dev, (n,)), n)
    return grads


def _step_shape(x: torch.Tensor, g: torch.Tensor):
    if x.dtype not in _DTYPES:
        raise ValueError(f"x must be one of {list(_DTYPES)}, got {x.dtype}")
    if x.dim() != 3 or (g.shape != x.shape and g.shape != x.shape[:-1]):
        raise ValueError(f"x must be [N,H,d] and g [N,H,d] or [N,H], got {tuple(x.shape)} and {tuple(g.shape)}")
    N, H, d = x.shape
    return N, H, d, (d if g.dim() == 3 else 1), _DTYPES[x.dtype]


def efla_scan_step(x, g, S, o=None, stream=None, rule: int = EFLA_RULE_EXACT) -> torch.Tensor:
    """One token of efla_scan_fwd's recurrence: x [N,H,d], g float32 [N,H,d] or [N,H]; S [N,H,d] float32 updated in
    place.  Returns o [N,H,d]."""
    if stream is None:
        out = _native.scan_step(lib.entries, x, g, S, o, rule)
        if _made(out, "efla_scan_step"):
            return out
    N, H, d, gw, dt = _step_shape(x, g)
    dev = x.device
    if o is None:
        with _made_on(stream, dev):
            o = torch.empty_like(x)
        _handed_over(stream, dev, o)
    _call(lib.efla_scan_step, "efla_scan_step", dev, stream, _tensor(x, "x", x.dtype, dev, x.shape),
          _tensor(g, "g", torch.float32, dev, g.shape), _tensor(S, "S", torch.float32, dev, x.shape),
          _tensor(o, "o", x.dtype, dev, x.shape), N, H, d, gw, dt, int(rule))
    return o


# ---------------------------------------------------------------- the state cache
class EflaPages:
    """The block of a state cache: which page holds the state of which slot.  `block` is an int32 tensor of
    efla_pages_bytes / 4 words: 64 of header, the table, the owners, scratch."""

    __slots__ = ("block", "n_pages", "n_slots")

    def __init__(self, block: torch.Tensor, n_pages: int, n_slots: int):
        need = 64 + 2 * n_slots + 3 * n_pages
        if n_pages < 1 or n_slots < 1:
            raise ValueError(f"a cache has at least one page and one slot, got {n_pages} and {n_slots}")
        if not block.is_cuda or block.dtype != torch.int32 or block.dim() != 1 or not block.is_contiguous() \
                or block.numel() < need:
            raise ValueError(f"block must be a contiguous CUDA int32 tensor of at least {need} words")
        self.block, self.n_pages, self.n_slots = block, n_pages, n_slots

    @property
    def table(self) -> torch.Tensor:
        """[n_slots] int32: the slot's page, -1 for none."""
        return self.block[64:64 + self.n_slots]

    @property
    def owner(self) -> torch.Tensor:
        """[n_pages] int32: the page's slot, -1 for a free page."""
        return self.block[64 + self.n_slots:64 + self.n_slots + self.n_pages]


def new_pages(n_pages: int, n_slots: int, device="cuda", stream=None) -> EflaPages:
    """The block of an empty cache of n_pages pages and n_slots slots."""
    n = int(lib.efla_pages_bytes(n_pages, n_slots))
    if n == 0:
        raise EflaError(EFLA_ERR_INVALID_ARG, "efla_pages_bytes")
    device = torch.device(device)
    if device.index is None and device.type == "cuda":
        device = torch.device("cuda", torch.cuda.current_device())
    with _made_on(stream, device):
        pages = EflaPages(torch.empty(n // 4, dtype=torch.int32, device=device), n_pages, n_slots)
    _handed_over(stream, device, pages.block)
    _call(lib.efla_pages_init, "efla_pages_init", pages.block.device, stream, pages.block.data_ptr(), n, n_pages,
          n_slots)
    return pages


def _pool(pool: torch.Tensor, pages: EflaPages, dtype=None) -> Tuple[int, int, int]:
    """(address, bytes between pages, bytes of a page's data) of a pool [n_pages, ...]: the pages may lie apart (a
    layer of a larger pool), each page's data is contiguous."""
    if not pool.is_cuda or pool.device != pages.block.device:
        raise ValueError(f"pool must be on {pages.block.device}, got {pool.device}")
    if dtype is not None and pool.dtype != dtype:
        raise ValueError(f"pool must be {dtype}, got {pool.dtype}")
    n, es = pages.n_pages, pool.element_size()
    if pool.dim() >= 2 and pool.shape[0] == n:
        data = pool.numel() // n * es
        if pool.is_contiguous():
            return pool.data_ptr(), data, data
        if pool[0].is_contiguous():
            return pool.data_ptr(), pool.stride(0) * es if n > 1 else data, data
    raise ValueError(f"pool must be [{n}, ...] with contiguous pages, got {tuple(pool.shape)}")


def _same_device(pages: EflaPages, name: str, device) -> None:
    if device != pages.block.device:
        raise ValueError(f"{name} must be on {pages.block.device}, where the cache is, got {device}")


def _slots(t: Optional[torch.Tensor], name: str, device, n: Optional[int] = None) -> Optional[int]:
    return None if t is None else _tensor(t, name, torch.int32, device, (t.numel() if n is None else n,))


def efla_pages_fork(pages: EflaPages, pool, source: torch.Tensor, dest: torch.Tensor, stream=None) -> None:
    """Every empty slot dest[i] gets a free page with a copy of slot source[i]'s page (-1: zeros).  pool [n_pages, ...]
    (any type), or None: pages are given without copying.  source, dest: int32, -1 in dest is padding."""
    if stream is None and _made(_native.pages_fork(lib.entries, pages.block, pages.n_pages, pages.n_slots, pool, source,
                                               dest), "efla_pages_fork"):
        return
    dev = pages.block.device
    ptr, stride, data = (None, 0, 0) if pool is None else _pool(pool, pages)
    _call(lib.efla_pages_fork, "efla_pages_fork", dev, stream, pages.block.data_ptr(), pages.n_pages, pages.n_slots, ptr,
          stride, data, _slots(source, "source", dev, dest.numel()), _slots(dest, "dest", dev), dest.numel())


def efla_pages_copy(pages: EflaPages, pool, source: torch.Tensor, dest: torch.Tensor, stream=None) -> None:
    """Slot dest[i]'s page becomes a copy of slot source[i]'s (-1: zeros), all entries as if at once."""
    if stream is None and _made(_native.pages_copy(lib.entries, pages.block, pages.n_pages, pages.n_slots, pool, source,
                                               dest), "efla_pages_copy"):
        return
    dev = pages.block.device
    ptr, stride, data = _pool(pool, pages)
    _call(lib.efla_pages_copy, "efla_pages_copy", dev, stream, pages.block.data_ptr(), pages.n_pages, pages.n_slots, ptr,
          stride, data, _slots(source, "source", dev, dest.numel()), _slots(dest, "dest", dev), dest.numel())


def efla_pages_free(pages: EflaPages, slots: torch.Tensor, stream=None) -> None:
    """The slots' pages are free again and the slots empty."""
    if stream is None and _made(_native.pages_free(lib.entries, pages.block, pages.n_pages, pages.n_slots, slots),
                                "efla_pages_free"):
        return
    dev = pages.block.device
    _call(lib.efla_pages_free, "efla_pages_free", dev, stream, pages.block.data_ptr(), pages.n_pages, pages.n_slots,
          _slots(slots, "slots", dev), slots.numel())


def efla_pages_compact(pages: EflaPages, pool, stream=None) -> None:
    """Moves pages so that the ones in use are the pool's first."""
    if stream is None and _made(_native.pages_compact(lib.entries, pages.block, pages.n_pages, pages.n_slots, pool),
                                "efla_pages_compact"):
        return
    ptr, stride, data = _pool(pool, pages)
    _call(lib.efla_pages_compact, "efla_pages_compact", pages.block.device, stream, pages.block.data_ptr(),
          pages.n_pages, pages.n_slots, ptr, stride, data)


def _pages_rows(fn, where, pages, pool, rows, slots, stream):
    dev = pages.block.device
    ptr, stride, data = _pool(pool, pages)
    _call(fn, where, dev, stream, pages.block.data_ptr(), pages.n_pages, pages.n_slots, ptr, stride,
          _tensor(rows, "rows", pool.dtype, dev, (slots.numel(), *pool.shape[1:])), data, _slots(slots, "slots", dev),
          slots.numel())


def efla_pages_write(pages: EflaPages, pool, rows: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
    """rows [n, ...] into the pages of slots[i]."""
    _pages_rows(lib.efla_pages_write, "efla_pages_write", pages, pool, rows, slots, stream)


def efla_pages_read(pages: EflaPages, pool, slots: torch.Tensor, rows: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """The pages of slots[i] as rows [n, ...] (zero rows for padding when `rows` is not given)."""
    if rows is None:
        rows = _zeros(pool, (slots.numel(), *pool.shape[1:]), stream)
    _pages_rows(lib.efla_pages_read, "efla_pages_read", pages, pool, rows, slots, stream)
    return rows


def efla_pages_status(pages: EflaPages, clear: bool = False, stream=None) -> int:
    """EFLA_OK, EFLA_ERR_SLOT or EFLA_ERR_FULL: what the calls on this cache met so far (waits for the stream)."""
    dev = pages.block.device
    with torch.cuda.device(dev):
        s = torch.cuda.current_stream(dev) if stream is None else stream
        return int(lib.efla_pages_status(pages.block.data_ptr(), int(clear),
                                         s.cuda_stream if hasattr(s, "cuda_stream") else int(s)))


def efla_scan_step_paged(x, g, pages: EflaPages, pool, slots, source=None, o=None, stream=None,
                         rule: int = EFLA_RULE_EXACT) -> torch.Tensor:
    """efla_scan_step on a state cache: row n's state is the page of slot slots[n] in pool [n_pages,H,d] float32.
    slots [N] int32, -1: a padded row, whose o is left as it was; source [N] int32: the slot a row's entering state is
    read from instead (-1: a zero state).  Returns o [N,H,d] (zeros for rows left out when `o` is not given)."""
    if stream is None:
        out = _native.scan_step_paged(lib.entries, x, g, pages.block, pages.n_pages, pages.n_slots, pool, slots, source, o,
                                      rule)
        if _made(out, "efla_scan_step_paged"):
            return out
    N, H, d, gw, dt = _step_shape(x, g)
    dev = x.device
    _same_device(pages, "x", dev)
    if pool.shape[1:] != x.shape[1:]:
        raise ValueError(f"pool must be [{pages.n_pages},{H},{d}], got {tuple(pool.shape)}")
    ptr, stride, _ = _pool(pool, pages, torch.float32)
    if o is None:
        o = _zeros(x, x.shape, stream)
    _call(lib.efla_scan_step_paged, "efla_scan_step_paged", dev, stream, _tensor(x, "x", x.dtype, dev, x.shape),
          _tensor(g, "g", torch.float32, dev, g.shape), pages.block.data_ptr(), pages.n_pages, pages.n_slots, ptr, stride,
          _slots(slots, "slots", dev, N), _slots(source, "source", dev, N), _tensor(o, "o", x.dtype, dev, x.shape), N, H,
          d, gw, dt, int(rule))
    return o


def efla_recurrent_step_paged(q, k, v, beta, pages: EflaPages, pool, slots, source=None, g=None, o=None, stream=None,
                              rule: int = EFLA_RULE_EXACT) -> torch.Tensor:
    """efla_recurrent_step (with g [N,H] float32: efla_recurrent_step_gated) on a state cache: row n's state is the
    page of slot slots[n] in pool [n_pages,H,d_k,d_v] float32.  slots, source and o as in efla_scan_step_paged."""
    if stream is None:
        out = _native.recurrent_step_paged(lib.entries, q, k, v, beta, pages.block, pages.n_pages, pages.n_slots, pool,
                                           slots, source, g, o, rule)
        if _made(out, "efla_recurrent_step_paged"):
            return out
    dt, dev = k.dtype, k.device
    if k.dim() != 3 or v.dim() != 3:
        raise ValueError(f"k must be [N,H,d_k] and v [N,H,d_v], got {tuple(k.shape)} and {tuple(v.shape)}")
    N, H, d_k = k.shape
    d_v = v.shape[-1]
    _same_device(pages, "k", dev)
    if pool.shape[1:] != (H, d_k, d_v):
        raise ValueError(f"pool must be [{pages.n_pages},{H},{d_k},{d_v}], got {tuple(pool.shape)}")
    ptr, stride, _ = _pool(pool, pages, torch.float32)
    if o is None:
        o = _zeros(v, v.shape, stream)
    _call(lib.efla_recurrent_step_paged, "efla_recurrent_step_paged", dev, stream, _tensor(q, "q", dt, dev, k.shape),
          _tensor(k, "k", dt, dev, k.shape), _tensor(v, "v", dt, dev, (N, H, d_v)), _tensor(beta, "beta", dt, dev, (N, H)),
          _tensor(g, "g", torch.float32, dev, (N, H)), pages.block.data_ptr(), pages.n_pages, pages.n_slots, ptr, stride,
          _slots(slots, "slots", dev, N), _slots(source, "source", dev, N), _tensor(o, "o", dt, dev, (N, H, d_v)), N, H,
          d_k, d_v, _DTYPES.get(dt, -1), int(rule))
    return o


__all__ = ["efla_scan_workspace_bytes", "efla_scan_fwd", "efla_scan_fwd_save", "efla_scan_backward", "efla_scan_step",
           "efla_scan_step_paged", "efla_recurrent_step_paged", "EflaPages", "new_pages", "efla_pages_fork",
           "efla_pages_copy", "efla_pages_free", "efla_pages_compact", "efla_pages_write", "efla_pages_read",
           "efla_pages_status", "EFLA_ERR_SLOT", "EFLA_ERR_FULL",
           "efla_train_saved_bytes", "efla_chunk_fwd_save", "efla_backward_saved", "efla_chunk_fwd_segmented", "efla_chunk_fwd_varlen", "efla_chunk_fwd_gated", "efla_recurrent_step_gated", "efla_backward", "efla_backward_workspace_bytes", "EFLA_RULE_EXACT", "EFLA_RULE_EULER", "efla_gate", "efla_chunk_fwd", "efla_chunk_fwd_noalloc", "efla_chunk_fwd_workspace_bytes", "efla_recurrent_step",
           "efla_workspace_status", "efla_noalloc_status", "efla_status_string", "load_checked", "efla_selftest_wait_timeout", "new_workspace", "EflaError", "lib",
           "LIB_PATH", "CHUNK"]
