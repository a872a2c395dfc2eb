"""GB300 (sm_103a) exact attention (forward, split-KV merge, e4m3 forward,
backward, sliding windows, rotary positions and a paged e4m3 cache): Python
binding of ``libfa_gb300.so``.

The functions below carry the names of the C ABI in ``include/fa.h`` and only
marshal arguments: every step of the computation runs in the library's CUDA
kernels. PyTorch supplies device memory and the current CUDA stream. The
library receives bare pointers and cannot see a buffer's size, so the binding
checks every tensor's dtype, shape, device and layout before the call. There is
no fallback: if the library is missing or a call fails, an exception says so.
"""

from __future__ import annotations

import contextlib
import ctypes
import math
import os
import struct
import warnings

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa_gb300.so")

FA_OK = 0
FA_ERR_SEQLENS = 12
STATUS_NAMES = {
    0: "FA_OK", 1: "FA_ERR_NULL", 2: "FA_ERR_ALIGN", 3: "FA_ERR_SHAPE", 4: "FA_ERR_HEADDIM",
    5: "FA_ERR_SPLITS", 6: "FA_ERR_WORKSPACE", 7: "FA_ERR_CUDA", 8: "FA_ERR_TIMEOUT",
    9: "FA_ERR_SCALE", 10: "FA_ERR_SCRATCH", 11: "FA_ERR_CAUSAL", 12: "FA_ERR_SEQLENS",
    13: "FA_ERR_TILE", 14: "FA_ERR_PAGES", 15: "FA_ERR_POSITIONS", 16: "FA_ERR_GROUP",
    17: "FA_ERR_WINDOW", 18: "FA_ERR_ROPE", 19: "FA_ERR_PAGE_SIZE", 20: "FA_ERR_STRIDE",
}
# Causal mask modes (include/fa.h): key j visible to query i iff j <= i (top-left)
# or j <= i + Nk - Nq (bottom-right).
CAUSAL_NONE, CAUSAL_TOP_LEFT, CAUSAL_BOTTOM_RIGHT = 0, 1, 2
_CAUSAL_NAMES = {"none": 0, "top_left": 1, "bottom_right": 2}
FA_MAX_SPLITS = 256
FA_MAX_AXES = 4

_lib = None
_compiled = None  # the module _calls, from load_library


class FAError(RuntimeError):
    """A library call returned a status other than FA_OK."""

    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {fa_status_string(status)}")


def load_library() -> ctypes.CDLL:
    """Load the in-tree CUDA library (build it with ``exact_attention_80_gb300.build``)."""
    global _lib, _compiled
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with `python -m exact_attention_80_gb300.build`")
    try:  # make torch's CUDA runtime the one the library binds to
        import torch  # noqa: F401
    except ImportError:
        pass
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
    lib.fa_fwd.restype = i
    lib.fa_fwd_rows.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
    lib.fa_fwd_rows.restype = i
    lib.fa_splitkv_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.fa_splitkv_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_fwd_splitkv.argtypes = [vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
    lib.fa_fwd_splitkv.restype = i
    lib.fa_combine.argtypes = [vp, vp, vp, i, i, i, i, i, vp]
    lib.fa_combine.restype = i
    lib.fa_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp]
    lib.fa_fwd_varlen.restype = i
    lib.fa_fwd_fp8.argtypes = [vp, vp, vp, f, f, f, vp, vp, i, i, i, i, i, f, i, vp]
    lib.fa_fwd_fp8.restype = i
    lib.fa_fwd_fp8_splitkv.argtypes = [vp, vp, vp, f, f, f, vp, i, i, i, i, i, f, i, i, vp]
    lib.fa_fwd_fp8_splitkv.restype = i
    lib.fa_bwd_workspace_bytes.argtypes = [i, i, i, i]
    lib.fa_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
    lib.fa_bwd.restype = i
    ll, packed = ctypes.c_longlong, ctypes.c_char_p  # packed: a struct of the interface, as bytes
    lib.fa_rope.argtypes = [packed, packed, packed, i, i, i, i, vp]
    lib.fa_rope.restype = i
    lib.fa_kv_append_fp8.argtypes = [vp, vp, vp, vp, packed, packed, vp, vp, vp, i, i, i, i, i, ll, ll, ll, vp]
    lib.fa_kv_append_fp8.restype = i
    lib.fa_paged_num_splits.argtypes = [i, i, i, i, i, i, i, i]
    lib.fa_paged_num_splits.restype = i
    lib.fa_paged_workspace_bytes.argtypes = [i, i, i, i]
    lib.fa_paged_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_fwd_paged_fp8.argtypes = [vp, packed, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, i, vp]
    lib.fa_fwd_paged_fp8.restype = i
    lib.fa_fwd_window.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, vp]
    lib.fa_fwd_window.restype = i
    lib.fa_fwd_window_splitkv.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, i, vp]
    lib.fa_fwd_window_splitkv.restype = i
    lib.fa_window_num_splits.argtypes = [i, i, i, i, i, i, i, i]
    lib.fa_window_num_splits.restype = i
    lib.fa_bwd_window_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i]
    lib.fa_bwd_window_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_bwd_window.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, vp]
    lib.fa_bwd_window.restype = i
    lib.fa_fwd_grid_ctas.argtypes = [i, i, i, i, i]
    lib.fa_fwd_grid_ctas.restype = ctypes.c_longlong
    lib.fa_device_status.argtypes = [vp, i]
    lib.fa_device_status.restype = i
    lib.fa_status_string.argtypes = [i]
    lib.fa_status_string.restype = ctypes.c_char_p
    _compiled = _load_calls(lib)
    _lib = lib  # only now: a load that failed is tried again by the next call
    return lib


def _load_calls(lib):
    """The compiled form of the calls that a few microseconds matter to (csrc/fa_calls.cpp). None, with a
    warning, where the module is missing or belongs to another PyTorch: the Python forms then take
    every call. None without PyTorch, or with one that has no CUDA."""
    try:
        import torch
    except ImportError:
        return None
    if torch.version.cuda is None:
        return None
    try:
        from . import _calls as calls  # type: ignore[attr-defined]

        if calls.torch_version != str(torch.__version__):
            raise ImportError(f"built against PyTorch {calls.torch_version}, this is {torch.__version__}")
    except (ImportError, AttributeError) as e:
        warnings.warn(f"exact_attention_80_gb300: the compiled calls are not there ({e}), short calls take longer; "
                      "build them with `python -m exact_attention_80_gb300.build`", RuntimeWarning, stacklevel=3)
        return None
    calls.init(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.fa_rope, lib.fa_kv_append_fp8, lib.fa_fwd_paged_fp8, lib.fa_paged_num_splits,
        lib.fa_paged_workspace_bytes, lib.fa_fwd_window, lib.fa_bwd_window, lib.fa_bwd_window_workspace_bytes,
        lib.fa_window_num_splits, lib.fa_fwd_window_splitkv, lib.fa_combine)))
    return calls


def fa_status_string(status: int) -> str:
    return load_library().fa_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != FA_OK:
        raise FAError(status, what)


def _int32(x):
    """``x`` where the interface's 32-bit int holds it: ctypes would pass on its low bits."""
    if not -(1 << 31) <= x < 1 << 31:
        raise OverflowError(f"{x} does not fit the library's 32-bit int")
    return x


def _stream_handle(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _allocating(stream, t):
    """What a call on ``stream`` allocates inside belongs to that stream (None: the current one). Memory of
    the current stream might still be in use there by work that ``stream`` does not wait for."""
    if stream is None:
        return contextlib.nullcontext()
    import torch

    if not hasattr(stream, "cuda_stream"):  # a handle; ExternalStream takes 0 for none at all
        stream = (torch.cuda.default_stream(t.device) if int(stream) in (0, 1) else
                  torch.cuda.ExternalStream(int(stream), device=t.device))
    return torch.cuda.stream(stream)


def _given(stream, *tensors):
    """Outputs of a call on ``stream``, which the caller uses on the current stream: their memory, once given
    back, waits for that stream as well."""
    if stream is not None:
        import torch

        for t in tensors:
            if t is not None:
                t.record_stream(torch.cuda.current_stream(t.device))
    return tensors


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _need(t, name, shape, dtype, device):
    """Raise unless ``t`` is a contiguous tensor of ``dtype`` and ``shape`` on
    ``device``: the library writes through a bare pointer."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on {device}")
    if tuple(t.shape) != tuple(int(x) for x in shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _need_workspace(t, nbytes: int, name: str, device):
    """Raise unless ``t`` is a contiguous float32 tensor on ``device`` of at least
    ``nbytes`` bytes (0: the arguments are out of range, for the library to
    reject)."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on {device}")
    if nbytes > 0 and t.numel() * 4 < nbytes:
        raise ValueError(f"{name} holds {t.numel() * 4} bytes; the call needs {nbytes}")


def _bhnd(q, k, v):
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
        if t.dim() != 4 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{name} must be a contiguous CUDA tensor [B, H, N, d]")
    if k.device != q.device or v.device != q.device:
        raise ValueError("q, k and v must be on the same device")
    B, H, Nq, d = q.shape
    if k.shape[:2] != (B, H) or k.shape[3] != d or v.shape != k.shape:
        raise ValueError(f"shape mismatch q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)}")
    return int(B), int(H), int(Nq), int(k.shape[2]), int(d)


def _need_o_lse(o, lse, B, H, Nq, d, device):
    import torch

    _need(o, "o", (B, H, Nq, d), torch.bfloat16, device)
    _need(lse, "lse", (B, H, Nq), torch.float32, device)


def causal_code(causal) -> int:
    """The C-ABI causal value: ``False``/``True`` (top-left), 0/1/2, or one of
    ``"none"``, ``"top_left"``, ``"bottom_right"``. Other values pass through as
    given, for the library to reject (FA_ERR_CAUSAL)."""
    if isinstance(causal, str):
        if causal not in _CAUSAL_NAMES:
            raise ValueError(f"unknown causal mode {causal!r}")
        return _CAUSAL_NAMES[causal]
    if isinstance(causal, bool):
        return CAUSAL_TOP_LEFT if causal else CAUSAL_NONE
    return _int32(int(causal))


def default_scale(d: int) -> float:
    """1/sqrt(d) rounded once to float32 (the value the kernel receives)."""
    return float(ctypes.c_float(d ** -0.5).value)


def fa_fwd(q, k, v, o, lse, causal=False, scale: float | None = None, stream=None):
    """Fused forward into caller-owned ``o`` (bf16 [B,H,Nq,d]) and ``lse`` (fp32 [B,H,Nq])."""
    B, H, Nq, Nk, d = _bhnd(q, k, v)
    _need_o_lse(o, lse, B, H, Nq, d, q.device)
    scale = default_scale(d) if scale is None else float(scale)
    st = load_library().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Nq, Nk, d,
                               scale, causal_code(causal), _stream_handle(stream))
    _check(st, "fa_fwd")


def fa_fwd_rows(q, k, v, o, lse, rows_per_cta: int, causal=False, scale: float | None = None,
                stream=None):
    """:func:`fa_fwd` with ``rows_per_cta`` query rows per CTA (include/fa.h,
    fa_fwd_rows: 64, 128 or 256 at d <= 128, 128 at d = 256)."""
    B, H, Nq, Nk, d = _bhnd(q, k, v)
    _need_o_lse(o, lse, B, H, Nq, d, q.device)
    scale = default_scale(d) if scale is None else float(scale)
    st = load_library().fa_fwd_rows(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Nq, Nk, d,
                                    scale, causal_code(causal), _int32(int(rows_per_cta)),
                                    _stream_handle(stream))
    _check(st, "fa_fwd_rows")


def _bhnd8(q, k, v):
    import torch

    ok_types = (torch.uint8, torch.float8_e4m3fn)
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype not in ok_types:
            raise TypeError(f"{name} must hold e4m3 codes (uint8 or float8_e4m3fn), got {t.dtype}")
        if t.dim() != 4 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{name} must be a contiguous CUDA tensor [B, H, N, d]")
    if k.device != q.device or v.device != q.device:
        raise ValueError("q, k and v must be on the same device")
    B, H, Nq, d = q.shape
    if k.shape[:2] != (B, H) or k.shape[3] != d or v.shape != k.shape:
        raise ValueError(f"shape mismatch q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)}")
    return int(B), int(H), int(Nq), int(k.shape[2]), int(d)


def fa_fwd_fp8(q, k, v, q_descale: float, k_descale: float, v_descale: float, o, lse,
               causal=False, scale: float | None = None, stream=None):
    """Fused forward on e4m3 inputs (include/fa.h, fa_fwd_fp8): ``q``, ``k``, ``v``
    hold e4m3 codes [B,H,N,d] (uint8 or float8_e4m3fn), the value of a code being
    its e4m3 value times the tensor's descale; ``o`` bf16 [B,H,Nq,d] and ``lse``
    fp32 [B,H,Nq] are written."""
    B, H, Nq, Nk, d = _bhnd8(q, k, v)
    _need_o_lse(o, lse, B, H, Nq, d, q.device)
    scale = default_scale(d) if scale is None else float(scale)
    st = load_library().fa_fwd_fp8(_ptr(q), _ptr(k), _ptr(v), float(q_descale), float(k_descale),
                                   float(v_descale), _ptr(o), _ptr(lse), B, H, Nq, Nk, d, scale,
                                   causal_code(causal), _stream_handle(stream))
    _check(st, "fa_fwd_fp8")


def fa_fwd_fp8_splitkv(q, k, v, q_descale: float, k_descale: float, v_descale: float, workspace,
                       num_splits: int, causal=False, scale: float | None = None, stream=None):
    """Split-KV forward on e4m3 inputs into ``workspace`` (fp32, at least
    ``fa_splitkv_workspace_bytes`` bytes); merge with :func:`fa_combine`."""
    B, H, Nq, Nk, d = _bhnd8(q, k, v)
    _need_workspace(workspace, fa_splitkv_workspace_bytes(B, H, Nq, d, int(num_splits)), "workspace",
                    q.device)
    scale = default_scale(d) if scale is None else float(scale)
    st = load_library().fa_fwd_fp8_splitkv(_ptr(q), _ptr(k), _ptr(v), float(q_descale),
                                           float(k_descale), float(v_descale), _ptr(workspace), B, H,
                                           Nq, Nk, d, scale, causal_code(causal), _int32(int(num_splits)),
                                           _stream_handle(stream))
    _check(st, "fa_fwd_fp8_splitkv")


def attention_fp8(q, k, v, q_descale: float = 1.0, k_descale: float = 1.0, v_descale: float = 1.0,
                  causal=False, scale: float | None = None, num_splits: int = 1, stream=None):
    """Allocate bf16 ``o`` and fp32 ``lse`` and run :func:`fa_fwd_fp8`, or, with
    ``num_splits > 1``, :func:`fa_fwd_fp8_splitkv` and :func:`fa_combine`."""
    import torch

    B, H, Nq, Nk, d = _bhnd8(q, k, v)
    with _allocating(stream, q):
        o = torch.empty((B, H, Nq, d), dtype=torch.bfloat16, device=q.device)
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
        if num_splits == 1:
            fa_fwd_fp8(q, k, v, q_descale, k_descale, v_descale, o, lse, causal, scale, stream)
        else:
            ws = torch.empty(fa_splitkv_workspace_bytes(B, H, Nq, d, num_splits) // 4,
                             dtype=torch.float32, device=q.device)
            fa_fwd_fp8_splitkv(q, k, v, q_descale, k_descale, v_descale, ws, num_splits, causal, scale,
                               stream)
            fa_combine(ws, o, lse, B, H, Nq, d, num_splits, stream)
    return _given(stream, o, lse)


def fa_bwd_workspace_bytes(B: int, H: int, Nq: int, d: int) -> int:
    return int(load_library().fa_bwd_workspace_bytes(*map(_int32, (B, H, Nq, d))))


def fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, workspace, causal=False,
           scale: float | None = None, stream=None):
    """Backward into caller-owned ``dq``, ``dk``, ``dv`` (bf16, shaped like q, k,
    v), from bf16 ``o`` and ``dout`` and the forward's fp32 ``lse``; ``workspace``
    fp32 of at least ``fa_bwd_workspace_bytes`` bytes (include/fa.h, fa_bwd)."""
    import torch

    B, H, Nq, Nk, d = _bhnd(q, k, v)
    dev = q.device
    _need(o, "o", (B, H, Nq, d), torch.bfloat16, dev)
    _need(dout, "dout", (B, H, Nq, d), torch.bfloat16, dev)
    _need(lse, "lse", (B, H, Nq), torch.float32, dev)
    _need(dq, "dq", (B, H, Nq, d), torch.bfloat16, dev)
    _need(dk, "dk", (B, H, Nk, d), torch.bfloat16, dev)
    _need(dv, "dv", (B, H, Nk, d), torch.bfloat16, dev)
    _need_workspace(workspace, fa_bwd_workspace_bytes(B, H, Nq, d), "workspace", dev)
    scale = default_scale(d) if scale is None else float(scale)
    st = load_library().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq),
                               _ptr(dk), _ptr(dv), _ptr(workspace), B, H, Nq, Nk, d, scale,
                               causal_code(causal), _stream_handle(stream))
    _check(st, "fa_bwd")


def attention_backward(q, k, v, o, lse, dout, causal=False, scale: float | None = None,
                       stream=None):
    """Allocate ``(dq, dk, dv)`` and the workspace and run :func:`fa_bwd`."""
    import torch

    B, H, Nq, Nk, d = _bhnd(q, k, v)
    with _allocating(stream, q):
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        ws = torch.empty(max(1, fa_bwd_workspace_bytes(B, H, Nq, d) // 4), dtype=torch.float32,
                         device=q.device)
        fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, ws, causal, scale, stream)
    return _given(stream, dq, dk, dv)


def fa_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, causal=False,
                  scale: float | None = None, stream=None):
    """Forward over packed variable-length sequences: ``q``/``o`` bf16
    [total_q, H, d], ``k``/``v`` bf16 [total_k, H, d], ``lse`` fp32 [H, total_q],
    ``cu_seqlens_*`` int32 [B+1] on the device (include/fa.h, fa_fwd_varlen)."""
    import torch

    for t in (q, k, v, o):
        if t.dtype != torch.bfloat16 or t.dim() != 3 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError("q, k, v, o must be contiguous CUDA bf16 [tokens, H, d]")
    for t in (cu_seqlens_q, cu_seqlens_k):
        if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError("cu_seqlens must be contiguous CUDA int32 [B+1]")
    if lse.dtype != torch.float32 or not lse.is_contiguous() or not lse.is_cuda:
        raise ValueError("lse must be contiguous CUDA fp32 [H, total_q]")
    if any(t.device != q.device for t in (k, v, o, lse, cu_seqlens_q, cu_seqlens_k)):
        raise ValueError("every tensor must be on q's device")
    total_q, H, d = (int(x) for x in q.shape)
    total_k = int(k.shape[0])
    if tuple(o.shape) != tuple(q.shape) or tuple(k.shape) != (total_k, H, d) or v.shape != k.shape:
        raise ValueError(f"shape mismatch q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)} "
                         f"o{tuple(o.shape)}")
    if tuple(lse.shape) != (H, total_q):
        raise ValueError(f"lse must have shape {(H, total_q)}, got {tuple(lse.shape)}")
    B = int(cu_seqlens_q.shape[0]) - 1
    if int(cu_seqlens_k.shape[0]) != B + 1 or B < 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must both have B+1 >= 2 entries")
    scale = default_scale(d) if scale is None else float(scale)
    st = load_library().fa_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                      _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), B, H, total_q,
                                      total_k, _int32(int(max_seqlen_q)), d, scale, causal_code(causal),
                                      _stream_handle(stream))
    _check(st, "fa_fwd_varlen")


def attention_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, causal=False,
                     scale: float | None = None, stream=None):
    """Allocate ``o`` [total_q, H, d] and ``lse`` [H, total_q] and run
    :func:`fa_fwd_varlen`. Returns ``(o, lse)``."""
    import torch

    with _allocating(stream, q):
        o = torch.empty_like(q)
        lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
        fa_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, causal, scale, stream)
    return _given(stream, o, lse)


def fa_splitkv_workspace_bytes(B: int, H: int, Nq: int, d: int, num_splits: int) -> int:
    return int(load_library().fa_splitkv_workspace_bytes(*map(_int32, (B, H, Nq, d, num_splits))))


def fa_fwd_splitkv(q, k, v, workspace, num_splits: int, causal=False,
                   scale: float | None = None, stream=None):
    """Split-KV partial states into ``workspace`` (see include/fa.h for the layout)."""
    B, H, Nq, Nk, d = _bhnd(q, k, v)
    _need_workspace(workspace, fa_splitkv_workspace_bytes(B, H, Nq, d, int(num_splits)), "workspace",
                    q.device)
    scale = default_scale(d) if scale is None else float(scale)
    st = load_library().fa_fwd_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(workspace), B, H, Nq, Nk,
                                       d, scale, causal_code(causal), _int32(int(num_splits)),
                                       _stream_handle(stream))
    _check(st, "fa_fwd_splitkv")


def fa_combine(workspace, o, lse, B: int, H: int, Nq: int, d: int, num_splits: int,
               stream=None):
    """Merge partial states from ``workspace`` into ``o`` and ``lse``."""
    _need_o_lse(o, lse, B, H, Nq, d, o.device if hasattr(o, "device") else None)
    _need_workspace(workspace, fa_splitkv_workspace_bytes(int(B), int(H), int(Nq), int(d), int(num_splits)),
                    "workspace", o.device)
    st = load_library().fa_combine(_ptr(workspace), _ptr(o), _ptr(lse), int(B), int(H), int(Nq),
                                   int(d), int(num_splits), _stream_handle(stream))
    _check(st, "fa_combine")


def fa_fwd_grid_ctas(B: int, H: int, Nq: int, d: int, num_splits: int = 1) -> int:
    return int(load_library().fa_fwd_grid_ctas(*map(_int32, (B, H, Nq, d, num_splits))))


def fa_device_status(clear: bool = True, stream=None) -> int:
    """Synchronises the stream and returns the device status (FA_OK, FA_ERR_TIMEOUT, or
    what a kernel found wrong in its device-side arguments: FA_ERR_SEQLENS,
    FA_ERR_PAGES, FA_ERR_POSITIONS)."""
    return int(load_library().fa_device_status(_stream_handle(stream), int(bool(clear))))


def attention(q, k, v, causal=False, scale: float | None = None, num_splits: int = 1,
              stream=None):
    """Allocate outputs and run the forward; ``num_splits > 1`` takes the split-KV +
    combine path. Returns ``(o, lse)``."""
    import torch

    B, H, Nq, Nk, d = _bhnd(q, k, v)
    with _allocating(stream, q):
        o = torch.empty((B, H, Nq, d), dtype=torch.bfloat16, device=q.device)
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
        if num_splits == 1:
            fa_fwd(q, k, v, o, lse, causal, scale, stream)
        else:
            nbytes = fa_splitkv_workspace_bytes(B, H, Nq, d, num_splits)
            if nbytes == 0:
                raise FAError(5, "fa_splitkv_workspace_bytes")
            ws = torch.empty(nbytes // 4, dtype=torch.float32, device=q.device)
            fa_fwd_splitkv(q, k, v, ws, num_splits, causal, scale, stream)
            fa_combine(ws, o, lse, B, H, Nq, d, num_splits, stream)
    return _given(stream, o, lse)


def fa_fwd_splitkv_static(q, k, v, o, lse, num_splits: int, causal=False,
                          scale: float | None = None, stream=None):
    """Split-KV forward + merge into caller-owned ``o``/``lse`` with no workspace
    argument: the partial states live in the library's static device buffer
    (``FA_STATIC_SCRATCH_BYTES``), so nothing is allocated. For callers that may
    not allocate device memory; calls that overlap on the GPU share that buffer
    and race (see include/fa.h)."""
    B, H, Nq, Nk, d = _bhnd(q, k, v)
    _need_o_lse(o, lse, B, H, Nq, d, q.device)
    scale = default_scale(d) if scale is None else float(scale)
    lib = load_library()
    fn = lib.fa_fwd_splitkv_static
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    fn.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
    fn.restype = i
    st = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Nq, Nk, d, scale,
            causal_code(causal), _int32(int(num_splits)), _stream_handle(stream))
    _check(st, "fa_fwd_splitkv_static")


# ------------------------------------------ rotary positions and the paged cache
# These calls are short (a decode step of a few sequences runs in a few
# microseconds on the GPU). On the current stream and with plain arguments rope,
# kv_append_fp8, attention_paged_fp8 and the window's two calls run in the
# compiled module _calls, where it is there; it answers None where an argument is
# anything else, and the forms below, whose checks touch each tensor once, say
# what is wrong or take the call.
_ROTATION = struct.Struct(f"PPii{FA_MAX_AXES}iii")   # fa_rotation
_ROPE_TENSOR = struct.Struct("PPi6q")                # fa_rope_tensor
_PAGED_CACHE = struct.Struct("PPPPiiii")             # fa_paged_cache


def _raw_stream(index):
    """Handle of the current stream of device ``index``."""
    import torch

    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the handle without a Stream object
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _on_stream(index, stream, fn, *args):
    """``fn(*args, handle)`` on device ``index`` and ``stream`` (None: the
    device's current stream), that device being the current one meanwhile."""
    import torch

    if stream is None:
        if torch.cuda.current_device() == index:
            return fn(*args, _raw_stream(index))
    else:
        on = getattr(stream, "device", None)
        if on is not None and on.index != index:
            raise ValueError(f"stream is on {on}, the tensors on device {index}")
    if index < 0:  # no device to make current
        return fn(*args, _raw_stream(index) if stream is None else int(getattr(stream, "cuda_stream", stream)))
    with torch.cuda.device(index):
        return fn(*args, _raw_stream(index) if stream is None else int(getattr(stream, "cuda_stream", stream)))


def _heads_view(t, name):
    """(B, H, N, d, batch, head and token strides) of a bf16 CUDA tensor [B, H, N, d] or, packed
    token-major, [N, H, d], whose columns are contiguous."""
    import torch

    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be a bfloat16 tensor")
    dim = t.dim()
    if dim == 4:
        B, H, N, d = t.shape
        sb, sh, sn, sd = t.stride()
    elif dim == 3:
        N, H, d = t.shape
        sn, sh, sd = t.stride()
        B, sb = 1, 0
    else:
        sd = 0
    if sd != 1 or not t.is_cuda or B * H * N * d == 0:
        raise ValueError(f"{name} must be a non-empty CUDA tensor [B, H, N, d] or [N, H, d] with contiguous columns")
    return B, H, N, d, sb if B > 1 else 0, sh if H > 1 else 0, sn if N > 1 else 0


def _rotation(table, positions, axes, sections, interleaved, tokens, index):
    """fa_rotation of a table and of positions that hold ``axes`` rows; ``tokens`` is the tokens' shape,
    (B, N) or (N,)."""
    import torch

    rows, rot = table.shape
    if table.dtype is not torch.float32 or not table.is_contiguous() or table.get_device() != index:
        raise ValueError(f"table must be contiguous float32 [max_pos, rot] on device {index}")
    at = 0
    if positions is not None:
        if positions.dtype is not torch.int32 or not positions.is_contiguous() or positions.get_device() != index:
            raise ValueError(f"positions must be contiguous int32 [axes, tokens] on device {index}")
        # One axis of [B, N] tensors may also come flat; [N, B], say, holds as many numbers for other tokens.
        shape, flat = tuple(positions.shape), (math.prod(tokens),)
        if shape not in (tokens, (axes, *tokens)) and (axes != 1 or shape not in (flat, (1, *flat))):
            raise ValueError(f"positions must have shape {tokens} or {('axes', *tokens)}, got {shape}")
        at = positions.data_ptr()
    if axes > FA_MAX_AXES:
        raise FAError(18, "rotation")
    if sections is None:
        sections = (rot // 2,) if axes == 1 else ()
    if len(sections) != axes:
        raise ValueError(f"sections must give the pairs of each of the {axes} axes")
    return _ROTATION.pack(table.data_ptr(), at, rot, axes, *sections, *(0,) * (FA_MAX_AXES - axes), rows,
                          1 if interleaved else 0)


def _rope(q, k, q_out, k_out, table, positions, sections, interleaved, inverse, stream):
    """The checks and the call of fa_rope; outputs None are allocated."""
    import torch

    index = q.get_device()
    B, H, N, d, sb, sh, sn = _heads_view(q, "q")
    dim = q.dim()
    outs, packed = [], []
    for t, out, name in ((q, q_out, "q"), (k, k_out, "k")):
        if t is None:
            if out is not None:
                raise ValueError(f"{name}_out without {name}")
            outs.append(None)
            packed.append(None)
            continue
        if t is not q:
            Bk, H, Nk, dk, sb, sh, sn = _heads_view(t, name)
            if (Bk, Nk, dk) != (B, N, d) or t.dim() != dim or t.get_device() != index:
                raise ValueError(f"shape or device mismatch: {name} {tuple(t.shape)}, q {tuple(q.shape)}")
        if out is None:
            out = torch.empty(t.shape, dtype=torch.bfloat16, device=t.device)
            ob, oh, on = (H * N * d, N * d, d) if dim == 4 else (0, d, H * d)
        elif out is t:
            ob, oh, on = sb, sh, sn
        else:
            if out.shape != t.shape or out.get_device() != index:
                raise ValueError(f"{name}_out must have {name}'s shape {tuple(t.shape)} and device")
            ob, oh, on = _heads_view(out, name + "_out")[4:]
        if (ob == 0 and B > 1) or (oh == 0 and H > 1) or (on == 0 and N > 1):
            raise ValueError(f"{name}_out must not be an expanded tensor")
        outs.append(out)
        packed.append(_ROPE_TENSOR.pack(t.data_ptr(), out.data_ptr(), H, sb, sh, sn, ob, oh, on))
    if positions is None:
        raise TypeError("positions must be a tensor")
    axes = positions.shape[0] if positions.dim() == dim - 1 else 1
    rope = _rotation(table, positions, axes, sections, interleaved, (B, N) if dim == 4 else (N,), index)
    st = _on_stream(index, stream, load_library().fa_rope, packed[0], packed[1], rope, B, N, d, 1 if inverse else 0)
    if st != FA_OK:
        raise FAError(st, "fa_rope")
    return outs


def fa_rope(q, k, q_out, k_out, table, positions, sections=None, interleaved=False, inverse=False, stream=None):
    """Rotates ``q`` and ``k`` (or ``q`` alone: ``k`` and ``k_out`` None) into caller-owned outputs
    (include/fa.h, fa_rope). Tensors are bf16 [B, H, N, d] or [N, H, d], of any strides that are
    multiples of 8 with contiguous columns; an output may be its input. ``table`` fp32
    [max_pos, rot] holds cosines, then sines; ``positions`` int32 [axes, B, N] or [axes, N] on the
    device ([B, N] or [N] for one axis); ``sections`` the pairs of each axis. ``inverse`` turns
    backwards: the rotation's gradient."""
    if q_out is None or (k is not None and k_out is None):
        raise TypeError("outputs must be tensors")
    _rope(q, k, q_out, k_out, table, positions, sections, interleaved, inverse, stream)


def rope(q, k, table, positions, sections=None, interleaved=False, inverse=False, stream=None):
    """:func:`fa_rope` into new contiguous outputs. Returns ``(q_out, k_out)``, or ``q_out`` where
    ``k`` is None."""
    if stream is None and _compiled is not None:
        out = _compiled.rope(q, k, table, positions, sections, interleaved, inverse)
        if out is not None:
            if type(out) is int:
                raise FAError(out, "fa_rope")
            return out
    with _allocating(stream, q):
        q_out, k_out = _rope(q, k, None, None, table, positions, sections, interleaved, inverse, stream)
    _given(stream, q_out, k_out)
    return q_out if k is None else (q_out, k_out)


def _tokens_view(t, name, index):
    """(tokens, heads, d, token stride) of a packed bf16 CUDA tensor [tokens, heads, d] whose heads
    and columns are contiguous (its tokens may be further apart)."""
    import torch

    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be a bfloat16 tensor")
    shape = t.shape
    if len(shape) != 3 or not t.is_cuda or t.get_device() != index or 0 in shape:
        raise ValueError(f"{name} must be a non-empty tensor [tokens, heads, d] on device {index}")
    n, h, d = shape
    sn, sh, sd = t.stride()
    if sd != 1 or (h > 1 and sh != d):
        raise ValueError(f"{name}: heads and columns of a token must be contiguous")
    return n, h, d, sn if n > 1 else h * d


def _cache_view(k_cache, v_cache, k_scale, v_scale, index):
    """(fa_paged_cache, Hkv, d) of a cache's tensors."""
    import torch

    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError(f"k_cache and v_cache must be [num_pages, Hkv, page_size, d], got {tuple(shape)} and "
                         f"{tuple(v_cache.shape)}")
    pages, heads, size, d = shape
    kt, vt, u8, f8, f32 = k_cache.dtype, v_cache.dtype, torch.uint8, torch.float8_e4m3fn, torch.float32
    if ((kt is u8 or kt is f8) and (vt is u8 or vt is f8) and k_scale.dtype is f32 and v_scale.dtype is f32
            and k_scale.shape == (pages, heads) == v_scale.shape and k_cache.is_contiguous()
            and v_cache.is_contiguous() and k_scale.is_contiguous() and v_scale.is_contiguous()
            and k_cache.get_device() == index == v_cache.get_device()
            and k_scale.get_device() == index == v_scale.get_device()):
        return _PAGED_CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages,
                                 heads, size, d), heads, d
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.dtype is not torch.float8_e4m3fn and t.dtype is not torch.uint8:
            raise TypeError(f"{name} must hold e4m3 codes (uint8 or float8_e4m3fn), got {t.dtype}")
        if not t.is_contiguous() or t.get_device() != index:
            raise ValueError(f"{name} must be contiguous on device {index}")
    for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if t.dtype is not torch.float32:
            raise TypeError(f"{name} must be float32, got {t.dtype}")
        if tuple(t.shape) != (pages, heads) or not t.is_contiguous() or t.get_device() != index:
            raise ValueError(f"{name} must be contiguous {(pages, heads)} on device {index}")
    raise ValueError("k_cache, v_cache, k_scale and v_scale do not agree")


def _batch_view(page_table, cu_seqlens, seqlens_k, index):
    """(B, max_pages) of a batch's device arrays."""
    import torch

    i32 = torch.int32
    shape = page_table.shape
    if (page_table.dtype is i32 and cu_seqlens.dtype is i32 and seqlens_k.dtype is i32 and len(shape) == 2
            and shape[0] > 0 and cu_seqlens.shape == (shape[0] + 1,) and seqlens_k.shape == (shape[0],)
            and page_table.is_contiguous() and cu_seqlens.is_contiguous() and seqlens_k.is_contiguous()
            and page_table.get_device() == index == cu_seqlens.get_device() and seqlens_k.get_device() == index):
        return shape
    for t, name in ((page_table, "page_table"), (cu_seqlens, "cu_seqlens"), (seqlens_k, "seqlens_k")):
        if t.dtype is not torch.int32 or not t.is_contiguous() or t.get_device() != index:
            raise ValueError(f"{name} must be contiguous int32 on device {index}")
    raise ValueError("page_table [B, max_pages], cu_seqlens [B+1] and seqlens_k [B] must agree on B >= 1")


def _check_out(t, name, shape, dtype, index):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"{name} must be contiguous {shape} on device {index}, got {tuple(t.shape)}")


def _append(q, k, v, q_out, make, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens, seqlens_k, max_seqlen,
            table, positions, sections, interleaved, stream):
    """The checks and the call of fa_kv_append_fp8; ``make``: allocate q_out."""
    import torch

    index = k.get_device()
    n, hkv, d, ks = _tokens_view(k, "k", index)
    vn, vh, vd, vs = _tokens_view(v, "v", index)
    cache, heads, width = _cache_view(k_cache, v_cache, k_scale, v_scale, index)
    if (vn, vh, vd) != (n, hkv, d) or (heads, width) != (hkv, d):
        raise ValueError(f"k {tuple(k.shape)}, v {tuple(v.shape)} and a cache of {heads} heads of {width} do not agree")
    B, max_pages = _batch_view(page_table, cu_seqlens, seqlens_k, index)
    H = qs = qp = op = 0
    if q is not None:
        qn, H, qd, qs = _tokens_view(q, "q", index)
        if (qn, qd) != (n, d):
            raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} do not agree")
        if make:
            q_out = torch.empty((n, H, d), dtype=torch.bfloat16, device=q.device)
        else:
            _check_out(q_out, "q_out", (n, H, d), torch.bfloat16, index)
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    rope = None
    if table is not None:
        axes = positions.shape[0] if positions is not None and positions.dim() == 2 else 1
        rope = _rotation(table, positions, axes, sections, interleaved, (n,), index)
    elif positions is not None:
        raise ValueError("positions without a table")
    st = _on_stream(index, stream, load_library().fa_kv_append_fp8, qp, k.data_ptr(), v.data_ptr(), op, rope, cache,
                    page_table.data_ptr(), cu_seqlens.data_ptr(), seqlens_k.data_ptr(), B, H, n, _int32(max_seqlen),
                    max_pages, qs, ks, vs)
    if st != FA_OK:
        raise FAError(st, "fa_kv_append_fp8")
    return q_out


def fa_kv_append_fp8(q, k, v, q_out, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens, seqlens_k,
                     max_seqlen: int, table=None, positions=None, sections=None, interleaved=False, stream=None):
    """Appends keys (rotated) and values to a paged e4m3 cache in place and rotates the queries
    (include/fa.h, fa_kv_append_fp8). ``q`` [total, H, d] into ``q_out`` (both may be None), ``k`` and
    ``v`` bf16 [total, Hkv, d], whose tokens may be strided (a fused projection's rows); ``k_cache``
    and ``v_cache`` [num_pages, Hkv, page_size, d] e4m3 codes, ``k_scale`` and ``v_scale`` fp32
    [num_pages, Hkv]; ``page_table`` int32 [B, max_pages], ``cu_seqlens`` int32 [B+1] of the new
    tokens (``max_seqlen`` the most of a sequence), ``seqlens_k`` int32 [B] the cache lengths with
    them. ``table`` None: no rotation; ``positions`` None: the cache positions."""
    _append(q, k, v, q_out, False, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens, seqlens_k, max_seqlen,
            table, positions, sections, interleaved, stream)


def kv_append_fp8(q, k, v, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens, seqlens_k, max_seqlen: int,
                  table=None, positions=None, sections=None, interleaved=False, stream=None):
    """:func:`fa_kv_append_fp8` into new rotated queries; returns them (None without ``q``). Tokens
    past ``cu_seqlens[B]`` are left as allocated."""
    if stream is None and _compiled is not None:
        out = _compiled.append(q, k, v, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens, seqlens_k, max_seqlen,
                            table, positions, sections, interleaved)
        if out is not None:
            if type(out) is int:
                raise FAError(out, "fa_kv_append_fp8")
            return None if out is True else out
    with _allocating(stream, k):
        q_out = _append(q, k, v, None, True, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens, seqlens_k,
                        max_seqlen, table, positions, sections, interleaved, stream)
    _given(stream, q_out)
    return q_out


def fa_paged_num_splits(B: int, H: int, Hkv: int, max_seqlen_q: int, max_seqlen_k: int, d: int, window: int = 0,
                        sinks: int = 0) -> int:
    """The key splits the library proposes for a paged call (0 for arguments out of range)."""
    return load_library().fa_paged_num_splits(
        *map(_int32, (B, H, Hkv, max_seqlen_q, max_seqlen_k, d, window, sinks)))


def fa_paged_workspace_bytes(total_q: int, H: int, d: int, num_splits: int) -> int:
    return load_library().fa_paged_workspace_bytes(*map(_int32, (total_q, H, d, num_splits)))


def _paged(q, k_cache, v_cache, k_scale, v_scale, o, lse, page_table, cu_seqlens_q, seqlens_k, max_seqlen_q,
           max_seqlen_k, workspace, num_splits, window, sinks, scale, stream):
    """The checks and the call of fa_fwd_paged_fp8; ``o`` None: outputs and the workspace are
    allocated (``num_splits`` None: the library's proposal). Returns ``(o, lse)``."""
    import torch

    index = q.get_device()
    n, H, d, qs = _tokens_view(q, "q", index)
    if qs != H * d:
        raise ValueError("q must be contiguous")
    cache, hkv, width = _cache_view(k_cache, v_cache, k_scale, v_scale, index)
    if width != d:
        raise ValueError(f"q has head dim {d}, the cache {width}")
    B, max_pages = _batch_view(page_table, cu_seqlens_q, seqlens_k, index)
    for x in (max_seqlen_q, max_seqlen_k, window, sinks, num_splits or 1):
        _int32(x)
    lib = load_library()
    if o is None:
        if num_splits is None:
            num_splits = lib.fa_paged_num_splits(B, H, hkv, max_seqlen_q, max_seqlen_k, d, window, sinks) or 1
        device = q.device
        o = torch.empty((n, H, d), dtype=torch.bfloat16, device=device)
        lse = torch.empty((H, n), dtype=torch.float32, device=device)
        if num_splits > 1:
            workspace = torch.empty(lib.fa_paged_workspace_bytes(n, H, d, num_splits) // 4, dtype=torch.float32,
                                    device=device)
    else:
        _check_out(o, "o", (n, H, d), torch.bfloat16, index)
        _check_out(lse, "lse", (H, n), torch.float32, index)
        if num_splits > 1:
            _need_workspace(workspace, fa_paged_workspace_bytes(n, H, d, num_splits), "workspace", q.device)
    st = _on_stream(index, stream, lib.fa_fwd_paged_fp8, q.data_ptr(), cache, page_table.data_ptr(),
                    cu_seqlens_q.data_ptr(), seqlens_k.data_ptr(), o.data_ptr(), lse.data_ptr(),
                    workspace.data_ptr() if num_splits > 1 else 0, B, H, n, max_seqlen_q, max_seqlen_k, max_pages,
                    default_scale(d) if scale is None else float(scale), window, sinks, num_splits)
    if st != FA_OK:
        raise FAError(st, "fa_fwd_paged_fp8")
    return o, lse


def fa_fwd_paged_fp8(q, k_cache, v_cache, k_scale, v_scale, o, lse, page_table, cu_seqlens_q, seqlens_k,
                     max_seqlen_q: int, max_seqlen_k: int, workspace=None, num_splits: int = 1, window: int = 0,
                     sinks: int = 0, scale: float | None = None, stream=None):
    """Attention of ``q`` bf16 [total_q, H, d] (the last tokens of each sequence) over a paged e4m3
    cache into caller-owned ``o`` bf16 [total_q, H, d] and ``lse`` fp32 [H, total_q] (include/fa.h,
    fa_fwd_paged_fp8). ``workspace`` fp32 of at least ``fa_paged_workspace_bytes`` bytes where
    ``num_splits > 1``."""
    if o is None:
        raise TypeError("o and lse must be tensors")
    _paged(q, k_cache, v_cache, k_scale, v_scale, o, lse, page_table, cu_seqlens_q, seqlens_k, max_seqlen_q,
           max_seqlen_k, workspace, num_splits, window, sinks, scale, stream)


def attention_paged_fp8(q, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens_q, seqlens_k,
                        max_seqlen_q: int, max_seqlen_k: int, window: int = 0, sinks: int = 0,
                        scale: float | None = None, num_splits: int | None = None, stream=None):
    """:func:`fa_fwd_paged_fp8` into new outputs, with a workspace of its own (``num_splits`` None:
    the library's proposal). Returns ``(o, lse)``; rows past ``cu_seqlens_q[B]`` are left as
    allocated."""
    if stream is None and _compiled is not None:
        out = _compiled.paged(q, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens_q, seqlens_k, max_seqlen_q,
                           max_seqlen_k, window, sinks, scale, num_splits)
        if out is not None:
            if type(out) is int:
                raise FAError(out, "fa_fwd_paged_fp8")
            return out
    with _allocating(stream, q):
        o, lse = _paged(q, k_cache, v_cache, k_scale, v_scale, None, None, page_table, cu_seqlens_q, seqlens_k,
                        max_seqlen_q, max_seqlen_k, None, num_splits, window, sinks, scale, stream)
    return _given(stream, o, lse)


# ------------------------------------------------ sliding windows, grouped heads
def _grouped(q, k, v):
    import torch

    index = q.get_device()
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if t.dtype is not torch.bfloat16:
            raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
        if t.dim() != 4 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{name} must be a contiguous CUDA tensor [B, H, N, d]")
        if t.get_device() != index:
            raise ValueError("q, k and v must be on the same device")
    B, H, Nq, d = q.shape
    Bk, Hkv, Nk, dk = k.shape
    if (Bk, dk) != (B, d) or v.shape != k.shape:
        raise ValueError(f"shape mismatch q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)}")
    return B, H, Hkv, Nq, Nk, d, index


def fa_fwd_window(q, k, v, o, lse, window: int, sinks: int = 0, scale: float | None = None, stream=None):
    """Sliding-window forward with sinks into caller-owned ``o`` (bf16 [B,H,Nq,d]) and ``lse`` (fp32
    [B,H,Nq]); ``k`` and ``v`` [B,Hkv,Nk,d], H a multiple of Hkv (include/fa.h, fa_fwd_window).
    ``window`` 0: no window, the bottom-right causal mask."""
    import torch

    B, H, Hkv, Nq, Nk, d, index = _grouped(q, k, v)
    _check_out(o, "o", (B, H, Nq, d), torch.bfloat16, index)
    _check_out(lse, "lse", (B, H, Nq), torch.float32, index)
    st = _on_stream(index, stream, load_library().fa_fwd_window, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                    o.data_ptr(), lse.data_ptr(), B, H, Hkv, Nq, Nk, d, default_scale(d) if scale is None else float(scale),
                    _int32(window), _int32(sinks))
    _check(st, "fa_fwd_window")


def fa_window_num_splits(B: int, H: int, Hkv: int, Nq: int, Nk: int, d: int, window: int, sinks: int = 0) -> int:
    """The key splits the library proposes for a windowed forward (0 for arguments out of range)."""
    return load_library().fa_window_num_splits(*map(_int32, (B, H, Hkv, Nq, Nk, d, window, sinks)))


def fa_fwd_window_splitkv(q, k, v, workspace, num_splits: int, window: int, sinks: int = 0,
                          scale: float | None = None, stream=None):
    """The windowed forward with split keys: partial states into ``workspace`` (fp32, at least
    ``fa_splitkv_workspace_bytes`` bytes), merged by :func:`fa_combine`."""
    B, H, Hkv, Nq, Nk, d, index = _grouped(q, k, v)
    _need_workspace(workspace, fa_splitkv_workspace_bytes(B, H, Nq, d, num_splits), "workspace", q.device)
    st = _on_stream(index, stream, load_library().fa_fwd_window_splitkv, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                    workspace.data_ptr(), B, H, Hkv, Nq, Nk, d, default_scale(d) if scale is None else float(scale),
                    _int32(window), _int32(sinks), _int32(num_splits))
    _check(st, "fa_fwd_window_splitkv")


def attention_window(q, k, v, window: int, sinks: int = 0, scale: float | None = None, num_splits: int | None = None,
                     stream=None):
    """Allocate ``o`` and ``lse`` and run :func:`fa_fwd_window`, or :func:`fa_fwd_window_splitkv` and the
    merge (``num_splits`` None: as the library proposes). Returns ``(o, lse)``."""
    if stream is None and _compiled is not None:
        out = _compiled.window(q, k, v, window, sinks, scale, num_splits)
        if out is not None:
            if type(out) is int:
                raise FAError(out, "fa_fwd_window")
            return out
    import torch

    B, H, Hkv, Nq, Nk, d, index = _grouped(q, k, v)
    if num_splits is None:
        num_splits = fa_window_num_splits(B, H, Hkv, Nq, Nk, d, window, sinks) or 1
    with _allocating(stream, q):
        o = torch.empty_like(q)
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
        if num_splits == 1:
            fa_fwd_window(q, k, v, o, lse, window, sinks, scale, stream)
        else:
            nbytes = fa_splitkv_workspace_bytes(B, H, Nq, d, num_splits)
            if nbytes == 0:
                raise FAError(5, "fa_fwd_window_splitkv")
            ws = torch.empty(nbytes // 4, dtype=torch.float32, device=q.device)
            fa_fwd_window_splitkv(q, k, v, ws, num_splits, window, sinks, scale, stream)
            st = _on_stream(index, stream, load_library().fa_combine, ws.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H,
                            Nq, d, num_splits)
            _check(st, "fa_combine")
    return _given(stream, o, lse)


def fa_bwd_window_workspace_bytes(B: int, H: int, Hkv: int, Nq: int, Nk: int, d: int, window: int,
                                  sinks: int = 0) -> int:
    return load_library().fa_bwd_window_workspace_bytes(*map(_int32, (B, H, Hkv, Nq, Nk, d, window, sinks)))


def fa_bwd_window(q, k, v, o, dout, lse, dq, dk, dv, workspace, window: int, sinks: int = 0,
                  scale: float | None = None, stream=None):
    """Backward of :func:`fa_fwd_window` into caller-owned ``dq``, ``dk``, ``dv`` (bf16, shaped like q,
    k, v); ``workspace`` fp32 of at least ``fa_bwd_window_workspace_bytes`` bytes."""
    import torch

    B, H, Hkv, Nq, Nk, d, index = _grouped(q, k, v)
    for t, name, like in ((o, "o", q), (dout, "dout", q), (dq, "dq", q), (dk, "dk", k), (dv, "dv", k)):
        _check_out(t, name, tuple(like.shape), torch.bfloat16, index)
    _check_out(lse, "lse", (B, H, Nq), torch.float32, index)
    _need_workspace(workspace, fa_bwd_window_workspace_bytes(B, H, Hkv, Nq, Nk, d, window, sinks), "workspace",
                    q.device)
    st = _on_stream(index, stream, load_library().fa_bwd_window, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                    o.data_ptr(), dout.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                    workspace.data_ptr(), B, H, Hkv, Nq, Nk, d, default_scale(d) if scale is None else float(scale),
                    _int32(window), _int32(sinks))
    _check(st, "fa_bwd_window")


def attention_window_backward(q, k, v, o, lse, dout, window: int, sinks: int = 0, scale: float | None = None,
                              stream=None):
    """Allocate ``(dq, dk, dv)`` and the workspace and run :func:`fa_bwd_window`."""
    if stream is None and _compiled is not None:
        out = _compiled.window_backward(q, k, v, o, lse, dout, window, sinks, scale)
        if out is not None:
            if type(out) is int:
                raise FAError(out, "fa_bwd_window")
            return out
    import torch

    B, H, Hkv, Nq, Nk, d, _ = _grouped(q, k, v)
    nbytes = fa_bwd_window_workspace_bytes(B, H, Hkv, Nq, Nk, d, window, sinks)
    with _allocating(stream, q):
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        ws = torch.empty(max(1, nbytes // 4), dtype=torch.float32, device=q.device)
        fa_bwd_window(q, k, v, o, dout, lse, dq, dk, dv, ws, window, sinks, scale, stream)
    return _given(stream, dq, dk, dv)


_SIDE_STREAMS = {}


def _side_streams(device):
    """Two streams per device, for host-to-device and device-to-host copies."""
    import torch

    key = torch.device(device).index
    if key not in _SIDE_STREAMS:
        _SIDE_STREAMS[key] = (torch.cuda.Stream(device=device), torch.cuda.Stream(device=device))
    return _SIDE_STREAMS[key]


def head_slices(BH: int, chunks: int):
    """The ``(h0, h1)`` bounds :func:`fa_fwd_from_host` cuts ``BH`` heads into:
    at most ``chunks`` non-empty slices of consecutive heads covering
    ``[0, BH)``. With three or more, the last two slices get a half and a
    quarter of the others' share: the last slice's kernel and copy back run
    after every copy in has finished, so a smaller last slice leaves less of
    the call uncovered."""
    chunks = max(1, min(int(chunks), BH))
    weights = [1.0] * (chunks - 2) + [0.5, 0.25] if chunks >= 3 else [1.0] * chunks
    total = sum(weights)
    bounds, acc, prev = [], 0.0, 0
    for w in weights:
        acc += w
        cur = min(BH, int(round(BH * acc / total)))
        if cur > prev:
            bounds.append((prev, cur))
            prev = cur
    if prev < BH:
        bounds.append((prev, BH))
    return bounds


def fa_fwd_from_host(q_host, k_host, v_host, o_host, lse_host, q, k, v, o, lse, causal=False,
                     scale: float | None = None, chunks: int = 4, stream=None):
    """The forward of :func:`fa_fwd` on inputs and outputs in pinned host memory.

    ``q_host``, ``k_host``, ``v_host`` (bf16 [B,H,N,d]) are copied into the
    device tensors ``q``, ``k``, ``v`` of the same shapes, the forward writes the
    device ``o``, ``lse``, and they are copied back into ``o_host``, ``lse_host``.
    The (b, h) heads are cut into at most ``chunks`` slices of consecutive heads
    (:func:`head_slices`; contiguous in every tensor, each slice runs as one
    forward over its heads) so that the copies of one slice overlap the kernel
    of another:
    host-to-device copies on one side stream, the kernels on ``stream``,
    device-to-host copies on another. Every call starts after the work already
    queued on ``stream`` and ``stream`` waits for the last copy back, so a caller
    synchronises on ``stream`` alone.
    """
    import torch

    B, H, Nq, Nk, d = _bhnd(q, k, v)
    _need_o_lse(o, lse, B, H, Nq, d, q.device)
    cpu = torch.device("cpu")
    for name, t, dev_t in (("q_host", q_host, q), ("k_host", k_host, k), ("v_host", v_host, v),
                           ("o_host", o_host, o), ("lse_host", lse_host, lse)):
        _need(t, name, tuple(dev_t.shape), dev_t.dtype, cpu)
        if not t.is_pinned():
            raise ValueError(f"{name} must be in pinned host memory")
    BH = B * H
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    s_in, s_out = _side_streams(q.device)
    s_in.wait_stream(stream)
    # Heads flattened: [1, B*H, N, d] views (contiguous tensors, checked above).
    flat = lambda t: t.view(1, BH, *t.shape[2:])  # noqa: E731
    qh, kh, vh, oh, lh = (flat(t) for t in (q_host, k_host, v_host, o_host, lse_host))
    qd, kd, vd, od, ld = (flat(t) for t in (q, k, v, o, lse))
    bounds = head_slices(BH, chunks)
    done_out = None
    for h0, h1 in bounds:
        with torch.cuda.stream(s_in):
            for src, dst in ((qh, qd), (kh, kd), (vh, vd)):
                dst[:, h0:h1].copy_(src[:, h0:h1], non_blocking=True)
            ev_in = torch.cuda.Event()
            ev_in.record(s_in)
        stream.wait_event(ev_in)
        fa_fwd(qd[:, h0:h1], kd[:, h0:h1], vd[:, h0:h1], od[:, h0:h1], ld[:, h0:h1], causal, scale, stream)
        ev_c = torch.cuda.Event()
        ev_c.record(stream)
        s_out.wait_event(ev_c)
        with torch.cuda.stream(s_out):
            oh[:, h0:h1].copy_(od[:, h0:h1], non_blocking=True)
            lh[:, h0:h1].copy_(ld[:, h0:h1], non_blocking=True)
            done_out = torch.cuda.Event()
            done_out.record(s_out)
    stream.wait_event(done_out)
