"""Python binding of the HIP library ``libtw.so`` (C ABI in ``include/tw.h``).

Argument marshalling only: every step of the forward runs in the library's
gfx950 kernels.  PyTorch provides device memory and the current HIP stream.
Importing this module fails loudly when the library has not been built
(``python -m activation_sparse_feed_gate_amd.build``); there is no fallback.

Low-level functions carry the C names and take preallocated tensors:
``tw_pack_gate`` (and ``tw_pack_gate_noalloc``, which takes no workspace),
``tw_sparse_ffn_fwd``, ``tw_ffn_fwd``, ``tw_workspace_bytes``,
``tw_ffn_workspace_bytes``, ``tw_gate_dense``, ``tw_pack_dense`` and the
hybrid training storage ``tw_hybrid_pack``, ``tw_hybrid_up``,
``tw_hybrid_down`` with its backward ``tw_hybrid_bwd_dh``, ``tw_hybrid_bwd_dx``,
``tw_hybrid_bwd_dw``.  ``pack_gate``, ``pack_unfused``, ``sparse_ffn``, ``ffn``,
``hybrid_forward`` and ``hybrid_backward`` allocate their outputs and return
them.

The layer norm in front of the block is ``tw_layernorm_fwd`` and
``tw_layernorm_bwd`` (allocating: ``layernorm``, ``layernorm_backward``); the
block's dense projections on 8-bit integers are ``tw_quant_rows``,
``tw_layernorm_quant``, ``tw_quant_linear`` and ``tw_quant_gateup``
(allocating: ``quantize_rows``, ``layernorm_quantize``, ``quant_linear``,
``quant_gateup``).

The dense training step is the RMS norm (``tw_rmsnorm_fwd``, ``tw_rmsnorm_quant``,
``tw_rmsnorm_bwd``; allocating: ``rmsnorm``, ``rmsnorm_quantize``,
``rmsnorm_backward``), the gated FFN (``tw_gated_ffn_fwd``, ``tw_gated_ffn_bwd``;
``gated_ffn``, ``gated_ffn_backward``), the cross entropy of the output projection
(``tw_linear_ce_fwd``, ``tw_linear_ce_bwd``; ``linear_ce``, ``linear_ce_backward``)
and gradient clipping (``tw_grad_norm``, ``tw_grad_clip``; ``grad_norm``,
``clip_grads``).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import warnings

import torch  # loads the HIP runtime the library links against

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(_HERE, "libtw.so")

if not os.path.exists(LIBRARY):
    raise ImportError(
        f"{LIBRARY} is missing: build it with `python -m activation_sparse_feed_gate_amd.build`")

_lib = ctypes.CDLL(LIBRARY)
# The small allocating calls (layernorm, quant_linear, ...) in native code: it
# checks, allocates and calls the library, and returns None for any argument
# that is not as the library needs it; the call is then made through the
# low-level function here, whose checks raise.  It is bound to one build of
# torch: where it does not load, every call takes the second way (the same
# kernels, with more host time a call).
try:
    from . import _tw_calls as _calls  # built beside the library
except ImportError as _e:
    warnings.warn(f"the native part of the binding does not load ({_e}): the allocating calls "
                  "take more host time each; build it with "
                  "`python -m activation_sparse_feed_gate_amd.build`", RuntimeWarning, stacklevel=2)

    class _calls:  # noqa: N801
        layernorm = layernorm_backward = quant_linear = quant_gateup = staticmethod(lambda *a: None)
        rmsnorm = rmsnorm_quantize = rmsnorm_backward = layernorm
        gated_ffn = gated_ffn_backward = linear_ce = linear_ce_backward = clip_grads = layernorm


_vp = ctypes.c_void_p
_i = ctypes.c_int
_sz = ctypes.c_size_t

_lib.tw_status_str.restype = ctypes.c_char_p
_lib.tw_status_str.argtypes = [_i]
_lib.tw_last_error.restype = ctypes.c_char_p
_lib.tw_last_error.argtypes = []
_lib.tw_workspace_bytes.restype = _sz
_lib.tw_workspace_bytes.argtypes = [_i] * 6
_lib.tw_ffn_workspace_bytes.restype = _sz
_lib.tw_ffn_workspace_bytes.argtypes = [_i] * 3
_lib.tw_pack_gate.restype = _i
_lib.tw_pack_gate.argtypes = [_vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp,
                              _vp, _sz, _vp, _vp]
_lib.tw_pack_gate_noalloc.restype = _i
_lib.tw_pack_gate_noalloc.argtypes = [_vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _i,
                                      _vp, _vp, _vp]
_lib.tw_sparse_ffn_fwd.restype = _i
_lib.tw_sparse_ffn_fwd.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp,
                                   _vp, _i, _vp, _vp, _sz, _vp, _vp]
_lib.tw_ffn_fwd.restype = _i
_lib.tw_ffn_fwd.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _sz, _vp, _vp]
_lib.tw_gate_dense.restype = _i
_lib.tw_gate_dense.argtypes = [_vp, _vp, _i, _i, _i, _vp, _vp, _vp]
_lib.tw_pack_dense_workspace_bytes.restype = _sz
_lib.tw_pack_dense_workspace_bytes.argtypes = [_i, _i]
_lib.tw_pack_dense.restype = _i
_lib.tw_pack_dense.argtypes = [_vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp, _sz, _vp,
                               _vp]
_lib.tw_hybrid_pack.restype = _i
_lib.tw_hybrid_pack.argtypes = [_i, _i, _i, _i, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp,
                                _i, _vp, _vp]
_lib.tw_hybrid_up.restype = _i
_lib.tw_hybrid_up.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _i,
                              _vp, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.tw_hybrid_down_workspace_bytes.restype = _sz
_lib.tw_hybrid_down_workspace_bytes.argtypes = [_i]
_lib.tw_hybrid_down.restype = _i
_lib.tw_hybrid_down.argtypes = [_vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp,
                                _vp, _sz, _vp, _vp]
_lib.tw_hybrid_bwd_dh.restype = _i
_lib.tw_hybrid_bwd_dh.argtypes = [_vp, _vp, _i, _i, _i, _i, ctypes.c_float, _vp, _vp, _vp, _vp,
                                  _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.tw_hybrid_bwd_dx_workspace_bytes.restype = _sz
_lib.tw_hybrid_bwd_dx_workspace_bytes.argtypes = [_i]
_lib.tw_hybrid_bwd_dx.restype = _i
_lib.tw_hybrid_bwd_dx.argtypes = [_vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                  _i, _vp, _vp, _vp, _vp, _sz, _vp, _vp]
_lib.tw_hybrid_bwd_dw_workspace_bytes.restype = _sz
_lib.tw_hybrid_bwd_dw_workspace_bytes.argtypes = [_i] * 5
_lib.tw_hybrid_bwd_dw.restype = _i
_lib.tw_hybrid_bwd_dw.argtypes = [_vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                  _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp]

_i64, _f = ctypes.c_int64, ctypes.c_float
_lib.tw_layernorm_fwd.restype = _i
_lib.tw_layernorm_fwd.argtypes = [_vp, _i, _i64, _vp, _i, _vp, _vp, _f, _i, _i, _vp, _vp, _i, _vp,
                                  _vp, _vp, _vp]
_lib.tw_layernorm_bwd_workspace_bytes.restype = _sz
_lib.tw_layernorm_bwd_workspace_bytes.argtypes = [_i, _i]
_lib.tw_layernorm_bwd.restype = _i
_lib.tw_layernorm_bwd.argtypes = [_vp, _i, _vp, _i, _i64, _vp, _vp, _vp, _vp, _i, _i, _vp, _i, _vp,
                                  _vp, _vp, _sz, _vp, _vp]
_lib.tw_quant_rows.restype = _i
_lib.tw_quant_rows.argtypes = [_vp, _i, _i64, _i, _i, _vp, _vp, _vp, _vp]
_lib.tw_layernorm_quant.restype = _i
_lib.tw_layernorm_quant.argtypes = [_vp, _i, _i64, _vp, _i, _vp, _vp, _f, _i, _i, _vp, _vp, _vp,
                                    _vp, _vp]
_lib.tw_quant_workspace_bytes.restype = _sz
_lib.tw_quant_workspace_bytes.argtypes = [_i, _i]
_lib.tw_quant_linear.restype = _i
_lib.tw_quant_linear.argtypes = [_vp, _i, _i64, _vp, _vp, _vp, _vp, _i, _i, _i, _vp, _i, _vp, _sz,
                                 _vp, _vp]
_lib.tw_quant_gateup.restype = _i
_lib.tw_quant_gateup.argtypes = [_vp, _i, _i64, _vp, _vp, _vp, _f, _vp, _vp, _vp, _vp, _i, _i, _i,
                                 _vp, _i, _vp, _sz, _vp, _vp]

_lib.tw_rmsnorm_fwd.restype = _i
_lib.tw_rmsnorm_fwd.argtypes = [_vp, _i, _i64, _vp, _i, _vp, _f, _i, _i, _vp, _vp, _i, _vp, _vp,
                                _vp]
_lib.tw_rmsnorm_quant.restype = _i
_lib.tw_rmsnorm_quant.argtypes = [_vp, _i, _i64, _vp, _i, _vp, _f, _i, _i, _vp, _vp, _vp, _vp, _vp]
_lib.tw_rmsnorm_bwd_workspace_bytes.restype = _sz
_lib.tw_rmsnorm_bwd_workspace_bytes.argtypes = [_i, _i]
_lib.tw_rmsnorm_bwd.restype = _i
_lib.tw_rmsnorm_bwd.argtypes = [_vp, _i, _vp, _i, _i64, _vp, _vp, _vp, _i, _i, _vp, _i, _vp, _vp,
                                _sz, _vp, _vp]
_lib.tw_gated_ffn_workspace_bytes.restype = _sz
_lib.tw_gated_ffn_workspace_bytes.argtypes = [_i] * 3
_lib.tw_gated_ffn_fwd.restype = _i
_lib.tw_gated_ffn_fwd.argtypes = [_vp, _i64, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _i, _vp,
                                  _sz, _vp, _vp]
_lib.tw_gated_ffn_bwd_workspace_bytes.restype = _sz
_lib.tw_gated_ffn_bwd_workspace_bytes.argtypes = [_i] * 3
_lib.tw_gated_ffn_bwd.restype = _i
_lib.tw_gated_ffn_bwd.argtypes = [_vp, _vp, _i64, _vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _vp, _i,
                                  _vp, _vp, _vp, _i, _vp, _sz, _vp, _vp]
_lib.tw_linear_ce_workspace_bytes.restype = _sz
_lib.tw_linear_ce_workspace_bytes.argtypes = [_i] * 3
_lib.tw_linear_ce_fwd.restype = _i
_lib.tw_linear_ce_fwd.argtypes = [_vp, _i64, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _sz, _vp, _vp]
_lib.tw_linear_ce_bwd_workspace_bytes.restype = _sz
_lib.tw_linear_ce_bwd_workspace_bytes.argtypes = [_i] * 3
_lib.tw_linear_ce_bwd.restype = _i
_lib.tw_linear_ce_bwd.argtypes = [_vp, _vp, _i64, _vp, _vp, _i, _vp, _i, _i, _i, _vp, _i, _vp, _i,
                                  _vp, _sz, _vp, _vp]
_lib.tw_grad_norm_workspace_bytes.restype = _sz
_lib.tw_grad_norm_workspace_bytes.argtypes = [_i, _vp]
_lib.tw_grad_norm.restype = _i
_lib.tw_grad_norm.argtypes = [_i, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp]
_lib.tw_grad_clip.restype = _i
_lib.tw_grad_clip.argtypes = [_i, _vp, _vp, _vp, _vp, _vp, _f, _f, _vp, _vp, _sz, _vp, _vp]

TW_OK, TW_EINVAL, TW_EUNSUPPORTED, TW_EHIP = 0, 1, 2, 3
TW_BF16, TW_F32, TW_INT8, TW_INT32, TW_INT64 = 0, 1, 2, 3, 4
TW_RELU, TW_SILU, TW_GELU = 0, 1, 2
_ACT = {"relu": TW_RELU, "silu": TW_SILU, "gelu": TW_GELU}


class TwError(RuntimeError):
    """A non-OK status from the library."""

    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.tw_last_error().decode(errors="replace")
        super().__init__(f"{where}: {_lib.tw_status_str(status).decode()}: {msg}")


def _check(status: int, where: str) -> None:
    if status != TW_OK:
        raise TwError(status, where)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous device tensors")
    return t.data_ptr()


def _rows_ptr(t):
    """Address of a tensor whose rows ``_Args.rows`` has checked."""
    if not t.is_cuda:
        raise ValueError("tensors passed to the library must be device tensors")
    return t.data_ptr()


_F32, _I32, _BF16, _U8T = torch.float32, torch.int32, torch.bfloat16, torch.uint8
_I8 = torch.int8
_I64 = torch.int64
_TYPE = {_BF16: TW_BF16, _F32: TW_F32, _I8: TW_INT8, _I32: TW_INT32, _I64: TW_INT64}
_FLOATS = (_BF16, _F32)


class _Args:
    """Checks every tensor of one call against the shape, dtype and device
    the kernels assume.  The C ABI receives bare pointers and cannot see a
    buffer's size, so a tensor of the wrong shape (say a packing made for
    another T or C) would be read or written out of bounds on the device:
    such calls raise here, before the library is called."""

    def __init__(self, where, ref):
        self.where = where
        self.device = ref.device

    def _common(self, t, name, dtype):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{self.where}: {name} must be a tensor, got {type(t).__name__}")
        if t.dtype != dtype:
            raise TypeError(f"{self.where}: {name} must be {dtype}, got {t.dtype}")
        if t.device != self.device:
            raise ValueError(f"{self.where}: {name} is on {t.device}, the inputs on {self.device}")

    def shape(self, t, name, dtype, shape):
        """t must have exactly this shape (None: t may be None)."""
        if (type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape
                and t.device == self.device):
            return
        if t is None:
            raise ValueError(f"{self.where}: {name} is required")
        self._common(t, name, dtype)
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{self.where}: {name} has shape {tuple(t.shape)}, "
                             f"expected {tuple(shape)}")

    def opt(self, t, name, dtype, shape):
        if t is not None:
            self.shape(t, name, dtype, shape)

    def overflow_list(self, ovf_rows, ovf_count, R_max):
        """The overflow list of tw_pack_gate: both tensors, or both None (no
        list is built)."""
        if ovf_rows is None and ovf_count is None:
            return
        self.room(ovf_rows, "ovf_rows", _I32, max(R_max, 1))
        self.room(ovf_count, "ovf_count", _I32, 1)

    def room(self, t, name, dtype, n):
        """t must be one-dimensional with at least n elements."""
        if t is None:
            raise ValueError(f"{self.where}: {name} is required")
        self._common(t, name, dtype)
        if t.dim() != 1 or t.numel() < n:
            raise ValueError(f"{self.where}: {name} has shape {tuple(t.shape)}, expected "
                             f"one dimension of at least {n} elements")

    def typed(self, t, name, dtypes, shape):
        """t has this shape and one of these dtypes; its tw_type."""
        if t is None:
            raise ValueError(f"{self.where}: {name} is required")
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{self.where}: {name} must be a tensor, got {type(t).__name__}")
        dtype = t.dtype
        if dtype not in dtypes:
            raise TypeError(f"{self.where}: {name} must be one of {dtypes}, got {dtype}")
        self.shape(t, name, dtype, shape)
        return _TYPE[dtype]

    def rows(self, t, name, dtypes):
        """t is [M][K] with contiguous rows, any distance apart (a single
        row's distance counts as K): its tw_type and the row distance."""
        M, K = t.shape
        kind = self.typed(t, name, dtypes, (M, K))
        if t.is_contiguous():
            return kind, K
        if K > 1 and t.stride(1) != 1:
            raise ValueError(f"{self.where}: {name} must have contiguous rows")
        return kind, (t.stride(0) if M > 1 else K)

    def bytes(self, t, name):
        """A workspace: any dtype, on the inputs' device (its size is checked
        by the library against the bytes it needs)."""
        if t is None:
            return
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{self.where}: {name} must be a tensor")
        if t.device != self.device:
            raise ValueError(f"{self.where}: {name} is on {t.device}, the inputs on {self.device}")

    def apart(self, out, name, others):
        """out and none of the named others, which the call reads after it has begun to
        write out, share memory (any of them may be None)."""
        if out is None or not out.numel():
            return
        begin, end = _span(out)
        for other, t in others.items():
            if t is None or not t.numel():
                continue
            b, e = _span(t)
            if begin < e and b < end:
                raise ValueError(f"{self.where}: {name} and {other} overlap")


def _span(t):
    """First and last address of a tensor's elements."""
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _dims2(t, name, where):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{where}: {name} must be a two-dimensional tensor")
    if max(t.shape) >= 2 ** 31:  # the library's sizes are 32-bit: it would see the rest of it
        raise ValueError(f"{where}: {name} has shape {tuple(t.shape)}, sizes must be below 2^31")
    return t.shape


def _tiles(N, T, where):
    if T <= 0 or N % T:
        raise ValueError(f"{where}: N={N} is not a multiple of the tile width T={T}")
    return N // T


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _on(t):
    """The device of a call's tensors made the current one, for the stream and
    the launches of the call."""
    if not t.is_cuda or t.device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(t.device)


def _events(events):
    if events is None:
        return None
    arr = (ctypes.c_void_p * len(events))(*[int(e) for e in events])
    return ctypes.cast(arr, ctypes.c_void_p), arr


# ----------------------------------------------------------------- C names --
def tw_workspace_bytes(M, K, N, T, C, R_max) -> int:
    return int(_lib.tw_workspace_bytes(M, K, N, T, C, R_max))


def tw_ffn_workspace_bytes(M, K, N) -> int:
    return int(_lib.tw_ffn_workspace_bytes(M, K, N))


def tw_pack_gate(x, wg_t, T, C, tw_val, tw_idx, tw_cnt, ovf_rows, ovf_count, R_max, ws,
                 z_debug=None, stream=None, events=None) -> None:
    M, K = _dims2(x, "x", "tw_pack_gate")
    N = _dims2(wg_t, "wg_t", "tw_pack_gate")[0]
    NT = _tiles(N, T, "tw_pack_gate")
    a = _Args("tw_pack_gate", x)
    a.shape(x, "x", _BF16, (M, K))
    a.shape(wg_t, "wg_t", _BF16, (N, K))
    a.shape(tw_val, "tw_val", _F32, (M, NT, C))
    a.shape(tw_idx, "tw_idx", _I32, (M, NT, C))
    a.shape(tw_cnt, "tw_cnt", _I32, (M, NT))
    a.overflow_list(ovf_rows, ovf_count, R_max)
    a.opt(z_debug, "z_debug", _F32, (M, N))
    a.bytes(ws, "ws")
    ev = _events(events)
    st = _lib.tw_pack_gate(_ptr(x), _ptr(wg_t), M, K, N, T, C, _ptr(tw_val), _ptr(tw_idx),
                           _ptr(tw_cnt), _ptr(ovf_rows), _ptr(ovf_count), R_max, _ptr(z_debug),
                           _ptr(ws), ws.numel() * ws.element_size(), _stream(stream),
                           ev[0] if ev else None)
    _check(st, "tw_pack_gate")


def tw_pack_gate_noalloc(x, wg_t, T, C, tw_val, tw_idx, tw_cnt, ovf_rows, ovf_count, R_max,
                         z_debug=None, stream=None, events=None) -> None:
    """tw_pack_gate on the library's static per-GPU scratch (no workspace)."""
    M, K = _dims2(x, "x", "tw_pack_gate_noalloc")
    N = _dims2(wg_t, "wg_t", "tw_pack_gate_noalloc")[0]
    NT = _tiles(N, T, "tw_pack_gate_noalloc")
    a = _Args("tw_pack_gate_noalloc", x)
    a.shape(x, "x", _BF16, (M, K))
    a.shape(wg_t, "wg_t", _BF16, (N, K))
    a.shape(tw_val, "tw_val", _F32, (M, NT, C))
    a.shape(tw_idx, "tw_idx", _I32, (M, NT, C))
    a.shape(tw_cnt, "tw_cnt", _I32, (M, NT))
    a.overflow_list(ovf_rows, ovf_count, R_max)
    a.opt(z_debug, "z_debug", _F32, (M, N))
    ev = _events(events)
    st = _lib.tw_pack_gate_noalloc(_ptr(x), _ptr(wg_t), M, K, N, T, C, _ptr(tw_val),
                                   _ptr(tw_idx), _ptr(tw_cnt), _ptr(ovf_rows), _ptr(ovf_count),
                                   R_max, _ptr(z_debug), _stream(stream), ev[0] if ev else None)
    _check(st, "tw_pack_gate_noalloc")


def tw_sparse_ffn_fwd(x, wg_t, wu_t, wd, T, C, tw_val, tw_idx, tw_cnt, ovf_rows, ovf_count,
                      R_max, y, ws, stream=None, events=None) -> None:
    M, K = _dims2(x, "x", "tw_sparse_ffn_fwd")
    N = _dims2(wg_t, "wg_t", "tw_sparse_ffn_fwd")[0]
    NT = _tiles(N, T, "tw_sparse_ffn_fwd")
    a = _Args("tw_sparse_ffn_fwd", x)
    a.shape(x, "x", _BF16, (M, K))
    for t, n in ((wg_t, "wg_t"), (wu_t, "wu_t"), (wd, "wd")):
        a.shape(t, n, _BF16, (N, K))
    a.shape(tw_val, "tw_val", _F32, (M, NT, C))
    a.shape(tw_idx, "tw_idx", _I32, (M, NT, C))
    a.shape(tw_cnt, "tw_cnt", _I32, (M, NT))
    a.room(ovf_rows, "ovf_rows", _I32, max(R_max, 1))
    a.room(ovf_count, "ovf_count", _I32, 1)
    a.shape(y, "y", _F32, (M, K))
    a.bytes(ws, "ws")
    ev = _events(events)
    st = _lib.tw_sparse_ffn_fwd(_ptr(x), _ptr(wg_t), _ptr(wu_t), _ptr(wd), M, K, N, T, C,
                                _ptr(tw_val), _ptr(tw_idx), _ptr(tw_cnt), _ptr(ovf_rows),
                                _ptr(ovf_count), R_max, _ptr(y), _ptr(ws),
                                ws.numel() * ws.element_size(), _stream(stream),
                                ev[0] if ev else None)
    _check(st, "tw_sparse_ffn_fwd")


def tw_ffn_fwd(x, wg_t, wu_t, wd, y, ws, stream=None, events=None) -> None:
    M, K = _dims2(x, "x", "tw_ffn_fwd")
    N = _dims2(wg_t, "wg_t", "tw_ffn_fwd")[0]
    a = _Args("tw_ffn_fwd", x)
    a.shape(x, "x", _BF16, (M, K))
    for t, n in ((wg_t, "wg_t"), (wu_t, "wu_t"), (wd, "wd")):
        a.shape(t, n, _BF16, (N, K))
    a.shape(y, "y", _F32, (M, K))
    a.bytes(ws, "ws")
    ev = _events(events)
    st = _lib.tw_ffn_fwd(_ptr(x), _ptr(wg_t), _ptr(wu_t), _ptr(wd), M, K, N, _ptr(y), _ptr(ws),
                         ws.numel() * ws.element_size(), _stream(stream), ev[0] if ev else None)
    _check(st, "tw_ffn_fwd")


def tw_gate_dense(x, wg_t, z, stream=None, events=None) -> None:
    M, K = _dims2(x, "x", "tw_gate_dense")
    N = _dims2(wg_t, "wg_t", "tw_gate_dense")[0]
    a = _Args("tw_gate_dense", x)
    a.shape(x, "x", _BF16, (M, K))
    a.shape(wg_t, "wg_t", _BF16, (N, K))
    a.shape(z, "z", _F32, (M, N))
    ev = _events(events)
    st = _lib.tw_gate_dense(_ptr(x), _ptr(wg_t), M, K, N, _ptr(z), _stream(stream),
                            ev[0] if ev else None)
    _check(st, "tw_gate_dense")


def tw_pack_dense_workspace_bytes(M, N) -> int:
    return int(_lib.tw_pack_dense_workspace_bytes(M, N))


def tw_pack_dense(z, T, C, tw_val, tw_idx, tw_cnt, ovf_rows, ovf_count, R_max, ws, stream=None,
                  events=None) -> None:
    M, N = _dims2(z, "z", "tw_pack_dense")
    NT = _tiles(N, T, "tw_pack_dense")
    a = _Args("tw_pack_dense", z)
    a.shape(z, "z", _F32, (M, N))
    a.shape(tw_val, "tw_val", _F32, (M, NT, C))
    a.shape(tw_idx, "tw_idx", _I32, (M, NT, C))
    a.shape(tw_cnt, "tw_cnt", _I32, (M, NT))
    a.room(ovf_rows, "ovf_rows", _I32, max(R_max, 1))
    a.room(ovf_count, "ovf_count", _I32, 1)
    a.bytes(ws, "ws")
    ev = _events(events)
    st = _lib.tw_pack_dense(_ptr(z), M, N, T, C, _ptr(tw_val), _ptr(tw_idx), _ptr(tw_cnt),
                            _ptr(ovf_rows), _ptr(ovf_count), R_max, _ptr(ws),
                            ws.numel() * ws.element_size(), _stream(stream),
                            ev[0] if ev else None)
    _check(st, "tw_pack_dense")


def tw_hybrid_pack(T, C, tw_val, tw_idx, tw_cnt, P, hy_val, hy_idx, hy_cnt, route, bk_rows,
                   bk_count, R_max, stream=None, events=None) -> None:
    M, NT = _dims2(tw_cnt, "tw_cnt", "tw_hybrid_pack")
    a = _Args("tw_hybrid_pack", tw_cnt)
    a.shape(tw_cnt, "tw_cnt", _I32, (M, NT))
    a.shape(tw_val, "tw_val", _F32, (M, NT, C))
    a.shape(tw_idx, "tw_idx", _I32, (M, NT, C))
    a.shape(hy_val, "hy_val", _F32, (M, P))
    a.shape(hy_idx, "hy_idx", _I32, (M, P))
    a.shape(hy_cnt, "hy_cnt", _I32, (M,))
    a.shape(route, "route", _U8T, (M,))
    a.room(bk_rows, "bk_rows", _I32, max(R_max, 1))
    a.room(bk_count, "bk_count", _I32, 1)
    ev = _events(events)
    st = _lib.tw_hybrid_pack(M, NT * T, T, C, _ptr(tw_val), _ptr(tw_idx), _ptr(tw_cnt), P,
                             _ptr(hy_val), _ptr(hy_idx), _ptr(hy_cnt), _ptr(route), _ptr(bk_rows),
                             _ptr(bk_count), R_max, _stream(stream), ev[0] if ev else None)
    _check(st, "tw_hybrid_pack")


def tw_hybrid_up(x, wg_t, wu_t, P, hy_g, hy_idx, hy_cnt, route, bk_rows, bk_count, R_max,
                 hy_u, hy_h, bk_g, bk_u, bk_h, stream=None, events=None) -> None:
    M, K = _dims2(x, "x", "tw_hybrid_up")
    N = _dims2(wg_t, "wg_t", "tw_hybrid_up")[0]
    R1 = max(R_max, 1)
    a = _Args("tw_hybrid_up", x)
    a.shape(x, "x", _BF16, (M, K))
    a.shape(wg_t, "wg_t", _BF16, (N, K))
    a.shape(wu_t, "wu_t", _BF16, (N, K))
    a.shape(hy_g, "hy_g", _F32, (M, P))
    a.shape(hy_idx, "hy_idx", _I32, (M, P))
    a.shape(hy_cnt, "hy_cnt", _I32, (M,))
    a.shape(route, "route", _U8T, (M,))
    a.room(bk_rows, "bk_rows", _I32, R1)
    a.room(bk_count, "bk_count", _I32, 1)
    a.opt(hy_u, "hy_u", _F32, (M, P))
    a.shape(hy_h, "hy_h", _F32, (M, P))
    a.opt(bk_g, "bk_g", _BF16, (R1, N))
    a.opt(bk_u, "bk_u", _BF16, (R1, N))
    a.shape(bk_h, "bk_h", _BF16, (R1, N))
    ev = _events(events)
    st = _lib.tw_hybrid_up(_ptr(x), _ptr(wg_t), _ptr(wu_t), M, K, N, P, _ptr(hy_g), _ptr(hy_idx),
                           _ptr(hy_cnt), _ptr(route), _ptr(bk_rows), _ptr(bk_count), R_max,
                           _ptr(hy_u), _ptr(hy_h), _ptr(bk_g), _ptr(bk_u), _ptr(bk_h),
                           _stream(stream), ev[0] if ev else None)
    _check(st, "tw_hybrid_up")


def tw_hybrid_down_workspace_bytes(R_max) -> int:
    return int(_lib.tw_hybrid_down_workspace_bytes(R_max))


def tw_hybrid_down(wd, M, P, hy_h, hy_idx, hy_cnt, route, bk_rows, bk_count, R_max, bk_h, y,
                   ws, stream=None, events=None) -> None:
    N, K = _dims2(wd, "wd", "tw_hybrid_down")
    R1 = max(R_max, 1)
    a = _Args("tw_hybrid_down", wd)
    a.shape(wd, "wd", _BF16, (N, K))
    a.shape(hy_h, "hy_h", _F32, (M, P))
    a.shape(hy_idx, "hy_idx", _I32, (M, P))
    a.shape(hy_cnt, "hy_cnt", _I32, (M,))
    a.shape(route, "route", _U8T, (M,))
    a.room(bk_rows, "bk_rows", _I32, R1)
    a.room(bk_count, "bk_count", _I32, 1)
    a.shape(bk_h, "bk_h", _BF16, (R1, N))
    a.shape(y, "y", _F32, (M, K))
    a.bytes(ws, "ws")
    ev = _events(events)
    nws = 0 if ws is None else ws.numel() * ws.element_size()
    st = _lib.tw_hybrid_down(_ptr(wd), M, K, N, P, _ptr(hy_h), _ptr(hy_idx), _ptr(hy_cnt),
                             _ptr(route), _ptr(bk_rows), _ptr(bk_count), R_max, _ptr(bk_h),
                             _ptr(y), _ptr(ws), nws, _stream(stream), ev[0] if ev else None)
    _check(st, "tw_hybrid_down")


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def tw_hybrid_bwd_dh(dy, wd, P, l1, hy_g, hy_u, hy_idx, hy_cnt, route, bk_rows, bk_count, R_max,
                     bk_g, bk_u, hy_du, hy_dz, bk_du, bk_dz, stream=None, events=None) -> None:
    M, K = _dims2(dy, "dy", "tw_hybrid_bwd_dh")
    N = _dims2(wd, "wd", "tw_hybrid_bwd_dh")[0]
    R1 = max(R_max, 1)
    a = _Args("tw_hybrid_bwd_dh", dy)
    a.shape(dy, "dy", _BF16, (M, K))
    a.shape(wd, "wd", _BF16, (N, K))
    for t, n in ((hy_g, "hy_g"), (hy_u, "hy_u"), (hy_du, "hy_du"), (hy_dz, "hy_dz")):
        a.shape(t, n, _F32, (M, P))
    a.shape(hy_idx, "hy_idx", _I32, (M, P))
    a.shape(hy_cnt, "hy_cnt", _I32, (M,))
    a.shape(route, "route", _U8T, (M,))
    a.room(bk_rows, "bk_rows", _I32, R1)
    a.room(bk_count, "bk_count", _I32, 1)
    for t, n in ((bk_g, "bk_g"), (bk_u, "bk_u"), (bk_du, "bk_du"), (bk_dz, "bk_dz")):
        a.shape(t, n, _BF16, (R1, N))
    ev = _events(events)
    st = _lib.tw_hybrid_bwd_dh(_ptr(dy), _ptr(wd), M, K, N, P, float(l1), _ptr(hy_g), _ptr(hy_u),
                               _ptr(hy_idx), _ptr(hy_cnt), _ptr(route), _ptr(bk_rows),
                               _ptr(bk_count), R_max, _ptr(bk_g), _ptr(bk_u), _ptr(hy_du),
                               _ptr(hy_dz), _ptr(bk_du), _ptr(bk_dz), _stream(stream),
                               ev[0] if ev else None)
    _check(st, "tw_hybrid_bwd_dh")


def tw_hybrid_bwd_dx_workspace_bytes(R_max) -> int:
    return int(_lib.tw_hybrid_bwd_dx_workspace_bytes(R_max))


def tw_hybrid_bwd_dx(wg_t, wu_t, M, P, hy_du, hy_dz, hy_idx, hy_cnt, route, bk_rows, bk_count,
                     R_max, bk_du, bk_dz, dx, ws, stream=None, events=None) -> None:
    N, K = _dims2(wg_t, "wg_t", "tw_hybrid_bwd_dx")
    R1 = max(R_max, 1)
    a = _Args("tw_hybrid_bwd_dx", wg_t)
    a.shape(wg_t, "wg_t", _BF16, (N, K))
    a.shape(wu_t, "wu_t", _BF16, (N, K))
    a.shape(hy_du, "hy_du", _F32, (M, P))
    a.shape(hy_dz, "hy_dz", _F32, (M, P))
    a.shape(hy_idx, "hy_idx", _I32, (M, P))
    a.shape(hy_cnt, "hy_cnt", _I32, (M,))
    a.shape(route, "route", _U8T, (M,))
    a.room(bk_rows, "bk_rows", _I32, R1)
    a.room(bk_count, "bk_count", _I32, 1)
    a.shape(bk_du, "bk_du", _BF16, (R1, N))
    a.shape(bk_dz, "bk_dz", _BF16, (R1, N))
    a.shape(dx, "dx", _F32, (M, K))
    a.bytes(ws, "ws")
    ev = _events(events)
    st = _lib.tw_hybrid_bwd_dx(_ptr(wg_t), _ptr(wu_t), M, K, N, P, _ptr(hy_du), _ptr(hy_dz),
                               _ptr(hy_idx), _ptr(hy_cnt), _ptr(route), _ptr(bk_rows),
                               _ptr(bk_count), R_max, _ptr(bk_du), _ptr(bk_dz), _ptr(dx), _ptr(ws),
                               _nbytes(ws), _stream(stream), ev[0] if ev else None)
    _check(st, "tw_hybrid_bwd_dx")


def tw_hybrid_bwd_dw_workspace_bytes(M, K, N, P, R_max) -> int:
    return int(_lib.tw_hybrid_bwd_dw_workspace_bytes(M, K, N, P, R_max))


def tw_hybrid_bwd_dw(x, dy, P, hy_h, hy_du, hy_dz, hy_idx, hy_cnt, route, bk_rows, bk_count,
                     R_max, bk_h, bk_du, bk_dz, dwg_t, dwu_t, dwd, ws, stream=None,
                     events=None) -> None:
    M, K = _dims2(x, "x", "tw_hybrid_bwd_dw")
    N = _dims2(dwd, "dwd", "tw_hybrid_bwd_dw")[0]
    R1 = max(R_max, 1)
    a = _Args("tw_hybrid_bwd_dw", x)
    a.shape(x, "x", _BF16, (M, K))
    a.shape(dy, "dy", _BF16, (M, K))
    for t, n in ((hy_h, "hy_h"), (hy_du, "hy_du"), (hy_dz, "hy_dz")):
        a.shape(t, n, _F32, (M, P))
    a.shape(hy_idx, "hy_idx", _I32, (M, P))
    a.shape(hy_cnt, "hy_cnt", _I32, (M,))
    a.shape(route, "route", _U8T, (M,))
    a.room(bk_rows, "bk_rows", _I32, R1)
    a.room(bk_count, "bk_count", _I32, 1)
    for t, n in ((bk_h, "bk_h"), (bk_du, "bk_du"), (bk_dz, "bk_dz")):
        a.shape(t, n, _BF16, (R1, N))
    for t, n in ((dwg_t, "dwg_t"), (dwu_t, "dwu_t"), (dwd, "dwd")):
        a.shape(t, n, _F32, (N, K))
    a.bytes(ws, "ws")
    ev = _events(events)
    st = _lib.tw_hybrid_bwd_dw(_ptr(x), _ptr(dy), M, K, N, P, _ptr(hy_h), _ptr(hy_du),
                               _ptr(hy_dz), _ptr(hy_idx), _ptr(hy_cnt), _ptr(route),
                               _ptr(bk_rows), _ptr(bk_count), R_max, _ptr(bk_h),
                               _ptr(bk_du), _ptr(bk_dz), _ptr(dwg_t), _ptr(dwu_t), _ptr(dwd),
                               _ptr(ws), _nbytes(ws), _stream(stream), ev[0] if ev else None)
    _check(st, "tw_hybrid_bwd_dw")


# ------------------------------------------- layer norm and int8 products --
def _norm_args(a, x, add, gamma, beta, total):
    M, K = x.shape
    kind, stride = a.rows(x, "x", _FLOATS)
    add_kind = 0 if add is None else a.typed(add, "add", _FLOATS, (M, K))
    a.shape(gamma, "gamma", _F32, (K,))
    a.opt(beta, "beta", _F32, (K,))
    a.opt(total, "total", x.dtype, (M, K))
    return kind, stride, add_kind


def tw_layernorm_fwd(x, gamma, beta, eps, y, add=None, total=None, mean=None, rstd=None,
                     stream=None, events=None) -> None:
    """y = layer norm of x (+ add); ``total`` receives x + add in x's type,
    ``mean`` and ``rstd`` what the backward reads."""
    M, K = _dims2(x, "x", "tw_layernorm_fwd")
    a = _Args("tw_layernorm_fwd", x)
    kind, stride, add_kind = _norm_args(a, x, add, gamma, beta, total)
    y_kind = a.typed(y, "y", _FLOATS, (M, K))
    a.opt(mean, "mean", _F32, (M,))
    a.opt(rstd, "rstd", _F32, (M,))
    ev = _events(events)
    st = _lib.tw_layernorm_fwd(_rows_ptr(x), kind, stride, _ptr(add), add_kind, _ptr(gamma),
                               _ptr(beta), eps, M, K, _ptr(total), _ptr(y), y_kind, _ptr(mean),
                               _ptr(rstd), _stream(stream), ev[0] if ev else None)
    _check(st, "tw_layernorm_fwd")


def tw_layernorm_bwd_workspace_bytes(M, K) -> int:
    return int(_lib.tw_layernorm_bwd_workspace_bytes(M, K))


def tw_layernorm_bwd(dy, x, gamma, mean, rstd, dx, dgamma=None, dbeta=None, dres=None, ws=None,
                     stream=None, events=None) -> None:
    M, K = _dims2(x, "x", "tw_layernorm_bwd")
    a = _Args("tw_layernorm_bwd", x)
    kind, stride = a.rows(x, "x", _FLOATS)
    dy_kind = a.typed(dy, "dy", _FLOATS, (M, K))
    a.shape(gamma, "gamma", _F32, (K,))
    a.shape(mean, "mean", _F32, (M,))
    a.shape(rstd, "rstd", _F32, (M,))
    dx_kind = a.typed(dx, "dx", _FLOATS, (M, K))
    a.opt(dres, "dres", dx.dtype, (M, K))
    a.opt(dgamma, "dgamma", _F32, (K,))
    a.opt(dbeta, "dbeta", _F32, (K,))
    a.bytes(ws, "ws")
    ev = _events(events)
    st = _lib.tw_layernorm_bwd(_ptr(dy), dy_kind, _rows_ptr(x), kind, stride, _ptr(gamma),
                               _ptr(mean), _ptr(rstd), _ptr(dres), M, K, _ptr(dx), dx_kind,
                               _ptr(dgamma), _ptr(dbeta), _ptr(ws), _nbytes(ws), _stream(stream),
                               ev[0] if ev else None)
    _check(st, "tw_layernorm_bwd")


def tw_quant_rows(x, q, scale, stream=None, events=None) -> None:
    """q, scale = the rows of x in int8 with one scale each."""
    M, K = _dims2(x, "x", "tw_quant_rows")
    a = _Args("tw_quant_rows", x)
    kind, stride = a.rows(x, "x", _FLOATS)
    a.shape(q, "q", _I8, (M, K))
    a.shape(scale, "scale", _F32, (M,))
    ev = _events(events)
    st = _lib.tw_quant_rows(_rows_ptr(x), kind, stride, M, K, _ptr(q), _ptr(scale),
                            _stream(stream), ev[0] if ev else None)
    _check(st, "tw_quant_rows")


def tw_layernorm_quant(x, gamma, beta, eps, q, scale, add=None, total=None, stream=None,
                       events=None) -> None:
    """The layer norm of x (+ add) in int8 with one scale per row."""
    M, K = _dims2(x, "x", "tw_layernorm_quant")
    a = _Args("tw_layernorm_quant", x)
    kind, stride, add_kind = _norm_args(a, x, add, gamma, beta, total)
    a.shape(q, "q", _I8, (M, K))
    a.shape(scale, "scale", _F32, (M,))
    ev = _events(events)
    st = _lib.tw_layernorm_quant(_rows_ptr(x), kind, stride, _ptr(add), add_kind, _ptr(gamma),
                                 _ptr(beta), eps, M, K, _ptr(total), _ptr(q), _ptr(scale),
                                 _stream(stream), ev[0] if ev else None)
    _check(st, "tw_layernorm_quant")


def tw_quant_workspace_bytes(M, K) -> int:
    return int(_lib.tw_quant_workspace_bytes(M, K))


def _quant_in(a, x, x_scale):
    """Rows of float (no x_scale), or int8 rows with their scales."""
    kind, stride = a.rows(x, "x", (_BF16, _F32, _I8))
    if kind == TW_INT8:
        a.shape(x_scale, "x_scale", _F32, (x.shape[0],))
    elif x_scale is not None:
        raise ValueError(f"{a.where}: x_scale is given, but x is not int8")
    return kind, stride


def tw_quant_linear(x, w, w_scale, y, bias=None, x_scale=None, ws=None, stream=None,
                    events=None) -> None:
    M, K = _dims2(x, "x", "tw_quant_linear")
    N = _dims2(w, "w", "tw_quant_linear")[0]
    a = _Args("tw_quant_linear", x)
    kind, stride = _quant_in(a, x, x_scale)
    a.shape(w, "w", _I8, (N, K))
    a.shape(w_scale, "w_scale", _F32, (N,))
    a.opt(bias, "bias", _F32, (N,))
    y_kind = a.typed(y, "y", _FLOATS, (M, N))
    a.bytes(ws, "ws")
    ev = _events(events)
    st = _lib.tw_quant_linear(_rows_ptr(x), kind, stride, _ptr(x_scale), _ptr(w), _ptr(w_scale),
                              _ptr(bias), M, K, N, _ptr(y), y_kind, _ptr(ws), _nbytes(ws),
                              _stream(stream), ev[0] if ev else None)
    _check(st, "tw_quant_linear")


def tw_quant_gateup(x, wg, g_scale, wu, u_scale, h, gamma=None, beta=None, eps=1e-5, x_scale=None,
                    ws=None, stream=None, events=None) -> None:
    M, K = _dims2(x, "x", "tw_quant_gateup")
    N = _dims2(wg, "wg", "tw_quant_gateup")[0]
    a = _Args("tw_quant_gateup", x)
    kind, stride = _quant_in(a, x, x_scale)
    a.shape(wg, "wg", _I8, (N, K))
    a.shape(g_scale, "g_scale", _F32, (N,))
    a.shape(wu, "wu", _I8, (N, K))
    a.shape(u_scale, "u_scale", _F32, (N,))
    a.opt(gamma, "gamma", _F32, (K,))
    a.opt(beta, "beta", _F32, (K,))
    h_kind = a.typed(h, "h", _FLOATS, (M, N))
    a.bytes(ws, "ws")
    ev = _events(events)
    st = _lib.tw_quant_gateup(_rows_ptr(x), kind, stride, _ptr(x_scale), _ptr(gamma), _ptr(beta),
                              eps, _ptr(wg), _ptr(g_scale), _ptr(wu), _ptr(u_scale), M, K, N,
                              _ptr(h), h_kind, _ptr(ws), _nbytes(ws), _stream(stream),
                              ev[0] if ev else None)
    _check(st, "tw_quant_gateup")


# ------------------------------------------------- dense training step --
def _act(act, where):
    if act not in _ACT:
        raise ValueError(f"{where}: act must be one of {sorted(_ACT)}, got {act!r}")
    return _ACT[act]


def tw_rmsnorm_fwd(x, gamma, eps, y, add=None, total=None, rstd=None, stream=None,
                   events=None) -> None:
    """y = RMS norm of x (+ add); ``total`` receives x + add in x's type,
    ``rstd`` what the backward reads."""
    M, K = _dims2(x, "x", "tw_rmsnorm_fwd")
    a = _Args("tw_rmsnorm_fwd", x)
    kind, stride, add_kind = _norm_args(a, x, add, gamma, None, total)
    y_kind = a.typed(y, "y", _FLOATS, (M, K))
    a.opt(rstd, "rstd", _F32, (M,))
    ev = _events(events)
    with _on(x):
        st = _lib.tw_rmsnorm_fwd(_rows_ptr(x), kind, stride, _ptr(add), add_kind, _ptr(gamma), eps,
                                 M, K, _ptr(total), _ptr(y), y_kind, _ptr(rstd), _stream(stream),
                                 ev[0] if ev else None)
    _check(st, "tw_rmsnorm_fwd")


def tw_rmsnorm_quant(x, gamma, eps, q, scale, add=None, total=None, stream=None,
                     events=None) -> None:
    """The RMS norm of x (+ add) in int8 with one scale per row."""
    M, K = _dims2(x, "x", "tw_rmsnorm_quant")
    a = _Args("tw_rmsnorm_quant", x)
    kind, stride, add_kind = _norm_args(a, x, add, gamma, None, total)
    a.shape(q, "q", _I8, (M, K))
    a.shape(scale, "scale", _F32, (M,))
    ev = _events(events)
    with _on(x):
        st = _lib.tw_rmsnorm_quant(_rows_ptr(x), kind, stride, _ptr(add), add_kind, _ptr(gamma),
                                   eps, M, K, _ptr(total), _ptr(q), _ptr(scale), _stream(stream),
                                   ev[0] if ev else None)
    _check(st, "tw_rmsnorm_quant")


def tw_rmsnorm_bwd_workspace_bytes(M, K) -> int:
    return int(_lib.tw_rmsnorm_bwd_workspace_bytes(M, K))


def tw_rmsnorm_bwd(dy, x, gamma, rstd, dx, dgamma=None, dres=None, ws=None, stream=None,
                   events=None) -> None:
    M, K = _dims2(x, "x", "tw_rmsnorm_bwd")
    a = _Args("tw_rmsnorm_bwd", x)
    kind, stride = a.rows(x, "x", _FLOATS)
    dy_kind = a.typed(dy, "dy", _FLOATS, (M, K))
    a.shape(gamma, "gamma", _F32, (K,))
    a.shape(rstd, "rstd", _F32, (M,))
    dx_kind = a.typed(dx, "dx", _FLOATS, (M, K))
    a.opt(dres, "dres", dx.dtype, (M, K))
    a.opt(dgamma, "dgamma", _F32, (K,))
    a.bytes(ws, "ws")
    ev = _events(events)
    with _on(x):
        st = _lib.tw_rmsnorm_bwd(_ptr(dy), dy_kind, _rows_ptr(x), kind, stride, _ptr(gamma),
                                 _ptr(rstd), _ptr(dres), M, K, _ptr(dx), dx_kind, _ptr(dgamma),
                                 _ptr(ws), _nbytes(ws), _stream(stream), ev[0] if ev else None)
    _check(st, "tw_rmsnorm_bwd")


def tw_gated_ffn_workspace_bytes(M, K, N) -> int:
    return int(_lib.tw_gated_ffn_workspace_bytes(M, K, N))


def tw_gated_ffn_fwd(x, wg_t, wu_t, wd, y, ws, act="silu", g=None, u=None, stream=None,
                     events=None) -> None:
    """y = (act(x W_g) * (x W_u)) W_d; g and u receive the projections before
    the activation."""
    M, K = _dims2(x, "x", "tw_gated_ffn_fwd")
    N = _dims2(wg_t, "wg_t", "tw_gated_ffn_fwd")[0]
    a = _Args("tw_gated_ffn_fwd", x)
    kind = _act(act, a.where)
    _, stride = a.rows(x, "x", (_BF16,))
    for t, name in ((wg_t, "wg_t"), (wu_t, "wu_t"), (wd, "wd")):
        a.shape(t, name, _BF16, (N, K))
    a.opt(g, "g", _BF16, (M, N))
    a.opt(u, "u", _BF16, (M, N))
    y_kind = a.typed(y, "y", _FLOATS, (M, K))
    a.bytes(ws, "ws")
    ev = _events(events)
    with _on(x):
        st = _lib.tw_gated_ffn_fwd(_rows_ptr(x), stride, _ptr(wg_t), _ptr(wu_t), _ptr(wd), kind, M,
                                   K, N, _ptr(g), _ptr(u), _ptr(y), y_kind, _ptr(ws), _nbytes(ws),
                                   _stream(stream), ev[0] if ev else None)
    _check(st, "tw_gated_ffn_fwd")


def tw_gated_ffn_bwd_workspace_bytes(M, K, N) -> int:
    return int(_lib.tw_gated_ffn_bwd_workspace_bytes(M, K, N))


def tw_gated_ffn_bwd(dy, x, wg_t, wu_t, wd, g, u, ws, act="silu", dx=None, dwg_t=None, dwu_t=None,
                     dwd=None, stream=None, events=None) -> None:
    """Gradient of ``tw_gated_ffn_fwd`` from its g and u; the weight gradients
    are of one type."""
    M, K = _dims2(x, "x", "tw_gated_ffn_bwd")
    N = _dims2(wg_t, "wg_t", "tw_gated_ffn_bwd")[0]
    a = _Args("tw_gated_ffn_bwd", x)
    kind = _act(act, a.where)
    _, stride = a.rows(x, "x", (_BF16,))
    a.shape(dy, "dy", _BF16, (M, K))
    for t, name in ((wg_t, "wg_t"), (wu_t, "wu_t"), (wd, "wd")):
        a.shape(t, name, _BF16, (N, K))
    a.shape(g, "g", _BF16, (M, N))
    a.shape(u, "u", _BF16, (M, N))
    dx_kind = TW_BF16 if dx is None else a.typed(dx, "dx", _FLOATS, (M, K))
    dw_kind = TW_BF16 if dwg_t is None else a.typed(dwg_t, "dwg_t", _FLOATS, (N, K))
    for t, name in ((dwu_t, "dwu_t"), (dwd, "dwd")):
        a.opt(t, name, _BF16 if dw_kind == TW_BF16 else _F32, (N, K))
    # dx is written from the gate's and up's weights, the weight gradients after it from x and dy
    a.apart(dx, "dx", {"wg_t": wg_t, "wu_t": wu_t, "dwg_t": dwg_t, "dwu_t": dwu_t, "dwd": dwd})
    if dwg_t is not None:
        a.apart(dx, "dx", {"x": x, "dy": dy})
    a.apart(dwg_t, "dwg_t", {"x": x, "dy": dy, "dwu_t": dwu_t, "dwd": dwd})
    a.apart(dwu_t, "dwu_t", {"x": x, "dy": dy, "dwd": dwd})
    a.apart(dwd, "dwd", {"x": x, "dy": dy})
    a.bytes(ws, "ws")
    ev = _events(events)
    with _on(x):
        st = _lib.tw_gated_ffn_bwd(_ptr(dy), _rows_ptr(x), stride, _ptr(wg_t), _ptr(wu_t),
                                   _ptr(wd), kind, _ptr(g), _ptr(u), M, K, N, _ptr(dx), dx_kind,
                                   _ptr(dwg_t), _ptr(dwu_t), _ptr(dwd), dw_kind, _ptr(ws),
                                   _nbytes(ws), _stream(stream), ev[0] if ev else None)
    _check(st, "tw_gated_ffn_bwd")


def tw_linear_ce_workspace_bytes(M, K, V) -> int:
    return int(_lib.tw_linear_ce_workspace_bytes(M, K, V))


def _ce_args(a, x, w, target):
    M, K = x.shape
    V = _dims2(w, "w", a.where)[0]
    _, stride = a.rows(x, "x", (_BF16,))
    a.shape(w, "w", _BF16, (V, K))
    return V, stride, a.typed(target, "target", (_I32, _I64), (M,))


def tw_linear_ce_fwd(x, w, target, loss, lse, ws, stream=None, events=None) -> None:
    """loss and log-sum-exp of every row of x w^T; a row whose target is
    outside [0, V) gets loss 0."""
    M, K = _dims2(x, "x", "tw_linear_ce_fwd")
    a = _Args("tw_linear_ce_fwd", x)
    V, stride, t_kind = _ce_args(a, x, w, target)
    a.shape(loss, "loss", _F32, (M,))
    a.shape(lse, "lse", _F32, (M,))
    a.bytes(ws, "ws")
    ev = _events(events)
    with _on(x):
        st = _lib.tw_linear_ce_fwd(_rows_ptr(x), stride, _ptr(w), _ptr(target), t_kind, M, K, V,
                                   _ptr(loss), _ptr(lse), _ptr(ws), _nbytes(ws), _stream(stream),
                                   ev[0] if ev else None)
    _check(st, "tw_linear_ce_fwd")


def tw_linear_ce_bwd_workspace_bytes(M, K, V) -> int:
    return int(_lib.tw_linear_ce_bwd_workspace_bytes(M, K, V))


def tw_linear_ce_bwd(dloss, x, w, target, lse, ws, dx=None, dw=None, stream=None,
                     events=None) -> None:
    """Gradient of ``tw_linear_ce_fwd`` from the gradient of every row's loss."""
    M, K = _dims2(x, "x", "tw_linear_ce_bwd")
    a = _Args("tw_linear_ce_bwd", x)
    V, stride, t_kind = _ce_args(a, x, w, target)
    a.shape(dloss, "dloss", _F32, (M,))
    a.shape(lse, "lse", _F32, (M,))
    dx_kind = TW_BF16 if dx is None else a.typed(dx, "dx", _FLOATS, (M, K))
    dw_kind = TW_BF16 if dw is None else a.typed(dw, "dw", _FLOATS, (V, K))
    # dx is written from w, a piece's dw after it from x
    a.apart(dx, "dx", {"w": w, "dw": dw})
    if dw is not None:
        a.apart(dx, "dx", {"x": x})
        a.apart(dw, "dw", {"x": x})
        if dw.data_ptr() != w.data_ptr() or dw.dtype != w.dtype:  # (else a piece replaces itself)
            a.apart(dw, "dw", {"w": w})
    a.bytes(ws, "ws")
    ev = _events(events)
    with _on(x):
        st = _lib.tw_linear_ce_bwd(_ptr(dloss), _rows_ptr(x), stride, _ptr(w), _ptr(target),
                                   t_kind, _ptr(lse), M, K, V, _ptr(dx), dx_kind, _ptr(dw),
                                   dw_kind, _ptr(ws), _nbytes(ws), _stream(stream),
                                   ev[0] if ev else None)
    _check(st, "tw_linear_ce_bwd")


class _Buffers:
    """The arrays of a call over many tensors: addresses, sizes, types."""

    def __init__(self, a, tensors, name):
        for t in tensors:
            if not isinstance(t, torch.Tensor) or t.dtype not in _FLOATS:
                raise TypeError(f"{a.where}: {name} must be tensors of {_FLOATS}")
            if t.device != a.device:
                raise ValueError(f"{a.where}: {name} are on {t.device} and {a.device}")
        self.count = len(tensors)
        self.p = (ctypes.c_void_p * self.count)(*[_ptr(t) for t in tensors])
        self.n = (ctypes.c_int64 * self.count)(*[t.numel() for t in tensors])
        self.type = (ctypes.c_int * self.count)(*[_TYPE[t.dtype] for t in tensors])


def tw_grad_norm_workspace_bytes(sizes) -> int:
    return int(_lib.tw_grad_norm_workspace_bytes(len(sizes), (ctypes.c_int64 * len(sizes))(*sizes)))


def tw_grad_norm(grads, norm, ws, stream=None, events=None) -> None:
    """norm (one fp32) = sqrt(sum of the squares of all elements)."""
    a = _Args("tw_grad_norm", norm)
    g = _Buffers(a, grads, "grads")
    a.shape(norm, "norm", _F32, ())
    a.bytes(ws, "ws")
    ev = _events(events)
    with _on(norm):
        st = _lib.tw_grad_norm(g.count, g.p, g.n, g.type, _ptr(norm), _ptr(ws), _nbytes(ws),
                               _stream(stream), ev[0] if ev else None)
    _check(st, "tw_grad_norm")


def tw_grad_clip(grads, out, max_norm, eps, norm, ws, stream=None, events=None) -> None:
    """out[i] = grads[i] min(1, max_norm / (norm + eps)); out may be grads."""
    a = _Args("tw_grad_clip", norm)
    g, o = _Buffers(a, grads, "grads"), _Buffers(a, out, "out")
    if [t.shape for t in out] != [t.shape for t in grads]:
        raise ValueError(f"{a.where}: out and grads have different shapes")
    a.shape(norm, "norm", _F32, ())
    a.bytes(ws, "ws")
    ev = _events(events)
    with _on(norm):
        st = _lib.tw_grad_clip(g.count, g.p, g.n, g.type, o.p, o.type, max_norm, eps, _ptr(norm),
                               _ptr(ws), _nbytes(ws), _stream(stream), ev[0] if ev else None)
    _check(st, "tw_grad_clip")


# ------------------------------------------------------------- allocating --
def alloc_pack(M, N, T, C, R_max, device="cuda"):
    """Output buffers of tw_pack_gate."""
    NT = N // T
    return {
        "tw_val": torch.empty((M, NT, C), dtype=torch.float32, device=device),
        "tw_idx": torch.empty((M, NT, C), dtype=torch.int32, device=device),
        "tw_cnt": torch.empty((M, NT), dtype=torch.int32, device=device),
        "ovf_rows": torch.empty((max(R_max, 1),), dtype=torch.int32, device=device),
        "ovf_count": torch.empty((1,), dtype=torch.int32, device=device),
    }


def workspace(M, K, N, T, C, R_max, device="cuda"):
    n = tw_workspace_bytes(M, K, N, T, C, R_max)
    if n == 0:
        raise ValueError("unsupported shape for the TwELL path")
    return torch.empty((n,), dtype=torch.uint8, device=device)


def pack_gate(x, wg_t, T, C, R_max=None, z_debug=False, ws=None):
    """Gate GEMM + ReLU + TwELL packing; returns the packing as a dict."""
    M, K = x.shape
    N = wg_t.shape[0]
    R_max = M if R_max is None else R_max
    out = alloc_pack(M, N, T, C, R_max, x.device)
    ws = workspace(M, K, N, T, C, R_max, x.device) if ws is None else ws
    z = torch.empty((M, N), dtype=torch.float32, device=x.device) if z_debug else None
    tw_pack_gate(x, wg_t, T, C, out["tw_val"], out["tw_idx"], out["tw_cnt"], out["ovf_rows"],
                 out["ovf_count"], R_max, ws, z_debug=z)
    if z_debug:
        out["z"] = z
    out.update(T=T, C=C, R_max=R_max)
    return out


def pack_unfused(x, wg_t, T, C, R_max=None):
    """The unfused equivalent of pack_gate: dense gate in memory, then packed."""
    M, K = x.shape
    N = wg_t.shape[0]
    R_max = M if R_max is None else R_max
    out = alloc_pack(M, N, T, C, R_max, x.device)
    z = torch.empty((M, N), dtype=torch.float32, device=x.device)
    ws = torch.empty((tw_pack_dense_workspace_bytes(M, N),), dtype=torch.uint8, device=x.device)
    tw_gate_dense(x, wg_t, z)
    tw_pack_dense(z, T, C, out["tw_val"], out["tw_idx"], out["tw_cnt"], out["ovf_rows"],
                  out["ovf_count"], R_max, ws)
    out.update(T=T, C=C, R_max=R_max, z=z)
    return out


def sparse_ffn(x, wg_t, wu_t, wd, packed, ws=None):
    """Sparse up+down (and dense fallback) from a packing; returns y fp32."""
    M, K = x.shape
    N = wg_t.shape[0]
    T, C, R_max = packed["T"], packed["C"], packed["R_max"]
    y = torch.empty((M, K), dtype=torch.float32, device=x.device)
    ws = workspace(M, K, N, T, C, R_max, x.device) if ws is None else ws
    tw_sparse_ffn_fwd(x, wg_t, wu_t, wd, T, C, packed["tw_val"], packed["tw_idx"],
                      packed["tw_cnt"], packed["ovf_rows"], packed["ovf_count"], R_max, y, ws)
    return y


def ffn(x, wg_t, wu_t, wd, ws=None):
    """Dense gated FFN over all rows; returns y fp32."""
    M, K = x.shape
    N = wg_t.shape[0]
    y = torch.empty((M, K), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = torch.empty((tw_ffn_workspace_bytes(M, K, N),), dtype=torch.uint8, device=x.device)
    tw_ffn_fwd(x, wg_t, wu_t, wd, y, ws)
    return y


def alloc_hybrid(M, N, P, R_max, keep=True, device="cuda"):
    """Buffers of the hybrid storage (sparse rows, routing, backup rows).
    ``keep`` also allocates the up values and the backup gate and up rows
    (what the backward reads); without it only the product h is stored."""
    R1 = max(R_max, 1)
    f32, i32, b16 = torch.float32, torch.int32, torch.bfloat16
    out = {
        "hy_cnt": torch.empty((M,), dtype=i32, device=device),
        "hy_idx": torch.empty((M, P), dtype=i32, device=device),
        "hy_g": torch.empty((M, P), dtype=f32, device=device),
        "hy_h": torch.empty((M, P), dtype=f32, device=device),
        "route": torch.empty((M,), dtype=torch.uint8, device=device),
        "bk_rows": torch.empty((R1,), dtype=i32, device=device),
        "bk_count": torch.empty((1,), dtype=i32, device=device),
        "bk_h": torch.empty((R1, N), dtype=b16, device=device),
        "hy_u": None, "bk_g": None, "bk_u": None,
    }
    if keep:
        out["hy_u"] = torch.empty((M, P), dtype=f32, device=device)
        out["bk_g"] = torch.empty((R1, N), dtype=b16, device=device)
        out["bk_u"] = torch.empty((R1, N), dtype=b16, device=device)
    out.update(P=P, R_max=R_max)
    return out


def hybrid_forward(x, wg_t, wu_t, wd, packed, P=128, R_max=None, keep=True, hy=None, ws=None):
    """Training forward over hybrid storage, from a TwELL packing of the gate
    (``pack_gate``'s output): TwELL -> hybrid, up at the stored entries, down
    to dense.  Returns (y fp32 [M][K], the hybrid storage dict)."""
    M, K = x.shape
    N = wg_t.shape[0]
    R_max = max(M // 8, 1) if R_max is None else R_max
    R_max = min(R_max, M)
    hy = alloc_hybrid(M, N, P, R_max, keep, x.device) if hy is None else hy
    tw_hybrid_pack(packed["T"], packed["C"], packed["tw_val"], packed["tw_idx"],
                   packed["tw_cnt"], P, hy["hy_g"], hy["hy_idx"], hy["hy_cnt"], hy["route"],
                   hy["bk_rows"], hy["bk_count"], R_max)
    tw_hybrid_up(x, wg_t, wu_t, P, hy["hy_g"], hy["hy_idx"], hy["hy_cnt"], hy["route"],
                 hy["bk_rows"], hy["bk_count"], R_max, hy["hy_u"], hy["hy_h"], hy["bk_g"],
                 hy["bk_u"], hy["bk_h"])
    y = torch.empty((M, K), dtype=torch.float32, device=x.device)
    nws = tw_hybrid_down_workspace_bytes(R_max)
    if ws is None and nws:
        ws = torch.empty((nws,), dtype=torch.uint8, device=x.device)
    tw_hybrid_down(wd, M, P, hy["hy_h"], hy["hy_idx"], hy["hy_cnt"], hy["route"], hy["bk_rows"],
                   hy["bk_count"], R_max, hy["bk_h"], y, ws)
    return y, hy


def hybrid_backward(x, wg_t, wu_t, wd, dy, hy, l1=0.0):
    """Backward over the hybrid storage ``hy`` of ``hybrid_forward`` (with
    ``keep=True``): returns a dict with dx [M][K], dwg_t, dwu_t, dwd [N][K]
    (fp32) and the activations' gradients (hy_du, hy_dz, bk_du, bk_dz)."""
    M, K = x.shape
    N = wg_t.shape[0]
    P, R_max = hy["P"], hy["R_max"]
    if hy["hy_u"] is None:
        raise ValueError("the forward did not keep u and g (keep=False)")
    dev = x.device
    R1 = max(R_max, 1)
    out = {
        "hy_du": torch.empty((M, P), dtype=torch.float32, device=dev),
        "hy_dz": torch.empty((M, P), dtype=torch.float32, device=dev),
        "bk_du": torch.empty((R1, N), dtype=torch.bfloat16, device=dev),
        "bk_dz": torch.empty((R1, N), dtype=torch.bfloat16, device=dev),
        "dx": torch.empty((M, K), dtype=torch.float32, device=dev),
        "dwg_t": torch.empty((N, K), dtype=torch.float32, device=dev),
        "dwu_t": torch.empty((N, K), dtype=torch.float32, device=dev),
        "dwd": torch.empty((N, K), dtype=torch.float32, device=dev),
    }
    tw_hybrid_bwd_dh(dy, wd, P, l1, hy["hy_g"], hy["hy_u"], hy["hy_idx"], hy["hy_cnt"],
                     hy["route"], hy["bk_rows"], hy["bk_count"], R_max, hy["bk_g"], hy["bk_u"],
                     out["hy_du"], out["hy_dz"], out["bk_du"], out["bk_dz"])
    nx = tw_hybrid_bwd_dx_workspace_bytes(R_max)
    wsx = torch.empty((nx,), dtype=torch.uint8, device=dev) if nx else None
    tw_hybrid_bwd_dx(wg_t, wu_t, M, P, out["hy_du"], out["hy_dz"], hy["hy_idx"], hy["hy_cnt"],
                     hy["route"], hy["bk_rows"], hy["bk_count"], R_max, out["bk_du"],
                     out["bk_dz"], out["dx"], wsx)
    wsw = torch.empty((tw_hybrid_bwd_dw_workspace_bytes(M, K, N, P, R_max),), dtype=torch.uint8,
                      device=dev)
    tw_hybrid_bwd_dw(x, dy, P, hy["hy_h"], out["hy_du"], out["hy_dz"], hy["hy_idx"],
                     hy["hy_cnt"], hy["route"], hy["bk_rows"], hy["bk_count"], R_max,
                     hy["bk_h"], out["bk_du"], out["bk_dz"], out["dwg_t"], out["dwu_t"],
                     out["dwd"], wsw)
    return out


def layernorm(x, gamma, beta=None, eps=1e-5, add=None, out_dtype=torch.bfloat16):
    """Layer norm of the rows of x (+ add).  Returns a dict: y, mean and rstd
    (fp32, for ``layernorm_backward``), and sum = x + add in x's type (None
    without add)."""
    got = _calls.layernorm(x, gamma, beta, eps, add, out_dtype)
    if got is not None:
        return got
    M, K = _dims2(x, "x", "layernorm")
    dev = x.device
    out = {
        "y": torch.empty((M, K), dtype=out_dtype, device=dev),
        "sum": None if add is None else torch.empty((M, K), dtype=x.dtype, device=dev),
        "mean": torch.empty((M,), dtype=_F32, device=dev),
        "rstd": torch.empty((M,), dtype=_F32, device=dev),
    }
    tw_layernorm_fwd(x, gamma, beta, eps, out["y"], add=add, total=out["sum"], mean=out["mean"],
                     rstd=out["rstd"])
    return out


def layernorm_backward(dy, x, gamma, mean, rstd, dres=None, dx_dtype=torch.float32):
    """Gradient of ``layernorm``: x is its input (``sum`` if there was an
    add), dres the gradient reaching x past the norm (dx's dtype).  Returns a
    dict with dx, dgamma, dbeta."""
    got = _calls.layernorm_backward(dy, x, gamma, mean, rstd, dres, dx_dtype)
    if got is not None:
        return got
    M, K = _dims2(x, "x", "layernorm_backward")
    dev = x.device
    out = {
        "dx": torch.empty((M, K), dtype=dx_dtype, device=dev),
        "dgamma": torch.empty((K,), dtype=_F32, device=dev),
        "dbeta": torch.empty((K,), dtype=_F32, device=dev),
    }
    ws = torch.empty((tw_layernorm_bwd_workspace_bytes(M, K),), dtype=_U8T, device=dev)
    tw_layernorm_bwd(dy, x, gamma, mean, rstd, out["dx"], out["dgamma"], out["dbeta"], dres=dres,
                     ws=ws)
    return out


def quantize_rows(x):
    """The rows of x in int8: (q [M][K], scale [M]).  For weights, x is the
    matrix with one row per output channel."""
    M, K = _dims2(x, "x", "quantize_rows")
    q = torch.empty((M, K), dtype=_I8, device=x.device)
    scale = torch.empty((M,), dtype=_F32, device=x.device)
    tw_quant_rows(x, q, scale)
    return q, scale


def layernorm_quantize(x, gamma, beta=None, eps=1e-5, add=None):
    """The layer norm of x (+ add) in int8.  Returns a dict: q, scale, and
    sum = x + add in x's type (None without add)."""
    M, K = _dims2(x, "x", "layernorm_quantize")
    out = {
        "q": torch.empty((M, K), dtype=_I8, device=x.device),
        "scale": torch.empty((M,), dtype=_F32, device=x.device),
        "sum": None if add is None else torch.empty((M, K), dtype=x.dtype, device=x.device),
    }
    tw_layernorm_quant(x, gamma, beta, eps, out["q"], out["scale"], add=add, total=out["sum"])
    return out


def _quant_ws(x):
    if x.dtype == _I8:
        return None
    return torch.empty((tw_quant_workspace_bytes(*x.shape),), dtype=_U8T, device=x.device)


def quant_linear(x, w, w_scale, bias=None, x_scale=None, out_dtype=torch.bfloat16, ws=None):
    """y = x w^T (+ bias) on int8 operands: x is bf16 or fp32 (quantised by
    the call) or int8 with x_scale; w [N][K] int8 with w_scale [N]."""
    got = _calls.quant_linear(x, w, w_scale, bias, x_scale, out_dtype, ws)
    if got is not None:
        return got
    M, N = _dims2(x, "x", "quant_linear")[0], _dims2(w, "w", "quant_linear")[0]
    y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    tw_quant_linear(x, w, w_scale, y, bias=bias, x_scale=x_scale,
                    ws=_quant_ws(x) if ws is None else ws)
    return y


def quant_gateup(x, wg, g_scale, wu, u_scale, gamma=None, beta=None, eps=1e-5, x_scale=None,
                 out_dtype=torch.bfloat16, ws=None):
    """h = ReLU(n wg^T) * (n wu^T) on int8 operands, n the layer norm of x
    (gamma given) or x itself; x as in ``quant_linear``."""
    got = _calls.quant_gateup(x, wg, g_scale, wu, u_scale, gamma, beta, eps, x_scale, out_dtype,
                              ws)
    if got is not None:
        return got
    M, N = _dims2(x, "x", "quant_gateup")[0], _dims2(wg, "wg", "quant_gateup")[0]
    h = torch.empty((M, N), dtype=out_dtype, device=x.device)
    tw_quant_gateup(x, wg, g_scale, wu, u_scale, h, gamma=gamma, beta=beta, eps=eps,
                    x_scale=x_scale, ws=_quant_ws(x) if ws is None else ws)
    return h


def _aligned(t):
    """A contiguous tensor of a value a row at an address that the library takes: copied
    where it begins at another row of a longer one (tokens[1:])."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous() and t.data_ptr() % 16:
        return t.clone()
    return t


def rmsnorm(x, gamma, eps=1e-5, add=None, out_dtype=torch.bfloat16):
    """RMS norm of the rows of x (+ add).  Returns a dict: y, rstd (fp32, for
    ``rmsnorm_backward``), and sum = x + add in x's type (None without add)."""
    got = _calls.rmsnorm(x, gamma, eps, add, out_dtype)
    if got is not None:
        return got
    M, K = _dims2(x, "x", "rmsnorm")
    dev = x.device
    out = {
        "y": torch.empty((M, K), dtype=out_dtype, device=dev),
        "sum": None if add is None else torch.empty((M, K), dtype=x.dtype, device=dev),
        "rstd": torch.empty((M,), dtype=_F32, device=dev),
    }
    tw_rmsnorm_fwd(x, gamma, eps, out["y"], add=add, total=out["sum"], rstd=out["rstd"])
    return out


def rmsnorm_backward(dy, x, gamma, rstd, dres=None, dx_dtype=torch.float32):
    """Gradient of ``rmsnorm``: x is its input (``sum`` if there was an add),
    dres the gradient reaching x past the norm (dx's dtype).  Returns a dict
    with dx, dgamma."""
    got = _calls.rmsnorm_backward(dy, x, gamma, rstd, dres, dx_dtype)
    if got is not None:
        return got
    M, K = _dims2(x, "x", "rmsnorm_backward")
    dev = x.device
    out = {
        "dx": torch.empty((M, K), dtype=dx_dtype, device=dev),
        "dgamma": torch.empty((K,), dtype=_F32, device=dev),
    }
    ws = torch.empty((tw_rmsnorm_bwd_workspace_bytes(M, K),), dtype=_U8T, device=dev)
    tw_rmsnorm_bwd(dy, x, gamma, _aligned(rstd), out["dx"], out["dgamma"], dres=dres, ws=ws)
    return out


def rmsnorm_quantize(x, gamma, eps=1e-5, add=None):
    """The RMS norm of x (+ add) in int8.  Returns a dict: q, scale, and
    sum = x + add in x's type (None without add)."""
    got = _calls.rmsnorm_quantize(x, gamma, eps, add)
    if got is not None:
        return got
    M, K = _dims2(x, "x", "rmsnorm_quantize")
    out = {
        "q": torch.empty((M, K), dtype=_I8, device=x.device),
        "scale": torch.empty((M,), dtype=_F32, device=x.device),
        "sum": None if add is None else torch.empty((M, K), dtype=x.dtype, device=x.device),
    }
    tw_rmsnorm_quant(x, gamma, eps, out["q"], out["scale"], add=add, total=out["sum"])
    return out


def _scratch(n, device):
    return torch.empty((n,), dtype=_U8T, device=device) if n else None


def gated_ffn(x, wg_t, wu_t, wd, act="silu", keep=False, out_dtype=torch.bfloat16, ws=None):
    """The dense gated FFN (act(x W_g) * (x W_u)) W_d, act "relu", "silu" or
    "gelu".  Returns a dict: y, and with ``keep`` g and u (what
    ``gated_ffn_backward`` reads; None without)."""
    got = _calls.gated_ffn(x, wg_t, wu_t, wd, act, keep, out_dtype, ws)
    if got is not None:
        return got
    M, K = _dims2(x, "x", "gated_ffn")
    N = _dims2(wg_t, "wg_t", "gated_ffn")[0]
    dev = x.device
    out = {
        "y": torch.empty((M, K), dtype=out_dtype, device=dev),
        "g": torch.empty((M, N), dtype=_BF16, device=dev) if keep else None,
        "u": torch.empty((M, N), dtype=_BF16, device=dev) if keep else None,
    }
    ws = _scratch(tw_gated_ffn_workspace_bytes(M, K, N), dev) if ws is None else ws
    tw_gated_ffn_fwd(x, wg_t, wu_t, wd, out["y"], ws, act=act, g=out["g"], u=out["u"])
    return out


def gated_ffn_backward(dy, x, wg_t, wu_t, wd, g, u, act="silu", dx_dtype=torch.bfloat16,
                       dw_dtype=torch.bfloat16, ws=None):
    """Gradient of ``gated_ffn`` from its g and u.  Returns a dict: dx, dwg_t,
    dwu_t, dwd."""
    got = _calls.gated_ffn_backward(dy, x, wg_t, wu_t, wd, g, u, act, dx_dtype, dw_dtype, ws)
    if got is not None:
        return got
    M, K = _dims2(x, "x", "gated_ffn_backward")
    N = _dims2(wg_t, "wg_t", "gated_ffn_backward")[0]
    dev = x.device
    out = {"dx": torch.empty((M, K), dtype=dx_dtype, device=dev)}
    for k in ("dwg_t", "dwu_t", "dwd"):
        out[k] = torch.empty((N, K), dtype=dw_dtype, device=dev)
    ws = _scratch(tw_gated_ffn_bwd_workspace_bytes(M, K, N), dev) if ws is None else ws
    tw_gated_ffn_bwd(dy, x, wg_t, wu_t, wd, g, u, ws, act=act, **out)
    return out


def linear_ce(x, w, target, ws=None):
    """Cross entropy of the logits x w^T against one target a row (w: [V][K];
    a target outside [0, V) leaves its row out).  The targets are contiguous and may
    begin anywhere in a longer tensor (tokens[1:]).  Returns a dict: loss and lse
    (log-sum-exp) of every row, fp32."""
    got = _calls.linear_ce(x, w, target, ws)
    if got is not None:
        return got
    M, K = _dims2(x, "x", "linear_ce")
    V = _dims2(w, "w", "linear_ce")[0]
    out = {k: torch.empty((M,), dtype=_F32, device=x.device) for k in ("loss", "lse")}
    ws = _scratch(tw_linear_ce_workspace_bytes(M, K, V), x.device) if ws is None else ws
    tw_linear_ce_fwd(x, w, _aligned(target), out["loss"], out["lse"], ws)
    return out


def linear_ce_backward(dloss, x, w, target, lse, dx_dtype=torch.bfloat16, dw_dtype=torch.bfloat16,
                       ws=None):
    """Gradient of ``linear_ce`` for dloss (fp32, one a row).  Returns a dict:
    dx, dw."""
    got = _calls.linear_ce_backward(dloss, x, w, target, lse, dx_dtype, dw_dtype, ws)
    if got is not None:
        return got
    M, K = _dims2(x, "x", "linear_ce_backward")
    V = _dims2(w, "w", "linear_ce_backward")[0]
    out = {"dx": torch.empty((M, K), dtype=dx_dtype, device=x.device),
           "dw": torch.empty((V, K), dtype=dw_dtype, device=x.device)}
    ws = _scratch(tw_linear_ce_bwd_workspace_bytes(M, K, V), x.device) if ws is None else ws
    tw_linear_ce_bwd(_aligned(dloss), x, w, _aligned(target), _aligned(lse), ws, **out)
    return out


def _grads(grads, where):
    grads = list(grads)
    if not grads:
        raise ValueError(f"{where}: there are no gradients")
    if not isinstance(grads[0], torch.Tensor):
        raise TypeError(f"{where}: grads must be tensors of {_FLOATS}")
    return grads


def grad_norm(grads):
    """The norm over all elements of a list of tensors (bf16 or fp32), as a
    scalar tensor."""
    grads = _grads(grads, "grad_norm")
    dev = grads[0].device
    norm = torch.empty((), dtype=_F32, device=dev)
    tw_grad_norm(grads, norm, _scratch(tw_grad_norm_workspace_bytes([t.numel() for t in grads]), dev))
    return norm


def clip_grads(grads, max_norm, eps=1e-6, out=None):
    """Scales the gradients by min(1, max_norm / (norm + eps)), in place or
    into ``out`` (a list of tensors of the same shapes, bf16 or fp32).  Returns the
    norm before, a scalar tensor."""
    got = _calls.clip_grads(grads, max_norm, eps, out)
    if got is not None:
        return got
    grads = _grads(grads, "clip_grads")
    dev = grads[0].device
    norm = torch.empty((), dtype=_F32, device=dev)
    tw_grad_clip(grads, grads if out is None else list(out), max_norm, eps, norm,
                 _scratch(tw_grad_norm_workspace_bytes([t.numel() for t in grads]), dev))
    return norm


def library_path() -> str:
    return LIBRARY
