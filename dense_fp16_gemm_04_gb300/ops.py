"""Operators beside the GEMM: the gated feed-forward block, its backward pass,
its products from 4-bit weights, and the orthogonalised update of its matrices.

Thin bindings over the C ABI in ``include/gemm_ops.h``: the block and the 4-bit
products through the compiled ``_binding`` (a call for one token costs the host
more than the GPU), ``orthogonalize`` through ctypes.  Every step runs in the
sm_103a kernels of ``libgb300gemm.so``.  Tensors are CUDA tensors of one device,
float16 or bfloat16; results and workspaces come from torch's allocator, on the
stream of the call (the current one, or ``stream``).  As with any work on another
stream, the caller orders it after what made the inputs and keeps them until it
has run (``Tensor.record_stream``).  There is no fallback: wrong arguments and
other devices raise.

The operators record no graph.  A tensor that requires grad (while gradients are
recorded) or has a forward-mode tangent is refused with a RuntimeError: call them
under ``torch.no_grad()`` or on detached tensors, or from the methods of a
``torch.autograd.Function``, whose backward is :func:`gated_ffn_backward`.

    >>> import torch, dense_fp16_gemm_04_gb300 as g
    >>> x = torch.randn(4096, 1024, device="cuda", dtype=torch.float16)
    >>> w_in = torch.randn(2 * 4096, 1024, device="cuda", dtype=torch.float16) / 32
    >>> w_down = torch.randn(1024, 4096, device="cuda", dtype=torch.float16) / 64
    >>> y, gu = g.gated_ffn(x, w_in, w_down, save=True)
    >>> dx, dw_in, dw_down = g.gated_ffn_backward(y, x, w_in, w_down, gu)
    >>> step = g.orthogonalize(dw_down)
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading

import torch

from . import GemmError, _build, _check, load as _load

__all__ = ["Ops", "default_ops", "gated_ffn", "gated_ffn_backward", "w4_linear", "w4_gated",
           "w4_quantize", "orthogonalize", "NEWTON_SCHULZ"]

_DTYPE = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}

#: Coefficients a, b, c of X <- a X + (b P + c P^2) X, P = X X^T.
NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)

_SIG = None
_sig_lock = threading.Lock()


def _lib():
    """The library, with the operators' signatures set."""
    global _SIG
    lib = _load()
    with _sig_lock:
        if _SIG is None:
            vp, i64, i32, u64, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint64,
                                     ctypes.c_size_t)
            st, f32 = ctypes.c_int, ctypes.c_float
            sig = {
                "gemm_ops_create": (st, [ctypes.POINTER(vp), ctypes.c_int]),
                "gemm_ops_destroy": (st, [vp]),
                "gemm_ops_check_error": (st, [vp]),
                "gemm_ops_last_error_detail": (st, [vp, ctypes.POINTER(ctypes.c_uint32)]),
                "gemm_ops_set_watchdog": (st, [vp, u64, i32]),
                "gemm_ops_launch_count": (u64, [vp]),
                "gemm_orthogonalize_workspace": (sz, [vp, i64, i64, i64]),
                "gemm_orthogonalize": (st, [vp, vp, i64, i64, vp, i64, i64, vp, sz, i64, i64, i64, i32,
                                            ctypes.POINTER(f32), f32, st, st, vp]),
            }
            for name, (res, args) in sig.items():
                fn = getattr(lib, name)
                fn.restype, fn.argtypes = res, args
            _SIG = sig
    return lib


def _current_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# The handle alone, without building a stream object (where torch has it).
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


_binding = None


def _load_binding():
    """The compiled binding, set up with torch's objects and the library's functions."""
    global _binding
    lib = _lib()
    with _sig_lock:
        if _binding is None:
            path = _build.binding_path()
            if path is None:
                raise ImportError("the operators need a torch with CUDA")
            if not os.path.exists(path):
                raise ImportError(f"{path} is missing: build it for this torch with "
                                  "dense_fp16_gemm_04_gb300.build()")
            spec = importlib.util.spec_from_file_location("_binding", path)
            mod = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(mod)
            fns = ("gemm_gated_ffn_workspace", "gemm_gated_ffn", "gemm_gated_ffn_backward_workspace",
                   "gemm_gated_ffn_backward", "gemm_w4_workspace", "gemm_w4_linear", "gemm_w4_gated")
            mod.setup(GemmError, *(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in fns))
            _binding = mod
    return _binding


class Ops:
    """Owns a ``gemm_ops_t`` bound to one CUDA device."""

    def __init__(self, device: int = 0):
        self._lib = _lib()
        self._h = ctypes.c_void_p()
        _check(self._lib.gemm_ops_create(ctypes.byref(self._h), int(device)), "gemm_ops_create")
        self.index = int(device)
        self.device = torch.device("cuda", self.index)
        self._addr = self._h.value
        self._b = _load_binding()

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            self._lib.gemm_ops_destroy(self._h)
            self._h = ctypes.c_void_p()
            self._addr = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def check_error(self) -> None:
        """Synchronize; raise GemmError if a kernel's watchdog fired."""
        _check(self._lib.gemm_ops_check_error(self._h), "gemm_ops_check_error")

    def last_error_detail(self):
        d = (ctypes.c_uint32 * 4)()
        _check(self._lib.gemm_ops_last_error_detail(self._h, d), "gemm_ops_last_error_detail")
        return list(d)

    def set_watchdog(self, timeout_ns: int = 0, skip_k_block: int = -1) -> None:
        _check(self._lib.gemm_ops_set_watchdog(self._h, int(timeout_ns), int(skip_k_block)),
               "gemm_ops_set_watchdog")

    @property
    def launch_count(self) -> int:
        return int(self._lib.gemm_ops_launch_count(self._h))

    # -- the gated block ----------------------------------------------------
    def gated_ffn(self, x, w_in, w_down, act="silu", save=False, out=None, stream=None):
        return self._b.gated_ffn(self._addr, self.index, x, w_in, w_down, act, save, out, stream)

    def gated_ffn_backward(self, dy, x, w_in, w_down, gu, act="silu", stream=None):
        return self._b.gated_ffn_backward(self._addr, self.index, dy, x, w_in, w_down, gu, act,
                                          stream)

    # -- 4-bit weights ------------------------------------------------------
    def w4_linear(self, x, codes, scales, zeros=None, out=None, stream=None):
        return self._b.w4(self._addr, self.index, x, codes, scales, zeros, None, out, stream)

    def w4_gated(self, x, codes, scales, zeros=None, act="silu", out=None, stream=None):
        if act is None:
            raise ValueError("act must be 'silu', 'gelu_tanh' or 'relu', got None")
        return self._b.w4(self._addr, self.index, x, codes, scales, zeros, act, out, stream)

    # -- the orthogonalised update -------------------------------------------
    def orthogonalize(self, m, steps=5, coeffs=NEWTON_SCHULZ, eps=1e-7, dtype=None, out=None, stream=None):
        for name, t in (("m", m), ("out", out)):
            if t is not None or name == "m":
                self._b.no_graph(t, name)
        if m.dtype not in _DTYPE:
            raise TypeError(f"m must be float16, bfloat16 or float32, got {m.dtype}")
        if m.device != self.device:
            raise ValueError(f"m must be on {self.device}, got {m.device}")
        if m.dim() not in (2, 3):
            raise ValueError(f"m must be [M, N] or [batch, M, N], got {list(m.shape)}")
        coeffs = tuple(float(c) for c in coeffs)
        if len(coeffs) != 3:
            raise ValueError(f"coeffs must be three numbers, got {len(coeffs)}")
        if dtype is None:
            dtype = out.dtype if out is not None else m.dtype
        if dtype not in _DTYPE:
            raise TypeError(f"dtype must be float16, bfloat16 or float32, got {dtype}")
        if stream is not None:  # what is allocated belongs to the stream that uses it
            if isinstance(stream, int):
                # The legacy default stream's handle is 1; torch knows it as 0.
                stream = torch.cuda.ExternalStream(0 if stream == 1 else stream, device=self.device)
            with torch.cuda.stream(stream):
                return self.orthogonalize(m, steps, coeffs, eps, dtype, out)
        given = out
        if out is None:
            out = torch.empty(m.shape, dtype=dtype, device=self.device)
        elif out.shape != m.shape or out.dtype != dtype or out.device != self.device:
            raise ValueError(f"out must be {dtype} {list(m.shape)} on {self.device}")
        m3, o3 = (m, out) if m.dim() == 3 else (m.unsqueeze(0), out.unsqueeze(0))
        B, M, N = m3.shape
        lds = []
        for name, t in (("m", m3), ("out", o3)):
            bs, ld, inner = t.stride()
            if N > 1 and inner != 1 or M > 1 and ld < N:
                raise ValueError(f"{name}'s rows must be contiguous")
            lds += [ld if M > 1 else N, bs if B > 1 else 0]
        need = self._lib.gemm_orthogonalize_workspace(self._h, B, M, N)
        ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        _check(self._lib.gemm_orthogonalize(
            self._h, m.data_ptr(), lds[0], lds[1], out.data_ptr(), lds[2], lds[3], ws.data_ptr(), need, B, M, N,
            int(steps), (ctypes.c_float * 3)(*coeffs), float(eps), _DTYPE[m.dtype], _DTYPE[dtype],
            _current_stream(self.index)), "gemm_orthogonalize")
        if given is not None:
            self._b.wrote(given)
        return out


_ops = {}
_ops_lock = threading.Lock()


def default_ops(device=None) -> Ops:
    """One shared handle per device, created on first use.  It holds no data
    between calls, so it serves every stream."""
    if device is None:
        device = torch.cuda.current_device()
    o = _ops.get(device)
    if o is None:
        with _ops_lock:
            o = _ops.get(device)
            if o is None:
                o = _ops[device] = Ops(device)
    return o


def _of(t, ops) -> Ops:
    if ops is not None:
        return ops
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"operands must be tensors, got {type(t)}")
    index = t.get_device()
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    return _ops.get(index) or default_ops(index)


def gated_ffn(x, w_in, w_down, act="silu", save=False, out=None, stream=None, ops: Ops | None = None):
    """The gated feed-forward block  y = (act(x Wg^T) * (x Wu^T)) Wd^T.

    x [T, D]; w_in [2 F, D], the rows of Wg, then those of Wu; w_down [D, F];
    act 'silu', 'gelu_tanh' or 'relu'.  Returns y [T, D], and with ``save`` also
    gu [T, 2 F], the two projections that :func:`gated_ffn_backward` takes.
    D and F are multiples of 8; rows may be strided by multiples of 8."""
    return _of(x, ops).gated_ffn(x, w_in, w_down, act, save, out, stream)


def gated_ffn_backward(dy, x, w_in, w_down, gu, act="silu", stream=None, ops: Ops | None = None):
    """Gradients (dx, dw_in, dw_down) of :func:`gated_ffn` from dy [T, D]."""
    return _of(x, ops).gated_ffn_backward(dy, x, w_in, w_down, gu, act, stream)


def w4_linear(x, codes, scales, zeros=None, out=None, stream=None, ops: Ops | None = None):
    """y [T, N] = x W^T with W[n, k] = scales[n, k // G] (q[n, k] - zeros[n, k // G]).

    codes [N, K / 2] uint8 holds two codes a byte, the even column's in the low
    half; scales [N, K / G] in x's type; zeros [N, K / G] uint8 (8 if None).  The
    group G is K / scales.shape[1], a power of two from 32 on."""
    return _of(x, ops).w4_linear(x, codes, scales, zeros, out, stream)


def w4_gated(x, codes, scales, zeros=None, act="silu", out=None, stream=None, ops: Ops | None = None):
    """act(x Wg^T) * (x Wu^T) from 4-bit weights of 2 N rows: Wg's, then Wu's."""
    return _of(x, ops).w4_gated(x, codes, scales, zeros, act, out, stream)


def w4_quantize(w, group=128, zero_point=False):
    """Codes, scales and zeros of w [N, K] for :func:`w4_linear`, by rounding to
    the nearest level: symmetric about code 8, or (``zero_point``) spread over
    each group's range, zero included.  No gradient goes back to w."""
    w = w.detach()
    N, K = w.shape
    if group < 32 or group & (group - 1) or K % group:
        raise ValueError(f"group must be a power of two from 32 on that divides K = {K}, got {group}")
    v = w.float().reshape(N, K // group, group)
    if zero_point:
        lo, hi = v.amin(-1).clamp_max(0), v.amax(-1).clamp_min(0)
        scales = ((hi - lo) / 15).to(w.dtype)
        s = scales.float().clamp_min(torch.finfo(torch.float32).tiny)
        zeros = (-lo / s).round().clamp_(0, 15)
    else:
        # The larger of the two ends lands on code 0 or 15.
        scales = torch.maximum(v.amax(-1) / 7, -v.amin(-1) / 8).to(w.dtype)
        s = scales.float().clamp_min(torch.finfo(torch.float32).tiny)
        zeros = torch.full_like(s, 8)
    q = ((v / s.unsqueeze(-1)).round() + zeros.unsqueeze(-1)).clamp_(0, 15).to(torch.uint8).reshape(N, K)
    codes = q[:, 0::2] | (q[:, 1::2] << 4)
    return codes.contiguous(), scales, zeros.to(torch.uint8) if zero_point else None


def orthogonalize(m, steps=5, coeffs=NEWTON_SCHULZ, eps=1e-7, dtype=None, out=None, stream=None,
                  ops: Ops | None = None):
    """The orthogonalised update of m [M, N] or [batch, M, N]: ``steps`` steps of
    X <- a X + (b P + c P^2) X, P = X X^T, from X = m / (|m| + eps), computed to
    fp32 accuracy.  m is float16, bfloat16 or float32; the result has ``dtype``
    (m's by default)."""
    return _of(m, ops).orthogonalize(m, steps, coeffs, eps, dtype, out, stream)
