"""Operators beside the GEMM: the gated feed-forward block, its backward pass,
its products from 4-bit weights, and the orthogonalised update of its matrices.

Thin ctypes bindings over the C ABI in ``include/gemm_ops.h``; every step runs
in the sm_103a kernels of ``libgb300gemm.so``.  Tensors are CUDA tensors of one
device, float16 or bfloat16; workspaces come from torch's allocator on the
current stream.  There is no fallback: wrong arguments and other devices raise.

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
import threading

import torch

from . import GemmError, _check, load as _load

__all__ = ["Ops", "default_ops", "gated_ffn", "gated_ffn_backward", "w4_linear", "w4_gated",
           "w4_quantize", "orthogonalize", "NEWTON_SCHULZ"]

_F16, _BF16 = torch.float16, torch.bfloat16
_DTYPE = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
_ACT = {"silu": 0, "gelu_tanh": 1, "relu": 2}

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
                "gemm_gated_ffn_workspace": (sz, [vp, i64, i64, i64]),
                "gemm_gated_ffn": (st, [vp, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, sz, i64, i64,
                                        i64, st, st, vp]),
                "gemm_gated_ffn_backward_workspace": (sz, [vp, i64, i64, i64]),
                "gemm_gated_ffn_backward": (st, [vp, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, i64,
                                                 vp, vp, vp, sz, i64, i64, i64, st, st, vp]),
                "gemm_w4_workspace": (sz, [vp, i64, i64, i64, i32]),
                "gemm_w4_linear": (st, [vp, vp, i64, vp, vp, vp, vp, i64, vp, sz, i64, i64, i64, i64, st,
                                        vp]),
                "gemm_w4_gated": (st, [vp, vp, i64, vp, vp, vp, vp, i64, vp, sz, i64, i64, i64, i64, st,
                                       st, vp]),
                "gemm_orthogonalize_workspace": (sz, [vp, i64, i64, i64]),
                "gemm_orthogonalize": (st, [vp, vp, i64, i64, vp, i64, i64, vp, sz, i64, i64, i64, i32,
                                            ctypes.POINTER(f32), f32, st, st, vp]),
            }
            for name, (res, args) in sig.items():
                fn = getattr(lib, name)
                fn.restype, fn.argtypes = res, args
            _SIG = sig
    return lib


def _act(act) -> int:
    try:
        return _ACT[act]
    except (KeyError, TypeError):
        raise ValueError(f"act must be one of {sorted(_ACT)}, got {act!r}") from None


def _matrix(t, name, dtype, index, shape, contiguous=False):
    """Checks one 2-D operand; returns its row distance in elements."""
    if t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous():
        return shape[1]  # the common case, in few calls: small products are bound by the host
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    rows, cols = shape
    ld, inner = t.stride()
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if (cols > 1 and inner != 1) or (rows > 1 and ld < cols):
        raise ValueError(f"{name}'s rows must be contiguous")
    # One row or none, or nothing in a row: the distance to the next is free.
    return ld if rows > 1 and cols else cols


def _operand(t, name):
    """Type, device index and shape of a call's first operand."""
    dt, index, shape = t.dtype, t.get_device(), t.shape
    if dt is not _F16 and dt is not _BF16:
        raise TypeError(f"{name} must be float16 or bfloat16, got {dt}")
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D, got {list(shape)}")
    return dt, index, shape


def _columns(t, name, rows):
    """Columns of a matrix that has to have `rows` rows."""
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows:
        raise ValueError(f"{name} must be a matrix of {rows} rows, got {list(shape)}")
    return shape[1]


def _current_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# The handle alone, without building a stream object (where torch has it).
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


def _stream(stream, index):
    if stream is None:
        return _current_stream(index)
    return stream if isinstance(stream, int) else stream.cuda_stream


class Ops:
    """Owns a ``gemm_ops_t`` bound to one CUDA device."""

    def __init__(self, device: int = 0):
        self._lib = _lib()
        self._h = ctypes.c_void_p()
        _check(self._lib.gemm_ops_create(ctypes.byref(self._h), int(device)), "gemm_ops_create")
        self.index = int(device)
        self.device = torch.device("cuda", self.index)
        self._needs = {}  # workspace bytes by operator and sizes

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            self._lib.gemm_ops_destroy(self._h)
            self._h = ctypes.c_void_p()

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

    def _workspace(self, query, *sizes):
        """A workspace of torch's allocator: (tensor, address, bytes)."""
        key = (query, sizes)
        need = self._needs.get(key)
        if need is None:
            if len(self._needs) >= 4096:
                self._needs.clear()
            need = self._needs[key] = getattr(self._lib, query)(self._h, *sizes)
        if not need:
            return None, None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        return ws, ws.data_ptr(), need

    def _same_device(self, index, name):
        if index != self.index:
            raise ValueError(f"{name} is on cuda:{index}, the handle on cuda:{self.index}")

    # -- the gated block ----------------------------------------------------
    def gated_ffn(self, x, w_in, w_down, act="silu", save=False, out=None, stream=None):
        dt, dev, (T, D) = _operand(x, "x")
        self._same_device(dev, "x")
        a = _act(act)
        ldx = _matrix(x, "x", dt, dev, (T, D))
        F = _columns(w_down, "w_down", D)
        ldd = _matrix(w_down, "w_down", dt, dev, (D, F))
        ldi = _matrix(w_in, "w_in", dt, dev, (2 * F, D))
        if out is None:
            out = torch.empty((T, D), dtype=dt, device=self.device)
            ldy = D
        else:
            ldy = _matrix(out, "out", dt, dev, (T, D))
        gu = torch.empty((T, 2 * F), dtype=dt, device=self.device) if save else None
        ws, wp, need = self._workspace("gemm_gated_ffn_workspace", T, D, F)
        st = self._lib.gemm_gated_ffn(
            self._h, x.data_ptr(), ldx, w_in.data_ptr(), ldi, w_down.data_ptr(), ldd, out.data_ptr(), ldy,
            gu.data_ptr() if save else None, wp, need, T, D, F, a, _DTYPE[dt], _stream(stream, dev))
        if st:
            _check(st, "gemm_gated_ffn")
        return (out, gu) if save else out

    def gated_ffn_backward(self, dy, x, w_in, w_down, gu, act="silu", stream=None):
        dt, dev, (T, D) = _operand(x, "x")
        self._same_device(dev, "x")
        a = _act(act)
        ldx = _matrix(x, "x", dt, dev, (T, D))
        F = _columns(w_down, "w_down", D)
        ldd = _matrix(w_down, "w_down", dt, dev, (D, F))
        ldi = _matrix(w_in, "w_in", dt, dev, (2 * F, D))
        ldy = _matrix(dy, "dy", dt, dev, (T, D))
        _matrix(gu, "gu", dt, dev, (T, 2 * F), contiguous=True)
        dx = torch.empty((T, D), dtype=dt, device=self.device)
        dw_in = torch.empty((2 * F, D), dtype=dt, device=self.device)
        dw_down = torch.empty((D, F), dtype=dt, device=self.device)
        ws, wp, need = self._workspace("gemm_gated_ffn_backward_workspace", T, D, F)
        st = self._lib.gemm_gated_ffn_backward(
            self._h, dy.data_ptr(), ldy, x.data_ptr(), ldx, w_in.data_ptr(), ldi, w_down.data_ptr(), ldd,
            gu.data_ptr(), dx.data_ptr(), D, dw_in.data_ptr(), dw_down.data_ptr(), wp, need,
            T, D, F, a, _DTYPE[dt], _stream(stream, dev))
        if st:
            _check(st, "gemm_gated_ffn_backward")
        return dx, dw_in, dw_down

    # -- 4-bit weights ------------------------------------------------------
    def _w4(self, x, codes, scales, zeros, gated, act, out, stream):
        dt, dev, (T, K) = _operand(x, "x")
        self._same_device(dev, "x")
        a = _act(act)
        ldx = _matrix(x, "x", dt, dev, (T, K))
        shape = codes.shape
        if len(shape) != 2 or shape[1] * 2 != K:
            raise ValueError(f"codes must be [N, {K // 2}] for x of {K} columns, got {list(shape)}")
        rows = shape[0]
        _matrix(codes, "codes", torch.uint8, dev, shape, contiguous=True)
        groups = _columns(scales, "scales", rows)
        if (groups == 0) != (K == 0) or (K and K % groups):
            raise ValueError(f"scales must be [{rows}, K / group], got {list(scales.shape)}")
        _matrix(scales, "scales", dt, dev, (rows, groups), contiguous=True)
        if zeros is not None:
            _matrix(zeros, "zeros", torch.uint8, dev, (rows, groups), contiguous=True)
        if gated and rows % 2:
            raise ValueError("gated weights have an even number of rows: gate rows, then up rows")
        N = rows // 2 if gated else rows
        if out is None:
            out = torch.empty((T, N), dtype=dt, device=self.device)
            ldy = N
        else:
            ldy = _matrix(out, "out", dt, dev, (T, N))
        ws, wp, need = self._workspace("gemm_w4_workspace", T, N, K, gated)
        zp = zeros.data_ptr() if zeros is not None else None
        group = K // groups if groups else 32
        if gated:
            st = self._lib.gemm_w4_gated(
                self._h, x.data_ptr(), ldx, codes.data_ptr(), scales.data_ptr(), zp, out.data_ptr(), ldy, wp,
                need, T, N, K, group, a, _DTYPE[dt], _stream(stream, dev))
        else:
            st = self._lib.gemm_w4_linear(
                self._h, x.data_ptr(), ldx, codes.data_ptr(), scales.data_ptr(), zp, out.data_ptr(), ldy, wp,
                need, T, N, K, group, _DTYPE[dt], _stream(stream, dev))
        if st:
            _check(st, "gemm_w4_gated" if gated else "gemm_w4_linear")
        return out

    def w4_linear(self, x, codes, scales, zeros=None, out=None, stream=None):
        return self._w4(x, codes, scales, zeros, False, "silu", out, stream)

    def w4_gated(self, x, codes, scales, zeros=None, act="silu", out=None, stream=None):
        return self._w4(x, codes, scales, zeros, True, act, out, stream)

    # -- the orthogonalised update -------------------------------------------
    def orthogonalize(self, m, steps=5, coeffs=NEWTON_SCHULZ, eps=1e-7, dtype=None, out=None, stream=None):
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
        ws, wp, need = self._workspace("gemm_orthogonalize_workspace", B, M, N)
        _check(self._lib.gemm_orthogonalize(
            self._h, m.data_ptr(), lds[0], lds[1], out.data_ptr(), lds[2], lds[3], wp, need, B, M, N,
            int(steps), (ctypes.c_float * 3)(*coeffs), float(eps), _DTYPE[m.dtype], _DTYPE[dtype],
            _stream(stream, self.index)), "gemm_orthogonalize")
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
    each group's range, zero included."""
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
