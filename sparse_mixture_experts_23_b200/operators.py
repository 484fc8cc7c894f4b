"""The experts' operators on torch tensors: matrix products grouped by expert and their gradients.

Like ``MoEBuffers`` these functions only marshal arguments: they check shapes, types and devices, allocate
what the caller did not pass, and call the C entry point of the same meaning (``moe_grouped_matmul`` ...) on
the current stream of the tensors' device.  Inputs made on another stream have to be ordered before the
call by the caller, as for any torch operator.  Bad arguments raise ``ValueError``; a status that the library
returns raises ``MoEError``.  They take part in no autograd graph: gradients are calls of their own, as
``MoEBuffers.backward`` is.
"""
from __future__ import annotations

import ctypes

import torch

import sparse_mixture_experts_23_b200 as _moe

_CODES = {torch.float32: 0, torch.bfloat16: 1}  # moe_dtype_t


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _dtype(t, name: str) -> int:
    code = _CODES.get(t.dtype)
    _need(code is not None, f"{name} must be float32 or bfloat16, not {t.dtype}")
    return code


def _rows(t, name: str, device) -> int:
    """A matrix whose rows are contiguous; returns the elements between them."""
    _need(t.device == device, f"{name} is on {t.device}, expected {device}")
    _need(t.dim() == 2, f"{name} must have two dimensions")
    if t.shape[0] <= 1:
        _need(t.shape[1] <= 1 or t.stride(1) == 1, f"the rows of {name} must be contiguous")
        return t.shape[1]
    _need((t.shape[1] <= 1 or t.stride(1) == 1) and t.stride(0) >= t.shape[1],
          f"the rows of {name} must be contiguous and must not overlap")
    return t.stride(0)


def _dense(t, name: str, device, dtype, shape):
    if t is None:
        return None
    _need(t.device == device, f"{name} is on {t.device}, expected {device}")
    _need(t.dtype == dtype, f"{name} must be {dtype}, not {t.dtype}")
    _need(tuple(t.shape) == tuple(shape), f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    _need(t.is_contiguous(), f"{name} must be contiguous")
    return t.data_ptr()


def _offsets(offsets, device):
    _need(offsets.device == device and offsets.dtype == torch.int32 and offsets.dim() == 1 and offsets.is_contiguous()
          and offsets.shape[0] >= 2, "offsets must be a contiguous int32 vector of E + 1 entries on x's device")
    return offsets.data_ptr(), offsets.shape[0] - 1


def _status(status, device):
    if status is None:
        return None
    _need(status.device == device and status.dtype == torch.int32 and status.numel() >= 1,
          "status must be an int32 tensor on x's device")
    return status.data_ptr()


def _call(where: str, device, fn, *args) -> None:
    """fn(*args, stream) with the tensors' device current."""
    _need(device.type == "cuda", f"{where} needs CUDA tensors, not {device}")
    if torch.cuda.current_device() == device.index:
        code = fn(*args, torch.cuda.current_stream().cuda_stream)
    else:
        with torch.cuda.device(device):
            code = fn(*args, torch.cuda.current_stream().cuda_stream)
    if code != 0:
        raise _moe.MoEError(code, where)


def grouped_matmul(x, W, offsets, bias=None, transpose_w: bool = False, out=None, out_dtype=None, status=None):
    """``out[r] = x[r] @ W[e] + bias[e]`` for the rows ``offsets[e] <= r < offsets[e + 1]`` of every expert.

    x ``[rows, K]`` (rows may be strided), W ``[E, K, N]`` -- or ``[E, N, K]`` with ``transpose_w``, which gives
    the data gradient ``dy @ W[e].T`` of a forward product -- bias ``[E, N]`` or None, all of one type (bf16 or
    f32); offsets int32 ``[E + 1]`` on the device.  ``out`` ``[rows, N]`` (rows may be strided) is made when not
    given, of x's type or ``out_dtype``; rows past ``offsets[E]`` are not written.  bf16 wants K, N and row
    pitches that are multiples of 8, f32 of 4.  ``status``: an int32 tensor, 0 at first, that a bad offset is
    recorded in (see ``moe_get_device_status``)."""
    device = x.device
    code = _dtype(x, "x")
    ldx = _rows(x, "x", device)
    optr, E = _offsets(offsets, device)
    rows, K = x.shape
    _need(W.dim() == 3, "W must have three dimensions")
    N = W.shape[1] if transpose_w else W.shape[2]
    wptr = _dense(W, "W", device, x.dtype, (E, N, K) if transpose_w else (E, K, N))
    bptr = _dense(bias, "bias", device, x.dtype, (E, N))
    if out is None:
        out = torch.empty((rows, N), dtype=out_dtype or x.dtype, device=device)
    else:
        _need(tuple(out.shape) == (rows, N), f"out must have shape {(rows, N)}, not {tuple(out.shape)}")
        _need(out_dtype is None or out.dtype == out_dtype, "out has another type than out_dtype")
    ldy = _rows(out, "out", device)
    m = _moe.Matmul(E, rows, K, N, code, _dtype(out, "out"), int(transpose_w), ldx, ldy)
    _call("moe_grouped_matmul", device, _moe.load_library().moe_grouped_matmul, ctypes.byref(m), optr, x.data_ptr(), wptr,
          bptr, out.data_ptr(), _status(status, device))
    return out


def grouped_wgrad(x, dy, offsets, bias_grad: bool = False, dW=None, db=None, status=None):
    """``dW[e] = x_e.T @ dy_e`` over every expert's rows (``[E, K, N]`` float32), and with ``bias_grad`` (or ``db``
    given) ``db[e] = dy_e.sum(0)`` (``[E, N]`` float32).  x ``[rows, K]`` and dy ``[rows, N]`` of one type, rows may
    be strided.  Returns dW, or (dW, db).  Both are overwritten; an expert without rows gets zeros."""
    device = x.device
    code = _dtype(x, "x")
    _need(dy.dtype == x.dtype, f"dy must be {x.dtype}, not {dy.dtype}")
    ldx, ldy = _rows(x, "x", device), _rows(dy, "dy", device)
    _need(dy.shape[0] == x.shape[0], "x and dy must have the same number of rows")
    optr, E = _offsets(offsets, device)
    (rows, K), N = x.shape, dy.shape[1]
    if dW is None:
        dW = torch.empty((E, K, N), dtype=torch.float32, device=device)
    if db is None and bias_grad:
        db = torch.empty((E, N), dtype=torch.float32, device=device)
    m = _moe.Matmul(E, rows, K, N, code, 0, 0, ldx, ldy)
    _call("moe_grouped_wgrad", device, _moe.load_library().moe_grouped_wgrad, ctypes.byref(m), optr, x.data_ptr(),
          dy.data_ptr(), _dense(dW, "dW", device, torch.float32, (E, K, N)),
          _dense(db, "db", device, torch.float32, (E, N)), _status(status, device))
    return dW if db is None else (dW, db)
