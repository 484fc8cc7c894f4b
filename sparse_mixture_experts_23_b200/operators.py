"""The experts' operators on torch tensors: matrix products grouped by expert, the activation with gate and
dropout between them, their gradients, and products with 4-bit weights.

Like ``MoEBuffers`` these functions only marshal arguments: they check shapes, types and devices, allocate
what the caller did not pass, and call the C entry point of the same meaning (``moe_grouped_matmul`` ...) on
the current stream of the tensors' device.  Inputs made on another stream have to be ordered before the
call by the caller, as for any torch operator.  Bad arguments raise ``ValueError``; a status that the library
returns raises ``MoEError``.  They take part in no autograd graph: gradients are calls of their own, as
``MoEBuffers.backward`` is, and a tensor that requires a gradient is refused while torch records gradients, since its
gradient would be lost without a word.  Call them under ``torch.no_grad()``, within the forward and backward of a
``torch.autograd.Function``, or on detached tensors (``q4_quantize`` takes any: codes have no gradient).
"""
from __future__ import annotations

import ctypes

import torch

import sparse_mixture_experts_23_b200 as _moe

_CODES = {torch.float32: 0, torch.bfloat16: 1}  # moe_dtype_t
try:  # the device and the stream as the numbers that the C calls take, without torch.cuda's objects in between
    from torch._C import _cuda_getCurrentRawStream as _raw_stream, _cuda_getDevice as _current_device
except ImportError:  # pragma: no cover
    from torch.cuda import current_device as _current_device

    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


_functions = {}


# The checks run on every call, ahead of a launch that takes a few microseconds: messages are put together only
# when one fails, and devices are compared as their numbers (-1: not a CUDA tensor).
def _place(t, name: str, index: int) -> None:
    raise ValueError(f"{name} is on {t.device}, expected " + (f"cuda:{index}" if index >= 0 else "cpu"))


def _no_graph(name: str) -> None:
    raise ValueError(f"{name} requires a gradient, which this operator does not record: call it under torch.no_grad() or "
                     f"with {name}.detach()")


def _dtype(t, name: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16, not {t.dtype}")
    return code


def _rows(t, name: str, index: int) -> int:
    """A matrix whose rows are contiguous; returns the elements between them."""
    if t.get_device() != index:
        _place(t, name, index)
    if t.requires_grad and torch.is_grad_enabled():
        _no_graph(name)
    strides = t.stride()
    if len(strides) != 2:
        raise ValueError(f"{name} must have two dimensions")
    rows, cols = t.shape
    pitch, step = strides
    if step != 1 and cols > 1:
        raise ValueError(f"the rows of {name} must be contiguous" + (" and must not overlap" if rows > 1 else ""))
    if rows <= 1:
        return cols
    if pitch < cols:
        raise ValueError(f"the rows of {name} must be contiguous and must not overlap")
    return pitch


def _dense(t, name: str, index: int, dtype, shape):
    if t is None:
        return None
    if t.get_device() != index:
        _place(t, name, index)
    if t.requires_grad and torch.is_grad_enabled():
        _no_graph(name)
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _offsets(offsets, index: int):
    shape = offsets.shape
    if (offsets.dtype is not torch.int32 or len(shape) != 1 or shape[0] < 2 or offsets.get_device() != index
            or not offsets.is_contiguous()):
        raise ValueError("offsets must be a contiguous int32 vector of E + 1 entries on x's device")
    return offsets.data_ptr(), shape[0] - 1


def _status(status, index: int):
    if status is None:
        return None
    if status.get_device() != index or status.dtype is not torch.int32 or status.numel() < 1:
        raise ValueError("status must be an int32 tensor on x's device")
    return status.data_ptr()


def _out(out, rows: int, N: int, like, out_dtype):
    """The result: the caller's, checked, or a new one."""
    if out is None:
        return torch.empty((rows, N), dtype=out_dtype or like.dtype, device=like.device)
    if out.shape != (rows, N):
        raise ValueError(f"out must have shape {(rows, N)}, not {tuple(out.shape)}")
    if out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out has another type than out_dtype")
    return out


def _call(where: str, index: int, *args) -> None:
    """The C call `where`(*args, stream) with the tensors' device current."""
    if index < 0:
        raise ValueError(f"{where} needs CUDA tensors")
    fn = _functions.get(where)
    if fn is None:
        fn = _functions[where] = getattr(_moe.load_library(), where)
    if _current_device() == index:
        code = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            code = fn(*args, _raw_stream(index))
    if code != 0:
        raise _moe.MoEError(code, where)


def grouped_matmul(x, W, offsets, bias=None, transpose_w: bool = False, out=None, out_dtype=None, status=None):
    """``out[r] = x[r] @ W[e] + bias[e]`` for the rows ``offsets[e] <= r < offsets[e + 1]`` of every expert.

    x ``[rows, K]`` (rows may be strided), W ``[E, K, N]`` -- or ``[E, N, K]`` with ``transpose_w``, which gives
    the data gradient ``dy @ W[e].T`` of a forward product -- bias ``[E, N]`` or None, all of one type (bf16 or
    f32); offsets int32 ``[E + 1]`` on the device.  ``out`` ``[rows, N]`` (rows may be strided) is made when not
    given, of x's type or ``out_dtype``, and must not overlap the inputs; rows past ``offsets[E]`` are not
    written.  bf16 wants K, N and row pitches that are multiples of 8, f32 of 4.  ``status``: an int32 tensor, 0 at
    first, that a bad offset is recorded in (see ``moe_get_device_status``)."""
    index = x.get_device()
    code = _dtype(x, "x")
    ldx = _rows(x, "x", index)
    optr, E = _offsets(offsets, index)
    rows, K = x.shape
    shape = W.shape
    if len(shape) != 3:
        raise ValueError("W must have three dimensions")
    N = shape[1] if transpose_w else shape[2]
    wptr = _dense(W, "W", index, x.dtype, (E, N, K) if transpose_w else (E, K, N))
    bptr = _dense(bias, "bias", index, x.dtype, (E, N))
    out = _out(out, rows, N, x, out_dtype)
    ldy = _rows(out, "out", index)
    m = _moe.Matmul(E, rows, K, N, code, _dtype(out, "out"), int(transpose_w), ldx, ldy)
    _call("moe_grouped_matmul", index, ctypes.byref(m), optr, x.data_ptr(), wptr,
          bptr, out.data_ptr(), _status(status, index))
    return out


def grouped_wgrad(x, dy, offsets, bias_grad: bool = False, dW=None, db=None, status=None):
    """``dW[e] = x_e.T @ dy_e`` over every expert's rows (``[E, K, N]`` float32), and with ``bias_grad`` (or ``db``
    given) ``db[e] = dy_e.sum(0)`` (``[E, N]`` float32).  x ``[rows, K]`` and dy ``[rows, N]`` of one type, rows may
    be strided.  Returns dW, or (dW, db).  Both are overwritten; an expert without rows gets zeros."""
    index = x.get_device()
    code = _dtype(x, "x")
    if dy.dtype is not x.dtype:
        raise ValueError(f"dy must be {x.dtype}, not {dy.dtype}")
    ldx, ldy = _rows(x, "x", index), _rows(dy, "dy", index)
    (rows, K), (dy_rows, N) = x.shape, dy.shape
    if dy_rows != rows:
        raise ValueError("x and dy must have the same number of rows")
    optr, E = _offsets(offsets, index)
    if dW is None:
        dW = torch.empty((E, K, N), dtype=torch.float32, device=x.device)
    if db is None and bias_grad:
        db = torch.empty((E, N), dtype=torch.float32, device=x.device)
    m = _moe.Matmul(E, rows, K, N, code, 0, 0, ldx, ldy)
    _call("moe_grouped_wgrad", index, ctypes.byref(m), optr, x.data_ptr(),
          dy.data_ptr(), _dense(dW, "dW", index, torch.float32, (E, K, N)),
          _dense(db, "db", index, torch.float32, (E, N)), _status(status, index))
    return dW if db is None else (dW, db)


def _activation(name) -> int:
    if name is None:
        return _moe.MOE_ACT_NONE
    code = _moe.ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"unknown activation {name!r}")
    return code


def _like(t, name: str, like, ld=None) -> int:
    """t has like's shape and type; with ld, also that row pitch."""
    if t.dtype is not like.dtype:
        raise ValueError(f"{name} must be {like.dtype}, not {t.dtype}")
    if t.shape != like.shape:
        raise ValueError(f"{name} must have shape {tuple(like.shape)}, not {tuple(t.shape)}")
    got = _rows(t, name, like.get_device())
    if ld is not None and got != ld and like.shape[0] > 1:
        raise ValueError(f"the rows of {name} must be {ld} elements apart, not {got}")
    return got


def _act(u, gate, activation, p, rng, rows):
    index = u.get_device()
    code = _dtype(u, "u")
    ld = _rows(u, "u", index)
    if gate is not None:
        _like(gate, "gate", u, ld)
    if rng is not None and (rng.get_device() != index or rng.dtype not in (torch.int64, torch.uint64) or rng.numel() != 2
                            or not rng.is_contiguous()):
        raise ValueError("rng must hold two 64-bit integers (seed, offset) on u's device")
    if rows is not None and (rows.get_device() != index or rows.dtype is not torch.int32 or rows.numel() != 1):
        raise ValueError("rows must be one int32 on u's device")
    shape = u.shape
    return _moe.Act(shape[0], None if rows is None else rows.data_ptr(), shape[1], code, _activation(activation), p,
                    None if rng is None else rng.data_ptr(), ld, 0, 0)


def act_dropout(u, gate=None, activation="gelu", p: float = 0.0, rng=None, rows=None, out=None):
    """``act(u) * gate``, with each element zeroed with probability p and the others scaled by ``1 / (1 - p)``.

    u and gate ``[rows, F]`` (bf16 or f32; rows may be strided, both by the same pitch, so they can be the two
    halves of one product's columns), activation "gelu", "silu" or None (plain dropout), rng two int64 on the
    device: seed and offset of the generator, of which the backward pass wants the same.  ``rows``: an int32
    on the device (``offsets[-1:]``), the rows in use; those behind it are left as they are in ``out``, which
    may be u or gate."""
    m = _act(u, gate, activation, p, rng, rows)
    if out is None:
        out = torch.empty(u.shape, dtype=u.dtype, device=u.device)
    m.ld_y = _like(out, "out", u)
    _call("moe_act_dropout", u.get_device(), ctypes.byref(m), u.data_ptr(),
          None if gate is None else gate.data_ptr(), out.data_ptr())
    return out


def act_dropout_backward(dy, u, gate=None, activation="gelu", p: float = 0.0, rng=None, rows=None, du=None, dgate=None):
    """Gradients of ``act_dropout`` for the same u, gate, activation, p and rng: du, or (du, dgate) with a gate.
    du and dgate may be strided (by the same pitch) and may be dy, u or gate."""
    m = _act(u, gate, activation, p, rng, rows)
    m.ld_y = _like(dy, "dy", u)
    if du is None:
        du = torch.empty(u.shape, dtype=u.dtype, device=u.device)
    m.ld_grad = _like(du, "du", u)
    if gate is None:
        if dgate is not None:
            raise ValueError("dgate without a gate")
    else:
        if dgate is None:
            dgate = torch.empty_strided(du.shape, du.stride(), dtype=u.dtype, device=u.device)
        _like(dgate, "dgate", u, m.ld_grad)
    _call("moe_act_dropout_backward", u.get_device(), ctypes.byref(m), dy.data_ptr(),
          u.data_ptr(), None if gate is None else gate.data_ptr(), du.data_ptr(), None if dgate is None else dgate.data_ptr())
    return du if gate is None else (du, dgate)


def q4_quantize(W, group: int = 64):
    """4-bit codes and scales of ``W [E, K, N]`` (bf16 or f32, contiguous): ``(codes uint8 [E, N, K / 2], scales bf16
    [E, K / group, N])``, with ``W[e, k, n]`` near ``scales[e, k // group, n] * (code - 8)`` and the code of an even k
    in the low half of its byte.  Symmetric: the scale is max |w| / 7 of the group, codes round to the nearest."""
    if W.dim() != 3:
        raise ValueError("W must have three dimensions")
    code = _dtype(W, "W")
    if not W.is_contiguous():
        raise ValueError("W must be contiguous")
    E, K, N = W.shape
    if group not in (32, 64, 128) or K == 0 or K % group != 0:
        raise ValueError("group must be 32, 64 or 128 and divide K")
    q = torch.empty((E, N, K // 2), dtype=torch.uint8, device=W.device)
    s = torch.empty((E, K // group, N), dtype=torch.bfloat16, device=W.device)
    _call("moe_q4_quantize", W.get_device(), E, K, N, group, code, W.data_ptr(), q.data_ptr(),
          s.data_ptr())
    return q, s


class Q4Weights:
    """Expert weights ``[E, K, N]`` in 4 bits, laid out for ``q4_matmul`` (once, from codes and scales as
    ``q4_quantize`` makes them; those are not kept)."""

    def __init__(self, codes, scales):
        index = codes.get_device()
        if codes.dim() != 3 or codes.dtype != torch.uint8:
            raise ValueError("codes must be a uint8 [E, N, K / 2] tensor")
        if scales.dim() != 3:
            raise ValueError("scales must have three dimensions")
        self.E, self.N, self.K = codes.shape[0], codes.shape[1], codes.shape[2] * 2
        groups = scales.shape[1]
        if groups == 0 or self.K % groups != 0 or self.K // groups not in (32, 64, 128):
            raise ValueError(f"scales must be [E, K / group, N] with a group of 32, 64 or 128, not {tuple(scales.shape)} for "
                             f"K = {self.K}")
        self.group = self.K // groups
        qptr = _dense(codes, "codes", index, torch.uint8, codes.shape)
        sptr = _dense(scales, "scales", index, torch.bfloat16, (self.E, groups, self.N))
        size = _moe.moe_q4_packed_size(self.E, self.K, self.N, self.group)
        if size == 0:
            raise _moe.MoEError(_moe.MOE_ERR_UNSUPPORTED, "moe_q4_packed_size")
        self.packed = torch.empty(size, dtype=torch.uint8, device=codes.device)
        _call("moe_q4_pack", index, self.E, self.K, self.N, self.group, qptr, sptr,
              self.packed.data_ptr())

    def dequantize(self, dtype=torch.bfloat16):
        """The weights ``[E, K, N]`` as they are computed with, rounded to dtype (exact in float32)."""
        W = torch.empty((self.E, self.K, self.N), dtype=dtype, device=self.packed.device)
        _call("moe_q4_dequantize", W.get_device(), self.E, self.K, self.N, self.group,
              self.packed.data_ptr(), _dtype(W, "W"), W.data_ptr())
        return W


def q4_workspace(device="cuda"):
    """A workspace for ``q4_matmul`` calls of any size."""
    return torch.zeros(_moe.moe_q4_workspace_size(), dtype=torch.uint8, device=device)


def q4_matmul(x, W: Q4Weights, offsets, bias=None, activation=None, out=None, out_dtype=None, ws=None):
    """``out[r] = act(x[r] @ W[e] + bias[e])`` for the rows ``offsets[e] <= r < offsets[e + 1]`` of every expert.

    x ``[rows, K]`` bf16 or f32 (rows may be strided), W a ``Q4Weights``, bias ``[E, N]`` of x's type or None,
    activation "gelu", "silu" or None, ``out`` ``[rows, N]`` of x's type or ``out_dtype`` (f32 or x's; rows may be
    strided; must not overlap the inputs); rows past ``offsets[E]`` are not written.  Made for a few rows an expert,
    right for any.  ws: a ``q4_workspace()`` (made for the call when not given); a bad offset is recorded in its first
    word (``moe_get_device_status(ws.data_ptr())``)."""
    index = x.get_device()
    code = _dtype(x, "x")
    ldx = _rows(x, "x", index)
    optr, E = _offsets(offsets, index)
    rows, K = x.shape
    if E != W.E:
        raise ValueError(f"offsets has {E} experts, W {W.E}")
    if K != W.K:
        raise ValueError(f"x must have {W.K} columns, not {K}")
    packed = W.packed
    if packed.get_device() != index:
        _place(packed, "W", index)
    bptr = _dense(bias, "bias", index, x.dtype, (E, W.N))
    out = _out(out, rows, W.N, x, out_dtype)
    ldy = _rows(out, "out", index)
    if ws is None:
        ws = q4_workspace(x.device)
    elif ws.get_device() != index or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on {x.device}")
    m = _moe.Q4(E, rows, K, W.N, W.group, code, _dtype(out, "out"), _activation(activation), ldx, ldy)
    _call("moe_q4_matmul", index, ctypes.byref(m), optr, x.data_ptr(), packed.data_ptr(),
          bptr, out.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size())
    return out
