"""The experts' operators on torch tensors: matrix products grouped by expert, the activation with gate and
dropout between them, their gradients, and products with 4-bit weights.

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


def _activation(name) -> int:
    if name is None:
        return _moe.MOE_ACT_NONE
    _need(name in _moe.ACTIVATIONS, f"unknown activation {name!r}")
    return _moe.ACTIVATIONS[name]


def _like(t, name: str, like, ld=None) -> int:
    """t has like's shape and type; with ld, also that row pitch."""
    _need(t.dtype == like.dtype, f"{name} must be {like.dtype}, not {t.dtype}")
    _need(t.shape == like.shape, f"{name} must have shape {tuple(like.shape)}, not {tuple(t.shape)}")
    got = _rows(t, name, like.device)
    _need(ld is None or like.shape[0] <= 1 or got == ld, f"the rows of {name} must be {ld} elements apart, not {got}")
    return got


def _act(u, gate, activation, p, rng, rows):
    device = u.device
    code = _dtype(u, "u")
    ld = _rows(u, "u", device)
    if gate is not None:
        _like(gate, "gate", u, ld)
    if rng is not None:
        _need(rng.device == device and rng.dtype in (torch.int64, torch.uint64) and rng.numel() == 2 and rng.is_contiguous(),
              "rng must hold two 64-bit integers (seed, offset) on u's device")
    if rows is not None:
        _need(rows.device == device and rows.dtype == torch.int32 and rows.numel() == 1,
              "rows must be one int32 on u's device")
    return _moe.Act(u.shape[0], None if rows is None else rows.data_ptr(), u.shape[1], code, _activation(activation), p,
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
    _call("moe_act_dropout", u.device, _moe.load_library().moe_act_dropout, ctypes.byref(m), u.data_ptr(),
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
    _need(gate is not None or dgate is None, "dgate without a gate")
    if gate is not None:
        if dgate is None:
            dgate = torch.empty_strided(du.shape, du.stride(), dtype=u.dtype, device=u.device)
        _like(dgate, "dgate", u, m.ld_grad)
    _call("moe_act_dropout_backward", u.device, _moe.load_library().moe_act_dropout_backward, ctypes.byref(m), dy.data_ptr(),
          u.data_ptr(), None if gate is None else gate.data_ptr(), du.data_ptr(), None if dgate is None else dgate.data_ptr())
    return du if gate is None else (du, dgate)


def q4_quantize(W, group: int = 64):
    """4-bit codes and scales of ``W [E, K, N]`` (bf16 or f32, contiguous): ``(codes uint8 [E, N, K / 2], scales bf16
    [E, K / group, N])``, with ``W[e, k, n]`` near ``scales[e, k // group, n] * (code - 8)`` and the code of an even k
    in the low half of its byte.  Symmetric: the scale is max |w| / 7 of the group, codes round to the nearest."""
    _need(W.dim() == 3, "W must have three dimensions")
    code = _dtype(W, "W")
    _need(W.is_contiguous(), "W must be contiguous")
    E, K, N = W.shape
    _need(group in (32, 64, 128) and K % group == 0 and K > 0, "group must be 32, 64 or 128 and divide K")
    q = torch.empty((E, N, K // 2), dtype=torch.uint8, device=W.device)
    s = torch.empty((E, K // group, N), dtype=torch.bfloat16, device=W.device)
    _call("moe_q4_quantize", W.device, _moe.load_library().moe_q4_quantize, E, K, N, group, code, W.data_ptr(), q.data_ptr(),
          s.data_ptr())
    return q, s


class Q4Weights:
    """Expert weights ``[E, K, N]`` in 4 bits, laid out for ``q4_matmul`` (once, from codes and scales as
    ``q4_quantize`` makes them; those are not kept)."""

    def __init__(self, codes, scales):
        device = codes.device
        _need(codes.dim() == 3 and codes.dtype == torch.uint8, "codes must be a uint8 [E, N, K / 2] tensor")
        _need(scales.dim() == 3, "scales must have three dimensions")
        self.E, self.N, self.K = codes.shape[0], codes.shape[1], codes.shape[2] * 2
        groups = scales.shape[1]
        _need(groups > 0 and self.K % groups == 0 and self.K // groups in (32, 64, 128),
              f"scales must be [E, K / group, N] with a group of 32, 64 or 128, not {tuple(scales.shape)} for K = {self.K}")
        self.group = self.K // groups
        qptr = _dense(codes, "codes", device, torch.uint8, codes.shape)
        sptr = _dense(scales, "scales", device, torch.bfloat16, (self.E, groups, self.N))
        size = _moe.moe_q4_packed_size(self.E, self.K, self.N, self.group)
        if size == 0:
            raise _moe.MoEError(_moe.MOE_ERR_UNSUPPORTED, "moe_q4_packed_size")
        self.packed = torch.empty(size, dtype=torch.uint8, device=device)
        _call("moe_q4_pack", device, _moe.load_library().moe_q4_pack, self.E, self.K, self.N, self.group, qptr, sptr,
              self.packed.data_ptr())

    def dequantize(self, dtype=torch.bfloat16):
        """The weights ``[E, K, N]`` as they are computed with, rounded to dtype (exact in float32)."""
        W = torch.empty((self.E, self.K, self.N), dtype=dtype, device=self.packed.device)
        _call("moe_q4_dequantize", W.device, _moe.load_library().moe_q4_dequantize, self.E, self.K, self.N, self.group,
              self.packed.data_ptr(), _dtype(W, "W"), W.data_ptr())
        return W


def q4_workspace(device="cuda"):
    """A workspace for ``q4_matmul`` calls that follow each other on one stream; it serves every size."""
    return torch.zeros(_moe.moe_q4_workspace_size(), dtype=torch.uint8, device=device)


def q4_matmul(x, W: Q4Weights, offsets, bias=None, activation=None, out=None, out_dtype=None, ws=None):
    """``out[r] = act(x[r] @ W[e] + bias[e])`` for the rows ``offsets[e] <= r < offsets[e + 1]`` of every expert.

    x ``[rows, K]`` bf16 or f32 (rows may be strided), W a ``Q4Weights``, bias ``[E, N]`` of x's type or None,
    activation "gelu", "silu" or None, ``out`` ``[rows, N]`` of x's type or ``out_dtype`` (f32 or x's; rows may be
    strided); rows past ``offsets[E]`` are not written.  Made for a few rows an expert, right for any.  ws: a
    ``q4_workspace()`` that no call on another stream uses meanwhile (made for the call when not given); a bad
    offset is recorded in its first word (``moe_get_device_status(ws.data_ptr())``)."""
    device = x.device
    code = _dtype(x, "x")
    ldx = _rows(x, "x", device)
    optr, E = _offsets(offsets, device)
    _need(E == W.E, f"offsets has {E} experts, W {W.E}")
    _need(x.shape[1] == W.K, f"x must have {W.K} columns, not {x.shape[1]}")
    _need(W.packed.device == device, f"W is on {W.packed.device}, expected {device}")
    bptr = _dense(bias, "bias", device, x.dtype, (E, W.N))
    if out is None:
        out = torch.empty((x.shape[0], W.N), dtype=out_dtype or x.dtype, device=device)
    else:
        _need(tuple(out.shape) == (x.shape[0], W.N), f"out must have shape {(x.shape[0], W.N)}, not {tuple(out.shape)}")
        _need(out_dtype is None or out.dtype == out_dtype, "out has another type than out_dtype")
    ldy = _rows(out, "out", device)
    if ws is None:
        ws = q4_workspace(device)
    else:
        _need(ws.device == device and ws.is_contiguous(), f"ws must be a contiguous tensor on {device}")
    m = _moe.Q4(E, x.shape[0], W.K, W.N, W.group, code, _dtype(out, "out"), _activation(activation), ldx, ldy)
    _call("moe_q4_matmul", device, _moe.load_library().moe_q4_matmul, ctypes.byref(m), optr, x.data_ptr(), W.packed.data_ptr(),
          bptr, out.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size())
    return out
