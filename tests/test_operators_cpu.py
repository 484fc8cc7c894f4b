"""Argument checks of the experts' operators: every refusal comes before any CUDA work, so none needs a GPU."""
import ctypes

import pytest
import torch

import sparse_mixture_experts_23_b200 as moe
from sparse_mixture_experts_23_b200 import build as moe_build

FAKE = 1 << 20  # an aligned non-null "device" address; never dereferenced by these calls


@pytest.fixture(scope="module", autouse=True)
def lib():
    moe_build.build()
    return moe.load_library()


def matmul(**kw):
    d = dict(E=4, rows_cap=100, K=64, N=128, dtype=1, out_dtype=1, transpose_w=0, ldx=0, ldy=0)
    d.update(kw)
    return moe.Matmul(**d)


BAD_SIZES = [
    (dict(E=0), moe.MOE_ERR_INVALID_ARG), (dict(E=257), moe.MOE_ERR_INVALID_ARG), (dict(rows_cap=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(K=0), moe.MOE_ERR_INVALID_ARG), (dict(N=0), moe.MOE_ERR_INVALID_ARG), (dict(N=-8), moe.MOE_ERR_INVALID_ARG),
    (dict(dtype=2), moe.MOE_ERR_INVALID_ARG), (dict(ldx=56), moe.MOE_ERR_INVALID_ARG), (dict(ldy=120), moe.MOE_ERR_INVALID_ARG),
    (dict(K=60), moe.MOE_ERR_UNSUPPORTED), (dict(N=100), moe.MOE_ERR_UNSUPPORTED), (dict(ldx=68), moe.MOE_ERR_UNSUPPORTED),
    (dict(ldy=132), moe.MOE_ERR_UNSUPPORTED), (dict(dtype=0, out_dtype=0, K=62), moe.MOE_ERR_UNSUPPORTED),
    (dict(rows_cap=(1 << 31) - 1024), moe.MOE_ERR_UNSUPPORTED), (dict(N=1 << 23), moe.MOE_ERR_UNSUPPORTED),
    (dict(rows_cap=1 << 30, N=1 << 20), moe.MOE_ERR_UNSUPPORTED), (dict(ldx=1 << 37), moe.MOE_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("bad,code", BAD_SIZES)
def test_matmul_sizes(bad, code):
    m = matmul(**bad)
    assert moe.moe_grouped_matmul(m, FAKE, FAKE, FAKE, None, FAKE) == code
    if "rows_cap" not in bad or bad["rows_cap"] != 1 << 30:  # the weight gradient has no tile per row block
        assert moe.moe_grouped_wgrad(m, FAKE, FAKE, FAKE, FAKE) == code
    assert moe.moe_last_launch_count() == 0


def test_matmul_types_and_pointers():
    for bad, code in ((dict(out_dtype=2), moe.MOE_ERR_INVALID_ARG), (dict(dtype=0, out_dtype=1), moe.MOE_ERR_UNSUPPORTED)):
        assert moe.moe_grouped_matmul(matmul(**bad), FAKE, FAKE, FAKE, None, FAKE) == code
    ok = [FAKE, FAKE, FAKE, None, FAKE]
    for i in (0, 1, 2, 4):  # offsets, x, W, y
        for p in (None, FAKE + 2):
            args = list(ok)
            args[i] = p
            assert moe.moe_grouped_matmul(matmul(), *args) == moe.MOE_ERR_INVALID_ARG, (i, p)
            assert moe.moe_grouped_wgrad(matmul(), *args[:3], args[4] if i == 4 else FAKE) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_grouped_matmul(matmul(), FAKE, FAKE, FAKE, FAKE + 8, FAKE) == moe.MOE_ERR_INVALID_ARG  # bias
    assert moe.moe_grouped_matmul(matmul(), FAKE, FAKE, FAKE, None, FAKE, FAKE + 1) == moe.MOE_ERR_INVALID_ARG  # status
    assert moe.moe_grouped_wgrad(matmul(), FAKE, FAKE, FAKE, FAKE, FAKE + 4) == moe.MOE_ERR_INVALID_ARG  # db
    lib = moe.load_library()
    assert lib.moe_grouped_matmul(None, FAKE, FAKE, FAKE, None, FAKE, None, None) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_grouped_matmul(matmul(rows_cap=0), None, None, None, None, None) == moe.MOE_OK
    assert moe.moe_last_launch_count() == 0


def test_matmul_result_in_place_of_an_input():
    OTHER, THIRD, FOURTH = FAKE + 4096, FAKE + 8192, FAKE + 12288
    for bias, y in ((None, OTHER), (None, THIRD), (FOURTH, FOURTH)):
        assert moe.moe_grouped_matmul(matmul(), FAKE, OTHER, THIRD, bias, y) == moe.MOE_ERR_INVALID_ARG
    for dW, db in ((OTHER, None), (THIRD, None), (FOURTH, OTHER), (FOURTH, THIRD), (FOURTH, FOURTH)):
        assert moe.moe_grouped_wgrad(matmul(), FAKE, OTHER, THIRD, dW, db) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_q4_matmul(q4(), FAKE, OTHER, THIRD, None, OTHER, FOURTH, WS) == moe.MOE_ERR_INVALID_ARG


def test_matmul_of_too_many_inputs():
    for dtype in (0, 1):
        m = matmul(K=(1 << 30) + 8, ldx=(1 << 30) + 8, dtype=dtype, out_dtype=dtype)
        assert moe.moe_grouped_matmul(m, FAKE, FAKE, FAKE, None, FAKE) == moe.MOE_ERR_UNSUPPORTED


def test_matmul_struct_layout():
    assert ctypes.sizeof(moe.Matmul) == 56 and moe.Matmul.ldx.offset == 40 and moe.Matmul.K.offset == 16


BF = torch.bfloat16


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("call,message", [
    (lambda: moe.grouped_matmul(z(4, 64, dtype=torch.float16), z(2, 64, 8), z(3, dtype=torch.int32)), "float32 or bfloat16"),
    (lambda: moe.grouped_matmul(z(4, 64), z(2, 64, 8, dtype=torch.float32), z(3, dtype=torch.int32)), "W must be"),
    (lambda: moe.grouped_matmul(z(4, 64), z(3, 64, 8), z(3, dtype=torch.int32)), "W must have shape"),
    (lambda: moe.grouped_matmul(z(4, 64), z(2, 64, 8), z(3, dtype=torch.int64)), "offsets"),
    (lambda: moe.grouped_matmul(z(4, 64), z(2, 64, 8), z(6, dtype=torch.int32)[::2]), "offsets"),
    (lambda: moe.grouped_matmul(z(64, 4).T, z(2, 64, 8), z(3, dtype=torch.int32)), "contiguous"),
    (lambda: moe.grouped_matmul(z(1, 64).expand(4, 64), z(2, 64, 8), z(3, dtype=torch.int32)), "overlap"),
    (lambda: moe.grouped_matmul(z(4, 64), z(2, 64, 8), z(3, dtype=torch.int32), bias=z(2, 16)), "bias must have shape"),
    (lambda: moe.grouped_matmul(z(4, 64), z(2, 64, 8), z(3, dtype=torch.int32), out=z(4, 16)), "out must have shape"),
    (lambda: moe.grouped_matmul(z(4, 64), z(2, 64, 8), z(3, dtype=torch.int32), out=z(4, 8), out_dtype=torch.float32),
     "another type"),
    (lambda: moe.grouped_matmul(z(4, 64), z(2, 64, 8), z(3, dtype=torch.int32)), "needs CUDA tensors"),
    (lambda: moe.grouped_wgrad(z(4, 64), z(5, 8), z(3, dtype=torch.int32)), "same number of rows"),
    (lambda: moe.grouped_wgrad(z(4, 64), z(4, 8, dtype=torch.float32), z(3, dtype=torch.int32)), "dy must be"),
    (lambda: moe.grouped_wgrad(z(4, 64), z(4, 8), z(3, dtype=torch.int32), dW=z(2, 64, 8)), "dW must be"),
    (lambda: moe.grouped_wgrad(z(4, 64), z(4, 8), z(3, dtype=torch.int32)), "needs CUDA tensors"),
])
def test_tensor_checks(call, message):
    with pytest.raises(ValueError, match=message):
        call()


# ---------------------------------------------------------------- activation with dropout
def act(**kw):
    d = dict(rows_cap=10, rows=None, F=64, dtype=1, activation=0, p=0.5, rng=FAKE, ld_in=0, ld_y=0, ld_grad=0)
    d.update(kw)
    return moe.Act(**d)


@pytest.mark.parametrize("bad,code", [
    (dict(rows_cap=-1), moe.MOE_ERR_INVALID_ARG), (dict(F=0), moe.MOE_ERR_INVALID_ARG), (dict(dtype=2), moe.MOE_ERR_INVALID_ARG),
    (dict(activation=2), moe.MOE_ERR_INVALID_ARG), (dict(activation=-2), moe.MOE_ERR_INVALID_ARG),
    (dict(p=-0.1), moe.MOE_ERR_INVALID_ARG), (dict(p=1.5), moe.MOE_ERR_INVALID_ARG), (dict(p=float("nan")), moe.MOE_ERR_INVALID_ARG),
    (dict(rng=None), moe.MOE_ERR_INVALID_ARG), (dict(rng=FAKE + 4), moe.MOE_ERR_INVALID_ARG), (dict(rows=FAKE + 2), moe.MOE_ERR_INVALID_ARG),
    (dict(ld_in=63), moe.MOE_ERR_INVALID_ARG), (dict(ld_y=8), moe.MOE_ERR_INVALID_ARG), (dict(ld_grad=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(rows_cap=1 << 32), moe.MOE_ERR_UNSUPPORTED), (dict(F=(1 << 30) + 1), moe.MOE_ERR_UNSUPPORTED),
])
def test_act_sizes(bad, code):
    m = act(**bad)
    assert moe.moe_act_dropout(m, FAKE, None, FAKE) == code
    assert moe.moe_act_dropout_backward(m, FAKE, FAKE, None, FAKE) == code
    assert moe.moe_last_launch_count() == 0


def test_act_pointers():
    assert moe.moe_act_dropout(act(), None, None, FAKE) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_act_dropout(act(), FAKE, None, None) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_act_dropout(act(), FAKE + 1, None, FAKE) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_act_dropout(act(dtype=0), FAKE, FAKE + 2, FAKE) == moe.MOE_ERR_INVALID_ARG
    for args in ((None, FAKE, None, FAKE, None), (FAKE, FAKE, FAKE, FAKE, None), (FAKE, FAKE, None, FAKE, FAKE)):
        assert moe.moe_act_dropout_backward(act(), *args) == moe.MOE_ERR_INVALID_ARG
    assert moe.load_library().moe_act_dropout(None, FAKE, None, FAKE, None) == moe.MOE_ERR_INVALID_ARG
    other = FAKE + (1 << 20)
    assert moe.moe_act_dropout(act(ld_y=72), FAKE, None, FAKE) == moe.MOE_ERR_INVALID_ARG  # in place at another pitch
    assert moe.moe_act_dropout(act(ld_y=72), FAKE, other, other) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_act_dropout_backward(act(ld_grad=72), FAKE, other, None, FAKE) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_act_dropout_backward(act(ld_grad=72), FAKE, FAKE, other, 2 * other, other) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_act_dropout_backward(act(), FAKE, FAKE, FAKE, other, other) == moe.MOE_ERR_INVALID_ARG  # du = dgate
    assert moe.moe_act_dropout(act(rows_cap=0), None, None, None) == moe.MOE_OK
    assert ctypes.sizeof(moe.Act) == 72 and moe.Act.p.offset == 32


def test_philox_known_answers():
    """The published known-answer vectors of Philox4x32-10, for the generator that the GPU tests compare with."""
    from philox import philox

    for ctr, key, want in (
            ([0] * 4, [0] * 2, "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
            ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
            ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
             "d16cfe09 94fdcceb 5001e420 24126ea1")):
        assert " ".join(f"{int(v):08x}" for v in philox(ctr, key)) == want


@pytest.mark.parametrize("call,message", [
    (lambda: moe.act_dropout(z(4, 8), activation="relu"), "unknown activation"),
    (lambda: moe.act_dropout(z(4, 8), gate=z(4, 9)), "gate must have shape"),
    (lambda: moe.act_dropout(z(4, 8), gate=z(4, 8, dtype=torch.float32)), "gate must be"),
    (lambda: moe.act_dropout(z(4, 8), gate=z(4, 16)[:, :8]), "rows of gate"),
    (lambda: moe.act_dropout(z(4, 8), rng=z(2)), "rng"),
    (lambda: moe.act_dropout(z(4, 8), rows=z(2, dtype=torch.int32)), "rows must be"),
    (lambda: moe.act_dropout(z(4, 8), out=z(4, 9)), "out must have shape"),
    (lambda: moe.act_dropout_backward(z(4, 9), z(4, 8)), "dy must have shape"),
    (lambda: moe.act_dropout_backward(z(4, 8), z(4, 8), dgate=z(4, 8)), "dgate without"),
    (lambda: moe.act_dropout_backward(z(4, 8), z(4, 8), gate=z(4, 8), du=z(4, 8), dgate=z(4, 16)[:, :8]), "rows of dgate"),
    (lambda: moe.act_dropout(z(4, 8)), "needs CUDA tensors"),
])
def test_act_tensor_checks(call, message):
    with pytest.raises(ValueError, match=message):
        call()


# ---------------------------------------------------------------- 4-bit weights
WS = 1 << 30


def q4(**kw):
    d = dict(E=4, rows_cap=10, K=128, N=100, group=64, dtype=1, out_dtype=1, activation=-1, ldx=0, ldy=0)
    d.update(kw)
    return moe.Q4(**d)


@pytest.mark.parametrize("bad,code", [
    (dict(E=0), moe.MOE_ERR_INVALID_ARG), (dict(E=257), moe.MOE_ERR_INVALID_ARG), (dict(rows_cap=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(K=0), moe.MOE_ERR_INVALID_ARG), (dict(N=0), moe.MOE_ERR_INVALID_ARG), (dict(group=16), moe.MOE_ERR_INVALID_ARG),
    (dict(group=0), moe.MOE_ERR_INVALID_ARG), (dict(dtype=2), moe.MOE_ERR_INVALID_ARG), (dict(out_dtype=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(activation=2), moe.MOE_ERR_INVALID_ARG), (dict(activation=-2), moe.MOE_ERR_INVALID_ARG),
    (dict(ldx=120), moe.MOE_ERR_INVALID_ARG), (dict(ldy=99), moe.MOE_ERR_INVALID_ARG), (dict(K=96), moe.MOE_ERR_UNSUPPORTED),
    (dict(K=1 << 25), moe.MOE_ERR_UNSUPPORTED), (dict(N=(1 << 24) + 1), moe.MOE_ERR_UNSUPPORTED), (dict(ldx=132), moe.MOE_ERR_UNSUPPORTED),
    (dict(dtype=0, out_dtype=0, ldx=130), moe.MOE_ERR_UNSUPPORTED), (dict(dtype=0), moe.MOE_ERR_UNSUPPORTED),
    (dict(rows_cap=(1 << 31) - 1024), moe.MOE_ERR_UNSUPPORTED), (dict(ldy=1 << 31), moe.MOE_ERR_UNSUPPORTED),
    (dict(K=1 << 24, N=1 << 24), moe.MOE_ERR_UNSUPPORTED), (dict(rows_cap=1 << 30, N=2048), moe.MOE_ERR_UNSUPPORTED),
    (dict(rows_cap=1 << 24, K=1 << 20, N=1024), moe.MOE_ERR_UNSUPPORTED),
])
def test_q4_sizes(bad, code):
    assert moe.moe_q4_matmul(q4(**bad), FAKE, FAKE, FAKE, None, FAKE, FAKE, WS) == code
    assert moe.moe_last_launch_count() == 0


def test_q4_pointers_and_workspace():
    ok = [FAKE, FAKE, FAKE, None, FAKE, FAKE]
    for i in (0, 1, 2, 4, 5):  # offsets, x, packed, y, ws
        for p in (None, FAKE + 1):
            args = list(ok)
            args[i] = p
            assert moe.moe_q4_matmul(q4(), *args, WS) == moe.MOE_ERR_INVALID_ARG, (i, p)
    assert moe.moe_q4_matmul(q4(), FAKE, FAKE + 8, FAKE, None, FAKE, FAKE, WS) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_q4_matmul(q4(), FAKE, FAKE, FAKE, FAKE + 1, FAKE, FAKE, WS) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_q4_matmul(q4(), *ok[:5], FAKE + 128, WS) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_q4_matmul(q4(), *ok, moe.moe_q4_workspace_size() - 1) == moe.MOE_ERR_WORKSPACE
    assert moe.moe_q4_matmul(q4(rows_cap=0), None, None, None, None, None, FAKE, WS) == moe.MOE_OK
    assert moe.load_library().moe_q4_matmul(None, *ok, WS, None) == moe.MOE_ERR_INVALID_ARG
    assert ctypes.sizeof(moe.Q4) == 56 and moe.Q4.ldx.offset == 40


def test_q4_layout_calls():
    assert moe.moe_q4_packed_size(2, 128, 16, 64) == 2 * 2 * (1024 + 64)  # 32 columns a block
    assert moe.moe_q4_packed_size(1, 160, 33, 32) == 2 * 2 * 2 * (1024 + 128)  # two steps of 128, two blocks of 32
    for E, K, N, group, code in ((0, 128, 8, 64, 1), (1, 128, 8, 48, 1), (1, 0, 8, 64, 1), (1, 128, 0, 64, 1), (1, 96, 8, 64, 2)):
        assert moe.moe_q4_packed_size(E, K, N, group) == 0
        assert moe.moe_q4_pack(E, K, N, group, FAKE, FAKE, FAKE) == code
        assert moe.moe_q4_quantize(E, K, N, group, 1, FAKE, FAKE, FAKE) == code
        assert moe.moe_q4_dequantize(E, K, N, group, FAKE, 1, FAKE) == code
    for bad in (None, FAKE + 1):
        for i in range(3):
            args = [FAKE] * 3
            args[i] = bad
            assert moe.moe_q4_pack(1, 128, 8, 64, *args) == moe.MOE_ERR_INVALID_ARG
            assert moe.moe_q4_quantize(1, 128, 8, 64, 1, *args) == moe.MOE_ERR_INVALID_ARG
        assert moe.moe_q4_dequantize(1, 128, 8, 64, bad, 1, FAKE) == moe.MOE_ERR_INVALID_ARG
        assert moe.moe_q4_dequantize(1, 128, 8, 64, FAKE, 1, bad) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_q4_quantize(1, 128, 8, 64, 2, FAKE, FAKE, FAKE) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_q4_dequantize(1, 128, 8, 64, FAKE, 7, FAKE) == moe.MOE_ERR_INVALID_ARG


def test_q4_layer_checks():
    shape = moe.make_shape(16, 128, 4, 2, 192, dtype="bf16")
    io = moe.IO(*([FAKE] * 14))

    def call(shape=shape, io=io, group=64, W1=FAKE, W2=FAKE, ws=FAKE, bytes=WS, combine=1):
        return moe.moe_expert_ffn_q4(shape, io, group, W1, W2, ws, bytes, combine)

    assert call(group=128) == moe.MOE_ERR_UNSUPPORTED  # does not divide F
    assert call(group=48) == moe.MOE_ERR_INVALID_ARG
    assert call(bytes=100) == moe.MOE_ERR_WORKSPACE
    for bad in (dict(W1=None), dict(W2=None), dict(W1=FAKE + 8), dict(ws=None), dict(ws=FAKE + 64)):
        assert call(**bad) == moe.MOE_ERR_INVALID_ARG, bad
    no_out = moe.IO(*([FAKE] * 14))
    no_out.out = None
    assert call(io=no_out) == moe.MOE_ERR_INVALID_ARG
    assert call(shape=moe.make_shape(0, 128, 4, 2, 192, dtype="bf16")) == moe.MOE_OK
    assert moe.moe_last_launch_count() == 0


def q4_weights(E=2, K=128, N=8, group=64):
    w = object.__new__(moe.Q4Weights)
    w.E, w.K, w.N, w.group, w.packed = E, K, N, group, torch.zeros(moe.moe_q4_packed_size(E, K, N, group), dtype=torch.uint8)
    return w


U8, I32 = torch.uint8, torch.int32


@pytest.mark.parametrize("call,message", [
    (lambda: moe.q4_quantize(z(128, 8)), "three dimensions"),
    (lambda: moe.q4_quantize(z(1, 128, 8, dtype=torch.float16)), "float32 or bfloat16"),
    (lambda: moe.q4_quantize(z(1, 128, 8), 48), "group"),
    (lambda: moe.q4_quantize(z(1, 96, 8), 64), "group"),
    (lambda: moe.q4_quantize(z(1, 8, 128).mT, 64), "contiguous"),
    (lambda: moe.q4_quantize(z(1, 128, 8), 64), "needs CUDA tensors"),
    (lambda: moe.Q4Weights(z(1, 8, 64), z(1, 2, 8)), "codes must be"),
    (lambda: moe.Q4Weights(z(1, 8, 64, dtype=U8), z(1, 3, 8)), "scales must be"),
    (lambda: moe.Q4Weights(z(1, 8, 64, dtype=U8), z(1, 2, 9)), "scales must have shape"),
    (lambda: moe.Q4Weights(z(1, 8, 64, dtype=U8), z(1, 2, 8, dtype=torch.float32)), "scales must be torch.bfloat16"),
    (lambda: moe.Q4Weights(z(1, 8, 64, dtype=U8), z(1, 2, 8)), "needs CUDA tensors"),
    (lambda: moe.q4_matmul(z(4, 128), q4_weights(), z(4, dtype=I32)), "experts"),
    (lambda: moe.q4_matmul(z(4, 64), q4_weights(), z(3, dtype=I32)), "128 columns"),
    (lambda: moe.q4_matmul(z(4, 128), q4_weights(), z(3, dtype=I32), bias=z(2, 9)), "bias must have shape"),
    (lambda: moe.q4_matmul(z(4, 128), q4_weights(), z(3, dtype=I32), activation="relu"), "unknown activation"),
    (lambda: moe.q4_matmul(z(4, 128), q4_weights(), z(3, dtype=I32), out=z(4, 9), ws=z(1)), "out must have shape"),
    (lambda: moe.q4_matmul(z(4, 128), q4_weights(), z(3, dtype=I32), out=z(4, 8), out_dtype=torch.float32, ws=z(1)), "another type"),
    (lambda: moe.q4_matmul(z(4, 128), q4_weights(), z(3, dtype=I32), ws=z(1)), "needs CUDA tensors"),
])
def test_q4_tensor_checks(call, message):
    with pytest.raises(ValueError, match=message):
        call()


def leaf(*shape):
    return z(*shape).requires_grad_()


OFF3 = z(3, dtype=I32)
GRAPH = {
    "x": lambda: moe.grouped_matmul(leaf(4, 64), z(2, 64, 8), OFF3),
    "W": lambda: moe.grouped_matmul(z(4, 64), leaf(2, 64, 8), OFF3),
    "bias": lambda: moe.grouped_matmul(z(4, 64), z(2, 64, 8), OFF3, bias=leaf(2, 8)),
    "out": lambda: moe.grouped_matmul(z(4, 64), z(2, 64, 8), OFF3, out=leaf(4, 8)),
    "dy": lambda: moe.grouped_wgrad(z(4, 64), leaf(4, 8), OFF3),
    "dW": lambda: moe.grouped_wgrad(z(4, 64), z(4, 8), OFF3, dW=z(2, 64, 8, dtype=torch.float32).requires_grad_()),
    "u": lambda: moe.act_dropout(leaf(4, 8)),
    "gate": lambda: moe.act_dropout(z(4, 8), gate=leaf(4, 8)),
    "du": lambda: moe.act_dropout_backward(z(4, 8), z(4, 8), du=leaf(4, 8)),
    "x of q4": lambda: moe.q4_matmul(leaf(4, 128), q4_weights(), OFF3, ws=z(1)),
    "bias of q4": lambda: moe.q4_matmul(z(4, 128), q4_weights(), OFF3, bias=leaf(2, 8), ws=z(1)),
}


@pytest.mark.parametrize("name", GRAPH)
def test_tensors_that_require_a_gradient_are_refused(name):
    """The operators record no graph: a gradient would be lost silently.  Without grad mode the call goes on."""
    with pytest.raises(ValueError, match=f"^{name.split()[0]} requires a gradient"):
        GRAPH[name]()
    for off in (torch.no_grad(), torch.inference_mode()):
        with off, pytest.raises(ValueError, match="needs CUDA tensors"):
            GRAPH[name]()


def test_matmul_form_query():
    """The dispatch rule of the bf16 product, for 148 SMs where there is no GPU to ask."""
    assert moe.moe_debug_matmul_form(matmul(E=0))[0] == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_debug_matmul_form(matmul(K=60))[0] == moe.MOE_ERR_UNSUPPORTED
    assert moe.moe_debug_matmul_form(matmul(dtype=0, out_dtype=0))[0] == moe.MOE_ERR_UNSUPPORTED
    assert moe.moe_debug_matmul_form(matmul(rows_cap=0))[0] == moe.MOE_ERR_UNSUPPORTED
    assert moe.load_library().moe_debug_matmul_form(ctypes.byref(matmul()), None) == moe.MOE_ERR_INVALID_ARG
    status, form = moe.moe_debug_matmul_form(matmul(E=8, rows_cap=8192, K=4096, N=14336))
    assert status == moe.MOE_OK and form == (1, 256, 0, 1)
    try:
        moe.moe_set_kernel_options(moe.MOE_KERNEL_NO_CTA_PAIR)
        assert moe.moe_debug_matmul_form(matmul(E=8, rows_cap=8192, K=4096, N=14336)) == (moe.MOE_OK, (0, 256, 0, 1))
    finally:
        moe.moe_set_kernel_options(moe.MOE_KERNEL_DEFAULT)
    assert moe.moe_debug_matmul_form(matmul(E=8, rows_cap=64, K=4096, N=14336))[1] == (0, 256, 16, 1)
    assert moe.moe_debug_matmul_form(matmul(E=128, rows_cap=8104, K=1024, N=4096))[1] == (0, 256, 8, 1)
    assert moe.moe_last_launch_count() == 0
