"""The operators on buffers of more than 2^31 elements: the rows and weights behind that border, against fp64."""
import pytest
import torch

import sparse_mixture_experts_23_b200 as moe
from oplib import SUM_STEP, offsets_of, round_bound, within
from philox import philox

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ROWS, WIDE = 262144 + 9000, 8192  # 2^31 elements end at row 262144


def filled(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0, std, generator=g)


def check_rows(y, x, W, r, what):
    ref, mag = x[r].double() @ W.double(), x[r].double().abs() @ W.double().abs()
    bound = (x.shape[1] + 2) * SUM_STEP * mag
    within(y[r], ref, bound + round_bound(ref.abs() + bound, y.dtype), what)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_past_the_border(dtype):
    off, last = offsets_of([ROWS - 1000, 1000]), slice(ROWS - 1000, ROWS)
    near = ((0, slice(262144 - 40, 262144 + 40)), (1, last))
    x, W = filled((ROWS, 64), dtype, 1), filled((2, 64, WIDE), dtype, 2, 0.125)
    y = moe.grouped_matmul(x, W, off)
    for e, r in near:
        check_rows(y, x, W[e], r, "result")
    dW, db = moe.grouped_wgrad(x, y, off, bias_grad=True)
    a, d = x[last].double(), y[last].double()
    within(dW[1], a.T @ d, 1002 * SUM_STEP * (a.abs().T @ d.abs()), "dW")
    within(db[1], d.sum(0), 1002 * SUM_STEP * d.abs().sum(0), "db")
    W2 = filled((2, WIDE, 64), dtype, 3, 0.01)
    z = moe.grouped_matmul(y, W2, off)
    for e, r in near:
        check_rows(z, y, W2[e], r, "from wide rows")
    p, seed, offset = 0.25, 5, 6
    kw = dict(activation=None, p=p, rng=torch.tensor([seed, offset], device="cuda"))
    kept = moe.act_dropout(y, **kw)
    back = moe.act_dropout_backward(y, y, **kw)
    r = ROWS - 1
    words = torch.tensor([int(w) for b in range(16) for w in philox((b, r, offset, 0), (seed, 0))], device="cuda")
    want = torch.where(words >= 2 ** 30, y[r, :64].float() / (1 - p), 0).to(dtype)
    for got in (kept, back):  # the scale 1 / (1 - p) in fp32 and its product: two halves of a step
        within(got[r, :64], want.double(), want.double().abs() * 2.0 ** -22 + round_bound(want.double(), dtype))


def test_weights_past_the_border():
    E, K, N, n = 40, WIDE, WIDE, 200
    counts = [5] + [0] * (E - 2) + [n]
    W, off, last = filled((E, K, N), BF, 4, K ** -0.5), offsets_of(counts), slice(5, 5 + n)
    x = filled((5 + n, K), BF, 5)
    for trans in (False, True):
        y = moe.grouped_matmul(x, W, off, transpose_w=trans)
        check_rows(y, x, W[-1].T if trans else W[-1], last, "many weights")
    dW = moe.grouped_wgrad(x, y, off)
    a, d = x[last].double(), y[last].double()
    within(dW[-1], a.T @ d, (n + 2) * SUM_STEP * (a.abs().T @ d.abs()), "dW")
    assert not dW[1].any() and not dW[-2].any()


def test_packed_weights_past_the_border():
    E, K, N, group = 70, WIDE, WIDE, 64
    q = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda")
    s = (torch.rand((E, K // group, N), device="cuda") + 0.5).to(BF)
    counts = [3] + [0] * (E - 2) + [20]
    x = filled((23, K), BF, 6)
    y = moe.q4_matmul(x, moe.Q4Weights(q, s), offsets_of(counts), out_dtype=F32)
    codes = torch.stack([q[-1] & 15, q[-1] >> 4], -1).flatten(1).double() - 8
    w = codes.T * s[-1].double().repeat_interleave(group, 0)
    within(y[3:], x[3:].double() @ w, (K + 162) * SUM_STEP * (x[3:].double().abs() @ w.abs()))
