"""moe_grouped_matmul and moe_grouped_wgrad against products in fp64, expert by expert.

The bounds are those of oplib: (n + 2) 2^-23 of the summed magnitudes, and the output type's rounding."""
import pytest
import torch

import sparse_mixture_experts_23_b200 as moe
from oplib import SUM_STEP, offsets_of, randn, round_bound, segments, strided, within

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def reference(x, W, counts, bias, trans):
    ref = torch.zeros((x.shape[0], W.shape[1] if trans else W.shape[2]), dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(ref)
    for e, r in segments(counts):
        w = W[e].double().T if trans else W[e].double()
        ref[r] = x[r].double() @ w
        mag[r] = x[r].double().abs() @ w.abs()
        if bias is not None:
            ref[r] += bias[e].double()
            mag[r] += bias[e].double().abs()
    return ref, mag


def check_forward(counts, K, N, dtype, out_dtype, trans, bias, pad=0, spare=0, seed=0):
    E, n = len(counts), sum(counts)
    x = randn((n + spare, K), dtype, seed)
    if spare:
        x[n:] = float("nan")  # rows behind the last segment must not reach any result
    W = randn((E, N, K) if trans else (E, K, N), dtype, seed + 1, K ** -0.5)
    b = randn((E, N), dtype, seed + 2) if bias else None
    ref, mag = reference(x, W, counts, b, trans)
    step = 8 if dtype == BF else 4
    xs = strided(x, step * pad)[0] if pad else x
    out, buf = strided(torch.full((n + spare, N), 7.0, dtype=out_dtype, device="cuda"), step * pad, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = moe.grouped_matmul(xs, W, offsets_of(counts), bias=b, transpose_w=trans, out=out, status=status)
    assert moe.moe_get_device_status(status.data_ptr()) == moe.MOE_OK
    assert y.data_ptr() == out.data_ptr()
    bound = (K + 2) * SUM_STEP * mag
    within(y[:n], ref[:n], bound[:n] + round_bound(ref[:n].abs() + bound[:n], out_dtype), f"{counts} {K} {N}")
    assert (buf[n:] == 7.0).all() and (buf[:, N:] == 7.0).all(), "wrote outside its rows or columns"


# short segments (16-row boxes), spread segments, full tiles, pair tiles; widths that end inside every tile
ROWS = [
    [1], [0, 1, 0], [5, 0, 31, 16, 17], [33, 64, 0, 100, 127], [128, 129, 130], [300, 1, 255, 0],
    [256, 257, 258], [1, 0, 900, 128], [511, 513],
]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts", ROWS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("K,N", [(64, 256), (8, 8), (72, 72), (200, 328), (136, 520)])
def test_bf16(counts, K, N, trans):
    check_forward(counts, K, N, BF, BF, trans, bias=N != 72)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts", ROWS, ids=lambda c: "-".join(map(str, c)))
def test_bf16_to_fp32(counts, trans):
    check_forward(counts, 136, 296, BF, F32, trans, bias=True, seed=3)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts", [[1], [0, 3, 64, 65, 0, 130], [63, 1, 300]], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("K,N", [(4, 4), (16, 128), (20, 132), (100, 260), (516, 68)])
def test_fp32(counts, K, N, trans):
    check_forward(counts, K, N, F32, F32, trans, bias=K != 16)


@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("counts", [[3, 0, 9], [40, 90], [700, 0, 400]], ids=lambda c: "-".join(map(str, c)))
def test_strides_and_spare_rows(counts, dtype, out):
    """Rows at a pitch, rows behind the last segment (NaN in x, untouched in y), columns past N untouched."""
    for trans in (False, True):
        check_forward(counts, 72, 200, dtype, out, trans, bias=True, pad=3, spare=70, seed=11)


def test_long_contraction_and_many_experts():
    check_forward([64] * 5, 14336, 264, BF, BF, False, True)
    check_forward([2] * 100 + [0] * 100 + [3] * 56, 64, 64, BF, BF, False, True)
    check_forward([1] + [0] * 254 + [1], 64, 64, BF, F32, True, True)
    check_forward([300] + [0] * 254 + [1], 64, 64, F32, F32, False, True)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinities_stay_in_their_rows(dtype):
    """A row that holds inf or NaN gives what its own sum gives; the rows beside it are unchanged."""
    counts = [5, 130]
    x = randn((135, 64), dtype, 1)
    W = randn((2, 64, 128), dtype, 2)
    off = offsets_of(counts)
    clean = moe.grouped_matmul(x, W, off)
    x[2, 3], x[70, 1], x[71, 0] = float("inf"), float("nan"), float("-inf")
    y = moe.grouped_matmul(x, W, off)
    rows = [2, 70, 71]
    keep = [r for r in range(135) if r not in rows]
    assert torch.equal(y[keep], clean[keep])
    assert torch.equal(y[2], torch.sign(W[0, 3]) * float("inf")) and y[70].isnan().all()
    assert torch.equal(y[71], torch.sign(W[1, 0]) * float("-inf"))


def check_wgrad(counts, K, N, dtype, bias, pad=0, spare=0, seed=0):
    E, n = len(counts), sum(counts)
    x, dy = randn((n + spare, K), dtype, seed), randn((n + spare, N), dtype, seed + 1)
    if spare:
        x[n:], dy[n:] = float("nan"), float("inf")
    step = 8 if dtype == BF else 4
    xs, dys = (strided(x, step * pad)[0], strided(dy, 2 * step * pad)[0]) if pad else (x, dy)
    dW = torch.full((E, K, N), float("nan"), device="cuda")
    db = torch.full((E, N), float("nan"), device="cuda") if bias else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = moe.grouped_wgrad(xs, dys, offsets_of(counts), dW=dW, db=db, status=status)
    assert moe.moe_get_device_status(status.data_ptr()) == moe.MOE_OK
    assert (got[0] if bias else got).data_ptr() == dW.data_ptr()
    for e, r in segments(counts):
        a, d, c = x[r].double(), dy[r].double(), counts[e]
        within(dW[e], a.T @ d, (c + 2) * SUM_STEP * (a.abs().T @ d.abs()), f"dW[{e}] {counts} {K} {N}")
        if bias:
            within(db[e], d.sum(0), (c + 2) * SUM_STEP * d.abs().sum(0), f"db[{e}] {counts}")
    again = moe.grouped_wgrad(xs, dys, offsets_of(counts), bias_grad=bias)
    assert torch.equal(again[0] if bias else again, dW) and (not bias or torch.equal(again[1], db))


@pytest.mark.parametrize("counts", [[1], [0, 1, 0], [5, 0, 16, 17], [127, 128, 129], [300, 0, 1], [1000]],
                         ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("K,N", [(64, 256), (8, 8), (72, 40), (264, 328)])
def test_wgrad_bf16(counts, K, N):
    check_wgrad(counts, K, N, BF, bias=True)


@pytest.mark.parametrize("counts", [[1], [0, 15, 16, 17, 0, 130]], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("K,N", [(4, 4), (64, 128), (68, 132), (100, 36)])
def test_wgrad_fp32(counts, K, N):
    check_wgrad(counts, K, N, F32, bias=True)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_wgrad_strides_and_spare_rows(dtype):
    check_wgrad([40, 0, 99], 72, 200, dtype, bias=True, pad=2, spare=130)
    check_wgrad([40, 0, 99], 72, 200, dtype, bias=False, spare=1)


def test_wgrad_without_rows_is_zero():
    for rows in (0, 8):  # an empty batch, and one whose rows belong to nobody
        x, dy = torch.ones((rows, 64), device="cuda", dtype=BF), torch.ones((rows, 32), device="cuda", dtype=BF)
        dW, db = moe.grouped_wgrad(x, dy, offsets_of([0, 0]), bias_grad=True)
        assert dW.shape == (2, 64, 32) and not dW.any() and not db.any()
    assert moe.grouped_matmul(torch.ones((0, 64), device="cuda", dtype=BF),
                              torch.ones((2, 64, 32), device="cuda", dtype=BF), offsets_of([0, 0])).shape == (0, 32)


def test_single_cta_kernels_agree():
    """The kernels without CTA pairs, on the shapes that would use pairs."""
    try:
        moe.moe_set_kernel_options(moe.MOE_KERNEL_NO_CTA_PAIR)
        check_forward([300, 0, 513], 136, 520, BF, BF, False, True, pad=1, spare=3)
        check_forward([300, 0, 513], 136, 520, BF, F32, True, True, pad=1, spare=3)
        check_wgrad([300, 0, 513], 136, 40, BF, True, pad=1, spare=3)
    finally:
        moe.moe_set_kernel_options(0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", [[0, 5, 3, 9], [1, 5, 7, 9], [0, 5, 7, 1000], [-4, 5, 7, 9], [0, -1, 7, 9]])
def test_bad_offsets_are_clamped_and_reported(dtype, bad):
    x, W = randn((9, 64), dtype, 1), randn((3, 64, 64), dtype, 2)
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.grouped_matmul(x, W, off, status=status)
    assert moe.moe_get_device_status(status.data_ptr()) == moe.MOE_ERR_INVALID_ARG
    moe.grouped_wgrad(x, x, off, status=status)
    assert moe.moe_get_device_status(status.data_ptr()) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_get_device_status(status.data_ptr()) == moe.MOE_OK


def test_graph_replay_and_side_stream():
    """Captured once, replayed on new inputs and new offsets; two calls at once on two streams."""
    counts, other = [30, 0, 70], [1, 98, 1]
    x, W = randn((100, 64), BF, 1), randn((3, 64, 128), BF, 2)
    off = offsets_of(counts)
    y, dW = torch.empty((100, 128), dtype=BF, device="cuda"), torch.empty((3, 64, 128), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        moe.grouped_matmul(x, W, off, out=y)
        moe.grouped_wgrad(x, y, off, dW=dW)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.grouped_matmul(x, W, off, out=y)
        moe.grouped_wgrad(x, y, off, dW=dW)
    x.copy_(randn((100, 64), BF, 5))
    off.copy_(offsets_of(other))
    g.replay()
    torch.cuda.synchronize()
    y2 = moe.grouped_matmul(x, W, off)
    assert torch.equal(y, y2) and torch.equal(dW, moe.grouped_wgrad(x, y2, off))
    ref, mag = reference(x, W, other, None, False)
    bound = 66 * SUM_STEP * mag
    within(y, ref, bound + round_bound(ref.abs() + bound, BF))


# fp32: a few rows an expert (more inputs than fit shared memory at once), 64-wide tiles with 8, 4 and 2 groups of threads
# a tile, 128-wide tiles
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts,K,N", [([2, 0, 9, 1], 2052, 132), ([1], 1028, 4), ([8, 8], 1024, 260), ([0, 40, 3], 260, 68),
                                        ([300, 0, 200], 68, 2100), ([300, 0, 200], 36, 4100), ([2000, 1900], 20, 2000)],
                         ids=lambda v: "-".join(map(str, v)) if isinstance(v, list) else str(v))
def test_fp32_forms(counts, K, N, trans):
    check_forward(counts, K, N, F32, F32, trans, bias=K != 1028, pad=1, spare=9)


@pytest.mark.parametrize("counts,K,N", [([3, 2], 132, 68), ([500, 200], 260, 300), ([90, 100, 0], 1000, 772), ([40] * 8, 516, 2052)],
                         ids=lambda v: "-".join(map(str, v[:3])) if isinstance(v, list) else str(v))
def test_wgrad_fp32_forms(counts, K, N):
    check_wgrad(counts, K, N, F32, bias=False)


# a tile's contraction shared by 2, 4 and 8 blocks, with shares that end early and tiles that end inside
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts,K,N", [([1], 1024, 4), ([3, 0, 6], 4100, 36), ([9], 2308, 300), ([5, 11], 1028, 1156), ([40], 516, 68),
                                        ([0, 70], 2052, 132), ([129], 1028, 700), ([33, 90], 8004, 60)],
                         ids=lambda v: "-".join(map(str, v)) if isinstance(v, list) else str(v))
def test_fp32_few_tiles_of_a_long_contraction(counts, K, N, trans):
    check_forward(counts, K, N, F32, F32, trans, bias=K != 1028, pad=1, spare=9)


@pytest.mark.parametrize("counts,K,N", [([513], 4, 4), ([2048], 68, 132), ([0, 3000], 64, 64), ([600, 1, 900], 132, 260)],
                         ids=lambda v: "-".join(map(str, v)) if isinstance(v, list) else str(v))
def test_wgrad_fp32_few_tiles_of_many_rows(counts, K, N):
    check_wgrad(counts, K, N, F32, bias=True, pad=1, spare=5)


@pytest.mark.parametrize("counts", [[769], [767, 768, 1], [1537, 0, 2305], [128, 3000]], ids=lambda c: "-".join(map(str, c)))
def test_wgrad_bf16_many_rows(counts):
    check_wgrad(counts, 264, 136, BF, bias=True, pad=1, spare=130)


def test_wgrad_of_many_rows_keeps_its_digits():
    """Positive terms, so that partial sums only grow: a sum of its own for every 768 rows is off by at most 48 steps of
    the tensor core, each cut at two steps of 2^-23 of the partial sum, and joining 11 of them by 11 more."""
    n = 8192
    x, dy = randn((n, 64), BF, 1).abs() + 0.5, randn((n, 256), BF, 2).abs() + 0.5
    dW = moe.grouped_wgrad(x, dy, offsets_of([n]))
    ref = x.double().T @ dy.double()
    within(dW[0], ref, (2 * 48 + 11) * SUM_STEP * ref)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_bias_gradient_of_long_segments(dtype):
    """Few strips and many rows: the rows of a strip shared by a cluster."""
    check_wgrad([1200, 0, 300], 8, 72, dtype, bias=True, pad=1, spare=7)
    check_wgrad([3000], 8, 520, dtype, bias=True)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts", [[1], [5, 0, 40], [128, 3], [300], [17, 100, 129]], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("K,N", [(512, 8), (520, 64), (1096, 72), (4104, 200), (2048, 520)])
def test_few_tiles_of_a_long_contraction(counts, K, N, trans):
    """K shared by the CTAs of a cluster, in 2, 4 or 8 parts."""
    check_forward(counts, K, N, BF, BF, trans, bias=N != 64, pad=1, spare=40)
    check_forward(counts, K, N, BF, F32, trans, bias=N != 72, spare=3, seed=4)


# every form of the bf16 product: K shared by a cluster, 64-wide tiles, 128 and 256 with spread rows, 256 with 16-row boxes,
# pair tiles (full and half)
LONG = [([64], 65544, 64), ([40] * 40, 6200, 128), ([40] * 128, 6200, 120), ([33, 64, 100, 127] * 10, 6200, 1000),
        ([8] * 8, 6200, 5000), ([1500, 300, 900], 6200, 3000)]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts,K,N", LONG, ids=lambda v: f"{len(v)}x{v[0]}" if isinstance(v, list) else str(v))
def test_long_sums_keep_their_digits(counts, K, N, trans):
    """Positive terms, so that partial sums only grow.  A tensor-core sum of 768 inputs is 48 steps, each cut at two steps of
    2^-23 of the partial sum at most; after i of them that is i / 48 of the part, within 15% (the terms' spread is 0.7 of
    their mean): 2 * 24.5 * 1.15 = 57.  Joining P sums rounds at half a step of the sum so far, (P + 1) / 4 (P = 9, or 11 and
    then 8 CTAs of a cluster: at most 20), the last rounding one more.  One sum over 6200 inputs loses about 160 steps, at either
    result type, and one over a CTA's 8200 more."""
    parts, E = 9 if K == 6200 else 20, len(counts)
    x = (randn((sum(counts), K), F32, 1).abs() + 0.5).to(BF)
    g = torch.Generator(device="cuda").manual_seed(2)
    W = (torch.randn((E, N, K) if trans else (E, K, N), generator=g, device="cuda").abs_() + 0.5).to(BF)
    off = offsets_of(counts)
    ref = torch.cat([x[r].double() @ (W[e].double().T if trans else W[e].double()) for e, r in segments(counts)])
    bound = (57 + (parts + 1) / 4 + 1) * SUM_STEP * ref
    within(moe.grouped_matmul(x, W, off, transpose_w=trans, out_dtype=F32), ref, bound, "fp32")
    within(moe.grouped_matmul(x, W, off, transpose_w=trans), ref, bound + round_bound(ref + bound, BF), "bf16")


@pytest.mark.parametrize("options", [moe.MOE_KERNEL_DEFAULT, moe.MOE_KERNEL_NO_CTA_PAIR])
def test_wgrad_of_very_many_rows_keeps_its_digits(options):
    """Positive terms as in test_long_sums_keep_their_digits: 57 steps of 2^-23 for the sums of 768 rows, (P + 1) / 4 for
    joining P = 86 of them, one for the last.  One sum over the 65541 rows loses more than a thousand."""
    n, parts = 65541, 86
    x, dy = (randn((n, 64), F32, 1).abs() + 0.5).to(BF), (randn((n, 264), F32, 2).abs() + 0.5).to(BF)
    ref = x.double().T @ dy.double()
    moe.moe_set_kernel_options(options)
    try:
        dW = moe.grouped_wgrad(x, dy, offsets_of([0, n, 0]))
    finally:
        moe.moe_set_kernel_options(moe.MOE_KERNEL_DEFAULT)
    assert not dW[0].any() and not dW[2].any()
    within(dW[1], ref, (57 + (parts + 1) / 4 + 1) * SUM_STEP * ref)


def test_wgrad_single_cta_kernel_of_many_rows():
    """Sums of 768 rows in the kernel without CTA pairs: none, one, an odd and an even number of them, tiles in sequence."""
    try:
        moe.moe_set_kernel_options(moe.MOE_KERNEL_NO_CTA_PAIR)
        check_wgrad([0, 1, 767, 769, 0, 1537, 2305, 768] * 4, 264, 520, BF, bias=False, pad=1, spare=3)
    finally:
        moe.moe_set_kernel_options(moe.MOE_KERNEL_DEFAULT)


# Shapes that reach every kernel of the bf16 product, as (CTA pairs, tile columns, box rows, CTAs that share K), with ragged N
# and K.  Those with whole K have more tiles than the GPU has SMs, most of them twice that, so that accumulators and stages
# are taken again.
FORMS = [
    ((1, 256, 0, 1), [1500, 300, 0, 900], 1288, 5000),
    ((0, 256, 16, 1), [9, 0, 1, 30, 16, 8, 17, 3] * 2, 200, 11000),
    ((0, 256, 8, 1), [33, 64, 0, 1, 100, 127, 128, 140] * 6, 840, 3000),
    ((0, 256, 0, 1), [200, 0, 129, 300] * 8, 136, 3000),
    ((0, 128, 16, 1), [40, 1, 0, 20, 3] * 50 + [4000], 72, 120),
    ((0, 128, 8, 1), [130, 129, 0, 200, 100] * 51, 72, 120),
    ((0, 128, 0, 1), [300, 0, 127, 128, 200] * 51, 72, 104),
    ((0, 64, 16, 1), [40, 1, 0, 20, 3] * 50 + [4000], 72, 56),
    ((0, 64, 8, 1), [130, 129, 0, 200, 100] * 51, 200, 64),
    ((0, 64, 0, 1), [300, 0, 127, 128, 200] * 51, 72, 8),
    ((0, 64, 0, 1), [40] * 40, 520, 120),  # fewer tiles than SMs
    ((0, 64, 0, 2), [64], 2056, 4040),
    ((0, 64, 0, 4), [64, 40], 4104, 904),
    ((0, 64, 0, 8), [100, 7], 7000, 200),
    ((0, 64, 16, 8), [10, 0, 3], 4104, 72),
]
FORM_IDS = ["pair" if f[0] else f"{f[1]}x{f[2]}x{f[3]}x{len(c)}" for f, c, _, _ in FORMS]


def form_of(rows, E, K, N, out_dtype, trans):
    m = moe.Matmul(E, rows, K, N, moe.MOE_DTYPE_BF16, int(out_dtype == BF), int(trans), K, N)
    status, form = moe.moe_debug_matmul_form(m)
    assert status == moe.MOE_OK
    return form


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("form,counts,K,N", FORMS, ids=FORM_IDS)
def test_every_bf16_kernel(form, counts, K, N, out_dtype, trans):
    """Against fp64, with a pitch, spare rows and a bias; the dispatch is asked, so that a later rule cannot drop one."""
    spare = 3
    assert form_of(sum(counts) + spare, len(counts), K, N, out_dtype, trans) == form
    check_forward(counts, K, N, BF, out_dtype, trans, bias=True, pad=1, spare=spare, seed=21)


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("trans", [False, True])
def test_single_cta_kernels_where_pairs_would_run(out_dtype, trans):
    counts, K, N = [1500, 300, 0, 900], 1288, 1400
    size = (sum(counts) + 3, len(counts), K, N, out_dtype, trans)
    assert form_of(*size)[0] == 1
    check_forward(counts, K, N, BF, out_dtype, trans, bias=True, pad=1, spare=3, seed=22)
    try:
        moe.moe_set_kernel_options(moe.MOE_KERNEL_NO_CTA_PAIR)
        assert form_of(*size)[0] == 0
        check_forward(counts, K, N, BF, out_dtype, trans, bias=True, pad=1, spare=3, seed=22)
    finally:
        moe.moe_set_kernel_options(moe.MOE_KERNEL_DEFAULT)


def test_wgrad_many_tiles_of_unlike_segments():
    """384 tiles for 74 pairs of CTAs: empty tiles, tiles of one sum and of an odd and an even number of them follow each
    other on a pair, whose two accumulators change hands at every sum."""
    base = [0, 1, 767, 769, 0, 0, 1537, 2305, 768, 5, 0, 130, 1536, 3, 0, 900]
    check_wgrad(base * 4, 264, 520, BF, bias=True, pad=1, spare=9)
    check_wgrad(base[::-1] + base, 1032, 264, BF, bias=False)
