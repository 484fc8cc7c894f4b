"""Products with 4-bit weights: quantise, pack, dequantise, moe_q4_matmul and the layer's FFN in 4 bits, against
fp64 products of the weights that the codes stand for.

Bounds.  The weights are exact (a code difference of 4 bits times a bf16 scale); a sum of K terms in fp32, cut or
rounded at each of its additions (three a term for fp32 rows, whose parts are summed apart), the joins of at most 16
warps' parts (162 allowed here) and the bias: (P K + 162) 2^-23 of the summed magnitudes, P = 1 or 3.  The activation's slope is at most 1.13
in size, and its own arithmetic is within 2^-13 (bf16 results) or 48 2^-24 (fp32) of the value's terms, as in the
tests of act_dropout (|v| <= 6 there: the inputs here are scaled to it).  Then the output type's rounding."""
import pytest
import torch

import sparse_mixture_experts_23_b200 as moe
from oplib import SUM_STEP, offsets_of, randn, round_bound, segments, strided, within

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def codes_and_scales(E, K, N, group, seed):
    """Codes of the whole range (no pattern that a wrong order could keep) and scales over a few octaves."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    s = (torch.rand((E, K // group, N), generator=g) + 0.5) * K ** -0.5 * 0.25
    return q.cuda(), s.to(BF).cuda()


def dense(q, s):
    """[E, K, N] in fp64 from codes and scales."""
    c = torch.stack([q & 15, q >> 4], -1).flatten(2).double() - 8  # [E, N, K]
    group = c.shape[2] // s.shape[1]
    return c.transpose(1, 2) * s.double().repeat_interleave(group, 1)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize(dtype, group):
    E, K, N = 3, 256, 37
    W = randn((E, K, N), dtype, 1, 0.3)
    W[0, :group, 5] = 0
    W[1, 3, 6], W[1, group + 1, 7], W[2, 0, 8] = float("inf"), float("nan"), -float("inf")
    W[2, :group, 9] = 1e-41 if dtype == F32 else 0  # a scale that rounds to zero
    q, s = moe.q4_quantize(W, group)
    w = W.float().view(E, K // group, group, N)
    finite = w.isfinite().all(2)
    sc = (w.abs().amax(2) / 7).to(BF)
    assert torch.equal(s[finite], sc[finite]) and s[~finite].isnan().all() and int((~finite).sum()) == 3
    live = (finite & (sc != 0))[:, :, None]
    want = torch.where(live, (w / sc.float()[:, :, None]).round().clamp(-8, 7), torch.zeros_like(w)) + 8
    got = torch.stack([q & 15, q >> 4], -1).flatten(2).transpose(1, 2).reshape(w.shape)
    assert torch.equal(got.float(), want)
    back = moe.Q4Weights(q, s).dequantize(F32)
    off = (back - W.float()).abs().view_as(w)
    # half a step of the code, the scale's own rounding (2^-8) at up to 7 codes, and the cut of codes above 7
    step = sc.float()[:, :, None].expand_as(w)
    ok = live.expand_as(w)
    assert (off[ok] <= (step * (0.5 + 7 * 2.0 ** -8) * 1.001)[ok]).all()
    assert back.view_as(w)[~finite[:, :, None].expand_as(w)].isnan().all()


SIZES = [(1, 32, 1, 32), (2, 128, 16, 128), (3, 64, 17, 64), (1, 160, 250, 32), (2, 384, 257, 128), (1, 448, 8, 64),
         (2, 1056, 530, 32), (4, 256, 48, 64)]


@pytest.mark.parametrize("E,K,N,group", SIZES)
def test_pack_keeps_every_weight(E, K, N, group):
    q, s = codes_and_scales(E, K, N, group, K + N)
    W = moe.Q4Weights(q, s)
    ref = dense(q, s)
    assert (W.E, W.K, W.N, W.group) == (E, K, N, group)
    assert torch.equal(W.dequantize(F32).double(), ref)  # 4 by 8 bits: exact
    assert torch.equal(W.dequantize(BF), ref.to(BF))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E,K,N,group", SIZES)
def test_unit_rows_bring_the_weights_back(E, K, N, group, dtype):
    """x = rows of the identity: every product picks one weight, exactly."""
    q, s = codes_and_scales(E, K, N, group, 7 * K + N)
    W = moe.Q4Weights(q, s)
    x = torch.eye(K, device="cuda", dtype=dtype).repeat(E, 1)
    y = moe.q4_matmul(x, W, offsets_of([K] * E), out_dtype=F32)
    assert torch.equal(y.view(E, K, N).double(), dense(q, s))


def test_fp32_rows_keep_all_bits():
    """Codes 7 and 9 (minus and plus one) and unit scales: every row has one fp32 value, which comes back whole."""
    K, N = 256, 40
    q = torch.where(torch.rand((1, N, K // 2), device="cuda") < 0.5, 0x79, 0x97).to(torch.uint8)
    W = moe.Q4Weights(q, torch.ones((1, K // 64, N), dtype=BF, device="cuda"))
    v = randn((K,), F32, 3, 100.0) * torch.logspace(-20, 20, K, device="cuda")
    v[:4] = torch.tensor([3.4028234e38, 1 + 2.0 ** -23, -(2.0 ** 24 - 1), 2.0 ** -100], device="cuda")
    y = moe.q4_matmul(torch.diag(v), W, offsets_of([K]))
    assert torch.equal(y.double(), torch.diag(v).double() @ dense(q, torch.ones((1, K // 64, N), dtype=BF, device="cuda"))[0])


def act64(v, act):
    if act == "gelu":
        return v * torch.special.ndtr(v)
    return v * torch.sigmoid(v) if act == "silu" else v


def check(counts, K, N, group, dtype=BF, out_dtype=None, act=None, bias=True, pad=0, spare=0, seed=0, ws=None):
    E, n = len(counts), sum(counts)
    out_dtype = out_dtype or dtype
    q, s = codes_and_scales(E, K, N, group, seed + 100)
    x = randn((n + spare, K), dtype, seed)
    if spare:
        x[n:] = float("nan")
    b = randn((E, N), dtype, seed + 2, 0.5) if bias else None
    ref = torch.zeros((n + spare, N), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    W = dense(q, s)
    for e, r in segments(counts):
        ref[r], mag[r] = x[r].double() @ W[e], x[r].double().abs() @ W[e].abs()
        if bias:
            ref[r] += b[e].double()
            mag[r] += b[e].double().abs()
    bound = ((3 if dtype == F32 else 1) * K + 162) * SUM_STEP * mag
    if act:
        assert ref.abs().max() <= 6
        bound = 1.13 * bound + (2.0 ** -13 if out_dtype == BF else 48 * 2.0 ** -24) * ref.abs()
        ref = act64(ref, act)
    xs = strided(x, 8 * pad)[0] if pad else x
    out, buf = strided(torch.full((n + spare, N), 7.0, dtype=out_dtype, device="cuda"), 5 * pad, 7.0)
    ws = moe.q4_workspace() if ws is None else ws
    y = moe.q4_matmul(xs, moe.Q4Weights(q, s), offsets_of(counts), bias=b, activation=act, out=out, ws=ws)
    assert moe.moe_get_device_status(ws.data_ptr()) == moe.MOE_OK
    assert y.data_ptr() == out.data_ptr()
    within(y[:n], ref[:n], bound[:n] + round_bound(ref[:n].abs() + bound[:n], out_dtype), f"{counts} {K} {N} {group}")
    assert (buf[n:] == 7.0).all() and (buf[:, N:] == 7.0).all(), "wrote outside its rows or columns"


ROWS = [[1], [0, 1, 0], [8, 0, 9, 1], [16, 17, 24, 25], [31, 32, 33], [0, 100, 7], [65]]


@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("counts", ROWS, ids=lambda c: "-".join(map(str, c)))
def test_rows(counts, dtype, out_dtype):
    check(counts, 256, 264, 64, dtype, out_dtype)
    check(counts, 96, 24, 32, dtype, out_dtype, bias=False, seed=5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K,N,group", [(32, 1, 32), (32, 8, 32), (128, 7, 128), (192, 255, 64), (4096, 16, 128), (2080, 40, 32),
                                       (14336, 8, 64), (512, 4104, 128)])
def test_sizes(K, N, group, dtype):
    check([3, 0, 12], K, N, group, dtype)


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (BF, F32), (F32, F32)])
def test_activation(act, dtype, out_dtype):
    check([2, 0, 20], 512, 100, 32, dtype, out_dtype, act=act)
    check([1], 128, 64, 128, dtype, out_dtype, act=act, bias=False, seed=9)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_and_spare_rows(dtype):
    check([5, 0, 30], 256, 72, 64, dtype, pad=1, spare=50)
    check([0, 0], 256, 72, 64, dtype, spare=9)
    W = moe.Q4Weights(*codes_and_scales(2, 64, 8, 32, 1))
    assert moe.q4_matmul(torch.ones((0, 64), device="cuda", dtype=dtype), W, offsets_of([0, 0])).shape == (0, 8)


def test_many_experts_and_rows():
    check([1] * 100 + [0] * 100 + [2] * 56, 128, 48, 64)
    check([1] + [0] * 254 + [1], 128, 48, 64, F32)
    check([500, 1, 300], 320, 300, 64)
    check([40, 0, 3, 1, 0, 0, 90, 2], 2048, 1000, 32)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinities_stay_in_their_rows(dtype):
    """A row that holds inf or NaN gives what its own sum gives; the rows beside it are unchanged."""
    counts = [5, 40]
    x = randn((45, 128), dtype, 1)
    q, s = codes_and_scales(2, 128, 48, 64, 2)
    W, off = moe.Q4Weights(q, s), offsets_of(counts)
    clean = moe.q4_matmul(x, W, off)
    x[2, 3], x[20, 1], x[21, 0] = float("inf"), float("nan"), float("-inf")
    y = moe.q4_matmul(x, W, off)
    rows = [2, 20, 21]
    keep = [r for r in range(45) if r not in rows]
    assert torch.equal(y[keep], clean[keep])
    w = dense(q, s)
    for r, e, k, sign in ((2, 0, 3, 1.0), (21, 1, 0, -1.0)):
        want = (sign * float("inf") * w[e, k]).to(dtype)  # NaN where the weight is zero
        assert torch.equal(y[r].isnan(), want.isnan()) and torch.equal(y[r][~want.isnan()], want[~want.isnan()])
    assert y[20].isnan().all()


def test_one_workspace_many_calls():
    """Calls of different sizes in a row on one workspace; the same call gives the same bits."""
    ws = moe.q4_workspace()
    for i, (K, N, group) in enumerate([(4096, 16, 128), (128, 520, 32), (2048, 264, 64), (4096, 16, 128)]):
        check([1, 0, 9], K, N, group, seed=i, ws=ws)
        check([40], K, N, group, F32, seed=i, ws=ws)
    x, W = randn((3, 4096), BF, 1), moe.Q4Weights(*codes_and_scales(1, 4096, 24, 64, 3))
    first = moe.q4_matmul(x, W, offsets_of([3]), ws=ws)
    for _ in range(20):
        assert torch.equal(moe.q4_matmul(x, W, offsets_of([3]), ws=ws), first)


@pytest.mark.parametrize("bad", [[0, 5, 3, 9], [1, 5, 7, 9], [0, 5, 7, 1000], [-4, 5, 7, 9]])
def test_bad_offsets_are_clamped_and_reported(bad):
    x, W, ws = randn((9, 64), BF, 1), moe.Q4Weights(*codes_and_scales(3, 64, 16, 32, 3)), moe.q4_workspace()
    moe.q4_matmul(x, W, torch.tensor(bad, dtype=torch.int32, device="cuda"), ws=ws)
    assert moe.moe_get_device_status(ws.data_ptr()) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_get_device_status(ws.data_ptr()) == moe.MOE_OK


def test_graph_replay_and_two_streams():
    """Captured once and replayed on new rows and offsets; calls at once on two streams, each with a workspace."""
    W = moe.Q4Weights(*codes_and_scales(3, 2048, 264, 64, 1))
    x, off, ws = randn((40, 2048), BF, 2), offsets_of([30, 0, 10]), moe.q4_workspace()
    y = moe.q4_matmul(x, W, off, ws=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.q4_matmul(x, W, off, out=y, ws=ws)
    x.copy_(randn((40, 2048), BF, 4))
    off.copy_(offsets_of([1, 38, 1]))
    g.replay()
    want = moe.q4_matmul(x, W, off)
    assert torch.equal(y, want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces, outs = [moe.q4_workspace() for _ in streams], [[], []]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(moe.q4_matmul(x, W, off, ws=spaces[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for row in outs for o in row)


@pytest.mark.parametrize("routing", ["token_choice", "expert_choice"])
@pytest.mark.parametrize("dtype,act,bias", [("bf16", "gelu", True), ("bf16", "silu", False), ("f32", "gelu", True)])
def test_layer_in_4_bits(dtype, act, bias, routing):
    """route, permute, expert_ffn_q4 against the definition in fp64 on the weights that the codes stand for, with
    the layer's own routing and tolerances (fp32: 1e-4 of the largest; bf16: 2e-2 of the root mean square)."""
    T, H, E, k, F, group = 50, 128, 8, 2, 192, 64
    dt = BF if dtype == "bf16" else F32
    inp = {"x": randn((T, H), dt, 1), "Wg": randn((H, E), dt, 2, H ** -0.5), "bg": None,
           "b1": randn((E, F), dt, 5, 0.1) if bias else None, "b2": randn((E, H), dt, 6, 0.1) if bias else None,
           "W1": None, "W2": None}
    q1, q2 = moe.q4_quantize(randn((E, H, F), dt, 3, H ** -0.5), group), moe.q4_quantize(randn((E, F, H), dt, 4, F ** -0.5), group)
    buf = moe.MoEBuffers(moe.make_shape(T, H, E, k, F, 1.25, dtype, act, routing), inp)
    W1, W2 = moe.Q4Weights(*q1), moe.Q4Weights(*q2)
    buf.out.fill_(float("nan"))
    buf.forward_q4(W1, W2)
    assert moe.moe_last_launch_count() == 3 and buf.device_status() == moe.MOE_OK
    ref = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    w1, w2, x = dense(*q1), dense(*q2), inp["x"].double()

    def expert(e, rows):
        h = act64(x[rows] @ w1[e] + (inp["b1"][e].double() if bias else 0), act)
        return h @ w2[e] + (inp["b2"][e].double() if bias else 0)

    for e in range(E):
        if routing == "expert_choice":
            rows = buf.topk_idx[e].long()
            ref.index_add_(0, rows, buf.topk_w[rows, e].double()[:, None] * expert(e, rows))
        else:
            for slot in range(k):
                rows = ((buf.topk_idx[:, slot] == e) & (buf.dropped[:, slot] == 0)).nonzero()[:, 0]
                ref[rows] += buf.topk_w[rows, slot].double()[:, None] * expert(e, rows)
    err = (buf.out.double() - ref).abs().max()
    assert err <= (2e-2 * ref.square().mean().sqrt() if dtype == "bf16" else 1e-4 * ref.abs().max())
    fused = buf.out.clone()  # without the combine, then moe_combine
    buf.expert_ffn_q4(W1, W2, combine=False)
    buf.combine()
    assert torch.equal(buf.out, fused)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_rows_near_the_largest_number(dtype, group):
    """Finite rows times small weights are finite: a group's sum before its scale must not overflow."""
    K, N, rows = 256, 40, 18
    q, _ = codes_and_scales(1, K, N, group, 3)
    s = torch.full((1, K // group, N), 2.0 ** -14, dtype=BF, device="cuda")
    x = (torch.rand((rows, K), device="cuda") * 2e38 + 1e38).to(dtype)
    x[1::2] *= torch.where(torch.rand((rows // 2, K), device="cuda") < 0.5, -1, 1).to(dtype)
    x[2] = torch.finfo(dtype).max
    w = dense(q, s)[0]
    ref, mag = x.double() @ w, x.double().abs() @ w.abs()
    assert mag.max() < torch.finfo(dtype).max
    y = moe.q4_matmul(x, moe.Q4Weights(q, s), offsets_of([rows]), out_dtype=F32)
    within(y, ref, ((3 if dtype == F32 else 1) * K + 162) * SUM_STEP * mag)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K,N,group", [(14336, 40, 64), (14336, 33, 128), (8224, 24, 32), (14272, 8, 64)])
@pytest.mark.parametrize("counts", [[1], [8, 0, 9], [17, 1]], ids=lambda c: "-".join(map(str, c)))
def test_long_sums_that_are_exact(counts, K, N, group, dtype):
    """Whole inputs up to 15 and scales 1 and 2: every product and every partial sum is a whole number below 2 * 8 * 15 * K <
    2^22, so that fp32 sums are exact in any order, and a step lost, doubled or taken from its neighbour shows."""
    E, n = len(counts), sum(counts)
    q, _ = codes_and_scales(E, K, N, group, K + N)
    g = torch.Generator().manual_seed(N)
    s = (torch.randint(0, 2, (E, K // group, N), generator=g) + 1).to(BF).cuda()
    x = (torch.randint(-15, 16, (n, K), generator=g)).to(dtype).cuda()
    w = dense(q, s)
    ref = torch.cat([x[r].double() @ w[e] for e, r in segments(counts)])
    assert torch.equal(moe.q4_matmul(x, moe.Q4Weights(q, s), offsets_of(counts), out_dtype=F32).double(), ref)


def test_long_sums_of_fp32_rows_keep_all_parts():
    """Rows of whole numbers up to 2^20 - 1, which take all three bf16 parts, against weights of one, minus one and zero: sums
    below 2^24 by pairing each input with its negative, but for the last two of a group."""
    K, N, group, rows = 14336, 24, 128, 9
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-(2 ** 20) + 1, 2 ** 20, (rows, K // 2), generator=g).double()
    x = torch.stack([x, -x], 2).view(rows, K)
    last = torch.arange(K) % (16 * group) >= 16 * group - 2
    x[:, last] = torch.randint(-(2 ** 20) + 1, 2 ** 20, (rows, int(last.sum())), generator=g).double()
    pair = torch.randint(7, 10, (1, N, K // 2), generator=g)  # one code for both inputs of a pair: 7, 8 or 9
    q = (pair | pair << 4).to(torch.uint8).cuda()
    s = torch.ones((1, K // group, N), dtype=BF, device="cuda")
    x = x.cuda()
    ref = x @ dense(q, s)[0]
    assert ref.abs().max() < 2 ** 24
    y = moe.q4_matmul(x.float(), moe.Q4Weights(q, s), offsets_of([rows]))
    assert torch.equal(y.double(), ref)
