"""The experts' operators together, as a program with gated experts uses them: the layer's own route and permute, one
product for u and gate, act_dropout between the halves, the second product into the layer's y, moe_combine; then the
gradients of every weight and of the rows, in a captured graph too.  Compared with autograd in fp64 on the same routing and
mask.  fp32: 1e-4 of the largest, as for the layer.  bf16 out: 2e-2 of the root mean square, as for the layer.  bf16
gradients: a Frobenius bound of 1e-2 as for the layer, and element by element what the roundings can do at most, with
q = 2^-8 a rounding (u, gate, h, dh, du, dgate are rounded; |SiLU'| <= 1.1, |SiLU''| <= 1/2):
    du = m dh gate act'(u):  |m dh| (3 q |gate act'| + q |u gate| / 2)      dgate = m dh act(u):  |m dh| (2 q |act| + 1.1 q |u|)
    h = m act(u) gate:       |m| (2 q |act gate| + 1.1 q |u gate|)
each times 1.02 for the products of two such errors and the fp32 sums, then through the magnitudes of the last product."""
import threading

import pytest
import torch

import sparse_mixture_experts_23_b200 as moe
from oplib import offsets_of, randn
from philox import keep_mask

pytestmark = pytest.mark.gpu


class GatedExperts:
    """Weights [E, H, 2F] and [E, F, H] on the rows that moe_permute has laid out in a layer's workspace."""

    def __init__(self, buf, W13, W2, p, rng):
        self.buf, self.W13, self.W2, self.p, self.rng = buf, W13, W2, p, rng
        s, v, dt = buf.shape, buf.view(), W13.dtype
        rows = s.T * s.k

        def at(ptr, n, dtype):
            start = ptr - buf.ws_ptr
            return buf.ws[start:start + n * dtype.itemsize].view(dtype)

        self.offsets = at(v.offsets, s.E + 1, torch.int32)
        self.x = at(v.x_perm, rows * s.H, dt).view(rows, s.H)
        self.y = at(v.y, rows * s.H, torch.float32).view(rows, s.H)
        self.row_token, self.row_slot = at(buf_row_map(buf)[0], rows, torch.int32), at(buf_row_map(buf)[1], rows, torch.int32)
        F = W2.shape[1]
        self.F, self.ug = F, torch.empty((rows, 2 * F), dtype=dt, device="cuda")
        self.h = torch.empty((rows, F), dtype=dt, device="cuda")
        self.kw = dict(activation="silu", p=p, rng=rng, rows=self.offsets[-1:])

    def forward(self):
        F = self.F
        moe.grouped_matmul(self.x, self.W13, self.offsets, out=self.ug)
        moe.act_dropout(self.ug[:, :F], gate=self.ug[:, F:], out=self.h, **self.kw)
        moe.grouped_matmul(self.h, self.W2, self.offsets, out=self.y)
        self.buf.combine()

    def backward(self, dy, g):
        F = self.F
        moe.grouped_wgrad(self.h, dy, self.offsets, dW=g["W2"])
        moe.grouped_matmul(dy, self.W2, self.offsets, transpose_w=True, out=g["h"])
        moe.act_dropout_backward(g["h"], self.ug[:, :F], gate=self.ug[:, F:], du=g["ug"][:, :F], dgate=g["ug"][:, F:], **self.kw)
        moe.grouped_wgrad(self.x, g["ug"], self.offsets, dW=g["W13"])
        moe.grouped_matmul(g["ug"], self.W13, self.offsets, transpose_w=True, out=g["x"])


def buf_row_map(buf):
    v = buf.view()
    return v.row_token, v.row_slot


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_training_step_of_gated_experts(dtype):
    T, H, E, k, F, p, seed, offset = 150, 128, 8, 2, 192, 0.2, 11, 5
    inp = {"x": randn((T, H), dtype, 1), "Wg": randn((H, E), dtype, 2, H ** -0.5)}
    name = "bf16" if dtype == torch.bfloat16 else "f32"
    buf = moe.MoEBuffers(moe.make_shape(T, H, E, k, F, 1.0, name, "silu"), inp)
    buf.route()
    buf.permute()
    W13, W2 = randn((E, H, 2 * F), dtype, 3, H ** -0.5), randn((E, F, H), dtype, 4, F ** -0.5)
    ex = GatedExperts(buf, W13, W2, p, torch.tensor([seed, offset], dtype=torch.int64, device="cuda"))
    rows = T * k
    dout = randn((T, H), torch.float32, 5)
    n = int(ex.offsets[-1])
    token, slot = ex.row_token[:n].long(), ex.row_slot[:n].long()
    weight = buf.topk_w[token, slot]
    dy = torch.full((rows, H), float("nan"), dtype=dtype, device="cuda")  # rows behind the last one are not read
    dy[:n] = (dout[token] * weight[:, None]).to(dtype)
    g = {"W2": torch.empty(W2.shape, device="cuda"), "W13": torch.empty(W13.shape, device="cuda"),
         "h": torch.empty((rows, F), dtype=dtype, device="cuda"), "ug": torch.empty((rows, 2 * F), dtype=dtype, device="cuda"),
         "x": torch.full((rows, H), 7.0, dtype=dtype, device="cuda")}

    # the definition in fp64 on the same rows
    x, w13, w2 = (t.double().requires_grad_() for t in (ex.x[:n].clone(), W13, W2))
    m = torch.from_numpy(keep_mask(rows, F, p, seed, offset)[:n] / (1 - p)).cuda()
    off, y = ex.offsets.tolist(), []
    for e in range(E):
        r = slice(off[e], off[e + 1])
        u, gate = (x[r] @ w13[e]).split(F, 1)
        y.append((u * torch.sigmoid(u) * gate * m[r]) @ w2[e])
    y = torch.cat(y)
    (y * dy[:n].double()).sum().backward()
    q, bounds = 1.02 * 2.0 ** -8, {"W2": [], "W13": [], "x": []}
    with torch.no_grad():
        for e in range(E):
            r = slice(off[e], off[e + 1])
            u, gate = (x[r] @ w13[e]).split(F, 1)
            s = torch.sigmoid(u)
            act, dact, mdh, d = u * s, s * (1 + u * (1 - s)), m[r] * (dy[r].double() @ w2[e].T).abs(), dy[r].double().abs()
            dug = q * torch.cat([mdh * (3 * (gate * dact).abs() + (u * gate).abs() / 2), mdh * (2 * act.abs() + 1.1 * u.abs())], 1)
            bounds["W2"].append((q * m[r] * (2 * (act * gate).abs() + 1.1 * (u * gate).abs())).T @ d)
            bounds["W13"].append(x[r].abs().T @ dug)
            bounds["x"].append(dug @ w13[e].abs().T + q * x.grad[r].abs())
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda").index_add_(0, token, weight.double()[:, None] * y.detach())

    def check(got, want, what, bound=None):
        err = (got.double() - want).abs()
        if dtype == torch.float32:
            assert err.max() <= 1e-4 * want.abs().max(), what
        elif bound is None:
            assert err.max() <= 2e-2 * want.square().mean().sqrt(), what
        else:
            assert (err <= bound).all() and err.norm() <= 1e-2 * want.norm(), what

    def verify():
        check(buf.out, out, "out")
        check(g["x"][:n], x.grad, "dx", torch.cat(bounds["x"]))
        assert (g["x"][n:] == 7.0).all()
        for e in range(E):
            if off[e] < off[e + 1]:
                check(g["W13"][e], w13.grad[e], f"dW13[{e}]", bounds["W13"][e])
                check(g["W2"][e], w2.grad[e], f"dW2[{e}]", bounds["W2"][e])
            else:
                assert not g["W13"][e].any() and not g["W2"][e].any()

    ex.forward()
    ex.backward(dy, g)
    verify()
    assert buf.device_status() == moe.MOE_OK
    # the same step captured and replayed
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            ex.forward()
            ex.backward(dy, g)
    torch.cuda.current_stream().wait_stream(s)
    for t in (buf.out, g["W13"], g["W2"]):
        t.fill_(float("nan"))
    g["x"].fill_(7.0)
    graph.replay()
    verify()


def test_calls_at_once():
    """The products, their gradients, the 4-bit product and the dropout from threads on streams of their own, and from two
    graphs replayed side by side (one error word between them): the bits of one call after the other.  Few rows, few tiles
    of a long contraction and long segments: every form that joins sums of several blocks is among them."""
    sets = []
    for i, (E, K, N, counts, dtype) in enumerate([
            (4, 2048, 64, [3, 0, 9, 1], torch.bfloat16), (8, 512, 1024, [64] * 8, torch.bfloat16), (2, 4096, 200, [50, 42], torch.float32),
            (1, 8192, 64, [10], torch.float32), (3, 64, 64, [3000, 1, 500], torch.float32), (1, 64, 520, [4000], torch.bfloat16)]):
        n = sum(counts)
        sets.append((randn((n, K), dtype, i), randn((E, K, N), dtype, i + 10), offsets_of(counts), randn((E, N), dtype, i + 20),
                     randn((n, N), dtype, i + 30)))
    q = moe.Q4Weights(*moe.q4_quantize(randn((4, 1024, 512), torch.float32, 50), group=64))
    ws, xq, oq = moe.q4_workspace(), randn((30, 1024), torch.bfloat16, 51), offsets_of([7, 0, 20, 3])
    rng = torch.tensor([3, 4], device="cuda")

    def work():
        r = [moe.q4_matmul(xq, q, oq, ws=ws), moe.act_dropout(sets[1][4], p=0.3, rng=rng)]
        for x, W, offsets, bias, dy in sets:
            r += [moe.grouped_matmul(x, W, offsets, bias), moe.grouped_matmul(dy, W, offsets, transpose_w=True)]
            r += moe.grouped_wgrad(x, dy, offsets, bias_grad=True)
        return r

    want = work()
    torch.cuda.synchronize()
    same = []

    def one():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(5):
                got = work()
                stream.synchronize()
                same.append(all(map(torch.equal, got, want)))

    threads = [threading.Thread(target=one) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert same == [True] * 15
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = work()
        graphs.append((g, got, torch.cuda.Stream()))
    for _ in range(5):
        for g, _, stream in graphs:
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    assert all(all(map(torch.equal, got, want)) for _, got, _ in graphs) and moe.moe_get_device_status(ws.data_ptr()) == 0
