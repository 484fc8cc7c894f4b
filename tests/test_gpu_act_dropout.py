"""moe_act_dropout and its backward pass against the definition in fp64, with the mask from a numpy Philox.

Bounds.  fp32: a result is a product of at most five factors (activation or its derivative, gate, dy, scale); each
factor and product is off by a few 2^-24, and the library's erfc and exp by up to 8 units in the last place, whose
arguments carry one more rounding that the steep tail multiplies by u^2 / 2 <= 18 at |u| <= 6: 48 * 2^-24 in all of
the value, or, where 1 + u (1 - s) or Phi + u phi cancels, of the terms' magnitudes.  bf16: the fast forms are
within 2^-13 (fitted tail 1e-5, exp and reciprocal a few 2^-22, times u^2 / 2), plus the rounding."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_23_b200 as moe
from oplib import randn, round_bound, strided, within
from philox import keep_mask, philox

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
REL = {F32: 48 * 2.0 ** -24, BF: 2.0 ** -13}


def act64(u, act):
    """act(u), act'(u) and the magnitude of the terms of act'."""
    if act is None:
        return u, torch.ones_like(u), torch.ones_like(u)
    if act == "gelu":
        cdf, pdf = 0.5 * torch.erfc(u * -(0.5 ** 0.5)), torch.exp(-u * u / 2) / (2 * np.pi) ** 0.5
        return u * cdf, cdf + u * pdf, cdf + (u * pdf).abs()
    s = torch.sigmoid(u)
    return u * s, s * (1 + u * (1 - s)), s * (1 + (u * (1 - s)).abs())


def rng_of(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def check(rows, F, dtype, act, gated, p, pad=0, used=None, seed=5, offset=(7 << 32) + 3):
    u = randn((rows, F), dtype, seed, 2.0).clamp_(-6, 6)
    gate = randn((rows, F), dtype, seed + 1) if gated else None
    dy = randn((rows, F), dtype, seed + 2)
    n = rows if used is None else used
    m = torch.from_numpy(keep_mask(rows, F, p, seed, offset) / (1 - p if p < 1 else 1.0)).cuda()
    a, da, mag = act64(u.double(), act)
    g64 = gate.double() if gated else torch.ones_like(a)
    if used is not None:  # what lies behind the rows in use is not read
        for t in (u, gate, dy):
            if t is not None:
                t[n:] = float("nan")

    def put(t, by):
        return strided(t, by)[0] if by else t

    def room(by):
        return strided(torch.full((rows, F), 9.0, dtype=dtype, device="cuda"), by, 9.0)

    kw = dict(gate=put(gate, pad) if gated else None, activation=act, p=p, rng=rng_of(seed, offset) if p else None,
              rows=None if used is None else torch.tensor([used], dtype=torch.int32, device="cuda"))
    us, (y, ybuf), (du, dubuf), (dg, dgbuf) = put(u, pad), room(2 * pad), room(3 * pad), room(3 * pad)
    moe.act_dropout(us, out=y, **kw)
    got = moe.act_dropout_backward(put(dy, 2 * pad), us, du=du, dgate=dg if gated else None, **kw)
    assert (got[0] if gated else got).data_ptr() == du.data_ptr()
    rel = REL[dtype]

    def same(name, v, ref, size, buf):
        bound = rel * size[:n] + round_bound(ref[:n].abs() + rel * size[:n], dtype)
        within(v[:n], ref[:n], bound, f"{name} {rows}x{F} {act} {p}")
        assert (buf[n:] == 9.0).all() and (buf[:, F:] == 9.0).all(), name
        if p:
            assert (v[:n][m[:n] == 0] == 0).all(), name

    same("y", y, m * a * g64, (m * a * g64).abs(), ybuf)
    same("du", du, m * dy.double() * g64 * da, (m * dy.double() * g64).abs() * mag, dubuf)
    if gated:
        same("dgate", dg, m * dy.double() * a, (m * dy.double() * a).abs(), dgbuf)
    else:
        assert (dgbuf == 9.0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["gelu", "silu", None])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5])
def test_against_the_definition(dtype, act, gated, p):
    check(67, 264, dtype, act, gated, p)
    check(5, 37, dtype, act, gated, p, pad=1)  # element by element


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,F", [(1, 1), (1, 3), (3, 4), (1, 8192), (513, 8), (2, 1030), (4100, 12)])
def test_sizes(dtype, rows, F):
    check(rows, F, dtype, "silu", True, 0.3)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pitches_and_rows_in_use(dtype):
    for used in (0, 1, 50, 64):
        check(64, 128, dtype, "gelu", True, 0.2, pad=8, used=used)
        check(64, 30, dtype, "gelu", True, 0.2, pad=1, used=used)
    u = torch.ones((4, 8), dtype=dtype, device="cuda")
    for beyond in (5, 1000, -3):  # a count outside [0, rows] is clamped
        y = moe.act_dropout(u, activation=None, rows=torch.tensor([beyond], dtype=torch.int32, device="cuda"),
                            out=torch.full_like(u, 9.0))
        assert (y == (9.0 if beyond < 0 else 1.0)).all()


def test_generator_known_answers():
    """The kernel's words, read off through the thresholds: an element is kept at p exactly while its word is at
    least p 2^32, so bisecting p finds the word; compared with the paper's generator."""
    F, rows, seed, offset = 8, 3, -0x123456789ABCDEF, 0x0F1E2D3C4B5A6978
    words = np.stack([np.stack(philox((b, r, offset & 0xFFFFFFFF, offset >> 32),
                                      ((seed % 2 ** 64) & 0xFFFFFFFF, (seed % 2 ** 64) >> 32)))
                      for r in range(rows) for b in range(2)]).reshape(rows, F)
    one = torch.ones((rows, F), device="cuda")
    for r in range(rows):
        for c in range(F):
            w = int(words[r, c])
            at = moe.act_dropout(one, activation=None, p=w / 2 ** 32, rng=rng_of(seed, offset))
            above = moe.act_dropout(one, activation=None, p=(w + 1) / 2 ** 32, rng=rng_of(seed, offset))
            assert at[r, c] != 0 and above[r, c] == 0, (r, c)


def test_all_and_nothing_dropped():
    u = randn((9, 40), BF, 1)
    u[2, 3], u[4, 5] = float("nan"), float("inf")
    for p in (1.0,):
        y = moe.act_dropout(u, gate=u, p=p, rng=rng_of(1, 2))
        du, dg = moe.act_dropout_backward(u, u, gate=u, p=p, rng=rng_of(1, 2))
        assert not y.any() and not du.any() and not dg.any()
    tiny = moe.act_dropout(u[:2], p=2.0 ** -40, rng=rng_of(1, 2))  # below one step of the generator
    assert torch.equal(tiny, moe.act_dropout(u[:2]))
    assert moe.act_dropout(u[:0]).shape == (0, 40)


def test_offsets_give_independent_masks_and_bits_repeat():
    u = torch.ones((64, 4096), device="cuda")
    y = [moe.act_dropout(u, activation=None, p=0.25, rng=rng_of(3, o)) != 0 for o in (0, 0, 1)]
    assert torch.equal(y[0], y[1])
    n = u.numel()
    sd = (0.25 * 0.75 / n) ** 0.5
    assert abs(y[0].double().mean() - 0.75) < 6 * sd
    both = (y[0] & y[2]).double().mean()  # independent: 0.75^2
    assert abs(both - 0.5625) < 6 * (0.5625 * 0.4375 / n) ** 0.5


def test_far_values():
    """Where the activation saturates or underflows; the bf16 and the fp32 forms."""
    for dtype in (BF, F32):
        u = torch.tensor([[0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 100.0, -100.0, 3e38, -3e38, 9.0, -9.0]], dtype=dtype,
                         device="cuda")
        for act in ("gelu", "silu"):
            y = moe.act_dropout(u, activation=act).double()
            du = moe.act_dropout_backward(torch.ones_like(u), u, activation=act).double()
            a, da, _ = act64(u.double(), act)
            assert y.isfinite().all() and du.isfinite().all()
            lim = 2.0 ** -7 if dtype == BF else 2.0 ** -14  # exp's argument error times its size, |u| <= 20
            near = u.double().abs() <= 20
            assert ((y - a).abs() <= lim * a.abs() + 1e-37)[near].all(), (act, y, a)
            assert ((du - da).abs() <= lim * da.abs() + 1e-37)[near].all(), (act, du, da)
            assert torch.equal(y[:, [6, 8]], u.double()[:, [6, 8]])
            assert (y[:, [7, 9]].abs() <= 1e-37).all() and (du[:, [7, 9]].abs() <= 1e-37).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("F", [64, 33])
def test_in_place(dtype, F):
    u, g, dy = (randn((50, F), dtype, s) for s in (1, 2, 3))
    kw = dict(activation="silu", p=0.2, rng=rng_of(4, 5))
    y = moe.act_dropout(u, gate=g, **kw)
    du, dg = moe.act_dropout_backward(dy, u, gate=g, **kw)
    for which in (0, 1):
        u2, g2 = u.clone(), g.clone()
        assert torch.equal(moe.act_dropout(u2, gate=g2, out=(u2, g2)[which], **kw), y)
    u2, g2 = u.clone(), g.clone()
    moe.act_dropout_backward(dy, u2, gate=g2, du=u2, dgate=g2, **kw)
    assert torch.equal(u2, du) and torch.equal(g2, dg)


def test_halves_of_one_product():
    """u and gate as the two halves of one buffer's columns, and their gradients in the halves of another."""
    F = 72
    both = randn((33, 2 * F), BF, 8)
    dy = randn((33, F), BF, 9)
    kw = dict(activation="silu", p=0.1, rng=rng_of(6, 7))
    y = moe.act_dropout(both[:, :F], gate=both[:, F:], **kw)
    grad = torch.empty_like(both)
    moe.act_dropout_backward(dy, both[:, :F], gate=both[:, F:], du=grad[:, :F], dgate=grad[:, F:], **kw)
    u, g = both[:, :F].contiguous(), both[:, F:].contiguous()
    assert torch.equal(y, moe.act_dropout(u, gate=g, **kw))
    assert torch.equal(grad, torch.cat(moe.act_dropout_backward(dy, u, gate=g, **kw), 1))


def test_gradient_against_differences():
    """Central differences of the forward pass in fp32, h = 2^-6: the rule's own error is h^2 / 6 of the third
    derivative (below 2 for both activations), and the forward results carry 2^-22 of values up to 8."""
    u = torch.linspace(-5, 5, 2000, device="cuda").view(4, 500).contiguous()
    g = randn((4, 500), F32, 3)
    h = 2.0 ** -6
    for act in ("gelu", "silu"):
        kw = dict(gate=g, activation=act, p=0.3, rng=rng_of(1, 1))
        d = (moe.act_dropout(u + h, **kw).double() - moe.act_dropout(u - h, **kw).double()) / (2 * h)
        du, dg = moe.act_dropout_backward(torch.ones_like(u), u, **kw)
        m = (d != 0) | (du != 0)
        bound = (h * h / 3 + 8 * 2.0 ** -22 / h) * g.abs().double() / 0.7 + 1e-6
        within(du * m, d * m, bound)
        within(dg * g, moe.act_dropout(u, **kw).double(), 1e-5 * g.abs().double() + 1e-6)


def test_graph_takes_new_numbers():
    u = torch.ones((16, 64), device="cuda")
    rng, y = rng_of(1, 0), torch.empty_like(u)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        moe.act_dropout(u, activation=None, p=0.5, rng=rng, out=y)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.act_dropout(u, activation=None, p=0.5, rng=rng, out=y)
    seen = []
    for o in range(2):
        rng[1] = o
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y != 0, torch.from_numpy(keep_mask(16, 64, 0.5, 1, o)).cuda())
        seen.append(y.clone())
    assert not torch.equal(*seen)
