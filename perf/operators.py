"""Workloads of the expert-level operators: grouped matrix products (forward, transposed, weight gradient),
the expert activation with dropout, and products with 4-bit expert weights.

``listed()`` names fixed cases, ``draw(rng)`` gives more of the same ranges, ``prepare`` makes what a
program holds before the call, ``run`` makes one pass, ``exact`` computes the same in 64 bits and ``work``
says what a pass cannot do without.  With ``own`` false, ``run`` uses elementary torch operations in 32 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # decode: 32 tokens, 2 experts each, of the Mixtral-style layer: every weight is read for a few rows
        dict(name="mm_decode", op="matmul", E=8, rows=64, K=4096, N=14336, dtype="bf16", out="bf16", trans=False,
             bias=True, spread="ragged"),
        # the Switch-style layer's first product: 128 experts, about 64 rows each, ragged
        dict(name="mm_switch", op="matmul", E=128, rows=8104, K=1024, N=4096, dtype="bf16", out="bf16", trans=False,
             bias=True, spread="ragged"),
        # the data gradient of the Mixtral-style layer's first product: the weights read transposed
        dict(name="mm_mixtral_t", op="matmul", E=8, rows=8192, K=14336, N=4096, dtype="bf16", out="bf16", trans=True,
             bias=False, spread="ragged"),
        # a skewed fp32 layer: few rows, odd widths, experts without rows
        dict(name="mm_f32_odd", op="matmul", E=16, rows=1003, K=516, N=780, dtype="f32", out="f32", trans=False,
             bias=True, spread="skewed"),
        # the weight gradient of the Mixtral-style layer's first product
        dict(name="wgrad_mixtral", op="wgrad", E=8, rows=8192, K=4096, N=14336, dtype="bf16", bias=False,
             spread="ragged"),
        # the weight gradient of a skewed layer of many small experts, with the bias gradient
        dict(name="wgrad_skewed", op="wgrad", E=64, rows=5003, K=1032, N=520, dtype="bf16", bias=True,
             spread="skewed"),
        # hidden rows of a training step of the Mixtral-style layer with gated experts
        dict(name="act_gated", op="act", rows=4099, F=14336, dtype="bf16", act="silu", gated=True, p=0.1),
        # the tiny fp32 layer's hidden rows, an odd width
        dict(name="act_small", op="act", rows=511, F=257, dtype="f32", act="gelu", gated=False, p=0.25),
        # one token, two experts: both halves of the Mixtral-style expert in 4 bits
        dict(name="q4_token", op="q4", E=8, rows=2, K=4096, N=14336, group=64, dtype="bf16", out="bf16", act="silu",
             bias=False, spread="one"),
        dict(name="q4_decode", op="q4", E=8, rows=64, K=14336, N=4096, group=128, dtype="bf16", out="bf16", act="none",
             bias=True, spread="ragged"),
        # a small step of a layer with many experts, some with dozens of rows, some with none
        dict(name="q4_skewed", op="q4", E=64, rows=301, K=2048, N=1992, group=32, dtype="bf16", out="bf16", act="gelu",
             bias=True, spread="skewed"),
        # the smallest call: a single fp32 row of one small expert
        dict(name="q4_tiny", op="q4", E=1, rows=1, K=512, N=256, group=32, dtype="f32", out="f32", act="none",
             bias=False, spread="one"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    return max(m, _log(rng, lo, hi) // m * m)


def draw(rng):
    op = rng.choice(["matmul", "matmul", "wgrad", "act", "q4", "q4"])
    if op == "act":
        return dict(op=op, rows=_log(rng, 1, 4096), F=_log(rng, 64, 14336), dtype=rng.choice(["bf16", "f32"]),
                    act=rng.choice(["gelu", "silu"]), gated=rng.random() < 0.5, p=rng.choice([0.0, 0.1, 0.25, 0.5]))
    while True:
        E = _log(rng, 1, 128)
        spread = rng.choice(["ragged", "skewed", "one"])
        if op == "q4":
            group = rng.choice([32, 64, 128])
            K, N, rows = _mult(rng, 256, 14336, group), _mult(rng, 64, 14336, 8), _log(rng, 1, 400)
            if E * K * N > 8 * 4096 * 14336:
                continue
            dtype = rng.choice(["bf16", "bf16", "f32"])
            return dict(op=op, E=E, rows=rows, K=K, N=N, group=group, dtype=dtype, out=dtype,
                        act=rng.choice(["none", "gelu", "silu"]), bias=rng.random() < 0.5, spread=spread)
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        m = 8 if dtype == "bf16" else 4
        K, N, rows = _mult(rng, 64, 8192, m), _mult(rng, 64, 8192, m), _log(rng, 1, 8192)
        if E * K * N > 8 * 4096 * 14336 or rows * K * N > (8192 * 4096 * 14336 if dtype == "bf16" else 2 ** 35):
            continue
        c = dict(op=op, E=E, rows=rows, K=K, N=N, dtype=dtype, bias=rng.random() < 0.5, spread=spread)
        if op == "matmul":
            c.update(out=dtype, trans=rng.random() < 0.5)
        return c


# ---------------------------------------------------------------- inputs
def _counts(case, seed):
    """Rows of each expert: an even choice for every row, a skewed one, or at most one row an expert."""
    E, rows = case["E"], case["rows"]
    r = np.random.default_rng(seed * 7919 + 17)
    if case["spread"] == "one":
        cnt = np.full(E, rows // E)
        cnt[r.permutation(E)[: rows % E]] += 1
    else:
        w = np.ones(E) if case["spread"] == "ragged" else 1.0 / np.arange(1, E + 1) ** 1.5
        cnt = r.multinomial(rows, w / w.sum())
    return [int(c) for c in cnt]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = _DT[case["dtype"]]

    def normal(shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dt)

    st = dict(case=case)
    if case["op"] == "act":
        rows, F = case["rows"], case["F"]
        st["u"] = normal((rows, F), 1.5)
        st["gate"] = normal((rows, F)) if case["gated"] else None
        st["dy"] = normal((rows, F), 0.1)
        st["rng"] = torch.tensor([seed * 1000003 + 12345, seed + 77], dtype=torch.int64, device="cuda")
        st["y"], st["du"] = torch.empty_like(st["u"]), torch.empty_like(st["u"])
        st["dgate"] = torch.empty_like(st["u"]) if case["gated"] else None
        return st
    E, rows, K, N = case["E"], case["rows"], case["K"], case["N"]
    st["counts"] = _counts(case, seed)
    st["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(st["counts"])]), dtype=torch.int32).cuda()
    st["x"] = normal((rows, K))
    if case["op"] == "wgrad":
        st["dy"] = normal((rows, N), 0.1)
        st["dW"] = torch.empty((E, K, N), device="cuda")
        st["db"] = torch.empty((E, N), device="cuda") if case["bias"] else None
        return st
    st["b"] = normal((E, N), 0.02) if case["bias"] else None
    st["y"] = torch.empty((rows, N), dtype=_DT[case["out"]], device="cuda")
    if case["op"] == "matmul":
        W = torch.empty((E, N, K) if case["trans"] else (E, K, N), dtype=dt, device="cuda")
        for e in range(E):
            W[e] = normal(W[e].shape, K ** -0.5)
        st["W"] = W
        return st
    # 4-bit codes (two a byte along k, the even k low) and a bf16 scale for each group of a column, as they are
    # made from normal weights; the program keeps them and the workspace of its calls
    G = case["group"]
    q = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.empty((E, K // G, N), dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        w = torch.randn((N, K // G, G), generator=g, device="cuda").mul_(K ** -0.5)
        sc = (w.abs().amax(-1) / 7).to(torch.bfloat16)
        c = (w / sc.float()[..., None]).round_().clamp_(-8, 7).add_(8).to(torch.uint8).view(N, K // 2, 2)
        q[e] = c[..., 0] | (c[..., 1] << 4)
        s[e] = sc.t()
    st["q"], st["s"] = q, s
    if own:
        import sparse_mixture_experts_23_b200 as moe

        st["qw"] = moe.Q4Weights(q, s)
        st["ws"] = moe.q4_workspace()
    return st


# ---------------------------------------------------------------- one pass
def _segments(counts):
    r = 0
    for e, c in enumerate(counts):
        if c:
            yield e, r, r + c
        r += c


_M0, _M1, _W0, _W1, _LOW = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85, 0xFFFFFFFF


def _keep(rng, rows, F, p):
    """Philox4x32-10 at counter (column // 4, row, offset), key seed: word column % 4 keeps the element when it
    is not below p * 2^32."""
    seed, off = rng[0], rng[1]
    c0 = torch.arange((F + 3) // 4, device="cuda").expand(rows, -1)
    c1 = torch.arange(rows, device="cuda")[:, None].expand_as(c0)
    c2, c3 = (off & _LOW).expand_as(c0), ((off >> 32) & _LOW).expand_as(c0)
    k0, k1 = seed & _LOW, (seed >> 32) & _LOW
    for _ in range(10):
        p0, p1 = c0 * _M0, c2 * _M1
        c0, c1, c2, c3 = ((p1 >> 32) & _LOW) ^ c1 ^ k0, p1 & _LOW, ((p0 >> 32) & _LOW) ^ c3 ^ k1, p0 & _LOW
        k0, k1 = (k0 + _W0) & _LOW, (k1 + _W1) & _LOW
    words = torch.stack([c0, c1, c2, c3], -1).reshape(rows, -1)[:, :F]
    return words >= int(p * 2.0 ** 32)


def _act32(u, act):
    """act(u) and act'(u) in 32 bits."""
    if act == "silu":
        sg = 1 / (1 + torch.exp(-u))
        return u * sg, sg * (1 + u * (1 - sg))
    phi = 0.5 * torch.erfc(u * -0.7071067811865476)
    return u * phi, phi + u * 0.3989422804014327 * torch.exp(-0.5 * u * u)


def _unpack(q, s):
    c = torch.stack([q & 15, q >> 4], -1).view(q.shape[0], -1).float() - 8
    return c * s.float().t().repeat_interleave(c.shape[1] // s.shape[0], 1)


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import sparse_mixture_experts_23_b200 as moe

        if op == "matmul":
            return moe.grouped_matmul(st["x"], st["W"], st["offsets"], bias=st["b"], transpose_w=case["trans"],
                                      out=st["y"])
        if op == "wgrad":
            return moe.grouped_wgrad(st["x"], st["dy"], st["offsets"], dW=st["dW"], db=st["db"])
        if op == "act":
            kw = dict(gate=st["gate"], activation=case["act"], p=case["p"], rng=st["rng"])
            y = moe.act_dropout(st["u"], out=st["y"], **kw)
            return y, moe.act_dropout_backward(st["dy"], st["u"], du=st["du"], dgate=st["dgate"], **kw)
        return moe.q4_matmul(st["x"], st["qw"], st["offsets"], bias=st["b"],
                             activation=None if case["act"] == "none" else case["act"], out=st["y"], ws=st["ws"])
    if op == "act":
        u, dy = st["u"].float(), st["dy"].float()
        a, da = _act32(u, case["act"])
        p = case["p"]
        m = 1.0
        if p > 0:
            m = _keep(st["rng"], case["rows"], case["F"], p) * (1.0 / (1.0 - p))
        if st["gate"] is None:
            return (m * a).to(st["u"].dtype), (m * dy * da).to(st["u"].dtype)
        gate = st["gate"].float()
        return ((m * a * gate).to(st["u"].dtype),
                ((m * dy * gate * da).to(st["u"].dtype), (m * dy * a).to(st["u"].dtype)))
    x = st["x"]
    if op == "wgrad":
        dW, db = st["dW"].zero_(), st["db"]
        if db is not None:
            db.zero_()
        for e, r0, r1 in _segments(st["counts"]):
            d = st["dy"][r0:r1].float()
            dW[e] = x[r0:r1].float().t() @ d
            if db is not None:
                db[e] = d.sum(0)
        return dW if db is None else (dW, db)
    y = st["y"]
    for e, r0, r1 in _segments(st["counts"]):
        if op == "matmul":
            W = st["W"][e].float()
            v = x[r0:r1].float() @ (W.t() if case["trans"] else W)
        else:
            v = x[r0:r1].float() @ _unpack(st["q"][e], st["s"][e]).t()
        if st["b"] is not None:
            v = v + st["b"][e].float()
        if op == "q4" and case["act"] != "none":
            v = _act32(v, case["act"])[0]
        y[r0:r1] = v.to(y.dtype)
    return y


# ---------------------------------------------------------------- the definition in 64 bits
def _philox_words(rng, rows, F):
    """The same generator from 16-bit halves of its products, row by row blocks (numpy, unsigned)."""
    seed, off = (int(v) & (2 ** 64 - 1) for v in rng.tolist())
    u64 = np.uint64

    def mul(a, m):  # high and low words of a 32 x 32 bit product
        pr = a * u64(m)
        return pr >> u64(32), pr & u64(_LOW)

    out = np.empty((rows, (F + 3) // 4, 4), dtype=np.uint32)
    step = max(1, (1 << 20) // max(1, F))
    for r0 in range(0, rows, step):
        n = min(step, rows - r0)
        c = [np.broadcast_to(v, (n, (F + 3) // 4)).astype(u64) for v in
             (np.arange((F + 3) // 4), np.arange(r0, r0 + n)[:, None], off & _LOW, off >> 32)]
        for i in range(10):
            key = u64((seed + i * _W0) & _LOW), u64(((seed >> 32) + i * _W1) & _LOW)
            (h0, l0), (h1, l1) = mul(c[0], _M0), mul(c[2], _M1)
            c = [h1 ^ c[1] ^ key[0], l1, h0 ^ c[3] ^ key[1], l0]
        for j in range(4):
            out[r0:r0 + n, :, j] = c[j]
    return out.reshape(rows, -1)[:, :F]


def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "act":
        rows, F, p = case["rows"], case["F"], case["p"]
        keep = torch.ones((rows, F), device="cuda", dtype=f64)
        if p > 0:
            words = _philox_words(st["rng"].cpu(), rows, F)
            keep = torch.from_numpy((words >= np.uint32(int(p * 2.0 ** 32))) / (1.0 - p)).cuda()
        u, dy = st["u"].to(f64), st["dy"].to(f64)
        if case["act"] == "gelu":
            cdf = torch.special.ndtr(u)
            a, da = u * cdf, cdf + u * torch.exp(-u.square() / 2) / math.sqrt(2 * math.pi)
        else:
            sg = torch.sigmoid(u)
            a, da = u * sg, sg + u * sg * torch.sigmoid(-u)
        if st["gate"] is None:
            return keep * a, keep * dy * da
        gate = st["gate"].to(f64)
        return keep * a * gate, (keep * dy * gate * da, keep * dy * a)
    bounds = st["offsets"].tolist()
    x = st["x"].to(f64)
    if case["op"] == "wgrad":
        dW = torch.empty(st["dW"].shape, device="cuda", dtype=f64)
        db = None if st["db"] is None else torch.empty(st["db"].shape, device="cuda", dtype=f64)
        for e in range(case["E"]):
            rows = slice(bounds[e], bounds[e + 1])
            d = st["dy"][rows].to(f64)
            torch.matmul(x[rows].mT, d, out=dW[e])
            if db is not None:
                db[e] = d.sum(0)
        return dW if db is None else (dW, db)
    y = torch.empty((case["rows"], case["N"]), device="cuda", dtype=f64)
    for e in range(case["E"]):
        rows = slice(bounds[e], bounds[e + 1])
        if bounds[e] == bounds[e + 1]:
            continue
        if case["op"] == "matmul":
            W = st["W"][e].to(f64)
            W = W.mT if case["trans"] else W
        else:
            codes = torch.empty((case["K"], case["N"]), device="cuda", dtype=f64)
            codes[0::2] = torch.remainder(st["q"][e], 16).mT
            codes[1::2] = torch.div(st["q"][e], 16, rounding_mode="floor").mT
            W = ((codes - 8).view(-1, case["group"], case["N"]) * st["s"][e].to(f64)[:, None]).view(case["K"], -1)
        v = x[rows] @ W
        if st["b"] is not None:
            v += st["b"][e].to(f64)
        if case["op"] == "q4" and case["act"] == "gelu":
            v = v * torch.special.ndtr(v)
        elif case["op"] == "q4" and case["act"] == "silu":
            v = v * torch.sigmoid(v)
        y[rows] = v
    return y


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    es = _ES[case["dtype"]]
    if case["op"] == "act":
        n, gated = case["rows"] * case["F"], case["gated"]
        # forward and backward of one pass: u, gate and dy are read once, y and the gradients written once
        return dict(bytes=n * es * (6 if gated else 4), flops=n * (30 if gated else 26))
    E, rows, K, N = case["E"], case["rows"], case["K"], case["N"]
    flops = 2 * rows * K * N
    if case["op"] == "wgrad":
        return dict(bytes=rows * (K + N) * es + 4 * E * K * N + (4 * E * N if case["bias"] else 0), flops=flops)
    touched = min(E, rows)  # experts with rows (an upper bound where the spread is uneven)
    if case["op"] == "matmul":
        b = touched * K * N * es
    else:
        b = touched * (K * N // 2 + 2 * (K // case["group"]) * N)
    b += rows * K * es + rows * N * _ES[case["out"]] + (touched * N * es if case["bias"] else 0)
    return dict(bytes=b, flops=flops)
