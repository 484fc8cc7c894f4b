"""Helpers of the operator tests: offsets, strided operands, and error bounds derived from the arithmetic.

A product is summed in fp32 over n terms: each of the n additions is off by at most one step of 2^-23 of its
partial sum (tensor cores may cut where CUDA cores round), and no partial sum exceeds S = sum |terms|, so the
sum is off by at most (n + 2) 2^-23 S, the 2 for the bias and the final addition.  Rounding the result to type
t adds at most finfo(t).eps / 2 of the value (and half the smallest subnormal)."""
import torch

SUM_STEP = 2.0 ** -23


def offsets_of(counts, device="cuda"):
    o = [0]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device=device)


def segments(counts):
    r = 0
    for e, c in enumerate(counts):
        yield e, slice(r, r + c)
        r += c


def randn(shape, dtype, seed, std=1.0, device="cuda"):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(device)


def strided(t, pad, fill=float("nan")):
    """The same values in a buffer whose rows are `pad` elements further apart; returns (view, buffer)."""
    buf = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=t.device)
    buf[:, : t.shape[1]] = t
    return buf[:, : t.shape[1]], buf


def round_bound(ref, dtype):
    """How far rounding to dtype may move a value."""
    fi = torch.finfo(dtype)
    return ref.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def within(got, ref, bound, what=""):
    """|got - ref| <= bound everywhere, both finite."""
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: got {got[i].item()}, "
                             f"expected {ref[i].item()} within {bound[i].item()}")
