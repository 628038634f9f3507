"""8-bit blocks, their products and experts' rows in 64 bits, for the tests."""
from __future__ import annotations

import torch

LARGEST = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


def up(n, to):
    return -(-n // to) * to


def sides(blocks):
    """Rows and columns of a block."""
    return {"rows": (1, 128), "columns": (128, 1), "tiles": (128, 128)}[blocks]


def spread(scales, like, blocks):
    """A scale for each number of `like`, in 64 bits."""
    h, w = sides(blocks)
    s = scales.double().repeat_interleave(h, -2).repeat_interleave(w, -1)
    return s[..., :like.shape[-2], :like.shape[-1]]


def quantize(x, blocks, dtype):
    """(codes, scales) by the definition: FP32 quotients and products are those of
    64 bits, rounded once more (exact for one operation on two FP32 numbers)."""
    h, w = sides(blocks)
    x = x.double()
    r, c = x.shape[-2:]
    good = torch.isfinite(x)
    a = torch.zeros((*x.shape[:-2], up(r, h), up(c, w)), dtype=torch.float64, device=x.device)
    a[..., :r, :c] = torch.where(good, x.abs(), 0.0)
    a = a.unflatten(-1, (-1, w)).amax(-1).unflatten(-2, (-1, h)).amax(-2).clamp(min=2.0 ** -100)
    big = LARGEST[dtype]
    scale, lift = (a / big).float(), (big / a).float()
    y = (x * spread(lift, x, blocks)).float().clamp(-big, big)
    return torch.where(good, y, torch.nan).to(dtype), scale


def kind_of(scales, codes):
    r, c = codes.shape[-2:]
    for blocks in ("tiles", "rows", "columns"):
        h, w = sides(blocks)
        if tuple(scales.shape[-2:]) == (-(-r // h), -(-c // w)):
            return blocks
    raise AssertionError("shapes of scales")


def values(b, blocks=None):
    """What Blocks stand for, in 64 bits."""
    return b.data.double() * spread(b.scales, b.data, blocks or kind_of(b.scales, b.data))


def half_step(t):
    return torch.finfo(t).eps / 2


def product_bound(a, b, dtype, extra=0):
    """How far C may be from a @ b (64 bits; a, b what the codes stand for).

    The codes' products are exact in FP32 (significands of at most 4 bits), and a
    block's 128 of them are added in FP32, in any order, each addition off by at
    most a whole step (2^-23) if the tensor core cuts instead of rounding.  Then
    the scales' product, the product with it and the addition to the sum round
    once each a block, and parts of a split inner dimension (8 at most, `extra`
    more for C's old value) once each: (128 + 3 + blocks + 8 + extra) 2^-23 of
    the sum of magnitudes.  FP32 below its normal range: two roundings a block,
    2^-149 each.  Then C's own rounding: half a step, or in its subnormal range
    half the smallest number.
    """
    k = a.shape[-1]
    blocks = -(-k // 128)
    size = a.abs() @ b.abs()
    err = (139 + blocks + extra) * 2.0 ** -23 * size + 2 * blocks * 2.0 ** -149
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    return err * (1 + half_step(dtype)) + half_step(dtype) * (a @ b).abs() + tiny


def check_product(c, a, b, extra=0, old=None):
    want = a @ b
    bound = product_bound(a, b, c.dtype, extra)
    if old is not None:
        bound = bound + 2.0 ** -23 * (want.abs() + old.abs()) * (1 + extra)
        want = want + old
    d = (c.double() - want).abs()
    assert c.isfinite().all()
    assert (d <= bound).all(), f"worst {(d / bound).max().item():.3g} of the bound"


def maps(picks, experts, align):
    """(starts, rows, source), counted on the host; `source` as long as needed."""
    flat = picks.reshape(-1).tolist()
    held = [[] for _ in range(experts)]
    for i, e in enumerate(flat):
        if 0 <= e < experts:
            held[e].append(i)
    starts, rows, source = [0], [-1] * len(flat), []
    for h in held:
        for i in h:
            rows[i] = len(source)
            source.append(i)
        source += [-1] * (up(len(source), align) - len(source))
        starts.append(len(source))
    most = up(len(flat) + min(experts, len(flat)) * (align - 1), align)
    return starts, rows, source + [-1] * (most - len(source))
