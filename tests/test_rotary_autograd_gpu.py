"""rotary in a graph of gradients: the backward pass is the rotation back."""
from __future__ import annotations

import pytest

from tests import paged_ref as ref

pytestmark = pytest.mark.gpu
D = ref.D


@pytest.fixture(scope="module")
def g():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import async_barrier_pipelined_gb300 as g
    from async_barrier_pipelined_gb300 import build
    build.build()
    return g


@pytest.fixture(scope="module")
def plan(g):
    with g.Plan(0) as p:
        yield p


def setup(g, tokens, heads, rot, seed):
    import torch
    gen = torch.Generator().manual_seed(seed)
    freq = torch.tensor(g.rope_frequencies(rot), dtype=torch.float64)
    x, dy = (torch.randn(tokens, heads, D, generator=gen).half().cuda() for _ in range(2))
    pos = torch.randint(0, 5000, (tokens,), generator=gen, dtype=torch.int32).cuda()
    return x, dy, pos, freq, g.rope_turns(freq).cuda()


def bound(dy, dx, factor):
    """Half a binary16 step of the result (half a step below the normal range);
    FP32: an angle off by pi 2^-24, cosine and sine by 2^-23 each, three
    roundings of the products and their sum, together under 8 * 2^-24 (|y0| +
    |y1|) * factor; a double angle of 5000 radians off by 2^-52 of it."""
    mag = dy.double().abs().amax(-1, keepdim=True) * 2 * abs(factor)
    return (2.0 ** -11 * dx.abs() + 8 * 2.0 ** -24 * mag + 2.0 ** -25
            + 5000 * 2.0 ** -51 * mag)


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,rot", [(1, 1, 256), (9, 3, 96), (0, 2, 16)])
def test_gradient_of_the_call(g, plan, layout, inverse, tokens, heads, rot):
    import torch
    x, dy, pos, freq, turns = setup(g, tokens, heads, rot, 1)
    kw = dict(layout=layout, factor=1.5, inverse=inverse)
    plain = g.rotary(plan, x, pos, turns, **kw)
    x.requires_grad_()
    y = g.rotary(plan, x, pos, turns, **kw)
    assert y.requires_grad and torch.equal(y, plain)
    y.backward(dy)
    torch.cuda.synchronize()
    assert plan.status() == 0
    x64 = x.detach().double().requires_grad_()
    (ref.rope_reference(x64, pos, freq, layout, 1.5, inverse) * dy.double()).sum().backward()
    assert ((x.grad.double() - x64.grad).abs() <= bound(dy, x64.grad, 1.5)).all()
    with torch.no_grad():
        assert not g.rotary(plan, x, pos, turns, **kw).requires_grad


@pytest.mark.parametrize("how", ["one number", "transposed", "odd address"])
def test_gradients_however_they_are_laid_out(g, plan, how):
    import torch
    x, dy, pos, freq, turns = setup(g, 6, 4, 64, 2)
    if how == "one number":
        dy = torch.ones((), dtype=torch.float16, device="cuda").expand(6, 4, D)
    elif how == "transposed":
        dy = dy.permute(2, 0, 1).contiguous().permute(1, 2, 0)
    else:
        buf = torch.empty(dy.numel() + 1, dtype=torch.float16, device="cuda")
        buf[1:] = dy.flatten()
        dy = buf[1:].view(dy.shape)
    want = g.rotary(plan, dy.contiguous().clone(), pos, turns, inverse=True)
    x.requires_grad_()
    g.rotary(plan, x, pos, turns).backward(dy)
    assert torch.equal(x.grad, want)


def test_through_a_graph_and_twice(g, plan):
    """A strided view of a larger leaf, on another stream, and the gradient of
    a gradient (the call is linear: that of dY is the rotation itself)."""
    import torch
    x, dy, pos, freq, turns = setup(g, 30, 5, 256, 3)
    leaf = torch.cat((x, x), 1).requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        y = g.rotary(plan, leaf[:, :5], pos, turns, stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        leaf.grad = None
        (y * dy).sum().backward()
        torch.cuda.synchronize()
        assert torch.equal(leaf.grad[:, :5], g.rotary(plan, dy, pos, turns, inverse=True))
        assert (leaf.grad[:, 5:] == 0).all()
    x.requires_grad_()
    dy.requires_grad_()
    dx, = torch.autograd.grad(g.rotary(plan, x, pos, turns), x, dy, create_graph=True)
    back, = torch.autograd.grad(dx, dy, x.detach())
    assert torch.equal(back, g.rotary(plan, x.detach(), pos, turns))
    assert plan.status() == 0


def test_an_output_cannot_be_given(g, plan):
    import torch
    x, dy, pos, freq, turns = setup(g, 3, 2, 64, 4)
    x.requires_grad_()
    for out in (torch.empty_like(dy), x):
        with pytest.raises(ValueError):
            g.rotary(plan, x, pos, turns, out=out)
    with torch.no_grad():
        out = torch.empty_like(dy)
        assert g.rotary(plan, x, pos, turns, out=out) is not None


def test_positions_of_a_step(g, plan):
    """Positions that paged_maps made are kept for the backward pass."""
    import torch
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    m = g.paged_maps(plan, i32([5, 0]), i32([2, 4]), i32([[0, 1], [2, 3]]), i32([4, 5, 6]),
                     i32([0]), 16, 6)
    x, dy, _, _, turns = setup(g, 6, 2, 64, 5)
    x.requires_grad_()
    g.rotary(plan, x, m.positions, turns).backward(dy)
    assert torch.equal(x.grad, g.rotary(plan, dy, i32([5, 6, 0, 1, 2, 3]), turns, inverse=True))
    torch.cuda.synchronize()
    assert plan.status() == 0
