"""Tokens sorted by expert and back, and 8-bit linear layers with their gradients,
on the GPU against 64 bits (f8_ref)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
from tests import f8_ref as ref  # noqa: E402
from tests.test_f8_gpu import E4, E5, BF16, F16, F32, g, gen, plan, rand  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def picks_of(seed, tokens, choices, experts, none=0.1, wide=False):
    r = gen(seed)
    p = torch.randint(0, experts, (tokens, choices), generator=r, device="cuda")
    p = torch.where(torch.rand(p.shape, generator=r, device="cuda") < none, -1 - p, p)
    return p if wide else p.int()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("align", [1, 16, 128])
@pytest.mark.parametrize("tokens,choices,experts", [
    (0, 2, 4), (1, 1, 1), (1, 8, 1024), (33, 1, 3), (48, 8, 64), (512, 8, 60), (513, 8, 256),
    (4096, 1, 1), (9000, 7, 128), (70000, 1, 1024)])
def test_maps(g, plan, tokens, choices, experts, align, wide):
    p = picks_of(tokens, tokens, choices, experts, wide=wide)
    m = g.expert_maps(plan, p, experts, align=align)
    starts, rows, source = ref.maps(p, experts, align)
    assert m.starts.tolist() == starts
    assert m.rows.shape == (tokens, choices) and m.rows.reshape(-1).tolist() == rows
    assert m.source.tolist() == source
    assert plan.status() == g.OK


def test_no_entry_of_any_expert_and_all_of_one(g, plan):
    for p in (torch.full((300, 2), -1, device="cuda"), torch.full((300, 2), 6, device="cuda")):
        m = g.expert_maps(plan, p, 7, align=16)
        assert [m.starts.tolist(), m.rows.reshape(-1).tolist(), m.source.tolist()] == list(
            ref.maps(p, 7, 16))


def test_an_expert_that_is_not_there_is_reported(g, plan):
    p = torch.tensor([[0, 4], [3, 1]], dtype=torch.int32, device="cuda")
    m = g.expert_maps(plan, p, 4)
    torch.cuda.synchronize()
    assert plan.status() == g.ERR_BAD_INDEX and plan.status() == g.OK
    assert m.rows.tolist() == [[0, -1], [2, 1]]


def test_bad_maps_are_reported_and_read_nothing(g, plan):
    """Entries outside the tokens (rows) count as none."""
    x = rand(1, 6, 40)
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    m = g.ExpertMaps(i(0, 12), i(*range(12)).view(6, 2), i(0, 3, 12, 5, -2, 10, 1, 2, 4, 6, 7, 8))
    y = g.expert_gather(plan, x, m)
    torch.cuda.synchronize()
    assert plan.status() == g.ERR_BAD_INDEX
    want = x[torch.div(m.source.clamp(0, 11), 2, rounding_mode="floor").long()]
    want[[2, 4]] = 0
    assert torch.equal(y, want)
    m = m._replace(rows=i(0, 1, 2, 3, 12, 5, -7, 7, 8, 9, 10, 11).view(6, 2))
    s = rand(2, 12, 40)
    y = g.expert_combine(plan, s, m)
    torch.cuda.synchronize()
    assert plan.status() == g.ERR_BAD_INDEX and plan.status() == g.OK
    want = s.view(6, 2, 40).clone()
    want[2, 0] = want[3, 0] = 0
    assert torch.equal(y, want.sum(1))


def forth(x, source, choices):
    at = source.long()
    return torch.where((at >= 0)[:, None], x[(at // choices).clamp(min=0)], 0)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("weights", ["none", "f32", "same"])
@pytest.mark.parametrize("tokens,choices,experts,cols,align", [
    (1, 1, 1, 1, 1), (7, 3, 4, 8, 16), (50, 5, 16, 333, 1), (200, 8, 64, 2048, 128),
    (300, 2, 3, 1028, 16)])
def test_there_and_back_with_gradients(g, plan, tokens, choices, experts, cols, align, weights, dtype):
    p = picks_of(cols, tokens, choices, experts)
    p[tokens // 2] = -1                               # a token that visits none
    x = rand(1, tokens, cols, dtype=F32).clamp(-60, 60).to(dtype).requires_grad_()
    w = None if weights == "none" else torch.rand(
        p.shape, generator=gen(5), device="cuda").to(F32 if weights == "f32" else dtype)
    if w is not None:
        w.requires_grad_()
    m = g.expert_maps(plan, p, experts, align=align)
    s = g.expert_gather(plan, x, m)
    assert torch.equal(s, forth(x.detach(), m.source, choices))
    # Rows of their own, not the tokens': one for each expert's answer.
    z = (s.detach() * 1).requires_grad_()
    with torch.no_grad():
        z += torch.rand(z.shape, generator=gen(6), device="cuda").to(dtype)
    y = g.expert_combine(plan, z, m, w)
    there = (p >= 0)[..., None]
    W = torch.ones(p.shape, dtype=torch.float64, device="cuda") if w is None else w.detach().double()
    Z = z.detach().double()[m.rows.clamp(min=0).long()] * there
    want, size = (Z * W[..., None]).sum(1), (Z * W[..., None]).abs().sum(1)
    # FP32: each addition, a fused multiply-add, rounds once; then the result.
    h = ref.half_step(dtype)
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    fp32 = choices * 2.0 ** -24 * size
    assert ((y.detach().double() - want).abs() <= fp32 * (1 + h) + h * want.abs() + tiny).all()

    dy = torch.randn(y.shape, generator=gen(8), device="cuda").to(dtype)
    grads = torch.autograd.grad(y, [z] if w is None else [z, w], dy, retain_graph=True)
    DY = dy.double()
    at = m.source.long()
    real = (at >= 0)[:, None]
    dz = torch.where(real, DY[(at // choices).clamp(min=0)] * W.reshape(-1)[at.clamp(min=0)][:, None], 0)
    # a product in FP32, then the type
    assert ((grads[0].double() - dz).abs() <= (h + 2.0 ** -24 * (1 + h)) * dz.abs() + tiny).all()
    assert (grads[0][at < 0] == 0).all()
    if w is not None:
        dw = (Z * DY[:, None]).sum(-1)
        size = (Z * DY[:, None]).abs().sum(-1)
        hw = ref.half_step(w.dtype)
        # cols fused additions in any order
        err = cols * 2.0 ** -24 * size
        assert ((grads[1].double() - dw).abs() <= err * (1 + hw) + hw * dw.abs()
                + torch.finfo(w.dtype).smallest_normal).all()
        assert (grads[1][p < 0] == 0).all()
    # the way there's gradient: the sum over a token's rows
    ds = torch.randn(s.shape, generator=gen(9), device="cuda").to(dtype)
    dx, = torch.autograd.grad(s, x, ds)
    DS = ds.double()[m.rows.clamp(min=0).long()] * there
    want, size = DS.sum(1), DS.abs().sum(1)
    assert ((dx.double() - want).abs() <= choices * 2.0 ** -24 * size * (1 + h) + h * want.abs()).all()
    assert plan.status() == g.OK


def test_gradients_against_differences(g, plan):
    """y is linear in the rows and in the weights: differences of integers, exact."""
    p = picks_of(1, 40, 3, 5)
    m = g.expert_maps(plan, p, 5, align=8)
    r = gen(2)
    ints = lambda *s: torch.randint(-8, 9, s, generator=r, device="cuda").float()
    x, w, ex, ew, dy = ints(40, 64), ints(40, 3), ints(40, 64), ints(40, 3), ints(40, 64)
    f = lambda x, w: g.expert_combine(plan, g.expert_gather(plan, x, m), m, w)
    x.requires_grad_(), w.requires_grad_()
    dx, dw = torch.autograd.grad(f(x, w), (x, w), dy)
    x, w = x.detach(), w.detach()
    assert ((f(x + ex, w) - f(x, w)) * dy).sum() == (dx * ex).sum()
    assert ((f(x, w + ew) - f(x, w)) * dy).sum() == (dw * ew).sum()


def test_gradients_of_gradients(g, plan):
    p = picks_of(3, 30, 2, 4, none=0.0)
    m = g.expert_maps(plan, p, 4)
    x = torch.randn(30, 16, device="cuda", requires_grad=True)
    y = g.expert_combine(plan, g.expert_gather(plan, x, m), m)       # 2 x
    dx, = torch.autograd.grad(y.pow(3).sum(), x, create_graph=True)
    ddx, = torch.autograd.grad(dx.sum(), x)
    torch.testing.assert_close(ddx, 48 * x.detach())
    w = torch.rand(30, 2, device="cuda", requires_grad=True)
    y = g.expert_combine(plan, g.expert_gather(plan, x, m), m, w)
    dw, = torch.autograd.grad(y.sum(), w, create_graph=True)
    with pytest.raises(RuntimeError):                  # torch's: no way from dw to x
        torch.autograd.grad(dw.sum(), x, retain_graph=True)
    with pytest.raises(RuntimeError, match="first gradients only"):
        dw.sum().backward()


# ------------------------------------------------------------------ linear layers

def linear_grads(x, w, dy, formats=(E4, E4)):
    """(Y, dX, dW) in 64 bits with bounds, from the codes that each product takes."""
    v = lambda t, kind, f: (lambda c, s: c.double() * ref.spread(s, c, kind))(*ref.quantize(t, kind, f))
    xr, xc, wq = v(x, "rows", formats[0]), v(x, "columns", formats[0]), v(w, "tiles", formats[0])
    gr, gc = v(dy, "rows", formats[1]), v(dy, "columns", formats[1])
    return (xr, wq.t()), (gr, wq), (gc.t(), xc)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("shape,n,formats", [((1, 64), 64, (E4, E4)), ((5, 3, 200), 300, (E4, E5)),
                                             ((300, 1000), 264, (E4, E4)), ((257, 129), 17, (E5, E5))])
def test_linear(g, plan, shape, n, formats, dtype):
    x = torch.randn(shape, generator=gen(1), device="cuda").to(dtype).requires_grad_()
    w = (torch.randn(n, shape[-1], generator=gen(2), device="cuda") * 0.1).to(dtype).requires_grad_()
    y = g.linear_f8(plan, x, w, dtype=formats[0], grad_dtype=formats[1])
    assert y.shape == (*shape[:-1], n) and y.dtype == dtype
    dy = torch.randn(y.shape, generator=gen(3), device="cuda").to(dtype)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    assert dx.shape == x.shape and dw.shape == w.shape
    flat = lambda t: t.detach().reshape(-1, t.shape[-1])
    for got, (a, b) in zip((flat(y), flat(dx), dw), linear_grads(flat(x), w.detach(), flat(dy), formats)):
        ref.check_product(got, a, b)
    # each gradient alone, and with W quantised beforehand: the same bits
    for inputs, want in (([x], dx), ([w], dw)):
        other = x.detach() if inputs[0] is w else x
        y2 = g.linear_f8(plan, other, w if inputs[0] is w else w.detach(), dtype=formats[0],
                         grad_dtype=formats[1])
        assert torch.equal(y2, y) and torch.equal(torch.autograd.grad(y2, inputs, dy)[0], want)
    q = g.quantize(plan, w.detach(), "tiles", formats[0])
    y3 = g.linear_f8(plan, x, q, dtype=formats[0], grad_dtype=formats[1])
    assert torch.equal(y3, y) and torch.equal(torch.autograd.grad(y3, x, dy)[0], dx)
    with torch.no_grad():
        assert not g.linear_f8(plan, x, w).requires_grad
    assert not g.linear_f8(plan, x.detach(), q, dtype=formats[0]).requires_grad


def test_linear_gradients_against_differences(g, plan):
    """Numbers that 8 bits hold exactly (each block's largest is 448, the others
    small whole numbers): Y is linear in them, and so its differences are exact."""
    r = gen(4)

    def exact(*shape):
        t = torch.randint(-8, 9, shape, generator=r, device="cuda").float()
        t[::1, ::128] = 448.0     # along rows; and with it in tiles
        t[::128] = 448.0          # along columns
        return t

    x, w, dy = exact(256, 256), exact(384, 256), exact(256, 384)
    change = torch.zeros_like(x)
    change[5, 9], change[200, 131] = 4.0, -3.0
    more = torch.zeros_like(w)
    more[70, 3], more[300, 200] = 2.0, 5.0
    x.requires_grad_(), w.requires_grad_()
    dx, dw = torch.autograd.grad(g.linear_f8(plan, x, w), (x, w), dy)
    x, w = x.detach(), w.detach()
    f = lambda x, w: g.linear_f8(plan, x, w).double()
    assert ((f(x + change, w) - f(x, w)) * dy).sum() == (dx * change).double().sum()
    assert ((f(x, w + more) - f(x, w)) * dy).sum() == (dw * more).double().sum()


def test_a_gradient_that_is_one_number_and_one_that_is_strided(g, plan):
    x = torch.randn(130, 200, device="cuda", requires_grad=True)
    w = torch.randn(96, 200, device="cuda", requires_grad=True)
    y = g.linear_f8(plan, x, w)
    for dy in (torch.ones((), device="cuda").expand(130, 96), torch.randn(96, 130, device="cuda").t()):
        got = torch.autograd.grad(y, (x, w), dy, retain_graph=True)
        want = torch.autograd.grad(y, (x, w), dy.contiguous(), retain_graph=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_second_gradient_is_refused(g, plan):
    x = torch.randn(20, 64, device="cuda", requires_grad=True)
    w = torch.randn(32, 64, device="cuda", requires_grad=True)
    dx, = torch.autograd.grad(g.linear_f8(plan, x, w).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="first gradients only"):
        dx.sum().backward()


def test_a_graph_keeps_its_plan_and_says_when_it_is_closed(g):
    x = torch.randn(20, 64, device="cuda", requires_grad=True)
    w = torch.randn(32, 64, device="cuda")
    p = g.Plan(0)
    first, second = (g.linear_f8(p, x, w) for _ in range(2))
    torch.autograd.grad(first.sum(), x)
    p.close()
    with pytest.raises(RuntimeError, match="closed"):
        torch.autograd.grad(second.sum(), x)
    y = g.linear_f8(g.Plan(0), x, w)
    torch.autograd.grad(y.sum(), x)


# ------------------------------------------------------------------ a layer of experts

def layer(g, plan, x, picks, w, up, down, align, stream=None):
    """Tokens to their experts, two 8-bit products with a square between, and back."""
    kw = dict(stream=stream)
    m = g.expert_maps(plan, picks, up.shape[0], align=align, **kw)
    s = g.expert_gather(plan, x, m, **kw)
    h = g.linear_f8(plan, s, up, starts=m.starts, **kw)
    return g.expert_combine(plan, g.linear_f8(plan, h, down, starts=m.starts, **kw), m, w, **kw), m, s, h


def layer_inputs(seed, tokens=150, choices=2, experts=5, k=136, n=200, dtype=BF16):
    r = gen(seed)
    t = lambda *s, f=1.0: (torch.randn(s, generator=r, device="cuda") * f).to(dtype)
    w = torch.softmax(torch.randn(tokens, choices, generator=r, device="cuda"), 1)
    picks = picks_of(seed, tokens, choices, experts)
    picks[picks == 3] = 0                             # an expert that no token visits
    return t(tokens, k), picks, w, t(experts, n, k, f=k ** -0.5), t(experts, k, n, f=n ** -0.5)


def test_a_layer_of_experts_and_its_gradients(g, plan):
    """Each call's result from what it was given, in 64 bits, through the whole
    layer forward and backward."""
    x, picks, w, up, down = layer_inputs(1)
    leaves = [t.requires_grad_() for t in (x, w, up, down)]
    y, m, s, h = layer(g, plan, x, picks, w, up, down, 128)
    z = g.linear_f8(plan, h, down, starts=m.starts)
    s.retain_grad(), h.retain_grad(), z.retain_grad()
    y = g.expert_combine(plan, z, m, w)
    dy = torch.randn(y.shape, generator=gen(2), device="cuda").to(y.dtype)
    got = torch.autograd.grad(y, (*leaves, s, h, z), dy)
    dx, dw, dup, ddown, ds, dh, dz = got
    at = m.starts.tolist()
    for e in range(up.shape[0]):
        r = slice(at[e], at[e + 1])
        for inp, weight, out, dout, din, dweight in ((s, up, h, dh, ds, dup),
                                                     (h, down, z, dz, dh, ddown)):
            if r.start == r.stop:
                assert (dweight[e] == 0).all()
                continue
            three = linear_grads(inp.detach()[r], weight.detach()[e], dout[r])
            for c, (a, b) in zip((out.detach()[r], din[r], dweight[e]), three):
                ref.check_product(c, a, b)
    assert (dz[at[-1]:] == 0).all() and (ds[at[-1]:] == 0).all()
    there = (picks >= 0)[..., None]
    want = (ds.double()[m.rows.clamp(min=0).long()] * there).sum(1)
    assert ((dx.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -22 * ds.abs().max()).all()
    assert plan.status() == g.OK


@pytest.mark.parametrize("tokens", [0, 1, 48])
def test_a_generation_step(g, plan, tokens):
    """No gradients, rows without filling: the same as token by token."""
    x, picks, w, up, down = layer_inputs(3, tokens=tokens, dtype=F16)
    ups, downs = g.quantize(plan, up, "tiles"), g.quantize(plan, down, "tiles")
    y, m, _, _ = layer(g, plan, x, picks, w, up, down, 1)
    s = g.quantize(plan, x, maps=m)                   # sorted and quantised in one
    hq = g.quantize(plan, g.matmul_f8(plan, s, ups.t(), starts=m.starts))
    z = g.matmul_f8(plan, hq, downs.t(), starts=m.starts)
    assert torch.equal(g.expert_combine(plan, z, m, w), y)
    for t in range(0, tokens, 7):
        one = layer(g, plan, x[t:t + 1], picks[t:t + 1], w[t:t + 1], up, down, 1)[0]
        assert torch.equal(one, y[t:t + 1])
    assert plan.status() == g.OK


def test_a_captured_layer_follows_its_tokens(g, plan):
    """A training step in a graph: other tokens, other choices, the same shapes."""
    fixed = [t.requires_grad_() if t.is_floating_point() else t for t in layer_inputs(5)]
    dy = torch.randn(150, 136, generator=gen(6), device="cuda").to(BF16)

    def step(x, picks, w, up, down):
        y = layer(g, plan, x, picks, w, up, down, 128)[0]
        return (y, *torch.autograd.grad(y, (x, w, up, down), dy))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step(*fixed)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        outs = step(*fixed)
    for seed in (7, 8):
        fresh = [t.requires_grad_() if t.is_floating_point() else t for t in layer_inputs(seed)]
        with torch.no_grad():
            for a, b in zip(fixed, fresh):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, step(*fresh)))
    assert plan.status() == g.OK


def test_on_a_stream_of_its_own(g, plan):
    """The calls' work, and the backward pass's, is on the given stream."""
    data = layer_inputs(9)
    want = layer(g, plan, *data, 128)[0]
    s = torch.cuda.Stream()
    leaves = [t.requires_grad_() if t.is_floating_point() else t for t in data]
    torch.cuda.synchronize()
    y = layer(g, plan, *leaves, 128, stream=s)[0]
    s.synchronize()
    assert torch.equal(y, want)
    with torch.cuda.stream(s):
        a = torch.autograd.grad(y.float().square().sum(), leaves[0])[0]
    torch.cuda.synchronize()
    b = torch.autograd.grad(layer(g, plan, *leaves, 128)[0].float().square().sum(), leaves[0])[0]
    assert torch.equal(a, b)


@pytest.mark.parametrize("m", [40, 300])
def test_linear_of_transposed_views(g, plan, m):
    """X and W as views of their transposes: the same bits, gradients too."""
    x = torch.randn(m, 200, generator=gen(21), device="cuda").to(BF16)
    w = torch.randn(130, 200, generator=gen(22), device="cuda").to(BF16)
    dy = torch.randn(m, 130, generator=gen(23), device="cuda").to(BF16)

    def run(x, w):
        x, w = x.detach().requires_grad_(), w.detach().requires_grad_()
        y = g.linear_f8(plan, x, w)
        return (y, *torch.autograd.grad(y, (x, w), dy))

    want = run(x, w)
    turned = lambda t: t.t().contiguous().t()
    for a, b in ((turned(x), w), (x, turned(w)), (turned(x), turned(w))):
        got = run(a, b)
        # another kernel may add a block's parts in another order
        for c, d in zip(got, want):
            assert c.shape == d.shape
        for c, (p, q) in zip(got, linear_grads(x, w, dy)):
            ref.check_product(c.detach(), p, q)


def test_no_tokens(g, plan):
    """Nothing to do forward; the gradients of weights are 0."""
    x = torch.zeros(0, 136, dtype=BF16, device="cuda", requires_grad=True)
    w = torch.randn(200, 136, device="cuda").to(BF16).requires_grad_()
    y = g.linear_f8(plan, x, w)
    dx, dw = torch.autograd.grad(y, (x, w), torch.zeros_like(y))
    assert y.shape == (0, 200) and dx.shape == (0, 136) and (dw == 0).all()
    _, _, _, up, down = layer_inputs(1)
    up.requires_grad_(), down.requires_grad_()
    picks = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    wt = torch.zeros(0, 2, device="cuda", requires_grad=True)
    y = layer(g, plan, x, picks, wt, up, down, 128)[0]
    got = torch.autograd.grad(y, (x, wt, up, down), torch.zeros_like(y))
    assert y.shape == (0, 136) and all((t == 0).all() for t in got)
    assert plan.status() == g.OK


@pytest.mark.parametrize("m,n,k", [(129, 300, 4100), (1000, 1024, 8192), (300, 2049, 2600)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_products_of_cut_tiles(g, plan, m, n, k, dtype):
    """Few tiles and many blocks: every kind of result, from parts joined after."""
    a = torch.randn(m, k, generator=gen(31), device="cuda") * k ** -0.5
    b = torch.randn(n, k, generator=gen(32), device="cuda")
    A = g.quantize(plan, a)
    for B in (g.quantize(plan, b, "tiles").t(), g.quantize(plan, b, "rows").t()):
        room = torch.full((m + 2, n + 24), 7.0, dtype=dtype, device="cuda")
        c = room[1:-1, 8:n + 8]
        g.matmul_f8(plan, A, B, c)
        ref.check_product(c, ref.values(A), ref.values(B))
        c.fill_(7.0)
        assert (room == 7.0).all()
