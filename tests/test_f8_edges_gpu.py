"""8-bit products, linear layers and experts' rows on the GPU where a call is at
the edge of what it takes: bad starts, mistakes that must not pass for results."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
from tests import f8_ref as ref  # noqa: E402
from tests.test_f8_gpu import E4, BF16, F16, F32, g, gen, operands, plan, rand  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ bad starts

@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("starts,bad", [
    ([0, 128, 200, 512, 640, 700], [1, 2]), ([0, 100, 100, 256, 384, 700], [0, 1, 2]),
    ([0, 128, 0, 256, 512, 700], [1]), ([0, 128, 256, 384, 512, 640], []),
    ([-128, 128, 256, 384, 512, 768], [0, 4])])
def test_the_matrix_of_an_expert_with_bad_inner_starts_is_nan(g, plan, starts, bad, dtype):
    """And the others' are right: an end inside a block spoils both its experts."""
    m, n, room = 300, 140, 700
    for turned in (False, True):
        x, y = rand(1, room, m) * 1e-3, rand(2, room, n) * 1e-3
        A = g.quantize(plan, x, "columns").t()
        B = g.quantize(plan, y, "tiles" if turned else "columns")
        a, b = ref.values(A, "rows"), ref.values(B, "tiles" if turned else "columns")
        A = A._replace(scales=(A.scales / (a.abs() @ b.abs()).max() * 1e3).float())
        a = ref.values(A, "rows")
        c = g.matmul_f8(plan, A, B, dtype=dtype, starts=i32(*starts))
        torch.cuda.synchronize()
        assert plan.status() == (g.ERR_BAD_INDEX if bad else g.OK) and plan.status() == g.OK
        for e, (lo, hi) in enumerate(zip(starts, starts[1:])):
            if e in bad:
                assert c[e].isnan().all()
            else:
                ref.check_product(c[e], a[:, lo:hi], b[lo:hi])
    old = torch.ones(len(starts) - 1, m, n, device="cuda")
    g.matmul_f8(plan, A, B, old, starts=i32(*starts), accumulate=True)
    torch.cuda.synchronize()
    assert plan.status() == (g.ERR_BAD_INDEX if bad else g.OK) and plan.status() == g.OK
    assert old.isnan().flatten(1).all(1).nonzero().flatten().tolist() == bad
    assert old.isnan().flatten(1).any(1).nonzero().flatten().tolist() == bad


def test_weights_of_experts_with_rows_out_of_step_have_no_gradient_of_zeros(g, plan):
    """Starts as they come from expert_maps without align=128."""
    x = torch.randn(50, 136, generator=gen(3), device="cuda")
    w = torch.randn(4, 64, 136, generator=gen(4), device="cuda", requires_grad=True)
    m = g.expert_maps(plan, torch.arange(100, device="cuda").view(50, 2) % 4, 4)
    y = g.linear_f8(plan, g.expert_gather(plan, x, m), w, starts=m.starts)
    dw, = torch.autograd.grad(y.sum(), w)
    torch.cuda.synchronize()
    assert dw.isnan().all()
    assert plan.status() == g.ERR_BAD_INDEX and plan.status() == g.OK


@pytest.mark.parametrize("times", [1, 20])         # the kernels for few and for many rows
@pytest.mark.parametrize("starts,good", [
    ([0, 40, 20], [0]), ([0, 40, -1], [0]), ([0, 40, 20, 60], [0]), ([0, 20, 40, 61], [0, 1]),
    ([-1, 20, 40, 60], [1, 2]), ([0, 30, 10, 30, 50], [0, 3]), ([0, 61, 5, 25, 60], [2, 3]),
    ([10, 30, 20, 25, 20, 40], [0]), ([70, 65, 3], []), ([5, 5, 3, 5, 60], [0, 3])])
def test_bad_starts_leave_the_other_experts_rows(g, plan, starts, good, times):
    """Rows of each expert whose starts are good, also where the last start is a
    bad one, or another expert's range would hold the same rows; 0 behind them."""
    room, experts = 60 * times, len(starts) - 1
    starts = [times * s for s in starts]
    A = g.quantize(plan, rand(1, room, 300))
    B = g.quantize(plan, rand(2, experts, 300, 200), "tiles")
    a, b = ref.values(A), ref.values(B)
    for _ in range(3):
        c = torch.full((room, 200), 7.0, device="cuda")
        g.matmul_f8(plan, A, B, c, starts=i32(*starts))
        torch.cuda.synchronize()
        assert plan.status() == g.ERR_BAD_INDEX and plan.status() == g.OK
        for e in good:
            lo, hi = starts[e:e + 2]
            ref.check_product(c[lo:hi], a[lo:hi], b[e])
        if good:
            assert (c[max(starts[e + 1] for e in good):] == 0).all()
        else:
            assert (c == 7.0).all()


def test_many_experts_whose_ranges_overlap(g, plan):
    """Every other range is all rows: the first of them is stored, once."""
    starts = [0, 500] * 200
    A = g.quantize(plan, rand(1, 500, 128))
    w = rand(2, len(starts) - 1, 128, 16)
    B = g.quantize(plan, w, "tiles")
    c = torch.full((500, 16), 7.0, device="cuda")
    g.matmul_f8(plan, A, B, c, starts=i32(*starts))
    torch.cuda.synchronize()
    assert plan.status() == g.ERR_BAD_INDEX and plan.status() == g.OK
    ref.check_product(c, ref.values(A), ref.values(B)[0])


def test_linear_of_maps_is_that_of_their_starts(g, plan):
    x = torch.randn(50, 136, generator=gen(3), device="cuda").to(BF16)
    w = torch.randn(4, 64, 136, generator=gen(4), device="cuda").to(BF16).requires_grad_()
    picks = torch.arange(100, device="cuda").view(50, 2) % 4
    m = g.expert_maps(plan, picks, 4, align=128)
    assert m.align == 128
    s = g.expert_gather(plan, x, m)
    got, want = (g.linear_f8(plan, s, w, starts=t) for t in (m, m.starts))
    assert torch.equal(got, want)
    assert all(torch.equal(torch.autograd.grad(y.float().sum(), w)[0],
                           torch.autograd.grad(want.float().sum(), w, retain_graph=True)[0])
               for y in (got,))
    m = g.expert_maps(plan, picks, 4)
    assert m.align == 1
    with pytest.raises(ValueError, match="align=128"):
        g.linear_f8(plan, g.expert_gather(plan, x, m), w, starts=m)
    assert g.linear_f8(plan, g.expert_gather(plan, x, m), w.detach(), starts=m).shape == (100, 64)
    assert plan.status() == g.OK


# ------------------------------------------------------------------ derivatives

def test_a_tangent_of_a_gradient_is_refused(g, plan):
    """Forward over reverse: the gradient that arrives carries a tangent."""
    import torch.autograd.forward_ad as fwd
    x = torch.randn(20, 64, device="cuda", requires_grad=True)
    w = torch.randn(32, 64, device="cuda", requires_grad=True)
    m = g.expert_maps(plan, torch.zeros(20, 2, dtype=torch.int32, device="cuda"), 2)
    weights = torch.ones(20, 2, device="cuda", requires_grad=True)
    s = g.expert_gather(plan, x, m)
    for y, leaf in ((g.linear_f8(plan, x, w), x), (s, x), (g.expert_combine(plan, s, m), x),
                    (g.expert_combine(plan, s.detach(), m, weights), weights)):
        with fwd.dual_level(), pytest.raises(RuntimeError, match="forward-mode"):
            dy = fwd.make_dual(torch.ones_like(y), torch.ones_like(y))
            torch.autograd.grad(y, leaf, dy, retain_graph=True)


# ------------------------------------------------------------------ few SMs

@pytest.mark.parametrize("limit", [1, 2, 3, 24])
def test_cut_tiles_and_shared_tiles_on_a_few_sms(g, limit):
    """Joined by fewer CTAs than there are pieces; experts' rows by one CTA an SM."""
    with g.Plan(0) as p:
        p.set_option(g.OPT_SM_LIMIT, limit)
        for m, n, k, kind in ((300, 700, 4100, "forward"), (300, 700, 4100, "weights"),
                              (5, 700, 4100, "forward")):
            A, B = operands(g, p, 71, m, n, k, kind)
            c = [g.matmul_f8(p, A, B, dtype=F32) for _ in range(2)]
            ref.check_product(c[0], ref.values(A), ref.values(B))
            assert torch.equal(*c)
        A = g.quantize(p, rand(1, 90, 400))
        B = g.quantize(p, rand(2, 3, 400, 300), "tiles")
        c = g.matmul_f8(p, A, B, dtype=F32, starts=i32(0, 40, 41, 90))
        for e, (lo, hi) in enumerate(((0, 40), (40, 41), (41, 90))):
            ref.check_product(c[lo:hi], ref.values(A)[lo:hi], ref.values(B)[e])
        assert p.status() == g.OK


def test_a_plan_launches_what_the_host_says(g, plan):
    """The choice for the device's own facts, and the workspace that goes with it."""
    for m, n, k in ((300, 700, 4100), (5, 700, 4100), (1000, 1024, 8192)):
        c = g.gemm_f8_run_choice(g.F8_DENSE, m, n, k, num_sms=plan.get_option(g.INFO_NUM_SMS))
        bytes_ = g.gemm_f8_workspace(plan.handle, g.F8_DENSE, m, n, k)
        assert (bytes_ > 0) == (c["join_ctas"] > 0)
        if bytes_:
            assert bytes_ == c["join_ctas"] // 16 * c["parts"] * 256 * 256 * 4


# ------------------------------------------------------------------ a given C

def test_a_given_result_that_a_graph_has_saved_is_noticed(g, plan):
    A, B = operands(g, plan, 5, 20, 64, 128)
    c, w = torch.randn(20, 64, device="cuda"), torch.randn(20, 64, device="cuda", requires_grad=True)
    y = (w * c).sum()
    g.matmul_f8(plan, A, B, c, accumulate=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        d = torch.zeros(20, 64, device="cuda")
    g.matmul_f8(plan, A, B, d)
    assert torch.equal(d, g.matmul_f8(plan, A, B, dtype=F32))


def test_a_result_whose_matrices_share_their_place_is_refused(g, plan):
    A, B = operands(g, plan, 6, 40, 64, 256, "weights")
    one = torch.full((1, 40, 64), 7.0, device="cuda")
    with pytest.raises(ValueError, match="place for each"):
        g.matmul_f8(plan, A, B, one.expand(2, 40, 64), starts=i32(0, 128, 256))
    g.matmul_f8(plan, A, B, one, starts=i32(0, 256))
    assert torch.equal(one[0], g.matmul_f8(plan, A, B, dtype=F32))
    beside = torch.full((40, 2, 64), 7.0, device="cuda").transpose(0, 1)     # rows in turn
    g.matmul_f8(plan, A, B, beside, starts=i32(0, 128, 256))
    for e in range(2):
        r = slice(128 * e, 128 * e + 128)
        ref.check_product(beside[e], ref.values(A, "rows")[:, r], ref.values(B, "columns")[r])


@pytest.mark.parametrize("experts", [0, 3])
def test_weights_without_rows(g, plan, experts):
    """A result of no columns: X's gradient is 0."""
    x = torch.randn(10, 72, device="cuda").to(BF16).requires_grad_()
    w = torch.zeros((experts, 0, 72) if experts else (0, 72), device="cuda", requires_grad=True)
    m = g.expert_maps(plan, torch.arange(5, device="cuda")[:, None] % 3, 3, align=128) if experts else None
    if experts:
        x = torch.randn(m.source.numel(), 72, device="cuda").to(BF16).requires_grad_()
    y = g.linear_f8(plan, x, w, starts=m)
    assert y.shape == (x.shape[0], 0) and y.dtype == BF16
    dx, dw = torch.autograd.grad(y, (x, w), torch.zeros_like(y))
    assert dx.shape == x.shape and dx.dtype == BF16 and (dx == 0).all()
    assert dw.shape == w.shape and dw.dtype == w.dtype
    dx, = torch.autograd.grad(g.linear_f8(plan, x, w.detach(), starts=m).sum(), x)
    assert (dx == 0).all()
    assert plan.status() == g.OK


# ------------------------------------------------------------------ launches that overlap

def test_a_chain_of_calls_through_the_same_buffers(g, plan):
    """Quantisation, product, quantisation into the same codes and scales, product,
    ..., nothing between: each launch starts beside the end of the one before."""
    s = torch.cuda.current_stream().cuda_stream
    m, k, n = 16, 4096, 2048
    W = g.quantize(plan, torch.randn(n, k, generator=gen(1), device="cuda"), "tiles").t()
    xs = [torch.randn(m, k, generator=gen(2 + i), device="cuda") * 10 ** i for i in range(4)]
    want = [g.matmul_f8(plan, g.quantize(plan, x), W, dtype=F32) for x in xs]
    q, outs = g.quantize(plan, xs[0]), [torch.empty(m, n, device="cuda") for _ in xs]
    torch.cuda.synchronize()
    for _ in range(50):
        for x, c in zip(xs, outs):
            g.gemm_f8_quantize(plan.handle, g.F8_ROWS, g.F8_E4M3, 2, 1, m, k, x.data_ptr(), k, 0, 0, 1,
                               0, q.data.data_ptr(), k, 0, q.scales.data_ptr(), stream=s)
            g.matmul_f8(plan, q, W, c)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert plan.status() == g.OK


# ------------------------------------------------------------------ the largest sizes

def test_matrices_of_more_numbers_than_32_bits_count(g, plan):
    """The last rows of 262,149 by 8200 numbers, of codes and of results."""
    rows, cols = 2 ** 18 + 5, 8200
    end = slice(rows - 300, rows)
    x = torch.zeros(rows, cols, dtype=F16, device="cuda")
    x[end] = torch.randn(300, cols, generator=gen(1), device="cuda").half()
    for blocks in ("rows", "both"):
        q = g.quantize(plan, x, blocks)
        q = q[0] if blocks == "both" else q
        codes, scales = ref.quantize(x[end], "rows", E4)
        assert torch.equal(q.data[end].view(torch.uint8), codes.view(torch.uint8))
        assert torch.equal(q.scales[end], scales)
    at = (rows - 300) // 128 * 128
    for b, kind in ((g.quantize(plan, x, "tiles"), "tiles"), (g.quantize(plan, x, "columns"), "columns")):
        codes, scales = ref.quantize(x[at:], kind, E4)
        assert torch.equal(b.data[at:].view(torch.uint8), codes.view(torch.uint8))
        assert torch.equal(b.scales[at // 128:], scales)
    del b, codes, scales
    # a result as large, dense and by experts' rows
    A = g.quantize(plan, torch.randn(rows, 130, generator=gen(2), device="cuda").half())
    B = g.quantize(plan, torch.randn(2, 130, cols, generator=gen(3), device="cuda"), "tiles")
    a, b = ref.values(g.Blocks(A.data[end], A.scales[end])), ref.values(B)
    c = g.matmul_f8(plan, A, g.Blocks(B.data[0], B.scales[0]), x)
    ref.check_product(c[end], a, b[0])
    x.zero_()
    c = g.matmul_f8(plan, A, B, x, starts=i32(0, rows - 200, rows))
    ref.check_product(c[end][:100], a[:100], b[0])
    ref.check_product(c[end][100:], a[100:], b[1])
    # rows there and back
    picks = torch.arange(rows, device="cuda").int()[:, None] % 2
    m = g.expert_maps(plan, picks, 2)
    s = g.expert_gather(plan, x, m)
    assert torch.equal(s[end], x[m.source[end].long()])
    assert torch.equal(g.expert_combine(plan, s, m)[end], x[end])
    assert plan.status() == g.OK


@pytest.mark.parametrize("m", [3000, 200000])
def test_as_many_experts_as_there_may_be(g, plan, m):
    """1024 experts, half of them without rows."""
    e = torch.arange(1024, device="cuda")
    lengths = torch.where(e % 2 == 0, 0, m // 512 - (e % 3))
    starts = torch.cat((torch.zeros(1, device="cuda"), lengths.cumsum(0))).int()
    A = g.quantize(plan, torch.randn(m, 130, generator=gen(1), device="cuda"))
    B = g.quantize(plan, torch.randn(1024, 130, 72, generator=gen(2), device="cuda"), "tiles")
    c = g.matmul_f8(plan, A, B, dtype=F32, starts=starts)
    at = starts.tolist()
    a, b = ref.values(A), ref.values(B)
    for i in list(range(0, 1024, 97)) + [1022, 1023]:
        ref.check_product(c[at[i]:at[i + 1]], a[at[i]:at[i + 1]], b[i])
    assert (c[at[-1]:] == 0).all()
    inner = torch.cat((torch.zeros(1, device="cuda"), torch.where(e % 2 == 0, 0, 128).cumsum(0))).int()
    k = 512 * 128
    A = g.quantize(plan, torch.randn(k, 40, generator=gen(3), device="cuda"), "columns").t()
    B = g.quantize(plan, torch.randn(k, 72, generator=gen(4), device="cuda"), "columns")
    c = g.matmul_f8(plan, A, B, dtype=F32, starts=inner)
    a, b = ref.values(A, "rows"), ref.values(B, "columns")
    for i in (0, 1, 2, 511, 777, 1023):
        r = slice(inner[i].item(), inner[i + 1].item())
        ref.check_product(c[i], a[:, r], b[r])
    assert plan.status() == g.OK


def test_one_kernel_time_for_each_product(g):
    """The product's, without the join of cut tiles."""
    with g.Plan(0) as p:
        calls = [operands(g, p, 7, m, n, k) for m, n, k in ((5, 300, 1000), (300, 700, 4100), (300, 700, 400))]
        p.set_option(g.OPT_KERNEL_TIMING, 1)
        for A, B in calls:
            g.matmul_f8(p, A, B)
            ms, count = p.kernel_time()
            assert count == 1 and 0 < ms < 1000


@pytest.mark.parametrize("m", [65, 300])
def test_linear_of_transposed_views_has_the_same_bits(g, plan, m):
    """Above 64 rows the same kernel takes X and W either way."""
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
        for c, d in zip(run(a, b), want):
            assert torch.equal(c, d)
