"""8-bit blocks and their products on the GPU against 64 bits (f8_ref)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
from tests import f8_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
E4, E5 = ref.E4, ref.E5
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g():
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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(seed, *shape, dtype=F32):
    """Numbers of sizes that differ by row and column, some of them 0."""
    r = gen(seed)
    x = torch.randn(shape, generator=r, device="cuda")
    x *= torch.exp2(3 * torch.randn(shape[-1:], generator=r, device="cuda"))
    x *= torch.exp2(3 * torch.randn((*shape[:-1], 1), generator=r, device="cuda"))
    return torch.where(torch.rand(shape, generator=r, device="cuda") < 0.02, 0.0, x).to(dtype)


def same_codes(got, want):
    """The same bits, but that any NaN is as good as another and -0 is not 0."""
    a, b = got.contiguous().view(torch.uint8), want.contiguous().view(torch.uint8)
    nan = got.float().isnan() & want.float().isnan()
    assert got.dtype == want.dtype and got.shape == want.shape
    assert ((a == b) | nan).all()


def check_blocks(got, x, blocks, dtype):
    codes, scales = ref.quantize(x, blocks, dtype)
    same_codes(got.data, codes)
    assert got.scales.shape == scales.shape and torch.equal(got.scales, scales)


# ------------------------------------------------------------------ quantize

@pytest.mark.parametrize("dtype", [E4, E5])
@pytest.mark.parametrize("type_", [F16, BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 129), (129, 16), (127, 300), (257, 1000)])
def test_quantize(g, plan, rows, cols, type_, dtype):
    x = rand(rows + cols, rows, cols, dtype=type_)
    for blocks in ("rows", "columns", "tiles"):
        check_blocks(g.quantize(plan, x, blocks, dtype), x, blocks, dtype)
    r, c = g.quantize(plan, x, "both", dtype)
    check_blocks(r, x, "rows", dtype)
    check_blocks(c, x, "columns", dtype)


@pytest.mark.parametrize("dtype", [E4, E5])
@pytest.mark.parametrize("type_", [F16, BF16, F32])
def test_quantize_of_unusual_numbers(g, plan, type_, dtype):
    """Zeros, the smallest and the largest numbers, infinities and NaN, alone in
    their blocks and beside others; a block of nothing but them."""
    x = rand(7, 300, 520, dtype=type_)
    inf, nan = float("inf"), float("nan")
    big, low = torch.finfo(type_).max, torch.finfo(type_).smallest_normal
    x[0, :128] = 0
    x[1, :128], x[1, 5] = 0, nan
    x[2, :128] = inf
    x[3, 130], x[3, 140], x[3, 150] = inf, -inf, nan
    x[4, :128], x[4, 7] = low / 2, -low
    x[5, :128], x[5, 9] = big, -big
    x[128:256, 256:384] = nan
    x[128:256, 384:512] = -inf
    x[256:, 512:] = 0
    x[:, 3] = nan
    x[:128, 4], x[17, 4] = -0.0, inf
    for blocks in ("rows", "columns", "tiles"):
        check_blocks(g.quantize(plan, x, blocks, dtype), x, blocks, dtype)
    r, c = g.quantize(plan, x, "both", dtype)
    check_blocks(r, x, "rows", dtype)
    check_blocks(c, x, "columns", dtype)


@pytest.mark.parametrize("blocks", ["rows", "columns", "tiles"])
def test_quantize_of_views_and_several_matrices(g, plan, blocks):
    room = rand(9, 3, 140, 300, dtype=BF16)
    for x in (room[0, :, 1:200], room[0, 5:, 8:264], room[0].t(), room[1, 3:77].t(), room,
              room[:, :131, 3:], room.transpose(1, 2), room[1:2], room[:, :1], room[:, :, :1]):
        check_blocks(g.quantize(plan, x, blocks), x, blocks, E4)
    r, c = g.quantize(plan, room[0].t(), "both")
    check_blocks(r, room[0].t(), "rows", E4)
    check_blocks(c, room[0].t(), "columns", E4)


@pytest.mark.parametrize("blocks", ["rows", "columns", "both"])
@pytest.mark.parametrize("cols", [40, 333])
def test_quantize_in_the_experts_order(g, plan, blocks, cols):
    x = rand(11, 50, cols, dtype=F16)
    picks = torch.randint(-1, 5, (50, 3), generator=gen(3), device="cuda").int()
    m = g.expert_maps(plan, picks, 5, align=128)
    want = g.expert_gather(plan, x, m)
    got = g.quantize(plan, x, blocks, maps=m)
    for b, kind in zip(got if blocks == "both" else (got,),
                       ("rows", "columns") if blocks == "both" else (blocks,)):
        check_blocks(b, want, kind, E4)
    assert plan.status() == g.OK


def test_quantize_of_nothing(g, plan):
    x = torch.zeros(0, 40, device="cuda")
    assert g.quantize(plan, x).data.shape == (0, 40)
    assert g.quantize(plan, x, "columns").scales.shape == (0, 40)
    with pytest.raises(ValueError):
        g.quantize(plan, torch.zeros(4, 0, device="cuda"))


# ------------------------------------------------------------------ products

def operands(g, plan, seed, m, n, k, kind="forward", a=E4, b=E4):
    """A [m, k] and B [k, n] as a program has them."""
    if kind == "weights":
        return (g.quantize(plan, rand(seed, k, m), "columns", a).t(),
                g.quantize(plan, rand(seed + 1, k, n), "columns", b))
    A = g.quantize(plan, rand(seed, m, k), "rows", a)
    if kind == "inputs":
        return A, g.quantize(plan, rand(seed + 1, k, n), "tiles", b)
    return A, g.quantize(plan, rand(seed + 1, n, k), "tiles", b).t()


def fit(g, A, B):
    """A with scales for which the largest result is 1000, in every type's range."""
    top = (ref.values(A) @ ref.values(B)).abs().max().clamp(min=1e-30)
    return g.Blocks(A.data, (A.scales.double() * (1000.0 / top)).float())


SIZES = [(1, 1, 1), (1, 100, 128), (2, 16, 127), (7, 300, 1000), (16, 128, 129), (17, 513, 256),
         (33, 129, 640), (64, 1000, 384), (65, 255, 2050), (100, 40, 300), (128, 256, 512),
         (129, 257, 513), (256, 256, 128), (300, 500, 1000), (513, 130, 100), (1000, 777, 3000)]


@pytest.mark.parametrize("kind", ["forward", "inputs", "weights"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product(g, plan, m, n, k, kind):
    formats = [(E4, E4), (E5, E4), (E4, E5), (E5, E5)][(m + n) % 4]
    A, B = operands(g, plan, m + k, m, n, k, kind, *formats)
    for dtype in (F32, BF16, F16):
        c = g.matmul_f8(plan, A, B, dtype=dtype)
        assert c.shape == (m, n) and c.dtype == dtype
        a, b = ref.values(A), ref.values(B)
        if dtype == F16:
            A = fit(g, A, B)
            c, a = g.matmul_f8(plan, A, B, dtype=dtype), ref.values(A)
        ref.check_product(c, a, b)
    assert plan.status() == g.OK


@pytest.mark.parametrize("m", [48, 300])
@pytest.mark.parametrize("sa", ["rows", "tiles"])
@pytest.mark.parametrize("sb", ["columns", "tiles"])
@pytest.mark.parametrize("turned_a", [False, True])
@pytest.mark.parametrize("turned_b", [False, True])
def test_product_with_each_kind_of_scales(g, plan, m, sa, sb, turned_a, turned_b):
    n, k = 260, 700
    x, y = rand(1, m, k), rand(2, k, n)
    turn = {"rows": "columns", "columns": "rows", "tiles": "tiles"}
    A = (g.quantize(plan, x.t().contiguous(), turn[sa]).t() if turned_a else g.quantize(plan, x, sa))
    B = (g.quantize(plan, y.t().contiguous(), turn[sb]).t() if turned_b else g.quantize(plan, y, sb))
    ref.check_product(g.matmul_f8(plan, A, B, dtype=F32), ref.values(A, sa), ref.values(B, sb))


@pytest.mark.parametrize("m", [5, 300])
@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("at", [0, 1, 8])
def test_product_into_a_larger_matrix(g, plan, m, dtype, at):
    """C's rows anywhere (aligned or not): nothing beside C is written."""
    A, B = operands(g, plan, 21, m, 203, 300)
    A = fit(g, A, B)
    room = torch.full((m + 2, 240), 7.0, dtype=dtype, device="cuda")
    c = room[1:-1, at:at + 203]
    assert g.matmul_f8(plan, A, B, c) is not None
    ref.check_product(c, ref.values(A), ref.values(B))
    c.fill_(7.0)
    assert (room == 7.0).all()


@pytest.mark.parametrize("m,n,k,kind", [(9, 300, 500, "forward"), (300, 300, 500, "inputs"),
                                        (300, 303, 5000, "weights")])
def test_accumulate(g, plan, m, n, k, kind):
    A, B = operands(g, plan, 31, m, n, k, kind)
    c = rand(5, m, n)
    old = c.double()
    for _ in range(2):
        g.matmul_f8(plan, A, B, c, accumulate=True)
    a, b = ref.values(A), ref.values(B)
    ref.check_product(c, torch.cat((a, a), 1), torch.cat((b, b), 0), extra=2, old=old)
    with pytest.raises(ValueError):
        g.matmul_f8(plan, A, B, accumulate=True)
    with pytest.raises(ValueError):
        g.matmul_f8(plan, A, B, c.half(), accumulate=True)


@pytest.mark.parametrize("m", [20, 300])
def test_not_a_number_stays_in_its_row_and_column(g, plan, m):
    x, y = rand(41, m, 300), rand(42, 200, 300)
    x[3, 299], y[7, 0] = float("nan"), float("inf")
    A, B = g.quantize(plan, x), g.quantize(plan, y, "rows").t()
    c = g.matmul_f8(plan, A, B, dtype=F32)
    bad = torch.zeros(m, 200, dtype=torch.bool, device="cuda")
    bad[3], bad[:, 7] = True, True
    assert torch.equal(c.isnan(), bad)


@pytest.mark.parametrize("m", [20, 300])
def test_scales_whose_product_leaves_fp32(g, plan, m):
    """2^-109 by 2^-40: sa * sb is below FP32's normal range, and yet the result,
    2^-149 by codes of up to 448 each, is not."""
    x, y = rand(43, m, 256) * 0 + 1, rand(44, 256, 130)
    A, B = g.quantize(plan, x), g.quantize(plan, y, "tiles")
    A = g.Blocks(A.data, torch.full_like(A.scales, 2.0 ** -109))
    B = g.Blocks(B.data, torch.full_like(B.scales, 2.0 ** -40))
    ref.check_product(g.matmul_f8(plan, A, B, dtype=F32), ref.values(A), ref.values(B))
    A = g.Blocks(A.data, torch.full_like(A.scales, 2.0 ** 100))
    B = g.Blocks(B.data, torch.full_like(B.scales, 2.0 ** 100))
    assert g.matmul_f8(plan, A, B, dtype=F32).isinf().any()    # as the number itself is


def test_products_of_nothing(g, plan):
    A, B = operands(g, plan, 51, 40, 60, 128)
    none = g.Blocks(A.data[:, :0], A.scales[:, :0])
    assert (g.matmul_f8(plan, none, g.Blocks(B.data[:0], B.scales[:0]), dtype=F32) == 0).all()
    assert g.matmul_f8(plan, g.Blocks(A.data[:0], A.scales[:0]), B).shape == (0, 60)


def test_the_same_bits_every_time_and_on_any_stream(g, plan):
    """Also where tiles are cut along the inner dimension, beside another call."""
    for m, n, k, kind in [(5, 700, 4096, "forward"), (1100, 800, 4096, "weights")]:
        A, B = operands(g, plan, 61, m, n, k, kind)
        first = g.matmul_f8(plan, A, B, dtype=F32)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        with g.Plan(0) as other:
            for _ in range(5):
                c = [g.matmul_f8(p, A, B, dtype=F32, stream=s) for p, s in zip((plan, other), streams)]
                torch.cuda.synchronize()
                assert all(torch.equal(x, first) for x in c)


@pytest.mark.parametrize("limit", [2, 16])
def test_on_a_few_sms(g, limit):
    with g.Plan(0) as p:
        p.set_option(g.OPT_SM_LIMIT, limit)
        for m, kind in ((9, "forward"), (600, "forward"), (600, "weights")):
            A, B = operands(g, p, 71, m, 500, 1500, kind)
            ref.check_product(g.matmul_f8(p, A, B, dtype=F32), ref.values(A), ref.values(B))


def test_a_captured_product_reads_new_inputs(g, plan):
    """Two graphs of products with cut tiles, replayed side by side."""
    A, B = operands(g, plan, 81, 1100, 800, 4096, "weights")
    s = torch.cuda.Stream()
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            outs.append(g.matmul_f8(plan, A, B, dtype=F32))
        graphs.append(gr)
    for seed in (1, 2):
        B.data.copy_(g.quantize(plan, rand(seed, 4096, 800), "columns").data)
        torch.cuda.synchronize()
        for gr in graphs:
            with torch.cuda.stream(torch.cuda.Stream()):
                gr.replay()
        torch.cuda.synchronize()
        for c in outs:
            ref.check_product(c, ref.values(A), ref.values(B))


# ------------------------------------------------------------------ by expert

def starts_of(lengths, first=0):
    t = [first]
    for n in lengths:
        t.append(t[-1] + n)
    return torch.tensor(t, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kind", ["forward", "inputs"])
@pytest.mark.parametrize("lengths,room,first", [
    ([0, 5, 0, 1, 33], 60, 0), ([0, 0, 0], 9, 0), ([130, 1, 0, 300], 431, 0), ([1000], 1003, 3),
    ([0, 700, 2, 128, 0], 2000, 0), ([17, 40], 57, 0), ([3000, 1, 1], 3002, 0)])
def test_product_by_experts_rows(g, plan, lengths, room, first, kind):
    n, k, e = 272, 400, len(lengths)
    A = g.quantize(plan, rand(1, room, k))
    w = rand(2, e, k, n)
    B = (g.quantize(plan, w, "tiles") if kind == "inputs"
         else g.quantize(plan, w.transpose(1, 2).contiguous(), "tiles").t())
    starts = starts_of(lengths, first)
    c = torch.full((room, n), 7.0, device="cuda")
    g.matmul_f8(plan, A, B, c, starts=starts)
    a, b = ref.values(A), ref.values(B)
    at = starts.tolist()
    assert (c[:first] == 7.0).all() and (c[at[-1]:] == 0).all()
    for i in range(e):
        ref.check_product(c[at[i]:at[i + 1]], a[at[i]:at[i + 1]], b[i])
    old = c.double()
    g.matmul_f8(plan, A, B, c, starts=starts, accumulate=True)
    assert (c[:first] == 7.0).all() and (c[at[-1]:] == 0).all()
    for i in range(e):
        r = slice(at[i], at[i + 1])
        ref.check_product(c[r], a[r], b[i], extra=2, old=old[r])
    assert plan.status() == g.OK


@pytest.mark.parametrize("lengths,room", [([128, 0, 384], 512), ([0, 0], 128), ([256], 300),
                                          ([128, 0, 256, 128], 700), ([256, 44], 300)])
@pytest.mark.parametrize("turned", [False, True])
def test_product_by_experts_inner_range(g, plan, lengths, room, turned):
    m, n = 300, 140
    x, y = rand(1, room, m), rand(2, room, n)
    A = g.quantize(plan, x, "columns").t()
    B = (g.quantize(plan, y.t().contiguous(), "rows").t() if turned
         else g.quantize(plan, y, "columns"))
    starts = starts_of(lengths)
    c = g.matmul_f8(plan, A, B, dtype=F32, starts=starts)
    assert c.shape == (len(lengths), m, n)
    a, b = ref.values(A, "rows"), ref.values(B, "columns")
    at = starts.tolist()
    for i in range(len(lengths)):
        ref.check_product(c[i], a[:, at[i]:at[i + 1]], b[at[i]:at[i + 1]])
    assert plan.status() == g.OK


@pytest.mark.parametrize("starts", [[0, 40, 20, 60], [-1, 20, 40, 60], [0, 20, 40, 61]])
def test_bad_starts_are_reported(g, plan, starts):
    A = g.quantize(plan, rand(1, 60, 128))
    B = g.quantize(plan, rand(2, 3, 128, 64), "tiles")
    g.matmul_f8(plan, A, B, starts=torch.tensor(starts, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert plan.status() == g.ERR_BAD_INDEX and plan.status() == g.OK


def test_inner_starts_inside_a_block_are_reported(g, plan):
    A, B = operands(g, plan, 91, 64, 64, 512, "weights")
    g.matmul_f8(plan, A, B, starts=torch.tensor([0, 100, 512], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert plan.status() == g.ERR_BAD_INDEX and plan.status() == g.OK


@pytest.mark.parametrize("m,kind", [(9, "forward"), (64, "forward"), (600, "forward"),
                                    (600, "weights")])
def test_a_copy_that_never_comes_is_reported(g, m, kind):
    """As for the other products: the first unit's first copy is not issued."""
    with g.Plan(0) as p:
        A, B = operands(g, p, 95, m, 512, 2048, kind)
        p.set_option(g.OPT_TIMEOUT_NS, 20_000_000)
        p.set_option(g.OPT_FAULT_UNIT, 0)
        g.matmul_f8(p, A, B, dtype=F32)
        torch.cuda.synchronize()
        assert p.status() == g.ERR_TIMEOUT and p.status() == g.OK
        p.set_option(g.OPT_FAULT_UNIT, -1)
        for _ in range(2):
            ref.check_product(g.matmul_f8(p, A, B, dtype=F32), ref.values(A), ref.values(B))
            assert p.status() == g.OK
