"""Calls at the edges of what the paged-cache calls accept."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu
D = 256


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


def i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("group", [1, 16, 17, 32, 33, 64])
def test_a_step_without_new_tokens_writes_zeros(g, plan, group):
    """max_q = 0 with padded rows, at every width of the few-token kernel."""
    import torch
    kc = torch.full((4, 16, 2, D), float("nan"), dtype=torch.float16, device="cuda")
    q = torch.full((5, 2 * group, D), float("nan"), dtype=torch.float16, device="cuda")
    out = torch.full_like(q, 3.0)
    g.paged_attention(plan, q, kc, kc.clone(), i32([[0, 1], [2, 3]]), i32([0, 0, 0]), i32([9, 0]),
                      0, out=out)
    torch.cuda.synchronize()
    assert plan.status() == 0
    assert (out == 0).all()


def test_maps_are_not_advanced_in_place(g, plan):
    """An earlier call's lengths or free head cannot be an input of the call
    that writes them again; nothing of a refused call is written."""
    import torch
    table, free = i32([[-1] * 4] * 3), torch.arange(9, dtype=torch.int32, device="cuda")
    m = g.paged_maps(plan, i32([0, 0, 0]), i32([20, 3, 0]), table, free, i32([0]), 16, 2000)
    kept = [x.clone() for x in (*m, table)]
    ones = i32([1, 1, 1])
    for change in (dict(cached=m.kv_lens), dict(free_head=m.free_head), dict(added=m.kv_lens),
                   dict(free_pages=m.positions), dict(added=m.starts[1:]),
                   dict(block_table=m.slots[:12].view(3, 4))):
        args = dict(cached=i32([20, 3, 0]), added=ones, block_table=table, free_pages=free,
                    free_head=i32([3]), page_size=16, max_tokens=2000)
        with pytest.raises(g.GemmError) as e:
            g.paged_maps(plan, **{**args, **change}, out=m)
        assert e.value.code == g.ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert plan.status() == 0
    assert all(torch.equal(a, b) for a, b in zip((*m, table), kept))


def step_calls(g, plan):
    """name -> call(stream, out), of each paged-cache call on the same inputs."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(7)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").half()
    cached, added = i32([30, 0, 7]), i32([1, 90, 2])
    free = torch.arange(20, dtype=torch.int32, device="cuda").flip(0).contiguous()
    start = g.paged_maps(plan, i32([0, 0, 0]), cached, i32([[-1] * 8] * 3), free, i32([0]), 16, 40)
    table = i32([[-1] * 8] * 3)
    g.paged_maps(plan, i32([0, 0, 0]), cached, table, free, i32([0]), 16, 40)
    m = g.paged_maps(plan, cached, added, table, free, start.free_head, 16, 100)
    kc, vc = rand(20, 16, 2, D), rand(20, 16, 2, D)
    q, k, v = rand(100, 8, D), rand(100, 2, D), rand(100, 2, D)
    turns = g.rope_turns(g.rope_frequencies(128)).cuda()
    own = kc.clone(), vc.clone()
    return {
        "maps": lambda stream, out: g.paged_maps(plan, cached, added, table, free,
                                                 start.free_head, 16, 100, out=out, stream=stream),
        "rotary": lambda stream, out: g.rotary(plan, q, m.positions, turns, out=out, stream=stream),
        "to cache": lambda stream, out: g.rotary_to_cache(plan, q, k, v, m.positions, m.slots,
                                                          turns, *own, out=out, stream=stream),
        "attention": lambda stream, out: g.paged_attention(plan, q, kc, vc, table, m.starts,
                                                           m.kv_lens, 90, out=out, stream=stream),
    }


@pytest.mark.parametrize("name", ["maps", "rotary", "to cache", "attention"])
def test_given_outputs_are_written(g, plan, name):
    """Into the tensors given, every number of them (they hold something else before)."""
    import torch
    call = step_calls(g, plan)[name]
    want = call(None, None)
    if name == "maps":
        out = type(want)(*[torch.full_like(x, -77) for x in want])
        got = call(None, out)
        assert all(a.data_ptr() == b.data_ptr() for a, b in zip(got, out))
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    else:
        out = torch.full_like(want, float("nan"))
        got = call(None, out)
        assert got.data_ptr() == out.data_ptr()
        assert torch.equal(out, want)
    torch.cuda.synchronize()
    assert plan.status() == 0


@pytest.mark.parametrize("name", ["maps", "rotary", "to cache", "attention"])
def test_given_streams_are_ordered(g, plan, name):
    """On another stream, given as an object or a handle: behind what that
    stream was told to wait for, with the tensors made here."""
    import torch
    call = step_calls(g, plan)[name]
    want = call(None, None)
    flat = lambda r: list(r) if name == "maps" else [r]
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        side.wait_stream(torch.cuda.current_stream())
        got = call(stream, None)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(flat(got), flat(want)))
    torch.cuda.synchronize()
    assert plan.status() == 0


@pytest.mark.parametrize("scale", [3e38, -3e38, 1e-44])
@pytest.mark.parametrize("new", [1, 90], ids=["few", "many"])
def test_scales_at_the_ends_of_their_range(g, plan, new, scale):
    """All scores 0: O is the mean of the values seen, whatever the scale (times
    log2 e the largest ones do not fit FP32).  Half a binary16 step of O, and
    FP32 sums of n numbers (2^-24 each of their magnitudes)."""
    import torch
    n = 200 + new
    gen = torch.Generator(device="cuda").manual_seed(8)
    kc, vc = (torch.randn(16, 32, 1, D, generator=gen, device="cuda").half() for _ in range(2))
    q = torch.zeros(new, 2, D, dtype=torch.float16, device="cuda")
    table = torch.arange(16, dtype=torch.int32, device="cuda")[None]
    o = g.paged_attention(plan, q, kc, vc, table, i32([0, new]), i32([n]), new, scale=scale)
    torch.cuda.synchronize()
    assert plan.status() == 0
    seen = torch.arange(n - new + 1, n + 1, device="cuda").double()[:, None]
    v = vc.view(-1, D)[:n].double()
    mean, mag = (x.cumsum(0)[n - new:] / seen for x in (v, v.abs()))
    bound = 2.0 ** -11 * mean.abs() + 2.0 ** -25 + 2 * n * 2.0 ** -24 * mag
    assert ((o.double() - mean[:, None]).abs() <= bound[:, None]).all()


@pytest.mark.parametrize("replay_first", [True, False])
@pytest.mark.parametrize("name", ["few", "many", "both"])
def test_a_plan_whose_first_call_is_captured(g, plan, name, replay_first):
    """Its workspace (all these steps cut tiles) serves the graph's replays and
    calls outside them, in either order."""
    import torch
    lens = {"few": [(3000, 1)], "many": [(900, 700)], "both": [(2000, 1), (500, 300)]}[name]
    gen = torch.Generator(device="cuda").manual_seed(9)
    kc, vc = (torch.randn(300, 16, 2, D, generator=gen, device="cuda").half() for _ in range(2))
    total = sum(n for _, n in lens)
    q = torch.randn(total, 4, D, generator=gen, device="cuda").half()
    table = torch.arange(300, dtype=torch.int32, device="cuda").view(1, 300).repeat(len(lens), 1)
    starts = i32([0] + [sum(n for _, n in lens[:b + 1]) for b in range(len(lens))])
    kv_lens, most = i32([c + n for c, n in lens]), max(n for _, n in lens)
    call = lambda p, out: g.paged_attention(p, q, kc, vc, table, starts, kv_lens, most, out=out)
    want = call(plan, None)
    torch.cuda.synchronize()
    with g.Plan(0) as fresh:
        out = torch.full_like(q, float("nan"))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(fresh, out)
        for replay in (replay_first, not replay_first, replay_first):
            if replay:
                out.fill_(float("nan"))
                graph.replay()
                got = out
            else:
                got = call(fresh, None)
            torch.cuda.synchronize()
            assert fresh.status() == 0
            assert torch.equal(got, want)
        del graph
