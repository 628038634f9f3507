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
