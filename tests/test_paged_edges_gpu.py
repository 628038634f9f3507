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
