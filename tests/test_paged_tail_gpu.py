"""One key far above a long flat tail: what the attention over a paged cache
keeps of weights that are tiny beside the row's largest."""
from __future__ import annotations

import math

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


@pytest.mark.parametrize("limit", [0, 2], ids=["all workers", "one"])
@pytest.mark.parametrize("new", [1, 80], ids=["few", "many"])
@pytest.mark.parametrize("below", [16.0, 25.5, 28.0])
def test_a_long_tail_counts(g, below, new, limit):
    """Key 0 scores `below` powers of two above all others and has the value 0,
    so O is the tail's alone.

    The bound of a row over n keys, with weights p relative to the largest,
    l = sum p and A = sum p v / l (v >= 0): O is rounded once (2^-11 |o|, 2^-25
    below the normal range); a weight is rounded to binary16 for the product
    with V, the largest being at least 2^7 there, so by 2^-11 of itself or, below
    the normal range, by 2^-25 / 2^7 = 2^-32 of the largest; a score is a sum of
    256 FP32 products of magnitude |s| in all (256 * 2^-24 |s|, a relative error
    of a weight, in numerator and denominator); the sums over n keys in FP32 are
    off by n * 2^-24 each; two units of 2^-22 for each exponential.
    """
    import torch
    n, page = 100_000 + new, 16
    pages = -(-n // page)
    gen = torch.Generator(device="cuda").manual_seed(5)
    c = torch.tensor(below * math.log(2.0) * 16.0 / D, dtype=torch.float16)
    kc = torch.zeros(pages, page, 1, D, dtype=torch.float16, device="cuda")
    kc[0, 0] = c
    vc = (torch.rand(kc.shape, generator=gen, device="cuda") + 0.5).half()
    vc[0, 0] = 0
    q = torch.ones(new, 1, D, dtype=torch.float16, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    with g.Plan(0) as plan:
        plan.set_option(g.OPT_SM_LIMIT, limit)
        o = g.paged_attention(plan, q, kc, vc, table, i32([0, new]), i32([n]), new)
        torch.cuda.synchronize()
        assert plan.status() == 0
    score = D * c.double().item() / 16.0
    p = math.exp(-score)
    seen = torch.arange(n - new + 1, n + 1, device="cuda").double()[:, None]
    v = vc.view(-1, D)[:n].double().cumsum(0)[n - new:]            # sums over the keys seen
    l = 1.0 + (seen - 1.0) * p
    want = p * v / l
    bound = (2.0 ** -11 * want + 2.0 ** -25 + 2.0 ** -32 * v / l
             + want * (2.0 ** -11 + 2 * 256 * 2.0 ** -24 * score + 2 * seen * 2.0 ** -24
                       + 4 * 2.0 ** -22))
    off = (o[:, 0].double() - want).abs()
    assert (off <= bound).all(), ((off / bound).max().item(), (off / want).max().item())
