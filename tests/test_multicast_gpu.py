"""OPT_MULTICAST: the CTA-pair kernel in place of the cluster-of-four kernel."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import async_barrier_pipelined_gb300 as g
    from async_barrier_pipelined_gb300 import build
    build.build()
    return g


@pytest.mark.parametrize("kernel", [0, 3])
def test_without_multicast_the_pair_kernel_runs(g, kernel, monkeypatch):
    import torch
    M, N, K = 2304, 2560, 2056      # a row pitch off 128-byte lines, 2^22 elements of A
    gen = torch.Generator(device="cuda").manual_seed(1)
    A, B = (torch.randn(s, generator=gen, device="cuda").half() for s in ((M, K), (K, N)))
    which = lambda p: g.gemm_f16_run_info(p.handle, 0, M, N, K, K)["kernel"]
    with g.Plan(0) as plan:
        plan.set_option(g.OPT_KERNEL, kernel)
        assert plan.get_option(g.OPT_MULTICAST) == 1 and which(plan) == 3
        plan.set_option(g.OPT_MULTICAST, 0)
        assert plan.get_option(g.OPT_MULTICAST) == 0 and which(plan) == 2
        C = g.matmul(plan, A, B)
        plan.set_option(g.OPT_KERNEL, 2)
        assert torch.equal(C, g.matmul(plan, A, B))
        torch.cuda.synchronize()
        assert plan.status() == 0
        plan.set_option(g.OPT_MULTICAST, 1)
        plan.set_option(g.OPT_KERNEL, kernel)
        assert which(plan) == 3
        for bad in (-1, 2):
            with pytest.raises(g.GemmError):
                plan.set_option(g.OPT_MULTICAST, bad)
    monkeypatch.setenv("WORLD_SIZE", "2")
    with g.Plan(0) as plan:
        plan.set_option(g.OPT_KERNEL, kernel)
        assert which(plan) == 2
