"""Multicast copies (the cluster-of-four GEMM kernel) are for runs on one GPU:
the plan of a process that is one of several leaves them out.  No GPU."""
from __future__ import annotations

import pytest

import async_barrier_pipelined_gb300 as g


@pytest.mark.parametrize("world,off", [(None, False), ("", False), ("1", False), ("2", True),
                                       ("8", True)])
def test_a_plan_among_several_processes(monkeypatch, world, off):
    options = []
    monkeypatch.setattr(g, "gemm_f16_plan", lambda device: 7)
    monkeypatch.setattr(g, "gemm_f16_destroy", lambda plan: None)
    monkeypatch.setattr(g, "gemm_f16_set_option", lambda *a: options.append(a))
    if world is None:
        monkeypatch.delenv("WORLD_SIZE", raising=False)
    else:
        monkeypatch.setenv("WORLD_SIZE", world)
    with g.Plan(0):
        assert options == ([(7, g.OPT_MULTICAST, 0)] if off else [])
