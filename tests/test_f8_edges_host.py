"""8-bit calls and experts' rows: calls that must be refused rather than answered
wrongly, on the host.  Nothing is computed here."""
from __future__ import annotations

import re
import types

import pytest

import async_barrier_pipelined_gb300 as g
from async_barrier_pipelined_gb300 import build as gbuild

PLAN = types.SimpleNamespace(handle=0, device=0)      # every call ends before it is used


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    return g.load()


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


# ------------------------------------------------------------------ maps and their align

def maps_of(torch, align):
    m = g.ExpertMaps(torch.zeros(5, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32),
                     torch.zeros(8, dtype=torch.int32))
    m.align = align
    return m


@pytest.mark.parametrize("align", [1, 16, 64, 192])
def test_weights_gradients_of_maps_that_cannot_give_them_are_refused(torch, align):
    """Before anything is computed, and only where W's gradient may be wanted."""
    x, w = torch.zeros(8, 32), torch.zeros(4, 16, 32)
    m = maps_of(torch, align)
    with pytest.raises(ValueError, match="align=128"):
        g.linear_f8(PLAN, x, w.requires_grad_(), starts=m)
    for call in (lambda: g.linear_f8(PLAN, x.requires_grad_(), w.detach(), starts=m),
                 lambda: g.linear_f8(PLAN, x, w.requires_grad_(), starts=m.starts)):
        with pytest.raises(ValueError, match="plan's device"):      # the next refusal
            call()
    with torch.no_grad(), pytest.raises(ValueError, match="plan's device"):
        g.linear_f8(PLAN, x, w, starts=m)


@pytest.mark.parametrize("align", [None, 128, 256, 1024])
def test_maps_that_can_are_taken(torch, align):
    x, w = torch.zeros(8, 32), torch.zeros(4, 16, 32, requires_grad=True)
    with pytest.raises(ValueError, match="plan's device"):
        g.linear_f8(PLAN, x, w, starts=maps_of(torch, align))


def test_maps_are_still_three_tensors(torch):
    m = maps_of(torch, 128)
    starts, rows, source = m
    assert len(m) == 3 and m._fields == ("starts", "rows", "source") and m[0] is starts
    assert m._replace(rows=rows).align is None      # others' maps: not known


# ------------------------------------------------------------------ forward mode

@pytest.mark.parametrize("which", ["X", "W", "gather", "S", "weights"])
@pytest.mark.parametrize("grad", [False, True])
def test_forward_mode_derivatives_are_refused(torch, which, grad):
    """Not dropped, whether or not a gradient is wanted as well."""
    import torch.autograd.forward_ad as fwd
    m = maps_of(torch, 128)
    with fwd.dual_level():
        def t(*shape, dual=False):
            x = torch.ones(shape, requires_grad=grad)
            return fwd.make_dual(x, torch.ones(shape)) if dual else x
        calls = {"X": lambda: g.linear_f8(PLAN, t(3, 4, 32, dual=True), t(16, 32)),
                 "W": lambda: g.linear_f8(PLAN, t(4, 32), t(16, 32, dual=True)),
                 "gather": lambda: g.expert_gather(PLAN, t(4, 32, dual=True), m),
                 "S": lambda: g.expert_combine(PLAN, t(8, 32, dual=True), m),
                 "weights": lambda: g.expert_combine(PLAN, t(8, 32), m, t(4, 2, dual=True))}
        with pytest.raises(NotImplementedError, match="forward-mode"):
            calls[which]()
        with fwd._set_fwd_grad_enabled(False), pytest.raises(ValueError, match="plan's device"):
            calls[which]()       # switched off: the next refusal


# ------------------------------------------------------------------ launches

SIZES = [(g.F8_DENSE, 1, 4096, 4096, 1), (g.F8_DENSE, 7, 100, 8192, 1), (g.F8_DENSE, 64, 12288, 4096, 1),
         (g.F8_DENSE, 129, 4096, 4096, 1), (g.F8_DENSE, 1000, 1024, 8192, 1),
         (g.F8_DENSE, 8192, 8192, 4096, 1), (g.F8_BY_ROWS, 96, 4096, 2048, 16),
         (g.F8_BY_ROWS, 16384, 4096, 2048, 16), (g.F8_BY_INNER, 2048, 2048, 4096, 8)]


@pytest.mark.parametrize("limit", [1, 2, 3, 7, 16, 40, 152])
@pytest.mark.parametrize("form,m,n,k,experts", SIZES)
def test_a_limit_of_sms_bounds_every_launch(form, m, n, k, experts, limit):
    """A CTA may have an SM of its own: there are no more of them than SMs, but
    for one cluster of two where a single SM is allowed."""
    kernel, parts, product, join = g.gemm_f8_run_choice(form, m, n, k, experts, sm_limit=limit).values()
    assert 1 <= product <= max(limit, 2 if kernel == 2 else 1)
    assert 0 <= join <= limit
    assert product % (parts if kernel == 1 else 2) == 0


@pytest.mark.parametrize("size,want", [
    ((g.F8_DENSE, 1, 4096, 4096), (1, 8, 256, 0)), ((g.F8_DENSE, 64, 12288, 4096), (1, 2, 192, 0)),
    ((g.F8_DENSE, 65, 4096, 4096), (2, 4, 128, 256)), ((g.F8_DENSE, 1000, 1024, 2048), (2, 1, 32, 0)),
    ((g.F8_DENSE, 8192, 8192, 4096), (2, 2, 152, 576)), ((g.F8_BY_ROWS, 96, 4096, 2048, 16), (1, 1, 304, 0)),
    ((g.F8_BY_ROWS, 16384, 4096, 2048, 16), (2, 1, 152, 0)),
    ((g.F8_BY_INNER, 100, 100, 4096, 8), (2, 1, 16, 0)), ((g.F8_DENSE, 40, 512, 512, 1, 1), (2, 1, 4, 0))])
def test_launches_without_a_limit(size, want):
    """On 152 SMs with 76 pairs of CTAs."""
    assert tuple(g.gemm_f8_run_choice(*size).values()) == want


@pytest.mark.parametrize("change", [dict(form=3), dict(M=0), dict(N=-1), dict(K=0), dict(num_sms=0),
                                    dict(max_pairs=0), dict(sm_limit=-1),
                                    dict(form=g.F8_BY_ROWS, experts=0),
                                    dict(form=g.F8_BY_INNER, experts=1025), dict(M=2 ** 31 - 1)])
def test_launches_of_bad_sizes_are_refused(change):
    with pytest.raises(g.GemmError):
        g.gemm_f8_run_choice(**{**dict(form=0, M=1, N=1, K=1), **change})


# ------------------------------------------------------------------ sources

def test_kernels_that_start_early_read_their_inputs_by_ordinary_loads():
    """A read-only load is for memory that nothing writes while the kernel runs.
    These kernels start before the one that writes their inputs has ended."""
    import glob
    import os
    found = []
    for path in glob.glob(os.path.join(gbuild.CSRC, "f8*")) + [os.path.join(gbuild.CSRC, "experts.cu")]:
        text = re.sub(r"//[^\n]*", "", open(path).read())
        found += [(os.path.basename(path), w) for w in ("__ldg", "global.nc", "__restrict__") if w in text]
    assert not found
