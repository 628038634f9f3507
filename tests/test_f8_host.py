"""8-bit products, their quantisation and experts' rows: what the header and the
binding declare, and the calls that are refused.  Nothing is computed here; the
addresses are never dereferenced."""
from __future__ import annotations

import ctypes
import os
import re
import types

import pytest

import async_barrier_pipelined_gb300 as g
from async_barrier_pipelined_gb300 import build as gbuild

P = 1 << 20
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    return g.load()


def test_header_binding_and_library_agree(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(gbuild.INCLUDE, "gemm_f8.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b((?:gemm_f8|experts)_\w+)\s*\(", text)))
    assert names == sorted(g.EXPORTED_SYMBOLS_F8)
    for n in names:
        assert ctypes.cast(getattr(lib, n), ctypes.c_void_p).value


QUANTIZE = dict(blocks=g.F8_ROWS, format=g.F8_E4M3, type=0, batch=1, rows=5, cols=300, X=P, ldx=300,
                x_batch=0, source=0, choices=1, x_rows=0, Q=P, ldq=304, q_batch=0, S=P, Q2=0, S2=0)


@pytest.mark.parametrize("change,code", [
    ({}, g.OK), (dict(blocks=4), g.ERR_INVALID_ARG), (dict(blocks=-1), g.ERR_INVALID_ARG),
    (dict(format=2), g.ERR_INVALID_ARG), (dict(type=3), g.ERR_INVALID_ARG),
    (dict(batch=65536), g.ERR_INVALID_ARG), (dict(batch=-1), g.ERR_INVALID_ARG),
    (dict(rows=-1), g.ERR_INVALID_ARG), (dict(rows=BIG), g.ERR_INVALID_ARG),
    (dict(cols=0), g.ERR_INVALID_ARG), (dict(ldx=299), g.ERR_INVALID_ARG),
    (dict(ldx=299, rows=1), g.OK), (dict(ldq=288), g.ERR_INVALID_ARG),
    (dict(ldq=305), g.ERR_MISALIGNED), (dict(Q=P + 8), g.ERR_MISALIGNED),
    (dict(X=P + 1), g.ERR_MISALIGNED), (dict(X=P + 2), g.OK), (dict(type=2, X=P + 2), g.ERR_MISALIGNED),
    (dict(S=P + 2), g.ERR_MISALIGNED), (dict(X=0), g.ERR_INVALID_ARG), (dict(S=0), g.ERR_INVALID_ARG),
    (dict(blocks=g.F8_BOTH), g.ERR_INVALID_ARG), (dict(blocks=g.F8_BOTH, Q2=P, S2=P), g.OK),
    (dict(blocks=g.F8_BOTH, Q2=P, S2=P, batch=2, x_batch=1500, q_batch=1520), g.ERR_INVALID_ARG),
    (dict(batch=2, x_batch=1500, q_batch=1528), g.ERR_MISALIGNED),
    (dict(source=P, choices=2, x_rows=3), g.OK), (dict(source=P, choices=0, x_rows=3), g.ERR_INVALID_ARG),
    (dict(source=P, choices=2, x_rows=0, X=0), g.OK), (dict(source=P, batch=2, x_rows=3), g.ERR_INVALID_ARG),
    (dict(rows=0, X=0, Q=0, S=0), g.OK), (dict(batch=0, X=0, Q=0, S=0), g.OK),
    (dict(rows=2 ** 30, cols=2 ** 30, ldx=2 ** 30, ldq=2 ** 30), g.ERR_INVALID_ARG),
])
def test_quantize_refusals(change, code):
    assert g.gemm_f8_quantize_validate(*{**QUANTIZE, **change}.values()) == code


def operand(**kw):
    return g.GemmF8Operand(**{**dict(data=P, ld=512, batch=0, scales=P, s_outer=4, s_inner=1,
                                     s_batch=0, format=0, transposed=0, tiles=0), **kw})


def product(a=None, b=None, form=g.F8_DENSE, M=100, N=512, K=512, experts=1, starts=0, C=P, ldc=512,
            c_batch=0, type=0, accumulate=0):
    return g.gemm_f8_validate(form, M, N, K, experts, starts, a or operand(), b or operand(), C, ldc,
                              c_batch, type, accumulate)


@pytest.mark.parametrize("kw,code", [
    ({}, g.OK), (dict(M=0, C=0), g.OK), (dict(K=0), g.OK), (dict(M=-1), g.ERR_INVALID_ARG),
    (dict(N=BIG), g.ERR_INVALID_ARG), (dict(form=3), g.ERR_INVALID_ARG),
    (dict(type=3), g.ERR_INVALID_ARG), (dict(accumulate=1), g.ERR_INVALID_ARG),
    (dict(accumulate=1, type=2), g.OK), (dict(accumulate=2, type=2), g.ERR_INVALID_ARG),
    (dict(ldc=511), g.ERR_INVALID_ARG), (dict(C=0), g.ERR_INVALID_ARG), (dict(C=P + 1), g.ERR_MISALIGNED),
    (dict(type=2, C=P + 2), g.ERR_MISALIGNED), (dict(a=dict(ld=511)), g.ERR_INVALID_ARG),
    (dict(a=dict(ld=520)), g.ERR_MISALIGNED), (dict(a=dict(data=P + 8)), g.ERR_MISALIGNED),
    (dict(b=dict(scales=P + 2)), g.ERR_MISALIGNED), (dict(b=dict(scales=0)), g.ERR_INVALID_ARG),
    (dict(b=dict(format=2)), g.ERR_INVALID_ARG), (dict(b=dict(transposed=2)), g.ERR_INVALID_ARG),
    (dict(b=dict(s_outer=-1)), g.ERR_INVALID_ARG),
    (dict(form=g.F8_BY_ROWS, experts=4, starts=P), g.OK),
    (dict(form=g.F8_BY_ROWS, experts=4), g.ERR_INVALID_ARG),
    (dict(form=g.F8_BY_ROWS, experts=0, starts=P), g.ERR_INVALID_ARG),
    (dict(form=g.F8_BY_ROWS, experts=1025, starts=P), g.ERR_INVALID_ARG),
    (dict(form=g.F8_BY_ROWS, experts=4, starts=P + 2), g.ERR_MISALIGNED),
    (dict(form=g.F8_BY_ROWS, experts=4, starts=P, a=dict(transposed=1)), g.ERR_INVALID_ARG),
    (dict(form=g.F8_BY_ROWS, experts=4, starts=P, b=dict(batch=8)), g.ERR_MISALIGNED),
    (dict(form=g.F8_BY_INNER, experts=4, starts=P), g.OK),
    (dict(form=g.F8_BY_INNER, experts=4, starts=P, c_batch=-1), g.ERR_INVALID_ARG),
])
def test_product_refusals(kw, code):
    kw = {k: operand(**v) if k in "ab" else v for k, v in kw.items()}
    assert product(**kw) == code


def test_product_without_operands_is_refused():
    assert g.load().gemm_f8_validate(0, 1, 1, 1, 1, 0, None, None, P, 1, 0, 0, 0) == g.ERR_INVALID_ARG


@pytest.mark.parametrize("entries,experts,align,want", [
    (0, 5, 128, 0), (1, 5, 1, 1), (1, 5, 128, 128), (7, 3, 16, 64), (100, 8, 1, 100),
    (100, 8, 128, 1152), (-1, 5, 1, None), (5, 0, 1, None), (5, 1025, 1, None), (5, 5, 0, None),
    (5, 5, 1025, None), (2 ** 26 + 1, 5, 1, None)])
def test_rows_of_any_choice(entries, experts, align, want):
    if want is None:
        with pytest.raises(g.GemmError):
            g.experts_max_rows(entries, experts, align)
    else:
        assert g.experts_max_rows(entries, experts, align) == want
        # enough where all experts that can have an entry have one, and one the rest
        used = min(experts, entries)
        if used:
            assert want >= (used - 1) * align + -(-(entries - used + 1) // align) * align


@pytest.mark.parametrize("change,code", [
    ({}, g.OK), (dict(max_rows=17), g.ERR_INVALID_ARG), (dict(wide=2), g.ERR_INVALID_ARG),
    (dict(starts=0), g.ERR_INVALID_ARG), (dict(rows=0), g.ERR_INVALID_ARG),
    (dict(source=0), g.ERR_INVALID_ARG), (dict(wide=1, experts=P + 4), g.ERR_MISALIGNED),
    (dict(rows=P + 2), g.ERR_MISALIGNED), (dict(num_experts=0), g.ERR_INVALID_ARG),
    (dict(entries=0, experts=0, rows=0, source=0, max_rows=0), g.OK)])
def test_maps_refusals(change, code):
    d = dict(entries=18, experts=P, wide=0, num_experts=4, align=1, max_rows=18, starts=P, rows=P,
             source=P)
    assert g.experts_maps_validate(*{**d, **change}.values()) == code


@pytest.mark.parametrize("change,code", [
    ({}, g.OK), (dict(type=3), g.ERR_INVALID_ARG), (dict(cols=0), g.ERR_INVALID_ARG),
    (dict(choices=0), g.ERR_INVALID_ARG), (dict(ldx=63), g.ERR_INVALID_ARG),
    (dict(ldy=63), g.ERR_INVALID_ARG), (dict(source=0), g.ERR_INVALID_ARG),
    (dict(X=P + 1), g.ERR_MISALIGNED), (dict(source=P + 1), g.ERR_MISALIGNED),
    (dict(x_rows=0, X=0), g.OK), (dict(rows=0, Y=0, source=0), g.OK)])
def test_gather_refusals(change, code):
    d = dict(type=0, rows=9, cols=64, X=P, ldx=64, x_rows=3, choices=3, source=P, Y=P, ldy=64)
    assert g.experts_gather_validate(*{**d, **change}.values()) == code


@pytest.mark.parametrize("change,code", [
    ({}, g.OK), (dict(weights=0), g.OK), (dict(weights_type=1), g.ERR_INVALID_ARG),
    (dict(weights_type=0), g.OK), (dict(tokens=2 ** 25, choices=3), g.ERR_INVALID_ARG),
    (dict(rows=0), g.ERR_INVALID_ARG), (dict(weights=P + 2), g.ERR_MISALIGNED),
    (dict(lds=63), g.ERR_INVALID_ARG), (dict(tokens=0, rows=0, Y=0), g.OK)])
def test_combine_refusals(change, code):
    d = dict(type=0, tokens=3, choices=3, cols=64, S=P, lds=64, s_rows=9, rows=P, weights=P,
             weights_type=2, Y=P, ldy=64)
    assert g.experts_combine_validate(*{**d, **change}.values()) == code


@pytest.mark.parametrize("change,code", [
    ({}, g.OK), (dict(dS=0, dw=0, dY=0, S=0, rows=0, source=0), g.OK), (dict(dY=0), g.ERR_INVALID_ARG),
    (dict(S=0), g.ERR_INVALID_ARG), (dict(S=0, dw=0), g.OK), (dict(rows=0), g.ERR_INVALID_ARG),
    (dict(source=0), g.ERR_INVALID_ARG), (dict(dw=P + 2), g.ERR_MISALIGNED),
    (dict(ldds=63), g.ERR_INVALID_ARG)])
def test_combine_gradient_refusals(change, code):
    d = dict(type=0, tokens=3, choices=3, cols=64, dY=P, lddy=64, S=P, lds=64, s_rows=9, rows=P,
             source=P, weights=P, weights_type=2, dS=P, ldds=64, dw=P)
    assert g.experts_combine_gradient_validate(*{**d, **change}.values()) == code


# ------------------------------------------------------------------ tensors
#
# A plan that is none: every call is refused before it is used.

PLAN = types.SimpleNamespace(handle=0, device=0)


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


def test_tensors_elsewhere_and_of_other_types_are_refused(torch):
    x = torch.zeros(4, 32, dtype=torch.float16)
    with pytest.raises(ValueError, match="plan's device"):
        g.quantize(PLAN, x)
    with pytest.raises(ValueError, match="float16, bfloat16 or float32"):
        g.quantize(PLAN, x.int())
    with pytest.raises(ValueError, match="blocks is"):
        g.quantize(PLAN, x, "row")
    with pytest.raises(TypeError):
        g.quantize(PLAN, x, dtype=torch.float16)
    q = torch.zeros(4, 32, dtype=torch.float8_e4m3fn)
    b = g.Blocks(q, torch.ones(4, 1))
    with pytest.raises(ValueError, match="inner dimension"):
        g.matmul_f8(PLAN, b, b)
    with pytest.raises(ValueError, match="plan's device"):
        g.matmul_f8(PLAN, b, b.t())
    with pytest.raises(TypeError):
        g.matmul_f8(PLAN, b, b.t(), dtype=torch.float64)
    with pytest.raises(ValueError, match="M, K"):
        g.matmul_f8(PLAN, g.Blocks(q[None], b.scales[None]), b.t())
    with pytest.raises(ValueError):
        g.linear_f8(PLAN, x, x[None])
    with pytest.raises(ValueError):
        g.linear_f8(PLAN, x[None], x[None], starts=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="tiles"):
        g.linear_f8(PLAN, x, b._replace(scales=torch.ones(4, 1)))
    picks = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        g.expert_maps(PLAN, picks, 4)
    with pytest.raises(ValueError):
        g.expert_maps(PLAN, picks.float(), 4)
    m = g.ExpertMaps(torch.zeros(5, dtype=torch.int32), picks, torch.zeros(8, dtype=torch.int32))
    with pytest.raises(ValueError):
        g.expert_gather(PLAN, x, m)
    with pytest.raises(ValueError):
        g.expert_combine(PLAN, torch.zeros(8, 32), m)
    with pytest.raises(ValueError, match="row for each token"):
        g.quantize(PLAN, x[:3], maps=m)


def test_blocks_are_transposed_without_a_copy(torch):
    b = g.Blocks(torch.zeros(4, 32, dtype=torch.float8_e4m3fn), torch.ones(4, 1))
    t = b.t()
    assert t.data.shape == (32, 4) and t.scales.shape == (1, 4)
    assert t.data.data_ptr() == b.data.data_ptr()
