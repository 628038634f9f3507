"""Host-side checks of the paged-cache calls (attn_f16.h, second half): the
argument checks of the C entry points and the frequency helpers.  No GPU."""
from __future__ import annotations

import ctypes
import math

import pytest

import async_barrier_pipelined_gb300 as g
from async_barrier_pipelined_gb300 import build as gbuild

P = 1 << 20  # a 16-byte-aligned fake address (never dereferenced)
D = 256


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    return g.load()


MAPS = dict(batch=4, cached=P, added=P, block_table=P, table_stride=10, max_pages=10,
            free_pages=P, num_free=5, free_head=P, page_size=16, max_tokens=8, starts=P,
            kv_lens=P, positions=P, slots=P, free_head_out=P + 4)


def test_maps_validate_accepts():
    for change in ({}, {"batch": 65535}, {"num_free": 0, "free_pages": 0}, {"page_size": 1},
                   {"max_tokens": 0, "positions": 0, "slots": 0}, {"table_stride": 1 << 40}):
        assert g.attn_f16_paged_maps_validate(*{**MAPS, **change}.values()) == g.OK, change


@pytest.mark.parametrize("change,code", [
    ({"batch": 0}, g.ERR_INVALID_ARG), ({"batch": 65536}, g.ERR_INVALID_ARG),
    ({"max_pages": 0}, g.ERR_INVALID_ARG), ({"table_stride": 9}, g.ERR_INVALID_ARG),
    ({"max_pages": (1 << 24) + 1, "table_stride": 1 << 30}, g.ERR_INVALID_ARG),
    ({"page_size": 0}, g.ERR_INVALID_ARG), ({"page_size": (1 << 20) + 1}, g.ERR_INVALID_ARG),
    ({"num_free": -1}, g.ERR_INVALID_ARG), ({"max_tokens": -1}, g.ERR_INVALID_ARG),
    ({"free_pages": 0}, g.ERR_INVALID_ARG), ({"positions": 0}, g.ERR_INVALID_ARG),
    ({"slots": 0}, g.ERR_INVALID_ARG), ({"free_head_out": P}, g.ERR_INVALID_ARG),
    *[({k: 0}, g.ERR_INVALID_ARG) for k in ("cached", "added", "block_table", "free_head",
                                            "starts", "kv_lens", "free_head_out")],
    *[({k: P + 2}, g.ERR_MISALIGNED) for k in ("cached", "added", "block_table", "free_pages",
                                               "free_head", "starts", "kv_lens", "positions",
                                               "slots", "free_head_out")],
], ids=lambda x: str(x))
def test_maps_validate_refuses(change, code):
    assert g.attn_f16_paged_maps_validate(*{**MAPS, **change}.values()) == code


ROPE = dict(tokens=3, q_heads=4, kv_heads=2, head_dim=D, rot_dim=128, layout=0, factor=1.0,
            turns=P, positions=P, Q=P, q_strides=(4 * D, D), Qo=P, qo_strides=(4 * D, D), K=P,
            k_strides=(2 * D, D), V=P, v_strides=(2 * D, D), slots=P, Kc=P,
            kc_strides=(32 * D, 2 * D, D), Vc=P, vc_strides=(32 * D, D, 16 * D), num_pages=9,
            page_size=16)


def test_rope_validate_accepts():
    none = {"K": 0, "V": 0, "slots": 0, "Kc": 0, "Vc": 0, "k_strides": None, "v_strides": None,
            "kc_strides": None, "vc_strides": None, "num_pages": 0, "page_size": 0}
    for change in ({}, {"layout": 1}, {"rot_dim": 16}, {"rot_dim": 256},
                   {"kv_heads": 0, **none}, {"q_heads": 0, "Q": 0, "Qo": 0, "q_strides": None,
                                             "qo_strides": None},
                   {"tokens": 0, "Q": 0, "Qo": 0, "K": 0, "V": 0, "positions": 0, "slots": 0},
                   {"q_heads": 1, "q_strides": (D, 5), "qo_strides": (D, 7)},
                   {"Qo": P + 4096, "qo_strides": (8 * D, D)}):
        assert g.attn_f16_rope_validate(*{**ROPE, **change}.values()) == g.OK, change


@pytest.mark.parametrize("change,code", [
    *[({k: v}, g.ERR_INVALID_ARG) for k, v in (
        ("tokens", -1), ("q_heads", -1), ("kv_heads", -1), ("q_heads", 65536), ("head_dim", 128),
        ("rot_dim", 0), ("rot_dim", 8), ("rot_dim", 24), ("rot_dim", 272), ("layout", 2),
        ("layout", -1), ("factor", math.inf), ("factor", math.nan), ("turns", 0),
        ("positions", 0), ("Q", 0), ("Qo", 0), ("K", 0), ("V", 0), ("slots", 0), ("Kc", 0),
        ("Vc", 0), ("num_pages", 0), ("page_size", 0), ("q_strides", None),
        ("q_strides", (4 * D, 0)), ("q_strides", (-8, D)), ("k_strides", (2 * D, 128)),
        ("kc_strides", None), ("kc_strides", (32 * D, 0, D)), ("vc_strides", (1 << 38, D, D)),
        ("qo_strides", (8 * D, D)))],          # in place with other strides
    ({"q_heads": 0, "kv_heads": 0}, g.ERR_INVALID_ARG),
    *[({k: v}, g.ERR_MISALIGNED) for k, v in (
        ("turns", P + 4), ("positions", P + 2), ("slots", P + 1), ("Q", P + 8), ("Qo", P + 8),
        ("K", P + 2), ("V", P + 4), ("Kc", P + 8), ("Vc", P + 8), ("q_strides", (4 * D + 4, D)),
        ("vc_strides", (32 * D, D + 2, 16 * D)))],
], ids=lambda x: str(x))
def test_rope_validate_refuses(change, code):
    assert g.attn_f16_rope_validate(*{**ROPE, **change}.values()) == code


PAGED = dict(batch=2, total_q=5, max_q=4, q_heads=8, kv_heads=2, head_dim=D, Q=P,
             q_strides=(8 * D, D), Kc=P, kc_strides=(32 * D, 2 * D, D), Vc=P,
             vc_strides=(32 * D, D, 16 * D), num_pages=7, page_size=16, block_table=P,
             table_stride=6, max_pages=6, starts=P, kv_lens=P, O=P, o_strides=(8 * D, D),
             scale=0.0625, window=0, sinks=0)


def test_paged_validate_accepts():
    for change in ({}, {"window": 5, "sinks": 2}, {"total_q": 0, "Q": 0, "O": 0}, {"max_q": 0},
                   {"q_heads": 2}, {"q_heads": 128}, {"page_size": 24}, {"page_size": 8},
                   {"num_pages": 1, "kc_strides": (0, 2 * D, D)}, {"scale": -1.0}):
        assert g.attn_f16_paged_validate(*{**PAGED, **change}.values()) == g.OK, change


@pytest.mark.parametrize("change,code", [
    *[({k: v}, g.ERR_INVALID_ARG) for k, v in (
        ("batch", 0), ("batch", 65536), ("total_q", -1), ("max_q", -1), ("q_heads", 7),
        ("q_heads", 0), ("q_heads", 130), ("kv_heads", 0), ("head_dim", 64), ("Q", 0), ("O", 0),
        ("Kc", 0), ("Vc", 0), ("block_table", 0), ("starts", 0), ("kv_lens", 0),
        ("num_pages", 0), ("page_size", 0), ("page_size", 4), ("page_size", 20),
        ("page_size", 32776), ("max_pages", 0), ("table_stride", 5), ("window", -1),
        ("sinks", -1), ("scale", math.nan), ("scale", -math.inf), ("q_strides", (8 * D, 8)),
        ("kc_strides", (32 * D, 0, D)), ("o_strides", None))],
    *[({k: v}, g.ERR_MISALIGNED) for k, v in (
        ("Q", P + 8), ("O", P + 2), ("Kc", P + 4), ("Vc", P + 8), ("block_table", P + 2),
        ("starts", P + 1), ("kv_lens", P + 2), ("o_strides", (8 * D + 2, D)),
        ("kc_strides", (32 * D, 2 * D + 4, D)))],
], ids=lambda x: str(x))
def test_paged_validate_refuses(change, code):
    assert g.attn_f16_paged_validate(*{**PAGED, **change}.values()) == code


def test_calls_without_a_plan_are_refused(lib):
    maps = [ctypes.c_void_p(v) if k in ("cached",) else v for k, v in MAPS.items()]
    assert lib.attn_f16_paged_maps(None, *maps, None) == g.ERR_INVALID_ARG
    with pytest.raises(g.GemmError):
        g.attn_f16_rope(0, 3, 4, 0, D, 128, 0, 0, 1.0, P, P, P, (4 * D, D), P, (4 * D, D))
    with pytest.raises(g.GemmError):
        g.attn_f16_paged_fwd(0, *PAGED.values())


def test_turns_are_parts_of_a_full_turn():
    two_pi = 2 * math.pi
    t = g.attn_f16_rope_turns([0.0, two_pi / 4, two_pi / 2, 1.0, 1e-6])
    assert t[:3] == [0, 1 << 62, 1 << 63]
    for w, bits in ((1.0, t[3]), (1e-6, t[4])):
        # a double has 53 bits: 2 roundings, and the cut to a whole number
        assert abs(bits / 2.0 ** 64 - w / two_pi) <= 2 * 2.0 ** -53 * w / two_pi + 2.0 ** -64
    for bad in (-0.1, two_pi, math.inf, math.nan):
        with pytest.raises(g.GemmError):
            g.attn_f16_rope_turns([0.5, bad])
    assert g.attn_f16_rope_turns([]) == []
    assert g.rope_turns([two_pi / 2]).tolist() == [-(1 << 63)]


def test_frequencies():
    f = g.rope_frequencies(64, 10000.0)
    assert len(f) == 32 and f[0] == 1.0
    assert f[16] == pytest.approx(0.01, rel=1e-14)
    assert g.rope_frequencies(64, scaling="linear", factor=8.0) == [w / 8.0 for w in f]
    b = g.rope_frequencies(64, scaling="base", factor=4.0)
    assert b[0] == 1.0 and b[-1] == pytest.approx(f[-1] / 4.0, rel=1e-12)
    p = g.rope_frequencies(64, scaling="parts", factor=16.0, original_len=4096)
    for w, x in zip(f, p):
        turns = 4096 * w / (2 * math.pi)
        if turns >= 32:
            assert x == w
        elif turns <= 1:
            assert x == pytest.approx(w / 16.0, rel=1e-14)
        else:
            assert w / 16.0 < x < w
    for bad in (dict(rot_dim=5), dict(rot_dim=64, base=1.0), dict(rot_dim=64, scaling="x"),
                dict(rot_dim=64, scaling="parts"), dict(rot_dim=2, scaling="base", factor=2.0)):
        with pytest.raises(ValueError):
            g.rope_frequencies(**bad)
