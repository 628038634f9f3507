"""Which buffers of a maps call may lie where (attn_f16_paged_maps_overlap).
Blocks of the call's kernel read lengths while others write maps, so a buffer
that is written may not serve as another one.  No GPU."""
from __future__ import annotations

import pytest

import async_barrier_pipelined_gb300 as g
from async_barrier_pipelined_gb300 import build as gbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    return g.load()


B, PAGES, FREE, TOKENS = 5, 7, 11, 13
AT = 1 << 20      # fake addresses, never dereferenced; buffers follow one another
SIZES = dict(cached=B, added=B, block_table=(B - 1) * 20 + PAGES, free_pages=FREE, free_head=1,
             starts=B + 1, kv_lens=B, positions=TOKENS, slots=TOKENS, free_head_out=1)
WRITTEN = ("block_table", "starts", "kv_lens", "positions", "slots", "free_head_out")


def where():
    at, out = AT, {}
    for name, n in SIZES.items():
        out[name] = at
        at += 4 * n
    return out


def overlap(stride=20, max_tokens=TOKENS, num_free=FREE, **moved):
    p = {**where(), **moved}
    return g.attn_f16_paged_maps_overlap(
        B, p["cached"], p["added"], p["block_table"], stride, PAGES, p["free_pages"], num_free,
        p["free_head"], max_tokens, p["starts"], p["kv_lens"], p["positions"], p["slots"],
        p["free_head_out"])


def test_buffers_side_by_side_are_fine():
    assert overlap() == g.OK
    assert overlap(stride=1 << 60, block_table=1 << 19) == g.OK
    # inputs may share memory
    assert overlap(added=where()["cached"]) == g.OK
    assert overlap(num_free=2 * B, free_pages=where()["cached"]) == g.OK
    # a buffer of no entries is nowhere
    assert overlap(max_tokens=0, positions=where()["cached"], slots=where()["cached"]) == g.OK
    assert overlap(max_tokens=0, num_free=0, positions=0, slots=0, free_pages=0) == g.OK


@pytest.mark.parametrize("name", WRITTEN)
@pytest.mark.parametrize("other", SIZES)
def test_a_written_buffer_serves_once(name, other):
    if name == other:
        return
    p = where()
    size = lambda x: 4 * SIZES[x]
    assert overlap(**{name: p[other]}) == g.ERR_INVALID_ARG
    # by one entry, at either end
    assert overlap(**{name: p[other] + size(other) - 4}) == g.ERR_INVALID_ARG
    assert overlap(**{name: p[other] - size(name) + 4}) == g.ERR_INVALID_ARG


@pytest.mark.parametrize("name", [n for n in SIZES if n != "block_table"])
def test_rows_of_a_table_with_room_between(name):
    """Every place of a buffer against the table's rows, 20 entries apart, of 7."""
    table = 1 << 24
    rows = {r * 20 + c for r in range(B) for c in range(PAGES)}
    n = SIZES[name]
    for at in range(-20, B * 20 + 20):
        meets = any(at + i in rows for i in range(n))
        want = g.ERR_INVALID_ARG if meets else g.OK
        assert overlap(block_table=table, **{name: table + 4 * at}) == want, at


def test_lengths_cannot_be_advanced_in_place():
    p = where()
    assert overlap(kv_lens=p["cached"]) == g.ERR_INVALID_ARG
    assert overlap(free_head_out=p["free_head"]) == g.ERR_INVALID_ARG
