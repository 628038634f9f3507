"""The paged-cache calls on the GPU against plain 64-bit forms: the maps of a
step, rotary positions (with the cache write, and the gradient), and causal
attention over pages, at the sizes and masks where they can go wrong."""
from __future__ import annotations

import random

import pytest

from tests import paged_ref as ref

pytestmark = pytest.mark.gpu
D = ref.D


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


def done(plan, want=0):
    import torch
    torch.cuda.synchronize()
    assert plan.status() == want


# ------------------------------------------------------------------ maps

def run_maps(g, plan, cached, added, table, free, head, page, most):
    import torch
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    tab = t(table)
    m = g.paged_maps(plan, t(cached), t(added), tab, t(free), t([head]), page, most)
    torch.cuda.synchronize()
    return (m.starts.tolist(), m.kv_lens.tolist(), m.positions.tolist(), m.slots.tolist(),
            tab.tolist(), m.free_head.item())


def maps_problem(batch, most_cached, most_added, page, seed):
    r = random.Random(seed)
    cached = [r.choice([0, r.randint(0, most_cached)]) for _ in range(batch)]
    added = [r.choice([0, 1, r.randint(0, most_added)]) for _ in range(batch)]
    wide = max(-(-(c + n) // page) for c, n in zip(cached, added)) + 1
    need = sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(cached, added))
    held = sum(-(-c // page) for c in cached)
    ids = list(range(held + need + 9))
    r.shuffle(ids)
    table, at = [], 0
    for c in cached:
        k = -(-c // page)
        table.append(ids[at:at + k] + [-5] * (wide - k))
        at += k
    return cached, added, table, ids[at:], need


@pytest.mark.parametrize("batch,most_cached,most_added,page", [
    (1, 0, 1, 16), (1, 50, 5000, 16), (7, 100, 40, 1), (64, 4000, 1, 16), (255, 90, 9, 8),
    (1024, 300, 20, 24), (1025, 300, 20, 32), (3000, 40, 3, 7), (5000, 0, 2, 1000),
    (20, 3000, 3000, 128)])
def test_maps(g, plan, batch, most_cached, most_added, page):
    cached, added, table, free, need = maps_problem(batch, most_cached, most_added, page, batch)
    for head, room in ((0, 0), (3, 5)):
        most = sum(added) + room
        want = ref.maps_reference(cached, added, table, free, head, page, most)
        got = run_maps(g, plan, cached, added, table, free, head, page, most)
        assert got == want[:6]
        done(plan, g.ERR_BAD_INDEX if want[6] else g.OK)
        assert not want[6]


@pytest.mark.parametrize("what", ["free list ends", "free head out", "negative", "too long",
                                  "too many tokens", "hole in the table", "far too many tokens"])
def test_maps_report_what_is_out_of_range(g, plan, what):
    cached, added, table, free, need = maps_problem(40, 200, 60, 16, 5)
    head, most = 0, sum(added) + 3
    if what == "free list ends":
        free = free[:need - 3]
    elif what == "free head out":
        head = len(free) + 4
    elif what == "negative":
        cached[3], added[5] = -4, -1
    elif what == "too long":
        cached[2], added[9] = 1 << 30, 1 << 30
        free = free + list(range(1000, 1100))
    elif what == "too many tokens":
        most = sum(added) // 2
    elif what == "hole in the table":
        b = next(b for b in range(40) if cached[b] % 16 and added[b])
        table[b][cached[b] // 16] = -1
    else:
        added[0], added[1], most = (1 << 31) - 1, (1 << 31) - 1, 100
    want = ref.maps_reference(cached, added, table, free, head, 16, most)
    assert want[6]
    assert run_maps(g, plan, cached, added, table, free, head, 16, most) == want[:6]
    done(plan, g.ERR_BAD_INDEX)


def test_maps_refuses(g, plan):
    import torch
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    ok = dict(cached=z(3), added=z(3), block_table=z(3, 4), free_pages=z(5), free_head=z(1),
              page_size=16, max_tokens=4)
    g.paged_maps(plan, **ok)
    for change in (dict(added=z(4)), dict(cached=z(3).long()), dict(block_table=z(2, 4)),
                   dict(free_head=z(2)), dict(added=z(3).cpu()), dict(block_table=z(4, 3).t())):
        with pytest.raises(ValueError):
            g.paged_maps(plan, **{**ok, **change})
    for change in (dict(page_size=0), dict(max_tokens=-1)):
        with pytest.raises(g.GemmError):
            g.paged_maps(plan, **{**ok, **change})
    with pytest.raises(g.GemmError):   # no request
        g.paged_maps(plan, **{**ok, "cached": z(0), "added": z(0), "block_table": z(0, 4)})
    done(plan)


# ------------------------------------------------------------------ rope

def rope_bound(x, y, factor):
    """Half a binary16 step of the result, and FP32: the angle is off by
    2^-24 of a half turn (pi 2^-24) and each cosine and sine by 2^-23, the
    products and their sum by three roundings: 8 * 2^-24 (|x0| + |x1|) * factor
    covers them; half a step below the normal range."""
    import torch
    mag = x.double().abs().amax(-1, keepdim=True) * 2 * abs(factor)
    return 2.0 ** -11 * y.abs() + 8 * 2.0 ** -24 * mag + 2.0 ** -25


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,rot,far,factor,inverse", [
    (1, 1, 16, 10, 1.0, False), (3, 5, 256, 1 << 20, 1.0, False), (129, 33, 64, 9000, 1.25, True),
    (17, 16, 240, 1 << 30, 0.5, False), (0, 4, 32, 5, 1.0, False), (1000, 2, 128, 70, 1.0, True)])
def test_rotary(g, plan, layout, tokens, heads, rot, far, factor, inverse):
    import torch
    gen = torch.Generator().manual_seed(tokens)
    freq = torch.tensor(g.rope_frequencies(rot), dtype=torch.float64)
    turns = g.rope_turns(freq).cuda()
    x = torch.randn(tokens, heads, D, generator=gen).half().cuda()
    pos = torch.randint(0, far, (tokens,), generator=gen, dtype=torch.int32).cuda()
    if tokens > 1:
        pos[0], pos[1] = 0, far - 1
    want = ref.rope_reference(x, pos, freq, layout, factor, inverse)
    kw = dict(layout=layout, factor=factor, inverse=inverse)
    y = g.rotary(plan, x, pos, turns, **kw)
    done(plan)
    # a double angle of p radians is itself off by 2^-52 p
    extra = far * 2.0 ** -51 * x.double().abs().amax().item() if tokens else 0
    assert ((y.double() - want).abs() <= rope_bound(x, want, factor) + extra).all()
    xs = ref.transposed_rows(x)                       # other strides, other output strides
    buf = torch.full((tokens, heads + 1, D), 3.0, dtype=torch.float16, device="cuda")
    z = g.rotary(plan, xs, pos, turns, out=buf[:, :heads], **kw)
    assert torch.equal(z, y) and (buf[:, heads] == 3.0).all()
    x2 = x.clone()
    assert torch.equal(g.rotary(plan, x2, pos, turns, out=x2, **kw), y)   # in place
    done(plan)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_gradient(g, plan, layout):
    """<dy, R x> has the gradient R^T dy: against the formula, and against
    differences of the 64-bit form."""
    import torch
    gen = torch.Generator().manual_seed(2)
    freq = torch.tensor(g.rope_frequencies(96), dtype=torch.float64)
    x = torch.randn(9, 3, D, generator=gen).half().cuda()
    dy = torch.randn(9, 3, D, generator=gen).half().cuda()
    pos = torch.randint(0, 5000, (9,), generator=gen, dtype=torch.int32).cuda()
    dx = g.rotary(plan, dy, pos, g.rope_turns(freq).cuda(), layout=layout, factor=1.5,
                  inverse=True)
    done(plan)
    x64 = x.double().requires_grad_()
    (ref.rope_reference(x64, pos, freq, layout, 1.5) * dy.double()).sum().backward()
    bound = rope_bound(dy, x64.grad, 1.5) + 5000 * 2.0 ** -51 * 8
    assert ((dx.double() - x64.grad).abs() <= bound).all()
    step, at = 2.0 ** -10, [(0, 0, 0), (3, 1, 47), (8, 2, 48), (5, 0, 95), (2, 2, 200)]
    for i in at:
        up, down = x.double(), x.double()
        up[i] += step
        down[i] -= step
        f = lambda v: (ref.rope_reference(v, pos, freq, layout, 1.5) * dy.double()).sum()
        diff = (f(up) - f(down)) / (2 * step)      # linear: exact to 64-bit rounding
        assert abs(diff - dx[i].double()) <= bound[i] + 1e-9


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,hq,hk,rot,page,head_major", [
    (1, 16, 4, 256, 16, False), (37, 8, 8, 64, 8, True), (300, 5, 1, 16, 24, False),
    (64, 0, 3, 128, 1, False), (50, 40, 20, 256, 64, True)])
def test_rotary_to_cache(g, plan, layout, tokens, hq, hk, rot, page, head_major):
    import torch
    gen = torch.Generator().manual_seed(tokens)
    freq = torch.tensor(g.rope_frequencies(rot, 500000.0), dtype=torch.float64)
    turns = g.rope_turns(freq).cuda()
    x = torch.randn(tokens, hq + 2 * hk, D, generator=gen).half().cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    pages = tokens // page + 4
    pos = torch.randint(0, 100000, (tokens,), generator=gen, dtype=torch.int32).cuda()
    slots = torch.randperm(pages * page, generator=gen)[:tokens].to(torch.int32).cuda()
    if tokens > 8:
        slots[3] = -1
    shape = (pages, hk, page, D) if head_major else (pages, page, hk, D)
    kc = torch.full(shape, 7.0, dtype=torch.float16, device="cuda")
    vc = torch.full(shape, 9.0, dtype=torch.float16, device="cuda")
    if head_major:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    if hq:
        qo = g.rotary_to_cache(plan, q, k, v, pos, slots, turns, kc, vc, layout=layout)
        want = ref.rope_reference(q, pos, freq, layout, 1.0)
        assert ((qo.double() - want).abs() <= rope_bound(q, want, 1.0) + 1e-9).all()
    else:
        g.attn_f16_rope(plan.handle, tokens, 0, hk, D, rot, ["half", "interleaved"].index(layout),
                        0, 1.0, turns.data_ptr(), pos.data_ptr(), 0, None, 0, None, k.data_ptr(),
                        k.stride()[:2], v.data_ptr(), v.stride()[:2], slots.data_ptr(),
                        kc.data_ptr(), kc.stride()[:3], vc.data_ptr(), vc.stride()[:3], pages,
                        page, torch.cuda.current_stream().cuda_stream)
    done(plan)
    wk = ref.rope_reference(k, pos, freq, layout, 1.0)
    written = torch.zeros(pages, page, dtype=torch.bool)
    for t in range(tokens):
        s = int(slots[t])
        if s < 0:
            continue
        written[s // page, s % page] = True
        got = kc[s // page, s % page].double()
        assert ((got - wk[t]).abs() <= rope_bound(k[t], wk[t], 1.0) + 1e-9).all()
        assert torch.equal(vc[s // page, s % page], v[t])
    rest = ~written.cuda()
    assert (kc[rest] == 7.0).all() and (vc[rest] == 9.0).all()


def test_rotary_reports_slots_out_of_range(g, plan):
    import torch
    turns = g.rope_turns(g.rope_frequencies(64)).cuda()
    x = torch.randn(3, 4, D, device="cuda").half()
    k = torch.randn(3, 2, D, device="cuda").half()
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    for bad in (64, -2, (1 << 31) - 1, -(1 << 31)):
        kc = torch.full((4, 16, 2, D), 7.0, dtype=torch.float16, device="cuda")
        vc = kc.clone()
        slots = torch.tensor([5, bad, 63], dtype=torch.int32, device="cuda")
        g.rotary_to_cache(plan, x, k, k, pos, slots, turns, kc, vc)
        done(plan, g.ERR_BAD_INDEX)
        flat = kc.view(64, 2, D)
        assert torch.equal(vc.view(64, 2, D)[5], k[0]) and torch.equal(
            vc.view(64, 2, D)[63], k[2])
        flat[5], flat[63] = 7.0, 7.0
        assert (flat == 7.0).all()


def test_rotary_refuses(g, plan):
    import torch
    turns = g.rope_turns(g.rope_frequencies(64)).cuda()
    x = torch.zeros(3, 4, D, dtype=torch.float16, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    g.rotary(plan, x, pos, turns)
    for args, kw in (((x.float(), pos, turns), {}), ((x, pos[:2], turns), {}),
                     ((x, pos.long(), turns), {}), ((x, pos, turns.int()), {}),
                     ((x[..., :128], pos, turns), {}), ((x.cpu(), pos, turns), {}),
                     ((x, pos, turns), {"layout": "both"}), ((x, pos, turns), {"out": x[:2]}),
                     ((x.transpose(1, 2), pos, turns), {})):
        with pytest.raises(ValueError):
            g.rotary(plan, *args, **kw)
    with pytest.raises(g.GemmError):
        g.rotary(plan, x, pos, turns[:20])      # 40 numbers: no multiple of 16
    with pytest.raises(g.GemmError):
        g.rotary(plan, x, pos, turns, factor=float("inf"))
    done(plan)


# ------------------------------------------------------------------ attention

def run_attention(g, plan, pr, **kw):
    return g.paged_attention(plan, kw.pop("q", pr.q.cuda()), pr.kc, pr.vc, pr.table, pr.starts,
                             pr.kv_lens, kw.pop("max_q", pr.max_q), window=pr.window,
                             sinks=pr.sinks, **kw)


def check(o, pr, **kw):
    want, bound = pr.reference(**kw)
    err = (o.double() - want).abs()
    assert (err <= bound).all(), (f"{int((~(err <= bound)).sum())} off, worst "
                                  f"{(err / bound).nan_to_num(1e9).max().item():.3g} of the bound")


def ragged(seed, batch, most_cached, most_new, few=0.3):
    r = random.Random(seed)
    return [(r.randint(0, most_cached), 0 if r.random() < few / 3 else
             (1 if r.random() < few else r.randint(1, most_new))) for _ in range(batch)]


ATTENTION = {
    "one key": dict(lens=[(0, 1)], q_heads=1, kv_heads=1, page=8),
    "one token": dict(lens=[(999, 1)], q_heads=4, kv_heads=1, page=16),
    "block edges": dict(lens=[(126, 1), (127, 1), (128, 1), (255, 1), (256, 1), (0, 1)],
                        q_heads=8, kv_heads=2, page=16),
    "decode": dict(lens=ragged(1, 40, 3000, 1, 0), q_heads=16, kv_heads=4, page=16),
    "decode shared by none": dict(lens=ragged(2, 9, 700, 1, 0), q_heads=3, kv_heads=3, page=32),
    "decode one key head": dict(lens=ragged(3, 5, 2000, 1, 0), q_heads=64, kv_heads=1, page=64),
    "decode odd group": dict(lens=ragged(4, 12, 900, 1, 0), q_heads=14, kv_heads=2, page=24),
    "decode large pages": dict(lens=ragged(5, 7, 3000, 1, 0), q_heads=8, kv_heads=2, page=1000),
    "decode empty requests": dict(lens=[(0, 0), (50, 1), (70, 0), (0, 1), (0, 0)], q_heads=4,
                                  kv_heads=2, page=16),
    "draft": dict(lens=ragged(6, 20, 1500, 6, 0.2), q_heads=16, kv_heads=4, page=16),
    "draft wide": dict(lens=ragged(7, 6, 1500, 4, 0.2), q_heads=32, kv_heads=2, page=8),
    "prompt": dict(lens=[(0, 300)], q_heads=4, kv_heads=2, page=16),
    "prompt odd": dict(lens=[(0, 257), (0, 1), (0, 129), (0, 515)], q_heads=3, kv_heads=1,
                       page=24),
    "chunk": dict(lens=[(1000, 513)], q_heads=8, kv_heads=4, page=64),
    "chunk seven": dict(lens=[(77, 200), (3, 91)], q_heads=7, kv_heads=1, page=40),
    "chunk wide group": dict(lens=[(333, 70), (3, 91)], q_heads=48, kv_heads=1, page=128),
    "mixed": dict(lens=ragged(8, 30, 1200, 300), q_heads=8, kv_heads=2, page=16),
    "mixed page 8": dict(lens=ragged(9, 15, 500, 200), q_heads=4, kv_heads=4, page=8),
    "mixed page 256": dict(lens=ragged(10, 12, 2500, 400), q_heads=6, kv_heads=2, page=256),
    "decode window": dict(lens=ragged(11, 30, 3000, 1, 0), q_heads=8, kv_heads=2, page=16,
                          window=300, sinks=4),
    "decode window 1": dict(lens=ragged(12, 9, 500, 1, 0), q_heads=4, kv_heads=2, page=8,
                            window=1),
    "decode window no sinks": dict(lens=ragged(13, 9, 3000, 1, 0), q_heads=4, kv_heads=2,
                                   page=32, window=129),
    "decode many sinks": dict(lens=ragged(14, 9, 3000, 2, 0), q_heads=4, kv_heads=1, page=16,
                              window=50, sinks=200),
    "chunk window": dict(lens=[(1500, 700), (0, 900), (40, 1)], q_heads=4, kv_heads=2, page=16,
                         window=200, sinks=5),
    "chunk narrow window": dict(lens=[(500, 300), (0, 400)], q_heads=2, kv_heads=2, page=8,
                                window=3, sinks=1),
    "chunk window over all": dict(lens=[(500, 300)], q_heads=4, kv_heads=1, page=48,
                                  window=5000, sinks=5000),
    "sinks without a window": dict(lens=[(300, 40)], q_heads=4, kv_heads=1, page=16, window=0,
                                   sinks=9),
}


@pytest.mark.parametrize("name", ATTENTION)
def test_attention(g, plan, name):
    pr = ref.PagedProblem(**ATTENTION[name], seed=len(name))
    o = run_attention(g, plan, pr)
    done(plan)
    check(o, pr)


@pytest.mark.parametrize("name", ["decode", "draft", "mixed", "chunk window"])
def test_attention_strides_padding_and_streams(g, plan, name):
    """Head-major caches, strided queries and outputs, rows past the last
    request, a max_q above the largest, and another stream."""
    import torch
    pr = ref.PagedProblem(**ATTENTION[name], seed=3, head_major=True, extra_rows=5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q = ref.transposed_rows(pr.q.cuda())
        buf = torch.full((q.shape[0], pr.q_heads + 1, D), 3.0, dtype=torch.float16,
                         device="cuda")
        o = run_attention(g, plan, pr, q=q, out=buf[:, 1:])
    done(plan)
    check(o, pr)
    assert (buf[:, 0] == 3.0).all()
    o2 = run_attention(g, plan, pr, max_q=pr.max_q + 3)
    done(plan)
    check(o2, pr)


@pytest.mark.parametrize("name", ["decode", "draft", "mixed", "chunk"])
def test_attention_is_the_same_again(g, plan, name):
    import torch
    pr = ref.PagedProblem(**ATTENTION[name], seed=4)
    first = run_attention(g, plan, pr)
    for _ in range(5):
        assert torch.equal(run_attention(g, plan, pr), first)
    done(plan)


@pytest.mark.parametrize("scale,q_scale", [(1.0, 3.0), (-0.0625, 1.0), (0.0, 1.0), (5.0, 20.0)])
def test_attention_scales(g, plan, scale, q_scale):
    """Weights on one key, spread evenly, and scores in the thousands."""
    for lens in ([(700, 1), (30, 1)], [(100, 260)]):
        pr = ref.PagedProblem(lens, 4, 2, 16, seed=6, q_scale=q_scale)
        o = run_attention(g, plan, pr, scale=scale)
        done(plan)
        check(o, pr, scale=scale)


def test_attention_infinite_scores(g, plan):
    """A key whose score overflows to -inf has no weight."""
    import torch
    for lens in ([(300, 1)], [(40, 300)]):
        pr = ref.PagedProblem(lens, 2, 1, 16, seed=8)
        pr.q.fill_(60000.0)
        for k in pr.keys:
            k.fill_(0.0)
            k[::3] = -60000.0
        c, n = lens[0]
        for i in range(-(-(c + n) // 16)):
            rows = pr.keys[0][16 * i:16 * i + 16]
            pr.kc[int(pr.table[0, i]), :rows.shape[0]] = rows.cuda()
        o = run_attention(g, plan, pr, scale=1e30)
        done(plan)
        v = pr.values[0].cuda().double()
        keep = torch.arange(c + n, device="cuda") % 3 != 0
        for i in (0, n // 2, n - 1):
            see = keep & (torch.arange(c + n, device="cuda") <= c + i)
            want = v[see].mean(0)[0]
            assert ((o[i, 0].double() - want).abs() <= 2.0 ** -10 * v[see].abs().mean(0)[0]
                    + (c + n) * 2.0 ** -23).all()


def test_attention_rows_that_see_nothing(g, plan):
    """More new tokens than keys: the first ones stand before the cache."""
    import torch
    for n, length in ((5, 3), (300, 200), (4, 0), (2, 0)):
        pr = ref.PagedProblem([(0, n), (20, 3)], 4, 2, 16, seed=9)
        pr.kv_lens[0] = length
        o = run_attention(g, plan, pr)
        done(plan)
        assert (o[:n - length] == 0).all()
        short = ref.PagedProblem([(0, n), (20, 3)], 4, 2, 16, seed=9)
        short.lens = [(0, length), (20, 3)]
        short.keys[0], short.values[0] = short.keys[0][:length], short.values[0][:length]
        short.q = short.q[n - length:]
        check(o[n - length:], short)


def test_attention_offsets_past_32_bits(g, plan):
    """Pages whose elements lie more than 2^32 bytes and 2^31 elements in."""
    import torch
    for lens in ([(900, 1), (5, 1)], [(300, 270)]):
        far = (1 << 31) // (64 * 4 * D) + 1
        pr = ref.PagedProblem(lens, 8, 4, 64, seed=10, far=far)
        o = run_attention(g, plan, pr)
        done(plan)
        check(o, pr)
        del pr, o
        torch.cuda.empty_cache()


def test_attention_reports_what_is_out_of_range(g, plan):
    import torch
    base = dict(q_heads=4, kv_heads=2, page=16, seed=11)
    for lens in ([(100, 1), (60, 1), (200, 1)], [(100, 70), (60, 90), (200, 80)]):
        good = ref.PagedProblem(lens, **base)
        want = run_attention(g, plan, good)
        done(plan)
        n0, n1 = lens[0][1], lens[1][1]
        keep = list(range(0, n0)) + list(range(n0 + n1, sum(n for _, n in lens)))

        def others_hold(pr, **kw):
            o = run_attention(g, plan, pr, **kw)
            done(plan, g.ERR_BAD_INDEX)
            assert torch.equal(o[keep], want[keep])

        for bad in (-1, good.pages, 1 << 30, -(1 << 31)):
            pr = ref.PagedProblem(lens, **base)
            pr.table[1, 2] = bad
            others_hold(pr)
        for length in (-5, 1 << 30, (1 << 31) - 1):
            pr = ref.PagedProblem(lens, **base)
            pr.kv_lens[1] = length
            pr.table[1] = pr.table[1].clamp(0, good.pages - 1)
            others_hold(pr)
        pr = ref.PagedProblem(lens, **base)
        pr.starts[3] = 1 << 30
        run_attention(g, plan, pr)
        done(plan, g.ERR_BAD_INDEX)
        pr = ref.PagedProblem(lens, **base)
        pr.starts[1], pr.starts[2] = n0 + n1, n0
        run_attention(g, plan, pr)
        done(plan, g.ERR_BAD_INDEX)
        if n0 > 1:
            pr = ref.PagedProblem(lens, **base)
            run_attention(g, plan, pr, max_q=3)
            done(plan, g.ERR_BAD_INDEX)
    o = run_attention(g, plan, good)       # and nothing is left behind
    done(plan)
    assert torch.equal(o, want)


def test_attention_refuses(g, plan):
    import torch
    pr = ref.PagedProblem([(30, 2)], 4, 2, 16)
    q = pr.q.cuda()
    ok = dict(Q=q, K_cache=pr.kc, V_cache=pr.vc, block_table=pr.table, starts=pr.starts,
              kv_lens=pr.kv_lens, max_q=2)
    g.paged_attention(plan, **ok)
    for change in (dict(Q=q.float()), dict(Q=q[..., :64]), dict(K_cache=pr.kc[:1]),
                   dict(starts=pr.starts[:1]), dict(block_table=pr.table.long()),
                   dict(kv_lens=pr.kv_lens.cpu()), dict(out=q[:1]),
                   dict(V_cache=pr.vc.transpose(2, 3))):
        with pytest.raises(ValueError):
            g.paged_attention(plan, **{**ok, **change})
    for change in (dict(Q=q[:, :3]), dict(max_q=-1), dict(window=-1), dict(sinks=-1),
                   dict(scale=float("nan")),
                   dict(K_cache=pr.kc[:, :12], V_cache=pr.vc[:, :12])):
        with pytest.raises(g.GemmError):
            g.paged_attention(plan, **{**ok, **change})
    empty = g.paged_attention(plan, **{**ok, "Q": q[:0]})
    assert empty.shape == (0, 4, D)
    done(plan)


def test_step_in_a_graph(g, plan):
    """Maps, rotation with the cache write, and attention, captured once and
    replayed for steps with other lengths."""
    import torch
    page, hq, hk, batch, wide = 16, 8, 2, 5, 12
    gen = torch.Generator().manual_seed(12)
    turns = g.rope_turns(g.rope_frequencies(128)).cuda()
    freq = torch.tensor(g.rope_frequencies(128), dtype=torch.float64)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cached, added = i32([0] * batch), i32([3] * batch)
    table = torch.full((batch, wide), -1, dtype=torch.int32, device="cuda")
    free, head = torch.randperm(100, generator=gen).to(torch.int32).cuda(), i32([0])
    kc = torch.full((100, page, hk, D), float("nan"), dtype=torch.float16, device="cuda")
    vc = kc.clone()
    x = torch.zeros(16, hq + 2 * hk, D, dtype=torch.float16, device="cuda")

    def step():
        m = g.paged_maps(plan, cached, added, table, free, head, page, 16)
        q = g.rotary_to_cache(plan, x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], m.positions,
                              m.slots, turns, kc, vc)
        return m, g.paged_attention(plan, q, kc, vc, table, m.starts, m.kv_lens, 4,
                                    window=20, sinks=2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        m, o = step()
    lens = [0] * batch
    keys = [torch.zeros(0, hk, D, dtype=torch.float64) for _ in range(batch)]
    values = [torch.zeros(0, hk, D, dtype=torch.float16) for _ in range(batch)]
    r = random.Random(1)
    for _ in range(8):
        new = [r.choice([0, 1, 1, 3, 4]) for _ in range(batch)]
        if sum(new) > 16:
            new = [3] * batch
        x.copy_(torch.randn(x.shape, generator=gen).half())
        cached.copy_(i32(lens))
        added.copy_(i32(new))
        graph.replay()
        done(plan)
        assert m.kv_lens.tolist() == [a + b for a, b in zip(lens, new)]
        pos = m.positions
        q64 = ref.rope_reference(x[:, :hq], pos, freq, "half", 1.0).half()
        k64 = ref.rope_reference(x[:, hq:hq + hk], pos, freq, "half", 1.0).cpu()
        at = 0
        for b, n in enumerate(new):
            keys[b] = torch.cat((keys[b], k64[at:at + n].half().double()))
            values[b] = torch.cat((values[b], x[at:at + n, hq + hk:].cpu()))
            at += n
        pr = ref.PagedProblem([(a, b) for a, b in zip(lens, new)], hq, hk, page, window=20,
                              sinks=2, extra_rows=16 - sum(new))
        pr.keys, pr.values, pr.q = keys, values, q64
        want, bound = pr.reference()
        # q and k may be rounded the other way: a step of 2^-10 in a factor of the scores
        assert ((o.double() - want).abs() <= bound + 0.05).all()
        assert ((o.double() - want).norm() <= 2e-3 * want.norm())
        lens = [a + b for a, b in zip(lens, new)]
        head.copy_(m.free_head)


@pytest.mark.parametrize("lens", [[(500, 1), (900, 1)], [(500, 3), (900, 700)], [(500, 400)]],
                         ids=["few", "both", "many"])
def test_attention_bounded_wait(g, lens):
    """The first copy of worker 0 or 1 is left out (the test-only fault option):
    the call must end with ERR_TIMEOUT, and the next ones must be right."""
    pr = ref.PagedProblem(lens, 8, 2, 16, seed=13)
    with g.Plan(0) as own:
        run_attention(g, own, pr)
        done(own)
        own.set_option(g.OPT_TIMEOUT_NS, 20_000_000)
        for unit in (0, 1):
            own.set_option(g.OPT_FAULT_UNIT, unit)
            run_attention(g, own, pr)
            done(own, g.ERR_TIMEOUT)
        own.set_option(g.OPT_FAULT_UNIT, -1)
        for _ in range(2):
            o = run_attention(g, own, pr)
            done(own)
            check(o, pr)


@pytest.mark.parametrize("limit", [1, 2, 7, 40])
def test_attention_sm_limit(g, limit):
    """Fewer workers: other cuts of the same tiles."""
    with g.Plan(0) as own:
        own.set_option(g.OPT_SM_LIMIT, limit)
        for lens in ([(300, 1), (0, 1), (700, 1)], [(100, 200), (5, 1), (600, 60)]):
            pr = ref.PagedProblem(lens, 8, 2, 16, seed=14)
            o = run_attention(g, own, pr)
            done(own)
            check(o, pr)


@pytest.mark.parametrize("what", [
    dict(lens=[(1300 + 37 * i, 700) for i in range(8)], q_heads=16, kv_heads=4, page=16),
    dict(lens=[(3000, 400), (0, 1), (10, 0), (2000, 1111), (50, 3), (2500, 600)], q_heads=12,
         kv_heads=6, page=64),
    dict(lens=[(2500, 2500), (100, 1)], q_heads=8, kv_heads=4, page=24, window=1500, sinks=9),
    dict(lens=[(1400 + i, 30) for i in range(300)], q_heads=8, kv_heads=1, page=32)],
    ids=["many", "mixed", "window", "short queries"])
@pytest.mark.parametrize("limit", [0, 6, 30])
def test_attention_many_long_tiles(g, limit, what):
    """Steps whose tiles are dealt out whole (with all workers or some of them)."""
    with g.Plan(0) as own:
        own.set_option(g.OPT_SM_LIMIT, limit)
        pr = ref.PagedProblem(**what, seed=16)
        o = run_attention(g, own, pr)
        done(own)
        check(o, pr)


def test_attention_many_requests(g, plan):
    """More requests than the kernels keep in shared memory, empty ones among them."""
    for most in (1, 90):
        pr = ref.PagedProblem(ragged(15, 700, 90, most, 0.6), 2, 1, 8, seed=15)
        o = run_attention(g, plan, pr)
        done(plan)
        check(o, pr)


def test_calls_take_a_stream_and_outputs(g, plan):
    """`stream` (an object or a handle) and `out` of every call; a tensor that a
    call allocates belongs to the call's stream."""
    import torch
    pr = ref.PagedProblem(ATTENTION["mixed"]["lens"], 8, 2, 16, seed=16)
    q = pr.q.cuda()
    want = run_attention(g, plan, pr, q=q)
    freq = torch.tensor(g.rope_frequencies(64), dtype=torch.float64)
    turns = g.rope_turns(freq).cuda()
    pos = torch.arange(q.shape[0], dtype=torch.int32, device="cuda")
    rotated = g.rotary(plan, q, pos, turns)
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    added = z(3) + 2
    table, free = z(3, 4) - 1, torch.arange(9, dtype=torch.int32, device="cuda")
    maps = g.paged_maps(plan, z(3), added, table, free, z(1), 16, 7)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        o = run_attention(g, plan, pr, q=q, stream=stream)
        y = g.rotary(plan, q, pos, turns, stream=stream)
        m = g.paged_maps(plan, z(3), added, table, free, z(1), 16, 7, stream=stream)
        side.synchronize()
        assert torch.equal(o, want) and torch.equal(y, rotated)
        assert all(torch.equal(a, b) for a, b in zip(m, maps))
    again = g.paged_maps(plan, z(3), added, table, free, z(1), 16, 7, out=maps)
    assert all(a.data_ptr() == b.data_ptr() for a, b in zip(again, maps))
    for bad in (maps._replace(slots=z(6)), maps._replace(starts=z(4).float())):
        with pytest.raises(ValueError):
            g.paged_maps(plan, z(3), added, table, free, z(1), 16, 7, out=bad)
    o = torch.empty_like(q)
    assert run_attention(g, plan, pr, q=q, out=o) is o or torch.equal(o, want)
    done(plan)
