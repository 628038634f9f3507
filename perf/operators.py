"""The operators of a serving step over a paged cache, as cases to be timed.

A step of a program that serves a model with 256-wide heads from a paged
key/value cache makes three kinds of calls:

  maps       once per step: from the requests' lengths, the pages that the new
             tokens take, and each token's request offset, position and slot;
  rope       once per layer: rotary positions of the new queries and keys, and
             the new keys and values into their slots (or, in training, the
             rotation alone and its gradient);
  attention  once per layer: the new tokens' queries over their request's
             pages, causal, with grouped heads, and with a sliding window and
             first tokens that stay visible where a layer has them.

``own`` false: the operators in plain torch operations.  ``own`` true: the
calls of async_barrier_pipelined_gb300.
"""
import math
import random

import torch

own = False

D = 256             # head dimension
PLAIN_SCORES = 1 << 28   # most scores the plain form holds at a time (FP32: 1 GB)
PLAIN_CACHE = 1 << 28    # most gathered key (or value) elements it holds at a time

_plans = []


def _plan():
    """The program's one plan, made on first use."""
    import async_barrier_pipelined_gb300 as g
    if not _plans:
        _plans.append(g.Plan(0))
    return _plans[0]


def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One token for each of a few dozen requests: what every step of token
        # generation begins with.  Latency.
        dict(name="maps-decode-48", op="maps", batch=48, new_lo=1, new_hi=1, ctx=4096, page=16,
             lens_seed=11),
        # A step that admits many prompts at once, next to running requests.
        dict(name="maps-prompts-600", op="maps", batch=600, new_lo=1, new_hi=1500, ctx=9000,
             page=32, lens_seed=12),
        # The new tokens of a generation step: queries and keys rotated, keys
        # and values into their slots.  Latency.
        dict(name="rope-decode-48", op="rope", tokens=48, q_heads=16, kv_heads=4, rot=256,
             layout="half", scaling="none", cache=True, inverse=False, page=16, far=8192),
        # A long prompt chunk, far positions with frequencies scaled by parts.
        dict(name="rope-chunk-8192", op="rope", tokens=8192, q_heads=16, kv_heads=8, rot=128,
             layout="half", scaling="parts", cache=True, inverse=False, page=64, far=131072),
        # Interleaved pairs, an odd token count, every head its own keys.
        dict(name="rope-chunk-2999", op="rope", tokens=2999, q_heads=16, kv_heads=16, rot=256,
             layout="interleaved", scaling="linear", cache=True, inverse=False, page=16,
             far=40000),
        # Training: the gradient of the rotation of a batch's queries.
        dict(name="rope-gradient-16384", op="rope", tokens=16384, q_heads=16, kv_heads=0, rot=64,
             layout="half", scaling="none", cache=False, inverse=True, page=16, far=4096),
        # Token generation for a few short conversations.  Latency.
        dict(name="attention-decode-6", op="attention", batch=6, new_lo=1, new_hi=1, ctx_lo=200,
             ctx_hi=1500, q_heads=16, kv_heads=4, page=16, window=0, sinks=0, lens_seed=21),
        # Token generation for a full batch of long ragged conversations.
        dict(name="attention-decode-64", op="attention", batch=64, new_lo=1, new_hi=1,
             ctx_lo=500, ctx_hi=16000, q_heads=16, kv_heads=4, page=16, window=0, sinks=0,
             lens_seed=22),
        # A few drafted tokens checked at once, on a layer with a window and
        # first tokens that stay visible.
        dict(name="attention-draft-40-window", op="attention", batch=40, new_lo=2, new_hi=5,
             ctx_lo=100, ctx_hi=20000, q_heads=16, kv_heads=2, page=32, window=2048, sinks=4,
             lens_seed=23),
        # Short prompts and running requests in one step.
        dict(name="attention-mixed-50", op="attention", batch=50, new_lo=1, new_hi=700, ctx_lo=1,
             ctx_hi=5000, q_heads=16, kv_heads=8, page=16, window=0, sinks=0, lens_seed=24),
        # A chunk of a long prompt on a layer with a window.
        dict(name="attention-chunk-4001-window", op="attention", batch=1, new_lo=4001,
             new_hi=4001, ctx_lo=6000, ctx_hi=6000, q_heads=16, kv_heads=4, page=64, window=1024,
             sinks=8, lens_seed=25),
        # The largest: a chunk of 4096 new tokens behind 8192 cached ones.
        dict(name="attention-chunk-4096", op="attention", batch=1, new_lo=4096, new_hi=4096,
             ctx_lo=8192, ctx_hi=8192, q_heads=16, kv_heads=16, page=128, window=0, sinks=0,
             lens_seed=26),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["maps", "rope", "rope", "attention", "attention", "attention"])
    page = rng.choice([8, 16, 24, 32, 64, 128, 256])
    if op == "maps":
        mixed = rng.random() < 0.5
        return dict(op="maps", batch=_log(rng, 1, 600), new_lo=1,
                    new_hi=_log(rng, 2, 1500) if mixed else 1, ctx=_log(rng, 10, 9000),
                    page=page, lens_seed=rng.randrange(1 << 30))
    heads = rng.choice([(16, 16), (16, 8), (16, 4), (16, 2), (16, 1), (12, 4), (8, 8), (5, 1),
                        (14, 2), (1, 1), (64, 8)])
    if op == "rope":
        cache = rng.random() < 0.7
        most = 8192 * 16 // heads[0]
        return dict(op="rope", tokens=_log(rng, 1, most), q_heads=heads[0],
                    kv_heads=heads[1] if cache else 0, rot=16 * rng.randint(1, 16),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "parts"]), cache=cache,
                    inverse=(not cache) and rng.random() < 0.5, page=page,
                    far=_log(rng, 100, 1000000))
    window = rng.choice([0, 0, _log(rng, 1, 4096)])
    sinks = rng.choice([0, 1, 4, 130]) if window else 0
    kind = rng.choice(["decode", "draft", "mixed", "chunk"])
    if kind in ("decode", "draft"):
        batch = _log(rng, 1, 200)
        hi = max(2, min(32000, 1 << 20, (1 << 21) // (batch * heads[1])))
        return dict(op="attention", batch=batch, new_lo=1,
                    new_hi=1 if kind == "decode" else rng.randint(2, 9), ctx_lo=1,
                    ctx_hi=_log(rng, 2, hi), q_heads=heads[0], kv_heads=heads[1], page=page,
                    window=window, sinks=sinks, lens_seed=rng.randrange(1 << 30))
    if kind == "mixed":
        batch = _log(rng, 2, 60)
        return dict(op="attention", batch=batch, new_lo=1, new_hi=_log(rng, 10, 700), ctx_lo=1,
                    ctx_hi=_log(rng, 10, 5000), q_heads=min(16, heads[0]),
                    kv_heads=max(1, min(16, heads[0]) * heads[1] // heads[0]),
                    page=page, window=window, sinks=sinks, lens_seed=rng.randrange(1 << 30))
    new = _log(rng, 64, 4096)
    ctx = new + _log(rng, 1, 8192)
    return dict(op="attention", batch=1, new_lo=new, new_hi=new, ctx_lo=ctx, ctx_hi=ctx,
                q_heads=min(16, heads[0]), kv_heads=max(1, min(16, heads[0]) * heads[1] // heads[0]),
                page=page, window=window, sinks=sinks, lens_seed=rng.randrange(1 << 30))


def _lens(case):
    """Per request (tokens cached before the step, new tokens), from the case alone."""
    r = random.Random(case["lens_seed"])
    out = []
    for _ in range(case["batch"]):
        lo, hi = case["new_lo"], case["new_hi"]
        # most requests of a mixed step are at one new token
        new = lo if hi > 9 and lo == 1 and r.random() < 0.6 else r.randint(lo, hi)
        if case["op"] == "maps":
            out.append((r.randint(0, case["ctx"]), new))
        else:
            out.append((r.randint(case["ctx_lo"], case["ctx_hi"]), new))
    return out


def _visible(cached, new, window, sinks):
    """(query, key) pairs a head computes, and the keys some query sees."""
    pairs = 0
    if not window:
        return new * cached + new * (new + 1) // 2, cached + new
    for i in range(new):
        pos = cached + i
        first = max(0, pos - window + 1)
        pairs += pos - first + 1 + min(sinks, first)
    first = max(0, cached - window + 1)
    return pairs, cached + new - first + min(sinks, first)


def work(case):
    if case["op"] == "maps":
        lens, p = _lens(case), case["page"]
        tokens = sum(n for _, n in lens)
        taken = sum(-(-(c + n) // p) - -(-c // p) for c, n in lens)
        old = sum(1 for c, _ in lens if c % p)
        b = len(lens)
        return {"bytes": 4 * (2 * b + 1 + 2 * taken + old + (b + 1) + b + 2 * tokens + 1),
                "flops": 4 * tokens}
    if case["op"] == "rope":
        t, rows = case["tokens"], case["q_heads"] + 2 * case["kv_heads"]
        turned = case["q_heads"] + case["kv_heads"]
        return {"bytes": t * rows * D * 2 * 2 + 4 * t * (2 if case["cache"] else 1)
                + 4 * case["rot"],
                "flops": t * turned * case["rot"] * 3}
    lens = _lens(case)
    pairs = keys = new = pages = 0
    for c, n in lens:
        a, k = _visible(c, n, case["window"], case["sinks"])
        pairs += a
        keys += k
        new += n
        pages += -(-k // case["page"])
    return {"bytes": new * case["q_heads"] * D * 2 * 2 + keys * case["kv_heads"] * D * 2 * 2
            + 4 * (pages + 2 * case["batch"] + 1),
            "flops": 4 * D * pairs * case["q_heads"]}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=_dev())
    g.manual_seed(seed)
    return g


def _frequencies(case):
    """FP64 radians per position of each pair, and the factor on the rotated
    values.  linear: positions of a context eight times the trained one
    squeezed into it.  parts: pairs that turn more than 32 times over the
    trained 4096 positions keep their frequency, those under one turn are
    slowed sixteenfold, a ramp between."""
    half = case["rot"] // 2
    f = 10000.0 ** (-torch.arange(half, dtype=torch.float64) * 2.0 / case["rot"])
    if case["scaling"] == "linear":
        return f / 8.0, 1.0
    if case["scaling"] == "parts":
        turns = 4096.0 * f / (2.0 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return f * keep + f / 16.0 * (1.0 - keep), 0.1 * math.log(16.0) + 1.0
    return f, 1.0


def _pages(tokens, page):
    return -(-tokens // page)


def prepare(case, seed):
    dev, gen = _dev(), _gen(seed)
    st = {"case": case}
    if own:
        st["plan"] = _plan()
    if case["op"] == "maps":
        lens, p = _lens(case), case["page"]
        need = [_pages(c + n, p) for c, n in lens]
        have = [_pages(c, p) for c, _ in lens]
        wide = max(max(need), 1) + 3
        total = sum(need) + 50
        order = torch.randperm(total, generator=gen, device=dev, dtype=torch.int32)
        table = torch.full((len(lens), wide), -1, dtype=torch.int32, device=dev)
        rows = torch.tensor(have, device=dev)
        cols = torch.arange(wide, device=dev)[None]
        firsts = (torch.cumsum(rows, 0) - rows)[:, None]
        held = cols < rows[:, None]
        table = torch.where(held, order[(firsts + cols).clamp(max=total - 1)], table)
        st["table"] = table.contiguous()
        st["cached"] = torch.tensor([c for c, _ in lens], dtype=torch.int32, device=dev)
        st["added"] = torch.tensor([n for _, n in lens], dtype=torch.int32, device=dev)
        st["free"] = order[sum(have):].contiguous()
        st["head"] = torch.full((1,), 7, dtype=torch.int32, device=dev)
        st["most"] = sum(n for _, n in lens) + 5   # the step's token buffers, padded
        return st
    if case["op"] == "rope":
        t, hq, hk = case["tokens"], case["q_heads"], case["kv_heads"]
        width = (hq + 2 * hk) * D
        x = torch.randn((t, width), generator=gen, device=dev, dtype=torch.float16)
        # queries, keys and values as one projection's output leaves them
        st["q"] = x[:, :hq * D].view(t, hq, D)
        start = int(torch.randint(0, max(1, case["far"] - t), (1,), generator=gen, device=dev))
        if t < 256:   # a token of each request, wherever that stands
            st["pos"] = torch.randint(0, case["far"], (t,), generator=gen, device=dev,
                                      dtype=torch.int32)
        else:
            st["pos"] = torch.arange(start, start + t, device=dev, dtype=torch.int32)
        if case["cache"]:
            st["k"] = x[:, hq * D:(hq + hk) * D].view(t, hk, D)
            st["v"] = x[:, (hq + hk) * D:].view(t, hk, D)
            pages = _pages(t, case["page"]) + 9
            slots = torch.randperm(pages, generator=gen, device=dev)[:_pages(t, case["page"])]
            slots = slots[:, None] * case["page"] + torch.arange(case["page"], device=dev)[None]
            st["slots"] = slots.reshape(-1)[:t].to(torch.int32).contiguous()
            shape = (pages, case["page"], hk, D)
            st["kc"] = torch.zeros(shape, device=dev, dtype=torch.float16)
            st["vc"] = torch.zeros(shape, device=dev, dtype=torch.float16)
        f, m = _frequencies(case)
        st["freq"], st["factor"] = f.to(dev), m
        if own:
            import async_barrier_pipelined_gb300 as g
            st["turns"] = g.rope_turns(f).to(dev)
        return st
    lens, p = _lens(case), case["page"]
    hq, hk = case["q_heads"], case["kv_heads"]
    need = [_pages(c + n, p) for c, n in lens]
    pages = sum(need) + 3
    kc = torch.randn((pages, p, hk, D), generator=gen, device=dev, dtype=torch.float16)
    vc = torch.randn((pages, p, hk, D), generator=gen, device=dev, dtype=torch.float16)
    # keys and values have a mean of their own in each channel
    kc += torch.randn((hk, D), generator=gen, device=dev, dtype=torch.float16)
    vc.mul_(0.5).add_(torch.randn((hk, D), generator=gen, device=dev, dtype=torch.float16) * 0.5)
    order = torch.randperm(pages, generator=gen, device=dev, dtype=torch.int32)
    table = torch.full((len(lens), max(need) + 2), -1, dtype=torch.int32, device=dev)
    rows = torch.tensor(need, device=dev)
    cols = torch.arange(table.shape[1], device=dev)[None]
    firsts = (torch.cumsum(rows, 0) - rows)[:, None]
    table = torch.where(cols < rows[:, None], order[(firsts + cols).clamp(max=pages - 1)], table)
    st["kc"], st["vc"], st["table"] = kc, vc, table.contiguous()
    total = sum(n for _, n in lens)
    st["q"] = torch.randn((total, hq, D), generator=gen, device=dev, dtype=torch.float16) * 1.5
    starts = [0]
    for _, n in lens:
        starts.append(starts[-1] + n)
    st["cu"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    st["lens"] = torch.tensor([c + n for c, n in lens], dtype=torch.int32, device=dev)
    st["most"] = max(n for _, n in lens)
    st["host"] = lens    # a serving program knows its requests' lengths
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    if case["op"] == "maps":
        return _run_maps(st)
    if case["op"] == "rope":
        return _run_rope(st)
    return _run_attention(st)


def _run_maps(st):
    page = st["case"]["page"]
    if own:
        import async_barrier_pipelined_gb300 as g
        m = g.paged_maps(st["plan"], st["cached"], st["added"], st["table"], st["free"],
                         st["head"], page, st["most"])
        return {"starts": m.starts, "lens": m.kv_lens, "positions": m.positions,
                "slots": m.slots, "head": m.free_head, "table": st["table"]}
    cached, added, table = st["cached"], st["added"], st["table"]
    dev = cached.device
    starts = torch.zeros(cached.numel() + 1, dtype=torch.int32, device=dev)
    starts[1:] = torch.cumsum(added, 0)
    lens = cached + added
    first = (cached + page - 1) // page
    last = (lens + page - 1) // page
    ends = torch.cumsum(last - first, 0)
    cols = torch.arange(table.shape[1], device=dev)[None]
    fresh = (cols >= first[:, None]) & (cols < last[:, None])
    at = st["head"] + (ends - (last - first))[:, None] + cols - first[:, None]
    at = at.clamp(0, st["free"].numel() - 1)
    table.copy_(torch.where(fresh, st["free"][at], table))
    t = torch.arange(st["most"], device=dev, dtype=torch.int32)
    real = t < starts[-1]
    b = (torch.searchsorted(starts, t, right=True) - 1).clamp(0, cached.numel() - 1)
    positions = torch.where(real, cached[b] + t - starts[b], 0).to(torch.int32)
    slots = table[b, (positions // page).long()] * page + positions % page
    slots = torch.where(real, slots, -1).to(torch.int32)
    head = st["head"] + ends[-1:].to(torch.int32)
    return {"starts": starts, "lens": lens, "positions": positions, "slots": slots,
            "head": head.to(torch.int32), "table": table}


def _run_rope(st):
    case = st["case"]
    if own:
        import async_barrier_pipelined_gb300 as g
        if case["cache"]:
            q = g.rotary_to_cache(st["plan"], st["q"], st["k"], st["v"], st["pos"], st["slots"],
                                  st["turns"], st["kc"], st["vc"], layout=case["layout"],
                                  factor=st["factor"])
            return {"q": q, "k_cache": st["kc"], "v_cache": st["vc"]}
        return {"q": g.rotary(st["plan"], st["q"], st["pos"], st["turns"], layout=case["layout"],
                              factor=st["factor"], inverse=case["inverse"])}
    angle = st["pos"].double()[:, None] * st["freq"][None]
    cos = (torch.cos(angle) * st["factor"]).float()[:, None]
    sin = (torch.sin(angle) * st["factor"]).float()[:, None]
    if case["inverse"]:
        sin = -sin
    rot = case["rot"]

    def turn(x):
        y = x.float().clone()
        if case["layout"] == "half":
            a, b = y[..., :rot // 2].clone(), y[..., rot // 2:rot].clone()
            y[..., :rot // 2] = a * cos - b * sin
            y[..., rot // 2:rot] = b * cos + a * sin
        else:
            a, b = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
            y[..., 0:rot:2] = a * cos - b * sin
            y[..., 1:rot:2] = b * cos + a * sin
        return y.half()

    q = turn(st["q"])
    if not case["cache"]:
        return {"q": q}
    at = st["slots"].long()
    st["kc"].view(-1, case["kv_heads"], D)[at] = turn(st["k"])
    st["vc"].view(-1, case["kv_heads"], D)[at] = st["v"]
    return {"q": q, "k_cache": st["kc"], "v_cache": st["vc"]}


def _pieces(st):
    """Groups of (request, first new token, new tokens) that the plain form
    computes padded to the same size."""
    case = st["case"]
    hq, hk = case["q_heads"], case["kv_heads"]
    pieces = []
    for b, (c, n) in enumerate(st["host"]):
        step = max(1, PLAIN_SCORES // (hq * (c + n)))
        for t in range(0, n, step):
            pieces.append((b, t, min(step, n - t), c + n))
    pieces.sort(key=lambda x: (x[2], x[3]))
    groups, group = [], []
    for x in pieces:
        most = max(x[2], max((y[2] for y in group), default=0))
        keys = max(x[3], max((y[3] for y in group), default=0))
        g = len(group) + 1
        if group and (g * hq * most * keys > PLAIN_SCORES or g * keys * hk * D > PLAIN_CACHE
                      or most > 2 * group[0][2]):
            groups.append(group)
            group = []
        group.append(x)
    groups.append(group)
    return groups


def _run_attention(st):
    case = st["case"]
    if own:
        import async_barrier_pipelined_gb300 as g
        return g.paged_attention(st["plan"], st["q"], st["kc"], st["vc"], st["table"], st["cu"],
                                 st["lens"], st["most"], window=case["window"],
                                 sinks=case["sinks"])
    q, kc, vc = st["q"], st["kc"], st["vc"]
    hq, hk, page = case["q_heads"], case["kv_heads"], case["page"]
    dev = q.device
    out = torch.empty((q.shape[0] + 1, hq, D), dtype=q.dtype, device=dev)  # and a row for padding
    for group in _pieces(st):
        keys = max(x[3] for x in group)
        most = max(x[2] for x in group)
        req = torch.tensor([x[0] for x in group], device=dev)
        t0 = torch.tensor([x[1] for x in group], device=dev)
        cnt = torch.tensor([x[2] for x in group], device=dev)
        idx = st["table"][req, :-(-keys // page)].clamp(min=0).long()
        k = kc[idx].flatten(1, 2)[:, :keys].permute(0, 2, 3, 1).float()    # g, hk, D, keys
        v = vc[idx].flatten(1, 2)[:, :keys].permute(0, 2, 1, 3).float()    # g, hk, keys, D
        i = t0[:, None] + torch.arange(most, device=dev)[None]             # new token, g x most
        real = torch.arange(most, device=dev)[None] < cnt[:, None]
        row = (st["cu"][req].long()[:, None] + i).clamp(max=q.shape[0] - 1)
        x = q[row].float().view(len(group), most, hk, hq // hk, D).permute(0, 2, 1, 3, 4)
        s = torch.matmul(x.reshape(len(group), hk, -1, D), k) * (D ** -0.5)
        length = st["lens"][req].long()
        new = st["cu"][req + 1].long() - st["cu"][req].long()
        pos = (length - new)[:, None] + i
        j = torch.arange(keys, device=dev)
        see = j[None, None] <= pos[..., None]
        if case["window"]:
            see &= (j[None, None] > pos[..., None] - case["window"]) | (j < case["sinks"])
        s = s.view(len(group), hk, most, hq // hk, keys)
        s.masked_fill_(~see[:, None, :, None], float("-inf"))
        s -= s.amax(-1, keepdim=True).clamp(min=-1e30)
        s.exp_()
        total = s.sum(-1, keepdim=True)
        o = torch.matmul(s.view(len(group), hk, -1, keys), v)
        o = o.view(len(group), hk, most, hq // hk, D) / total
        o = o.permute(0, 2, 1, 3, 4).reshape(len(group), most, hq, D)
        out[torch.where(real, row, q.shape[0])] = o.half()
    return out[:-1]


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "maps":
        return None
    if case["op"] == "rope":
        half, rot = case["rot"] // 2, case["rot"]
        theta = torch.outer(st["pos"].double(), st["freq"])
        if case["inverse"]:
            theta = -theta
        wheel = torch.polar(torch.full_like(theta, st["factor"]), theta)[:, None]

        def spin(x):
            x = x.double()
            pair = x[..., :rot]
            pair = (pair.unflatten(-1, (2, half)).transpose(-1, -2) if case["layout"] == "half"
                    else pair.unflatten(-1, (half, 2)))
            z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * wheel)
            z = z.transpose(-1, -2) if case["layout"] == "half" else z
            return torch.cat((z.flatten(-2), x[..., rot:]), -1)

        if not case["cache"]:
            return {"q": spin(st["q"])}
        kc, vc = st["kc"].double(), st["vc"].double()
        where = (st["slots"].long() // case["page"], st["slots"].long() % case["page"])
        kc[where] = spin(st["k"])
        vc[where] = st["v"].double()
        return {"q": spin(st["q"]), "k_cache": kc, "v_cache": vc}
    if work(case)["flops"] > 4e12:
        return None
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    share = case["q_heads"] // case["kv_heads"]
    row = 0
    for b, (cached, new) in enumerate(_lens(case)):
        used = _pages(cached + new, case["page"])
        pages = st["table"][b, :used].long()
        k = st["kc"][pages].double().reshape(-1, case["kv_heads"], D)[:cached + new]
        v = st["vc"][pages].double().reshape(-1, case["kv_heads"], D)[:cached + new]
        at = torch.arange(cached + new, device=k.device)
        step = max(1, (1 << 26) // (share * (cached + new)))
        for lo in range(0, new, step):
            hi = min(new, lo + step)
            stand = torch.arange(cached + lo, cached + hi, device=k.device)[:, None]
            hidden = at > stand
            if case["window"]:
                hidden |= (stand - at >= case["window"]) & (at >= case["sinks"])
            for h in range(case["kv_heads"]):
                x = st["q"][row + lo:row + hi, h * share:(h + 1) * share].double()
                w = torch.einsum("tgd,jd->gtj", x, k[:, h]) / math.sqrt(D)
                w = torch.softmax(w.masked_fill(hidden, -math.inf), -1)
                out[row + lo:row + hi, h * share:(h + 1) * share] = torch.einsum(
                    "gtj,jd->tgd", w, v[:, h])
        row += new
    return out
