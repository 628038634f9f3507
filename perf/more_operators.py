"""Products in 8-bit floating point and layers of experts, as cases to be timed.

A program that runs its large products in 8 bits, and whose layers may hold
several experts of which each token visits a few, makes four kinds of calls:

  quantize   before a product: numbers to 8-bit codes with a scale for each
             block of 128 (along a row, along a column, or 128 x 128);
  product    C = A B from codes and scales, dense or expert by expert over
             rows that are sorted by expert;
  trip       tokens to their experts and back: the sort's maps, the rows in
             sorted order, and the experts' rows brought back with weights,
             with its gradient in training;
  train      a layer's forward and backward pass in 8 bits, dense or through
             the experts (all of the above together).

The scale of a block is its largest finite magnitude (at least 2^-100) over
the format's largest number, both rounded to FP32; a code is the number times
FP32(largest number / largest magnitude), rounded to FP32 and then to the
format.  Infinities and NaN become NaN.

``own`` false: the operators in plain torch operations.  ``own`` true: the
calls of async_barrier_pipelined_gb300.
"""
import math
import random

import torch

own = False

BLOCK = 128
FLOOR = 2.0 ** -100
FORMATS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
MOST_WORK = 2 * 8192 * 8192 * 4096    # operations of the largest listed product

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
        # The new tokens of a generation step, before a projection.  Latency.
        dict(name="quantize-decode-48", op="quantize", rows=48, cols=4096, blocks="rows",
             type="f16", format="e4m3"),
        # A training batch's activations: along rows for the forward product, along
        # columns for the weights' gradient, from one reading.  Ragged on both sides.
        dict(name="quantize-both-16001x4104", op="quantize", rows=16001, cols=4104,
             blocks="both", type="bf16", format="e4m3"),
        # One projection of a generation step for a few requests: the weights' bytes.
        dict(name="product-decode-7", op="product", m=7, n=4096, k=4096, kind="forward",
             a="e4m3", b="e4m3", out="f16"),
        # Odd sizes on every side.
        dict(name="product-4000x4104x3000", op="product", m=4000, n=4104, k=3000,
             kind="forward", a="e4m3", b="e4m3", out="bf16"),
        # A weight gradient: both operands along the tokens, gradients in e5m2, FP32 out.
        dict(name="product-weights-gradient-4096", op="product", m=4096, n=4096, k=4096,
             kind="weights", a="e5m2", b="e4m3", out="f32"),
        # The largest: a wide projection of a long batch.
        dict(name="product-8192x8192x4096", op="product", m=8192, n=8192, k=4096,
             kind="forward", a="e4m3", b="e4m3", out="f16"),
        # A generation step through a layer of experts: most of them see a few rows.
        dict(name="experts-decode-48", op="experts", tokens=48, choices=2, experts=16, n=4096,
             k=2048, kind="forward", align=1, out="f16", skew=1.0, pick_seed=31),
        # Prompts through the same layer, experts unevenly loaded.
        dict(name="experts-prompt-8192", op="experts", tokens=8192, choices=2, experts=16,
             n=4096, k=2048, kind="forward", align=1, out="f16", skew=1.0, pick_seed=32),
        # To many experts and back in a generation step.  Latency.
        dict(name="trip-decode-48", op="trip", tokens=48, choices=8, experts=64, cols=2048,
             type="f16", align=1, grad=False, drop=False, skew=0.5, pick_seed=41),
        # A training batch to its experts and back, with the gradients; padding tokens
        # that visit none.
        dict(name="trip-gradient-8192", op="trip", tokens=8192, choices=4, experts=64,
             cols=4096, type="bf16", align=128, grad=True, drop=True, skew=0.5, pick_seed=42),
        # A dense layer's training step on a small ragged batch.
        dict(name="train-1000", op="train", tokens=1000, n=1024, k=2048, experts=0, choices=1,
             type="f16", skew=0.0, pick_seed=51),
        # A layer of experts in training: sort, products, weighted way back, gradients.
        dict(name="train-experts-4096", op="train", tokens=4096, n=2048, k=2048, experts=8,
             choices=2, type="bf16", skew=1.0, pick_seed=52),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "product", "experts", "experts", "trip",
                     "train"])
    fmt = lambda: rng.choice(["e4m3", "e4m3", "e5m2"])
    if op == "quantize":
        cols = _log(rng, 16, 8192)
        return dict(op=op, rows=min(_log(rng, 1, 16384), (1 << 26) // cols), cols=cols,
                    blocks=rng.choice(["rows", "columns", "tiles", "both"]),
                    type=rng.choice(["f16", "bf16", "f32"]), format=fmt())
    if op == "product":
        kind = rng.choice(["forward", "forward", "inputs", "weights"])
        m, n, k = _log(rng, 1, 8192), _log(rng, 16, 8192), _log(rng, 16, 8192)
        while 2 * m * n * k > MOST_WORK:
            m = max(1, m // 2)
        return dict(op=op, m=m, n=n, k=k, kind=kind, a=fmt(), b=fmt(),
                    out=rng.choice(["f16", "bf16", "f32"]))
    if op == "experts":
        experts = rng.choice([1, 2, 4, 8, 16, 60, 64, 128])
        choices = rng.randint(1, min(8, experts))
        kind = rng.choice(["forward", "forward", "inputs", "weights"])
        wide = 1 << 28     # most weights of a layer
        n = _log(rng, 64, 4096)
        k = min(_log(rng, 64, 4096), wide // (experts * n))
        return dict(op=op, tokens=max(1, min(_log(rng, 1, 8192), 16384 // choices)),
                    choices=choices, experts=experts, n=n, k=k, kind=kind,
                    align=128 if kind == "weights" else rng.choice([1, 1, 128]),
                    out=rng.choice(["f16", "bf16", "f32"]), skew=rng.choice([0.0, 0.5, 1.5]),
                    pick_seed=rng.randrange(1 << 30))
    if op == "trip":
        experts = rng.choice([2, 8, 16, 60, 64, 128, 256])
        choices = rng.randint(1, min(8, experts))
        cols = 8 * _log(rng, 2, 640)
        return dict(op=op, tokens=max(1, min(_log(rng, 1, 16384), (1 << 27) // (choices * cols))),
                    choices=choices, experts=experts, cols=cols,
                    type=rng.choice(["f16", "bf16", "f32"]), align=rng.choice([1, 16, 128]),
                    grad=rng.random() < 0.5, drop=rng.random() < 0.5,
                    skew=rng.choice([0.0, 0.5, 1.5]), pick_seed=rng.randrange(1 << 30))
    experts = rng.choice([0, 0, 4, 8])
    return dict(op=op, tokens=_log(rng, 1, 4096), n=_log(rng, 64, 2048), k=8 * _log(rng, 8, 256),
                experts=experts, choices=rng.randint(1, 2) if experts else 1,
                type=rng.choice(["f16", "bf16"]), skew=rng.choice([0.0, 1.0]),
                pick_seed=rng.randrange(1 << 30))


def _blocks(n):
    return -(-n // BLOCK)


def _up(n, to):
    return -(-n // to) * to


def _capacity(entries, experts, align):
    """Rows that hold any choice of experts, each one's rows filled up to `align`."""
    return _up(entries + min(experts, entries) * (align - 1), align)


def _picks(case):
    """The experts of each token, [tokens, choices] (a router's best ones; all -1 for a
    padding token), and each expert's rows, from the case alone."""
    g = torch.Generator().manual_seed(case["pick_seed"])
    e, t = case["experts"], case["tokens"]
    score = torch.randn((t, e), generator=g) + case["skew"] * torch.randn((e,), generator=g)
    picks = score.topk(case["choices"], 1).indices.int()
    if case.get("drop"):
        picks[torch.rand((t,), generator=g) < 0.06] = -1
    return picks, torch.bincount(picks[picks >= 0].long(), minlength=e)


_ELEMENT = {"f16": 2, "bf16": 2, "f32": 4}


def work(case):
    op = case["op"]
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        scales = {"rows": r * _blocks(c), "columns": _blocks(r) * c,
                  "tiles": _blocks(r) * _blocks(c), "both": r * _blocks(c) + _blocks(r) * c}
        sets = 2 if case["blocks"] == "both" else 1
        return {"bytes": r * c * (_ELEMENT[case["type"]] + sets) + 4 * scales[case["blocks"]],
                "flops": 3 * sets * r * c}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        sa = m * _blocks(k)
        sb = _blocks(k) * (n if case["kind"] == "weights" else _blocks(n))
        return {"bytes": m * k + k * n + 4 * (sa + sb) + m * n * _ELEMENT[case["out"]],
                "flops": 2 * m * n * k}
    if op == "experts":
        _, counts = _picks(case)
        rows, n, k, e = int(counts.sum()), case["n"], case["k"], case["experts"]
        seen = int((counts > 0).sum())
        weights = seen * (n * k + 4 * _blocks(n) * _blocks(k))
        size = _ELEMENT[case["out"]]
        if case["kind"] == "forward":
            moved = rows * (k + 4 * _blocks(k)) + weights + rows * n * size
        elif case["kind"] == "inputs":
            moved = rows * (n + 4 * _blocks(n)) + weights + rows * k * size
        else:
            moved = rows * (n + k) + 4 * (n + k) * _blocks(rows) + e * n * k * size
        return {"bytes": moved + 4 * (e + 1), "flops": 2 * rows * n * k}
    t, j, size = case["tokens"], case["choices"], _ELEMENT[case["type"]]
    if op == "trip":
        _, counts = _picks(case)
        rows, c = int(counts.sum()), case["cols"]
        cap = _capacity(t * j, case["experts"], case["align"])
        there = 4 * (2 * t * j + cap + case["experts"] + 1) + t * c * size + cap * c * size
        back = rows * c * size + t * c * size + 4 * 2 * t * j
        if not case["grad"]:
            return {"bytes": there + back, "flops": 2 * rows * c}
        # the way back's gradients (of its rows and weights), and the way there's
        again = t * c * size + rows * c * size + cap * c * size + 4 * 3 * t * j
        first = rows * c * size + t * c * size
        return {"bytes": there + back + again + first, "flops": 2 * rows * c * 3 + rows * c}
    n, k, e = case["n"], case["k"], max(1, case["experts"])
    rows = t * j
    # inputs, weights, output and its gradient, both gradients
    return {"bytes": size * (2 * t * k + 2 * e * n * k + 2 * t * n), "flops": 6 * rows * n * k}


# ------------------------------------------------------------------ plain forms

def _spread(s, blocks, rows, cols):
    """A scale for each number of a [.., rows, cols] matrix."""
    if blocks in ("columns", "tiles"):
        s = s.repeat_interleave(BLOCK, -2)
    if blocks in ("rows", "tiles"):
        s = s.repeat_interleave(BLOCK, -1)
    return s[..., :rows, :cols]


def _plain_quantize(x, blocks, fmt):
    """(codes, scales) of x [.., rows, cols]."""
    x = x.float()
    rows, cols = x.shape[-2:]
    size = x.abs()
    size = torch.where(torch.isfinite(size), size, torch.zeros_like(size))
    size = torch.nn.functional.pad(size, (0, _up(cols, BLOCK) - cols, 0, _up(rows, BLOCK) - rows))
    if blocks == "rows":
        top = size[..., :rows, :].unflatten(-1, (-1, BLOCK)).amax(-1)
    elif blocks == "columns":
        top = size[..., :cols].unflatten(-2, (-1, BLOCK)).amax(-2)
    else:
        top = size.unflatten(-1, (-1, BLOCK)).amax(-1).unflatten(-2, (-1, BLOCK)).amax(-2)
    top = top.clamp(min=FLOOR)
    largest = torch.full((), LARGEST[fmt], dtype=torch.float32, device=x.device)
    y = x * _spread(largest / top, blocks, rows, cols)
    y = torch.where(torch.isfinite(x), y.clamp(-LARGEST[fmt], LARGEST[fmt]),
                    torch.full_like(y, math.nan))
    return y.to(FORMATS[fmt]), top / largest


def _values(codes, scales, blocks):
    """The FP32 numbers that codes and scales stand for."""
    return codes.float() * _spread(scales, blocks, *codes.shape[-2:])


def _pitched(codes):
    """Codes with rows a multiple of 16 bytes apart, as the products take them."""
    cols = codes.shape[-1]
    room = torch.zeros((*codes.shape[:-1], _up(cols, 16)), dtype=torch.uint8, device=codes.device)
    room[..., :cols] = codes.view(torch.uint8)
    return room.view(codes.dtype)[..., :cols]


def _plain_maps(picks, experts, align):
    t, j = picks.shape
    flat = picks.reshape(-1).long()
    cap = _capacity(flat.numel(), experts, align)
    dev = picks.device
    there = (flat >= 0) & (flat < experts)
    key = torch.where(there, flat, experts)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(experts + 1, dtype=torch.long, device=dev).scatter_add_(
        0, key, torch.ones_like(key))
    ends = torch.cumsum((counts[:-1] + align - 1) // align * align, 0)
    starts = torch.cat((torch.zeros(1, dtype=torch.long, device=dev), ends))
    first = torch.cumsum(counts, 0) - counts
    rank = torch.arange(flat.numel(), device=dev) - first[key[order]]
    at = starts[key[order]] + rank
    rows = torch.empty_like(flat)
    rows[order] = torch.where(key[order] < experts, at, -1)
    source = torch.full((cap + 1,), -1, dtype=torch.long, device=dev)
    source[torch.where(rows >= 0, rows, cap)] = torch.arange(flat.numel(), device=dev)
    return starts.int(), rows.int().view(t, j), source[:cap].int()


def _plain_gather(x, source, choices):
    at = source.long()
    y = x[(at // choices).clamp(min=0)]
    return torch.where((at >= 0)[:, None], y, torch.zeros_like(y))


def _plain_combine(s, rows, weights):
    """FP32 sum over a token's rows, in order."""
    y = torch.zeros((rows.shape[0], s.shape[1]), dtype=torch.float32, device=s.device)
    for j in range(rows.shape[1]):
        at = rows[:, j].long()
        w = torch.ones_like(at, dtype=torch.float32) if weights is None else weights[:, j].float()
        part = s[at.clamp(min=0)].float() * w[:, None]
        y += torch.where((at >= 0)[:, None], part, torch.zeros_like(part))
    return y


def _plain_combine_gradient(dy, s, rows, source, weights):
    at, j = source.long(), rows.shape[1]
    real = (at >= 0)[:, None]
    token = dy.float()[(at // j).clamp(min=0)]
    ds = torch.where(real, token * weights.float().reshape(-1)[at.clamp(min=0)][:, None], 0.0)
    dw = torch.zeros(weights.numel() + 1, dtype=torch.float32, device=s.device)
    dot = (torch.where(real, token, 0.0) * s.float()).sum(1)
    dw[torch.where(at >= 0, at, weights.numel())] = dot
    return ds.to(s.dtype), dw[:-1].view(weights.shape).to(weights.dtype)


def _by_expert(starts, a, w, out):
    """out[rows of e] = a[rows of e] @ w[e]; rows past the last expert's are 0."""
    out.zero_()
    for e in range(w.shape[0]):
        if starts[e] < starts[e + 1]:
            torch.matmul(a[starts[e]:starts[e + 1]], w[e], out=out[starts[e]:starts[e + 1]])
    return out


# ------------------------------------------------------------------ inputs

def _activations(gen, rows, cols, type_):
    """Normal numbers with a few channels ten times larger."""
    x = torch.randn((rows, cols), generator=gen, device=_dev())
    loud = torch.rand((cols,), generator=gen, device=_dev()) < 0.01
    return (x * torch.where(loud, 10.0, 1.0)).to(TYPES[type_])


def _weights(gen, *shape, type_="f32"):
    return (torch.randn(shape, generator=gen, device=_dev()) * shape[-1] ** -0.5).to(TYPES[type_])


def _gradients(gen, rows, cols, type_):
    """Small numbers, each token's of its own size."""
    x = torch.randn((rows, cols), generator=gen, device=_dev())
    return (x * 0.01 * torch.exp(torch.randn((rows, 1), generator=gen, device=_dev()))).to(
        TYPES[type_])


def prepare(case, seed):
    gen = torch.Generator(device=_dev())
    gen.manual_seed(seed)
    st = {"case": case}
    if own:
        st["plan"] = _plan()
    op = case["op"]
    if op == "quantize":
        st["x"] = _activations(gen, case["rows"], case["cols"], case["type"])
        return st
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        if case["kind"] == "weights":       # gradients [k, m] and inputs [k, n] along tokens
            pair = (_plain_quantize(_gradients(gen, k, m, "f32"), "columns", case["a"]),
                    _plain_quantize(_activations(gen, k, n, "f32"), "columns", case["b"]))
        elif case["kind"] == "inputs":      # gradients [m, k] and weights stored [k, n]
            pair = (_plain_quantize(_gradients(gen, m, k, "f32"), "rows", case["a"]),
                    _plain_quantize(_weights(gen, k, n), "tiles", case["b"]))
        else:                               # activations [m, k] and weights stored [n, k]
            pair = (_plain_quantize(_activations(gen, m, k, "f32"), "rows", case["a"]),
                    _plain_quantize(_weights(gen, n, k), "tiles", case["b"]))
        st["a"], st["b"] = [(_pitched(c), s) for c, s in pair]
        return st
    if op == "experts":
        picks, _ = _picks(case)
        starts, _, source = _plain_maps(picks.to(_dev()), case["experts"], case["align"])
        st["starts"] = starts
        st["host"] = starts.tolist()     # the plain form's loop; the kernels read `starts`
        rows, n, k = source.numel(), case["n"], case["k"]
        real = (source >= 0)[:, None]
        if case["kind"] == "forward":
            x = _activations(gen, rows, k, "f32") * real
            st["a"] = _plain_quantize(x, "rows", "e4m3")
        else:
            x = _gradients(gen, rows, n, "f32") * real
            st["a"] = _plain_quantize(x, "rows" if case["kind"] == "inputs" else "columns", "e5m2")
        if case["kind"] == "weights":
            y = _activations(gen, rows, k, "f32") * real
            st["b"] = _plain_quantize(y, "columns", "e4m3")
        else:
            st["b"] = _plain_quantize(_weights(gen, case["experts"], n, k), "tiles", "e4m3")
        st["a"], st["b"] = [(_pitched(c), s) for c, s in (st["a"], st["b"])]
        return st
    picks = _picks(case)[0] if case["experts"] else None
    t = case["tokens"]
    if op == "trip":
        st["picks"] = picks.to(_dev())
        st["x"] = _activations(gen, t, case["cols"], case["type"])
        st["w"] = torch.softmax(torch.randn(picks.shape, generator=gen, device=_dev()), 1)
        if case["grad"]:
            st["dy"] = _gradients(gen, t, case["cols"], case["type"])
        return st
    st["x"] = _activations(gen, t, case["k"], case["type"])
    st["dy"] = _gradients(gen, t, case["n"], case["type"])
    if case["experts"]:
        st["picks"] = picks.to(_dev())
        st["weights"] = _weights(gen, case["experts"], case["n"], case["k"], type_=case["type"])
        # a router whose weights have the activations' type
        st["w"] = torch.softmax(torch.randn(picks.shape, generator=gen, device=_dev()), 1).to(
            TYPES[case["type"]])
    else:
        st["weights"] = _weights(gen, case["n"], case["k"], type_=case["type"])
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    return {"quantize": _run_quantize, "product": _run_product, "experts": _run_experts,
            "trip": _run_trip, "train": _run_train}[st["case"]["op"]](st)


def _run_quantize(st):
    case = st["case"]
    if own:
        import async_barrier_pipelined_gb300 as g
        got = g.quantize(st["plan"], st["x"], case["blocks"], FORMATS[case["format"]])
        got = got if case["blocks"] == "both" else (got,)
        return [t for b in got for t in (b.data, b.scales)]
    kinds = ("rows", "columns") if case["blocks"] == "both" else (case["blocks"],)
    return [t for b in kinds for t in _plain_quantize(st["x"], b, case["format"])]


def _run_product(st):
    case, kind = st["case"], st["case"]["kind"]
    (a, sa), (b, sb) = st["a"], st["b"]
    if own:
        import async_barrier_pipelined_gb300 as g
        a, b = g.Blocks(a, sa), g.Blocks(b, sb)
        a = a.t() if kind == "weights" else a
        b = b.t() if kind == "forward" else b
        return g.matmul_f8(st["plan"], a, b, dtype=TYPES[case["out"]])
    if kind == "weights":
        c = torch.matmul(_values(a, sa, "columns").t(), _values(b, sb, "columns"))
    elif kind == "inputs":
        c = torch.matmul(_values(a, sa, "rows"), _values(b, sb, "tiles"))
    else:
        c = torch.matmul(_values(a, sa, "rows"), _values(b, sb, "tiles").t())
    return c.to(TYPES[case["out"]])


def _run_experts(st):
    case, kind = st["case"], st["case"]["kind"]
    (a, sa), (b, sb) = st["a"], st["b"]
    if own:
        import async_barrier_pipelined_gb300 as g
        a, b = g.Blocks(a, sa), g.Blocks(b, sb)
        a = a.t() if kind == "weights" else a
        b = b.t() if kind == "forward" else b
        return g.matmul_f8(st["plan"], a, b, dtype=TYPES[case["out"]], starts=st["starts"])
    e, n, k = case["experts"], case["n"], case["k"]
    if kind == "weights":
        c = torch.zeros((e, n, k), device=a.device)
        va, vb = _values(a, sa, "columns"), _values(b, sb, "columns")
        for i in range(e):
            lo, hi = st["host"][i:i + 2]
            if lo < hi:
                torch.matmul(va[lo:hi].t(), vb[lo:hi], out=c[i])
    else:
        w = _values(b, sb, "tiles")
        w = w.transpose(1, 2) if kind == "forward" else w
        c = _by_expert(st["host"], _values(a, sa, "rows"), w,
                       torch.empty((a.shape[0], w.shape[2]), device=a.device))
    return c.to(TYPES[case["out"]])


def _run_trip(st):
    case = st["case"]
    x, w, picks = st["x"], st["w"], st["picks"]
    if own:
        import async_barrier_pipelined_gb300 as g
        if case["grad"]:
            x, w = x.detach().requires_grad_(), w.detach().requires_grad_()
        maps = g.expert_maps(st["plan"], picks, case["experts"], align=case["align"])
        s = g.expert_gather(st["plan"], x, maps)
        y = g.expert_combine(st["plan"], s, maps, w)
        got = {"starts": maps.starts, "rows": maps.rows, "source": maps.source, "sorted": s.detach(),
               "y": y.detach()}
        if case["grad"]:
            got["dx"], got["dw"] = torch.autograd.grad(y, (x, w), st["dy"])
        return got
    starts, rows, source = _plain_maps(picks, case["experts"], case["align"])
    s = _plain_gather(x, source, case["choices"])
    got = {"starts": starts, "rows": rows, "source": source, "sorted": s,
           "y": _plain_combine(s, rows, w).to(x.dtype)}
    if case["grad"]:
        ds, dw = _plain_combine_gradient(st["dy"], s, rows, source, w)
        got["dx"], got["dw"] = _plain_combine(ds, rows, None).to(x.dtype), dw
    return got


def _run_train(st):
    case = st["case"]
    x, dy, weights = st["x"], st["dy"], st["weights"]
    if own:
        import async_barrier_pipelined_gb300 as g
        x, weights = x.detach().requires_grad_(), weights.detach().requires_grad_()
        if not case["experts"]:
            y = g.linear_f8(st["plan"], x, weights)
            dx, dweights = torch.autograd.grad(y, (x, weights), dy)
            return {"y": y.detach(), "dx": dx, "dweights": dweights}
        w = st["w"].detach().requires_grad_()
        maps = g.expert_maps(st["plan"], st["picks"], case["experts"], align=BLOCK)
        s = g.expert_gather(st["plan"], x, maps)
        y = g.expert_combine(st["plan"], g.linear_f8(st["plan"], s, weights, starts=maps.starts),
                             maps, w)
        dx, dweights, dw = torch.autograd.grad(y, (x, weights, w), dy)
        return {"y": y.detach(), "dx": dx, "dweights": dweights, "dw": dw}
    qw = _values(*_plain_quantize(weights, "tiles", "e4m3"), "tiles")
    if not case["experts"]:
        s, ds = x, dy
    else:
        starts, rows, source = _plain_maps(st["picks"], case["experts"], BLOCK)
        host = starts.tolist()
        s = _plain_gather(x, source, case["choices"])
    xr = _values(*_plain_quantize(s, "rows", "e4m3"), "rows")
    xc = _values(*_plain_quantize(s, "columns", "e4m3"), "columns")
    got = {}
    if not case["experts"]:
        got["y"] = torch.matmul(xr, qw.t()).to(x.dtype)
    else:
        z = _by_expert(host, xr, qw.transpose(1, 2),
                       torch.empty((s.shape[0], case["n"]), device=s.device)).to(x.dtype)
        got["y"] = _plain_combine(z, rows, st["w"]).to(x.dtype)
        ds, dw = _plain_combine_gradient(dy, z, rows, source, st["w"])
    gr = _values(*_plain_quantize(ds, "rows", "e4m3"), "rows")
    gc = _values(*_plain_quantize(ds, "columns", "e4m3"), "columns")
    if not case["experts"]:
        got["dx"] = torch.matmul(gr, qw).to(x.dtype)
        got["dweights"] = torch.matmul(gc.t(), xc).to(x.dtype)
        return got
    dsx = _by_expert(host, gr, qw, torch.empty((s.shape[0], case["k"]), device=s.device))
    got["dx"] = _plain_combine(dsx.to(x.dtype), rows, None).to(x.dtype)
    dweights = torch.zeros(weights.shape, device=x.device)
    for e in range(case["experts"]):
        if host[e] < host[e + 1]:
            torch.matmul(gc[host[e]:host[e + 1]].t(), xc[host[e]:host[e + 1]], out=dweights[e])
    got["dweights"], got["dw"] = dweights.to(x.dtype), dw
    return got


# ------------------------------------------------------------------ in 64 bits

def _exact_codes(x, kind, fmt):
    """Codes and scales by the definition, block by block size: FP32 steps computed in
    64 bits and rounded (a quotient or product of two FP32 numbers, rounded from 64 bits
    to 32, is the correctly rounded one)."""
    x = x.double()
    rows, cols = x.shape[-2:]
    high = BLOCK if kind in ("columns", "tiles") else 1
    wide = BLOCK if kind in ("rows", "tiles") else 1
    good = torch.isfinite(x)
    padded = torch.zeros((*x.shape[:-2], _up(rows, high), _up(cols, wide)), dtype=torch.float64,
                         device=x.device)
    padded[..., :rows, :cols] = torch.where(good, x, 0.0).abs()
    cut = padded.reshape(*x.shape[:-2], padded.shape[-2] // high, high,
                         padded.shape[-1] // wide, wide)
    peak = torch.maximum(cut.amax((-3, -1)), torch.tensor(FLOOR, dtype=torch.float64,
                                                          device=x.device))
    scale = (peak / LARGEST[fmt]).float()
    lift = (LARGEST[fmt] / peak).float().double()
    lift = lift.repeat_interleave(high, -2).repeat_interleave(wide, -1)[..., :rows, :cols]
    y = (x * lift).float().clamp(-LARGEST[fmt], LARGEST[fmt])
    y = torch.where(good, y, torch.full_like(y, math.nan)).to(FORMATS[fmt])
    return y, scale


def _exact_values(codes, scale):
    """What codes stand for, in 64 bits; the blocks' sides follow from the shapes."""
    s = scale.double()
    for d in (-2, -1):
        if s.shape[d] != codes.shape[d]:
            s = s.repeat_interleave(BLOCK, d)
    return codes.double() * s[..., :codes.shape[-2], :codes.shape[-1]]


def _exact_maps(case, picks):
    """Rows of each (token, choice), by counting on the host."""
    e, align = case["experts"], case.get("align", BLOCK)
    flat = picks.reshape(-1).tolist()
    held = [[] for _ in range(e)]
    for i, p in enumerate(flat):
        if 0 <= p < e:
            held[p].append(i)
    rows, starts = [-1] * len(flat), [0]
    for p in range(e):
        for r, i in enumerate(held[p]):
            rows[i] = starts[-1] + r
        starts.append(starts[-1] + _up(len(held[p]), align))
    return starts, torch.tensor(rows, device=_dev()).view(picks.shape)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if work(case)["flops"] > 2e12:
        return None
    if op == "quantize":
        kinds = ("rows", "columns") if case["blocks"] == "both" else (case["blocks"],)
        return [t for b in kinds for t in _exact_codes(st["x"], b, case["format"])]
    if op == "product":
        a, b = _exact_values(*st["a"]), _exact_values(*st["b"])
        how = {"forward": "mk,nk->mn", "inputs": "mk,kn->mn", "weights": "km,kn->mn"}
        return torch.einsum(how[case["kind"]], a, b)
    if op == "experts":
        a, b = _exact_values(*st["a"]), _exact_values(*st["b"])
        cut = st["starts"].tolist()
        if case["kind"] == "weights":
            return torch.stack([torch.einsum("rn,rk->nk", a[lo:hi], b[lo:hi])
                                for lo, hi in zip(cut, cut[1:])])
        width = case["n"] if case["kind"] == "forward" else case["k"]
        c = torch.zeros((a.shape[0], width), dtype=torch.float64, device=a.device)
        for e, (lo, hi) in enumerate(zip(cut, cut[1:])):
            c[lo:hi] = torch.einsum("rk,nk->rn" if case["kind"] == "forward" else "rn,nk->rk",
                                    a[lo:hi], b[e])
        return c
    x = st["x"].double()
    if op == "trip":
        cut, rows = _exact_maps(case, st["picks"])
        c, j = case["cols"], case["choices"]
        cap = _capacity(rows.numel(), case["experts"], case["align"])
        there = rows >= 0
        s = torch.zeros((cap, c), dtype=torch.float64, device=x.device)
        s[rows[there]] = x.repeat_interleave(j, 0)[there.view(-1)]
        w = st["w"].double() * there
        got = {"starts": None, "rows": None, "source": None, "sorted": s, "y": x * w.sum(1)[:, None]}
        if case["grad"]:
            dy = st["dy"].double()
            # y = (sum of w) x, but each row's gradient w dy is rounded to the rows' type
            part = (dy[:, None] * w[:, :, None]).float().to(st["x"].dtype).double()
            got["dx"] = part.sum(1)
            got["dw"] = (dy * x).sum(1)[:, None] * there
        return got
    small = st["x"].dtype
    wv = _exact_values(*_exact_codes(st["weights"], "tiles", "e4m3"))
    dy = st["dy"]
    if not case["experts"]:
        return {"y": _exact_values(*_exact_codes(st["x"], "rows", "e4m3")) @ wv.t(),
                "dx": _exact_values(*_exact_codes(dy, "rows", "e4m3")) @ wv,
                "dweights": _exact_values(*_exact_codes(dy, "columns", "e4m3")).t()
                @ _exact_values(*_exact_codes(st["x"], "columns", "e4m3"))}
    # Through experts the rounding of what passes between the calls belongs to the
    # definition (its codes decide): those numbers are rounded as the calls hand them on.
    cut, rows = _exact_maps(case, st["picks"])
    y = torch.zeros((case["tokens"], case["n"]), dtype=torch.float64, device=x.device)
    dx = torch.zeros_like(x)
    dw = torch.zeros(rows.shape, dtype=torch.float64, device=x.device)
    dwv = torch.zeros(wv.shape, dtype=torch.float64, device=x.device)
    for e, (lo, hi) in enumerate(zip(cut, cut[1:])):
        if lo == hi:
            continue
        token, choice = ((rows >= lo) & (rows < hi)).nonzero(as_tuple=True)
        xe = torch.zeros((hi - lo, case["k"]), dtype=small, device=x.device)
        at = rows[token, choice] - lo
        xe[at] = st["x"][token]
        z = _exact_values(*_exact_codes(xe, "rows", "e4m3")) @ wv[e].t()
        y.index_add_(0, token, z[at] * st["w"][token, choice].double()[:, None])
        dw[token, choice] = (z[at] * dy[token].double()).sum(1)
        de = torch.zeros((hi - lo, case["n"]), dtype=small, device=x.device)
        de[at] = (dy[token].float() * st["w"][token, choice].float()[:, None]).to(small)
        dwv[e] = (_exact_values(*_exact_codes(de, "columns", "e4m3")).t()
                  @ _exact_values(*_exact_codes(xe, "columns", "e4m3")))
        dx.index_add_(0, token, (_exact_values(*_exact_codes(de, "rows", "e4m3")) @ wv[e])[at])
    return {"y": y, "dx": dx, "dweights": dwv, "dw": dw}
