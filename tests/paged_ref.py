"""Plain 64-bit forms of the paged-cache calls, and the problems the GPU tests
run them on.  Test infrastructure only."""
from __future__ import annotations

import math
import random

D = 256


def maps_reference(cached, added, table, free, head, page, max_tokens):
    """(starts, kv_lens, positions, slots, table, free_head, reported) as the
    header describes them, on Python lists."""
    rows = len(table[0]) * page
    table = [list(r) for r in table]
    starts, lens, pos, slots, bad = [0], [], [], [], False
    at = head if 0 <= head <= len(free) else len(free)
    bad |= at != head
    for b, (c, n) in enumerate(zip(cached, added)):
        cc = min(max(c, 0), rows)
        nn = min(max(n, 0), rows - cc)
        bad |= cc != c or nn != n
        left = min(nn, max_tokens - starts[-1])
        bad |= left != nn
        nn = left
        for i in range(-(-cc // page), -(-(cc + nn) // page)):
            table[b][i] = free[at] if at < len(free) else -1
            at += 1
        for i in range(nn):
            p = cc + i
            e = table[b][p // page]
            bad |= e < 0
            pos.append(p)
            slots.append(e * page + p % page if e >= 0 else -1)
        starts.append(starts[-1] + nn)
        lens.append(cc + nn)
    pos += [0] * (max_tokens - len(pos))
    slots += [-1] * (max_tokens - len(slots))
    return starts, lens, pos, slots, table, min(at, len(free)), bad


def rope_reference(x, positions, freq, layout, factor, inverse=False):
    """Rotation of [tokens, heads, 256] in 64 bits; freq: FP64 radians."""
    import torch
    x = x.double()
    ang = positions.double()[:, None] * freq.to(x.device)[None]
    c, s = (torch.cos(ang) * factor)[:, None], (torch.sin(ang) * factor)[:, None]
    if inverse:
        s = -s
    half = freq.numel()
    y = x.clone()
    ia = torch.arange(half, device=x.device)
    ia, ib = (ia, ia + half) if layout == "half" else (2 * ia, 2 * ia + 1)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


class PagedProblem:
    """A step over a paged cache: everything that no query may look at is NaN
    (rows past a request's length, pages of no request, pages that no query
    sees) or, for table entries, out of range."""

    def __init__(self, lens, q_heads, kv_heads, page, window=0, sinks=0, seed=0, extra_rows=0,
                 head_major=False, spare_pages=3, device="cuda", q_scale=1.0, far=0):
        import torch
        self.lens, self.page, self.window, self.sinks = lens, page, window, sinks
        self.q_heads, self.kv_heads = q_heads, kv_heads
        g = torch.Generator(device="cpu").manual_seed(seed)
        r = random.Random(seed)
        need = [-(-(c + n) // page) for c, n in lens]
        pages = sum(need) + spare_pages + far
        ids = list(range(far, pages))
        r.shuffle(ids)
        nan = float("nan")
        shape = ((pages, kv_heads, page, D) if head_major else (pages, page, kv_heads, D))
        alloc = (torch.empty if far else torch.full)
        args = () if far else (nan,)
        kc = alloc(shape, *args, dtype=torch.float16, device=device)
        vc = alloc(shape, *args, dtype=torch.float16, device=device)
        if far:
            kc[far:] = nan
            vc[far:] = nan
        if head_major:
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
        table = torch.full((len(lens), max(need + [1]) + 2), -7, dtype=torch.int32)
        table[:, -1] = 1 << 30
        self.keys, self.values = [], []
        at = 0
        for b, (c, n) in enumerate(lens):
            total = c + n
            k = torch.randn(total, kv_heads, D, generator=g).half()
            v = (torch.randn(total, kv_heads, D, generator=g) * 0.5 + 0.25).half()
            self.keys.append(k)
            self.values.append(v)
            first = max(0, c - window + 1) if window else 0
            for i in range(need[b]):
                page_id = ids[at]
                at += 1
                lo, hi = i * page, min(total, (i + 1) * page)
                seen = n > 0 and (hi > first or lo < sinks)
                if not seen:
                    continue
                table[b, i] = page_id
                kc[page_id, :hi - lo] = k[lo:hi].to(device)
                vc[page_id, :hi - lo] = v[lo:hi].to(device)
        total_q = sum(n for _, n in lens) + extra_rows
        self.q = (torch.randn(total_q, q_heads, D, generator=g) * q_scale).half()
        self.kc, self.vc, self.pages = kc, vc, pages
        starts = [0]
        for _, n in lens:
            starts.append(starts[-1] + n)
        i32 = torch.int32
        self.table = table.to(device)
        self.starts = torch.tensor(starts, dtype=i32, device=device)
        self.kv_lens = torch.tensor([c + n for c, n in lens], dtype=i32, device=device)
        self.max_q = max([n for _, n in lens] + [0])
        self.device = device

    def reference(self, scale=1 / 16):
        """(O, bound): the rows in 64 bits and how far a binary16 result may
        be off, element by element.

        With A = sum p|v| / sum p: O is rounded once (half a step, 2^-11 |o|,
        or 2^-25 below the normal range); each weight is rounded to binary16
        for the product with V (2^-11 A, and 2^-25 |v| for a weight below the
        normal range, the largest being at least 1); a score is a sum of 256
        FP32 products (256 * 2^-24 of the sum of their magnitudes), taken by
        the exponent as a relative error, in numerator and denominator; the
        sums over k keys in FP32 are off by at most k * 2^-24 each; two units
        of 2^-22 for the exponential.
        """
        import torch
        dev = self.device
        out = torch.zeros(self.q.shape, dtype=torch.float64, device=dev)
        bound = torch.full(self.q.shape, 2.0 ** -25, dtype=torch.float64, device=dev)
        share = self.q_heads // self.kv_heads
        row = 0
        for (c, n), k, v in zip(self.lens, self.keys, self.values):
            k, v = k.to(dev).double(), v.to(dev).double()
            j = torch.arange(c + n, device=dev)
            step = max(1, (1 << 25) // max(1, self.q_heads * (c + n)))
            for lo in range(0, n, step):
                hi = min(n, lo + step)
                pos = torch.arange(c + lo, c + hi, device=dev)[:, None]
                see = j <= pos
                if self.window:
                    see &= (j > pos - self.window) | (j < self.sinks)
                for h in range(self.q_heads):
                    q = self.q[row + lo:row + hi, h].to(dev).double()
                    kk, vv = k[:, h // share], v[:, h // share]
                    s = (q @ kk.T) * scale
                    mag = (q.abs() @ kk.abs().T) * abs(scale)
                    s = s.masked_fill(~see, -math.inf)
                    p = torch.exp(s - s.amax(1, keepdim=True))
                    l = p.sum(1, keepdim=True)
                    o = p @ vv / l
                    a = p @ vv.abs() / l
                    eps = 256 * 2.0 ** -24 * mag.masked_fill(~see, 0).amax(1, keepdim=True)
                    keys = see.sum(1, keepdim=True).double()
                    tol = (2.0 ** -11 * o.abs() + a * (2.0 ** -11 + 2 * eps + 2 * keys * 2.0 ** -24
                                                      + 4 * 2.0 ** -22)
                           + 2.0 ** -25 * (see.double() @ vv.abs()) / l)
                    out[row + lo:row + hi, h] = o
                    bound[row + lo:row + hi, h] += tol
            row += n
        return out, bound


def transposed_rows(x):
    """The same [tokens, heads, 256] tensor stored [heads, tokens, 256]."""
    return x.transpose(0, 1).contiguous().transpose(0, 1)
