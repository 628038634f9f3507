"""Serving a small stack of attention layers from a paged cache.

Prompts of different lengths enter in one step, are continued one token per
request from a captured CUDA graph, and a request's pages are taken from the
free list on the GPU as it grows.  Per step: the maps (paged_maps); per layer:
the projections (matmul), rotary positions with the new keys and values into
their slots (rotary_to_cache), attention over the pages (paged_attention) and
the output projection.  Every second layer sees a sliding window and the
first tokens.  Weights are random; a step's output is the next step's input.

    python examples/paged_serving.py [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import async_barrier_pipelined_gb300 as g  # noqa: E402

HEAD = 256


class Layers:
    """Attention layers with a residual each, and their paged caches."""

    def __init__(self, plan, layers=2, width=1024, q_heads=8, kv_heads=2, pages=512,
                 page_size=16, window=64, sinks=4, seed=0):
        import torch
        self.plan, self.page_size = plan, page_size
        self.q_heads, self.kv_heads = q_heads, kv_heads
        self.windows = [(window, sinks) if i % 2 else (0, 0) for i in range(layers)]
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=gen, device="cuda") * rows ** -0.5).half()

        self.w_in = [weight(width, (q_heads + 2 * kv_heads) * HEAD) for _ in range(layers)]
        self.w_out = [weight(q_heads * HEAD, width) for _ in range(layers)]
        shape = (pages, page_size, kv_heads, HEAD)
        self.caches = [(torch.zeros(shape, dtype=torch.float16, device="cuda"),
                        torch.zeros(shape, dtype=torch.float16, device="cuda"))
                       for _ in range(layers)]
        # positions scaled to four times a trained length of 256, by parts
        self.frequencies = g.rope_frequencies(HEAD, scaling="parts", factor=4.0, original_len=256)
        self.turns = g.rope_turns(self.frequencies).cuda()

    @staticmethod
    def normed(x):
        return (x.float() * x.float().square().mean(-1, keepdim=True).add(1e-6).rsqrt()).half()

    def __call__(self, x, maps, table, max_q):
        """One step: x [tokens, width] of all requests' new tokens."""
        hq, hk = self.q_heads, self.kv_heads
        for w_in, w_out, (kc, vc), (window, sinks) in zip(self.w_in, self.w_out, self.caches,
                                                          self.windows):
            qkv = g.matmul(self.plan, self.normed(x), w_in).view(x.shape[0], hq + 2 * hk, HEAD)
            q = g.rotary_to_cache(self.plan, qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:],
                                  maps.positions, maps.slots, self.turns, kc, vc)
            o = g.paged_attention(self.plan, q, kc, vc, table, maps.starts, maps.kv_lens, max_q,
                                  window=window, sinks=sinks)
            x = x + g.matmul(self.plan, o.view(x.shape[0], hq * HEAD), w_out)
        return x


def serve(prompts, steps, **kw):
    """Run the prompts' lengths and `steps` generated tokens; returns the
    layers, and per request all inputs and outputs in order."""
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    with g.Plan(0) as plan:
        layers = Layers(plan, **kw)
        pages = layers.caches[0][0].shape[0]
        width = layers.w_in[0].shape[0]
        batch = len(prompts)
        gen = torch.Generator(device="cuda").manual_seed(1)
        free = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        head = torch.zeros(1, **i32)
        table = torch.full((batch, -(-(max(prompts) + steps) // layers.page_size)), -1, **i32)
        cached = torch.zeros(batch, **i32)
        added = torch.tensor(prompts, **i32)

        # The prompts, all in one step.
        x = torch.randn(sum(prompts), width, generator=gen, device="cuda").half()
        maps = g.paged_maps(plan, cached, added, table, free, head, layers.page_size, x.shape[0])
        y = layers(x, maps, table, max(prompts))
        inputs = [list(t) for t in x.split(prompts)]
        outputs = [list(t) for t in y.split(prompts)]
        cached += added
        head.copy_(maps.free_head)
        added.fill_(1)

        # One token per request and step, from a graph: an eager step first
        # sets up what the plan keeps, without moving the state on.
        token = layers.normed(torch.stack([t[-1] for t in outputs]))
        result = torch.empty_like(token)

        def step():
            m = g.paged_maps(plan, cached, added, table, free, head, layers.page_size, batch)
            result.copy_(layers(token, m, table, 1))
            return m

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m = step()
            cached.add_(added)
            head.copy_(m.free_head)
        for _ in range(steps):
            graph.replay()
            for b in range(batch):
                inputs[b].append(token[b].clone())
                outputs[b].append(result[b].clone())
            token.copy_(layers.normed(result))
        torch.cuda.synchronize()
        status = plan.status()
        if status != 0:
            raise RuntimeError(g.gemm_f16_strerror(status))
        return layers, [torch.stack(t) for t in inputs], [torch.stack(t) for t in outputs]


def plain(layers, x):
    """All of a request's tokens at once, in FP32, without a cache."""
    import torch
    n, hq, hk = x.shape[0], layers.q_heads, layers.kv_heads
    x = x.float()
    pos = torch.arange(n, device=x.device)
    angle = pos.double()[:, None] * torch.tensor(layers.frequencies, dtype=torch.float64,
                                                 device=x.device)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turn(t):
        a, b = t.chunk(2, -1)
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)

    for w_in, w_out, (window, sinks) in zip(layers.w_in, layers.w_out, layers.windows):
        qkv = (layers.normed(x).float() @ w_in.float()).view(n, hq + 2 * hk, HEAD)
        q, k = turn(qkv[:, :hq]), turn(qkv[:, hq:hq + hk])
        k = k.repeat_interleave(hq // hk, 1)
        v = qkv[:, hq + hk:].repeat_interleave(hq // hk, 1)
        s = torch.einsum("ihd,jhd->hij", q, k) / 16.0
        hidden = pos[None] > pos[:, None]
        if window:
            hidden |= (pos[:, None] - pos[None] >= window) & (pos[None] >= sinks)
        p = s.masked_fill(hidden, float("-inf")).softmax(-1)
        o = torch.einsum("hij,jhd->ihd", p, v)
        x = x + o.reshape(n, hq * HEAD) @ w_out.float()
    return x


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=40)
    args = ap.parse_args(argv)
    layers, inputs, outputs = serve([5, 130, 1, 333, 64], args.steps)
    worst = 0.0
    for b, (x, y) in enumerate(zip(inputs, outputs)):
        want = plain(layers, x)
        off = ((y.float() - want).norm() / want.norm()).item()
        worst = max(worst, off)
        print(f"request {b}: {x.shape[0]} tokens, relative difference from FP32 {off:.2e}")
    return worst


if __name__ == "__main__":
    # Per layer a handful of binary16 roundings of 2^-11 relative each.
    sys.exit(0 if main() < 1e-2 else 1)
