"""Decoding on a mapped cache held in 8 bits.

A source model's cache of a prompt is mapped into the target model's (kvmap_apply), enters 8-bit pages
(kvmap_q8_write), and the target model goes on from there: it reads a question on top of the prompt, all of its tokens
at once, and then decodes token by token.  A decode step over all layers -- each layer's new keys and values written,
its attention computed -- is captured into a graph once and replayed while the sequence grows.

The models are stand-ins: caches, maps, queries and new keys and values are random.  Prints what the cache takes, how
long the steps take, and how far attention over the 8-bit cache is from attention over the 16-bit one, and over what the
8-bit one holds.

    python examples/decode_on_mapped_cache.py [--tokens 32768] [--layers 16] [--steps 64]
"""

from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from cross_model_kv_amd import Context


def mapped_cache(ctx, tokens, layers, heads, d, k, gen):
    """Keys and values [layers][heads][tokens][d] of the target model, mapped from a random source cache."""
    def rand(*shape, scale=1.0):
        return (scale * torch.randn(shape, generator=gen, device="cuda")).bfloat16()
    n, f = heads * d, k * heads * d
    src_layers = max(k, layers // 2)
    sel = [sorted((t + j) % src_layers for j in range(k)) for t in range(layers)]
    return ctx.apply(rand(src_layers, heads, tokens, d), rand(src_layers, heads, tokens, d), sel,
                     rand(layers, n, f, scale=f ** -0.5), rand(layers, n, scale=0.1),
                     rand(layers, n, f, scale=f ** -0.5), rand(layers, n, scale=0.1), 1e6, 1e6)


def attention_16_bit(q, k, v):
    """The same attention over a cache that stays in 16 bits: q [n][H_q][d], k, v [H][T][d] -> [n][H_q][d]."""
    n, hq, d = q.shape
    h, t = k.shape[:2]
    rows = q.float().view(n, h, hq // h, d).permute(1, 2, 0, 3)
    y = rows @ k.float().transpose(1, 2).contiguous()[:, None] * d ** -0.5
    ahead = torch.arange(t, device=q.device) > torch.arange(t - n, t, device=q.device)[:, None]
    p = torch.softmax(y.masked_fill(ahead, float("-inf")), -1)
    return (p @ v.float()[:, None]).permute(2, 0, 1, 3).reshape(n, hq, d)


def run(tokens=32768, layers=16, heads=8, group=8, d=128, k=4, question=256, steps=64, page=64, seed=0):
    """The whole walk; returns what it prints as a dict."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ctx = Context(0)
    key, val = mapped_cache(ctx, tokens, layers, heads, d, k, gen)

    # one sequence whose pages lie anywhere in the pool
    total = tokens + question + steps
    n_pages = -(-total // page)
    cache = ctx.q8_cache(layers, n_pages, heads, page, d)
    pages = torch.randperm(n_pages, generator=gen, device="cuda").int()[None].contiguous()
    at = lambda t: torch.tensor([t], dtype=torch.int32, device="cuda")
    ctx.q8_write(cache, key.unsqueeze(1), val.unsqueeze(1), pages, at(0))
    ctx.q8_reserve(cache, 1, question, heads * group, total)

    # the question: its tokens' keys and values enter the cache, then they attend, layer by layer
    new = torch.randn((2, layers, 1, heads, question, d), generator=gen, device="cuda").bfloat16()
    q = 1.5 * torch.randn((layers, 1, question, heads * group, d), generator=gen, device="cuda")
    q = q.bfloat16()
    worst = own = 0.0
    far = lambda got, want: float((got.float() - want).norm() / want.norm())
    for l in range(layers):
        ctx.q8_write(cache, new[0, l], new[1, l], pages, at(tokens), layer=l)
        out = ctx.q8_attend(cache, q[l], pages, at(tokens + question), total, layer=l)
        if l in (0, layers - 1):
            last = q[l, 0, -8:]
            want = attention_16_bit(last, torch.cat([key[l], new[0, l, 0]], 1), torch.cat([val[l], new[1, l, 0]], 1))
            worst = max(worst, far(out[0, -8:], want))
            held_k, held_v = ctx.q8_read(cache, pages, at(0), tokens + question, layer=l, n_layers=1)
            own = max(own, far(out[0, -8:], attention_16_bit(last, held_k[0, 0], held_v[0, 0])))

    # decoding: one step captured, the position kept on the device
    kv = torch.zeros((2, layers, 1, heads, 1, d), dtype=torch.bfloat16, device="cuda")
    qs = torch.zeros((layers, 1, 1, heads * group, d), dtype=torch.bfloat16, device="cuda")
    outs = torch.zeros_like(qs)
    start, length = at(tokens + question), at(tokens + question + 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for l in range(layers):
            ctx.q8_write(cache, kv[0, l], kv[1, l], pages, start, layer=l)
            ctx.q8_attend(cache, qs[l], pages, length, total, layer=l, out=outs[l])
        start += 1
        length += 1
    torch.cuda.synchronize()
    # (timed on the device, around the graph alone: drawing the next token's inputs is not part of a step)
    around = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)) for _ in range(steps)]
    for begin, end in around:
        kv.normal_(generator=gen)
        qs.normal_(generator=gen)
        begin.record()
        graph.replay()
        end.record()
    torch.cuda.synchronize()
    step_us = sum(begin.elapsed_time(end) for begin, end in around) / steps * 1e3
    assert int(start) == total and ctx.q8_dropped() == 0 and bool(torch.isfinite(outs).all())
    held = sum(t.numel() * t.element_size() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale))
    result = dict(bytes_8=held, bytes_16=2 * 2 * layers * heads * n_pages * page * d, error=worst, own_error=own,
                  step_us=step_us, layer_us=step_us / layers, outs=outs)
    # the last step again, outside the graph, on the same cache
    eager = ctx.q8_attend(cache, qs[-1], pages, at(total), total, layer=layers - 1)
    result["graph_is_eager"] = bool(torch.equal(eager, outs[-1]))
    ctx.close()
    return result


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=32768)
    ap.add_argument("--layers", type=int, default=16)
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    r = run(tokens=a.tokens, layers=a.layers, steps=a.steps)
    print(f"cache: {r['bytes_8'] / 1e9:.2f} GB in 8 bits ({r['bytes_16'] / 1e9:.2f} GB in 16)")
    print(f"attention over it: {100 * r['error']:.2f} % from attention over the 16-bit cache (Frobenius, worst layer looked at),\n"
          f"  {100 * r['own_error']:.2f} % from attention over the values that the 8-bit cache holds")
    print(f"decode step: {r['step_us']:.0f} us for {a.layers} layers ({r['layer_us']:.1f} us a layer: write and attention)")


if __name__ == "__main__":
    main()
