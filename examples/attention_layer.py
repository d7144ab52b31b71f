#!/usr/bin/env python3
"""One attention layer served from a paged E4M3 cache, on one MI355X.

A layer's QKV projection, rotation, append, attention and output projection
run as a serving program would chain them: the projections as block-scaled
FP8 GEMMs, the cache in E4M3 with a scale a page and head.  A few requests'
prompts go in packed, then every request decodes token by token:

    python examples/attention_layer.py [--requests 8] [--prompt 700] [--tokens 16]

It prints the time of the prompt pass and of a decoding step, and how far the
attention of a request decoded token by token is from the same tokens passed
as one prompt (both read the cache's E4M3 values, whose scales grow at
different moments on the two ways).
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fp8_fine_grained_fp8bs_amd import fp8bs  # noqa: E402


class Layer:
    """Weights (quantized once), rotary table and page pool of one layer."""

    def __init__(self, hidden=2048, heads=16, kv_heads=4, dim=128, page=64, pages=1024, positions=8192, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.page = heads, kv_heads, dim, page
        rows = (heads + 2 * kv_heads) * dim
        draw = lambda n, k: torch.randn((n, k), generator=g, device="cuda").mul_(k ** -0.5).bfloat16()  # noqa: E731
        self.w_qkv = fp8bs.quant_w_128x128(draw(rows, hidden))
        self.w_out = fp8bs.quant_w_128x128(draw(hidden, heads * dim))
        self.angles = fp8bs.rope_table(positions, dim, base=500000.0)
        self.cache = fp8bs.paged_cache(pages, kv_heads, page, dim)
        self.free = list(range(pages))

    def attention(self, x, table, kv_len, q_off, max_q):
        """x bf16 [T][hidden], packed rows of the requests -> the heads' outputs."""
        qkv = fp8bs.gemm(*fp8bs.quant_act_1x128(x), *self.w_qkv).view(x.shape[0], -1, self.dim)
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), dim=1)
        q = fp8bs.kv_append(k, v, *self.cache, table, kv_len, q_off, max_q, q=q, cs=self.angles)
        return fp8bs.attn_paged(q, *self.cache, table, kv_len, q_off, max_q)

    def __call__(self, x, table, kv_len, q_off=None, max_q=1):
        o = self.attention(x, table, kv_len, q_off, max_q)
        return fp8bs.gemm(*fp8bs.quant_act_1x128(o.view(x.shape[0], -1)), *self.w_out)


class Batch:
    """Requests with their pages: lengths and page table on the device."""

    def __init__(self, layer, count, longest):
        self.layer = layer
        width = -(-longest // layer.page)
        pages = [[layer.free.pop() for _ in range(width)] for _ in range(count)]
        self.table = torch.tensor(pages, dtype=torch.int32, device="cuda")
        self.kv_len = torch.zeros(count, dtype=torch.int32, device="cuda")

    def prompt(self, x, lengths):
        q_off = torch.tensor([0] + lengths, device="cuda").cumsum(0).int()
        self.kv_len += q_off[1:] - q_off[:-1]
        return self.layer(x, self.table, self.kv_len, q_off, max(lengths))

    def step(self, x):
        self.kv_len += 1
        return self.layer(x, self.table, self.kv_len)


def run(requests=8, prompt=700, tokens=16, hidden=2048, verbose=True):
    layer = Layer(hidden=hidden)
    lengths = [max(1, prompt - 61 * i) for i in range(requests)]
    total = prompt + tokens
    batch = Batch(layer, requests, total)
    x = torch.randn((sum(lengths), hidden), device="cuda").bfloat16()

    def timed(f):
        torch.cuda.synchronize()
        t = time.perf_counter()
        y = f()
        torch.cuda.synchronize()
        return y, (time.perf_counter() - t) * 1e6

    Batch(layer, requests, total).prompt(x, lengths)   # a first call loads the kernels
    _, t_prompt = timed(lambda: batch.prompt(x, lengths))
    steps = [torch.randn((requests, hidden), device="cuda").bfloat16() for _ in range(tokens)]
    outs, times = [], []
    for s in steps:
        y, t = timed(lambda: batch.step(s))
        outs.append(y)
        times.append(t)

    # the first request's tokens again, all of them as one prompt
    again = Batch(layer, 1, total)
    rows = torch.cat([x[:lengths[0]]] + [s[:1] for s in steps])
    whole = again.prompt(rows, [len(rows)])[-tokens:] if tokens else rows[:0]
    mine = torch.cat([y[:1] for y in outs]) if outs else rows[:0]
    off = float((mine.float() - whole.float()).norm() / whole.float().norm()) if tokens else 0.0
    if verbose:
        print(f"prompts of {lengths} tokens: {t_prompt:.0f} us")
        if times:
            print(f"a decoding step of {requests} requests: {sorted(times)[len(times) // 2]:.0f} us")
        print(f"token by token against one prompt: relative difference {off:.2e}")
    return off


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=700)
    ap.add_argument("--tokens", type=int, default=16)
    a = ap.parse_args()
    run(a.requests, a.prompt, a.tokens)
