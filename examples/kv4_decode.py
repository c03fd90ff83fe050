"""Continuous batching of one attention layer with 4-bit weights and a 4-bit cache.

    python examples/kv4_decode.py [--steps 6]

A step takes the new tokens of all requests at once: kv_maps hands out pages and
says where each token goes, qmm gives its queries, keys and values from 4-bit
weights, kv4_write puts the last two into the cache, kv4_attention reads it, and
qmm projects the result.  The first step takes whole prompts; the others, of one
token a request, are one HIP graph, replayed over the same buffers.  Every step
is held against attention in float64 on what kv4_read says the cache holds.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matmul_affine_qmv_amd as qmx  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, PAGE = 512, 8, 2, 64, 16
DEV = "cuda:0"


def quantised(rows, cols, gen, bits=4, group=64):
    """Random weights as qmm takes them: packed words, scales, biases."""
    w = torch.randn(rows, cols, generator=gen, device=DEV) * cols ** -0.5
    g = w.view(rows, -1, group)
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    s = ((hi - lo) / 15).bfloat16()
    b = lo.bfloat16()
    c = ((g - b.float()) / s.float()).round().clamp(0, 15).long().view(rows, -1, 8)
    words = (c << (4 * torch.arange(8, device=DEV))).sum(-1)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).int()
    return words, s[..., 0].contiguous(), b[..., 0].contiguous()


class Layer:
    """The layer's weights and cache, and the requests' pages."""

    def __init__(self, requests, most_tokens, gen):
        self.wqkv = quantised((HEADS + 2 * KV_HEADS) * DIM, HIDDEN, gen)
        self.wo = quantised(HIDDEN, HEADS * DIM, gen)
        self.columns = -(-most_tokens // PAGE)
        pages = requests * self.columns
        self.cache = qmx.Kv4Cache.zeros(pages, KV_HEADS, DIM, page_size=PAGE, group_size=32, device=DEV)
        self.table = torch.full((requests, self.columns), -1, dtype=torch.int32, device=DEV)
        self.free = torch.randperm(pages, generator=gen, device=DEV).int()

    def take_pages(self, maps):
        """The pages a step used leave the front of the free list (on the device: no copy to the host)."""
        n = self.free.numel()
        at = torch.arange(n, device=DEV) + maps.counts[1]
        self.free.copy_(self.free[at.clamp(max=n - 1)])

    def step(self, x, past, new, maps, most_new):
        m = qmx.kv_maps(past, new, self.table, self.free, page_size=PAGE, out=maps)
        qkv = qmx.qmm(*self.wqkv, x).view(x.shape[0], HEADS + 2 * KV_HEADS, DIM)
        q, k, v = qkv.split((HEADS, KV_HEADS, KV_HEADS), 1)
        qmx.kv4_write(self.cache, k, v, m.slots)
        o = qmx.kv4_attention(self.cache, q, self.table, m.kv_lens, m.query_offsets, max_query_len=most_new,
                              max_kv_len=self.columns * PAGE)
        return q, o, qmx.qmm(*self.wo, o.view(x.shape[0], HEADS * DIM))


def expected(layer, q, maps, request):
    """Attention of one request's new tokens in float64, on what its cached tokens stand for."""
    first, last = maps.query_offsets[request].item(), maps.query_offsets[request + 1].item()
    kv = maps.kv_lens[request].item()
    at = torch.arange(kv, device=DEV)
    slots = layer.table[request, at // PAGE] * PAGE + (at % PAGE).int()
    k, v = (t.double().repeat_interleave(HEADS // KV_HEADS, 1).transpose(0, 1).contiguous()
            for t in qmx.kv4_read(layer.cache, slots))
    s = q[first:last].double().transpose(0, 1) @ k.transpose(1, 2).contiguous() * DIM ** -0.5
    seen = at <= (kv - (last - first) + torch.arange(last - first, device=DEV))[:, None]
    return first, last, (s.masked_fill(~seen, -torch.inf).softmax(-1) @ v).transpose(0, 1)


def worst(layer, q, o, maps, requests):
    """The largest error of a step, relative to the largest output of its token and head."""
    most = 0.0
    for r in range(requests):
        first, last, want = expected(layer, q, maps, r)
        off = (o[first:last].double() - want).abs().amax(-1) / want.abs().amax(-1)
        most = max(most, off.max().item() if last > first else 0.0)
    return most


def main(steps=6, prompts=(37, 5, 120), seed=0):
    """Runs the loop; returns the largest error of each step."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    R, T = len(prompts), sum(prompts)
    layer = Layer(R, max(prompts) + steps + 1, gen)
    past = torch.zeros(R, dtype=torch.int32, device=DEV)
    new = torch.tensor(prompts, dtype=torch.int32, device=DEV)
    x = torch.randn(T, HIDDEN, generator=gen, device=DEV).bfloat16()
    maps = qmx.KvMaps.empty(R, T, DEV)
    q, o, _ = layer.step(x, past, new, maps, max(prompts))
    errors = [worst(layer, q, o, maps, R)]
    layer.take_pages(maps)
    past += new
    new.fill_(1)

    maps = qmx.KvMaps.empty(R, R, DEV)
    x = torch.empty(R, HIDDEN, dtype=torch.bfloat16, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, o, y = layer.step(x, past, new, maps, 1)
        layer.take_pages(maps)
        past += new
    for _ in range(steps):
        x.normal_(generator=gen)
        graph.replay()
        errors.append(worst(layer, q, o, maps, R))
    return errors


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=6)
    for i, e in enumerate(main(ap.parse_args().steps)):
        print(f"step {i}: {'prompts' if i == 0 else 'one token each'}, largest error {e:.2e} of the row's largest output")
