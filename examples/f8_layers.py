"""Continuous batching of a small model's layers in 8-bit floats, with a 4-bit cache.

A step takes the new tokens of all requests at once.  Per layer: rms_norm_f8 adds the
last product to the residual stream and norms it into 8 bits, qmm_f8 gives queries, keys
and values, rope turns them where they are by the positions that kv_maps wrote,
kv4_write and kv4_attention use the cache, f8_quantize brings what is not behind a norm
into 8 bits, and qmm_f8 does the projection and the gated feed-forward's two products.
The first step takes whole prompts; the others, of one token a request, are one HIP
graph, replayed over the same buffers.  In every step products and rotations are held
against float64 on their own operands, attention on what kv4_read says the cache holds.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matmul_affine_qmv_amd as qmx  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, FEED, PAGE, EPS = 512, 8, 2, 64, 1024, 16, 1e-5
DEV = "cuda:0"


class Weight:
    """An 8-bit matrix [rows, cols] with a scale for each block of 128 x 128."""

    def __init__(self, rows, cols, gen):
        w = torch.randn(rows, cols, generator=gen, device=DEV) * cols ** -0.5
        self.codes, self.scales = qmx.f8_quantize(w.bfloat16(), block_rows=128)

    def __call__(self, codes, scales):
        self.x = codes, scales  # kept for the check
        self.y = qmx.qmm_f8(self.codes, self.scales, codes, scales)
        return self.y

    def error(self):
        """The largest error of the last product, relative to the largest output of its row."""
        x, w = (qmx.f8_dequantize(c, s).double() for c, s in (self.x, (self.codes, self.scales)))
        want = x @ w.T
        return ((self.y.double() - want).abs().amax(-1) / want.abs().amax(-1).clamp(min=1e-30)).max().item()


class Layer:
    def __init__(self, requests, columns, gen):
        self.norms = [(1 + 0.1 * torch.randn(HIDDEN, generator=gen, device=DEV)).bfloat16() for _ in range(2)]
        self.qkv = Weight((HEADS + 2 * KV_HEADS) * DIM, HIDDEN, gen)
        self.out = Weight(HIDDEN, HEADS * DIM, gen)
        self.up = Weight(2 * FEED, HIDDEN, gen)
        self.down = Weight(HIDDEN, FEED, gen)
        self.cache = qmx.Kv4Cache.zeros(requests * columns, KV_HEADS, DIM, page_size=PAGE, group_size=32, device=DEV)

    def __call__(self, delta, stream, m, table, frequencies, most_new, most_kv):
        codes, scales, _ = qmx.rms_norm_f8(delta, self.norms[0], stream, eps=EPS, sum_out=stream)
        qkv = self.qkv(codes, scales).view(-1, HEADS + 2 * KV_HEADS, DIM)
        self.before = qkv.clone()
        q, k, v = qkv.split((HEADS, KV_HEADS, KV_HEADS), 1)
        qmx.rope(q, k, m.positions, frequencies, out=(q, k))
        self.qkv.y, self.after = self.before.flatten(1), qkv
        qmx.kv4_write(self.cache, k, v, m.slots)
        self.o = qmx.kv4_attention(self.cache, q, table, m.kv_lens, m.query_offsets, max_query_len=most_new,
                                   max_kv_len=most_kv)
        delta = self.out(*qmx.f8_quantize(self.o.flatten(1)))
        codes, scales, _ = qmx.rms_norm_f8(delta, self.norms[1], stream, eps=EPS, sum_out=stream)
        gate, up = self.up(codes, scales).split(FEED, 1)
        return self.down(*qmx.f8_quantize(torch.nn.functional.silu(gate) * up))

    def errors(self, m, table, frequencies, requests):
        turn = torch.polar(torch.ones_like(frequencies), m.positions.double()[:, None] * frequencies)[:, None]
        a, b = self.before[:, :HEADS + KV_HEADS].double().chunk(2, -1)
        want = torch.complex(a.contiguous(), b.contiguous()) * turn
        got = self.after[:, :HEADS + KV_HEADS].double()
        off = (got - torch.cat((want.real, want.imag), -1)).abs().amax() / got.abs().amax()
        worst = [off.item(), *(w.error() for w in (self.qkv, self.out, self.up, self.down))]
        for r in range(requests):  # attention of the request's new tokens
            first, last, kv = m.query_offsets[r].item(), m.query_offsets[r + 1].item(), m.kv_lens[r].item()
            at = torch.arange(kv, device=DEV)
            keys, values = (t.double().repeat_interleave(HEADS // KV_HEADS, 1).transpose(0, 1).contiguous()
                            for t in qmx.kv4_read(self.cache, table[r, at // PAGE] * PAGE + (at % PAGE).int()))
            q = self.after[first:last, :HEADS].double().transpose(0, 1).contiguous()
            s = q @ keys.transpose(1, 2).contiguous() * DIM ** -0.5
            s = s.masked_fill(at > (kv - last + torch.arange(first, last, device=DEV))[:, None], -torch.inf)
            want = (s.softmax(-1) @ values).transpose(0, 1)
            off = (self.o[first:last].double() - want).abs().amax(-1) / want.abs().amax(-1)
            worst.append(off.max().item())
        return max(worst)


def main(steps=6, prompts=(37, 5, 120), layers=2, seed=0):
    """Runs the loop; returns the largest error of each step."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    R, T = len(prompts), sum(prompts)
    columns = -(-(max(prompts) + steps + 1) // PAGE)
    model = [Layer(R, columns, gen) for _ in range(layers)]
    frequencies = qmx.rope_frequencies(DIM, scaling="linear", factor=2.0, device=DEV)
    table = torch.full((R, columns), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(R * columns, generator=gen, device=DEV).int()
    final = torch.ones(HIDDEN, dtype=torch.bfloat16, device=DEV)

    def step(x, past, new, maps, most_new):
        m = qmx.kv_maps(past, new, table, free, page_size=PAGE, out=maps)
        stream, delta = torch.zeros_like(x), x
        for layer in model:
            delta = layer(delta, stream, m, table, frequencies, most_new, columns * PAGE)
        y, _ = qmx.rms_norm(delta, final, stream, eps=EPS, sum_out=stream)
        # the pages that the step used leave the front of the free list, and tokens are past ones
        at = torch.arange(free.numel(), device=DEV) + m.counts[1]
        free.copy_(free[at.clamp(max=free.numel() - 1)])
        past.add_(new)
        return y

    past = torch.zeros(R, dtype=torch.int32, device=DEV)
    new = torch.tensor(prompts, dtype=torch.int32, device=DEV)
    x = torch.randn(T, HIDDEN, generator=gen, device=DEV).bfloat16()
    maps = qmx.KvMaps.empty(R, T, DEV)
    step(x, past, new, maps, max(prompts))
    errors = [max(layer.errors(maps, table, frequencies, R) for layer in model)]
    new.fill_(1)

    maps = qmx.KvMaps.empty(R, R, DEV)
    x = torch.empty(R, HIDDEN, dtype=torch.bfloat16, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(x, past, new, maps, 1)
    for _ in range(steps):
        x.normal_(generator=gen)
        graph.replay()
        assert torch.isfinite(y).all()
        errors.append(max(layer.errors(maps, table, frequencies, R) for layer in model))
    return errors


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=6)
    for i, e in enumerate(main(ap.parse_args().steps)):
        print(f"step {i}: {'prompts' if i == 0 else 'one token each'}, largest error {e:.2e} of the row's largest output")
