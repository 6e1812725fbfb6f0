#!/usr/bin/env python3
"""Decoding steps of one decoder layer on the library's operators.

    python examples/decode_layer.py [--batch 8] [--context 2000] [--steps 64] [--kv int8|16bit] [--check]

A step takes one new token of every sequence through the layer:

    rmsnorm (+ residual) -> W4A16 product (q, k, v) -> rotation -> kv_write
    -> attention over the paged cache -> W4A16 product
    -> rmsnorm_a8 (+ residual) -> W4A8 product (gate, up) -> silu_mul_a8 -> W4A8 product (down)

Weights, prompts and inputs are random. The prompts' keys and values are
written to the cache in one kv_write, as a prefill would write them. The step
is captured into a HIP graph once and replayed; the lengths grow on the GPU.
``--check`` compares the first step with the same layer in plain fp32.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import mixed_precision_w4a16_repack_amd as w4  # noqa: E402

EPS = 1e-5
GROUP = 128


def random_weight(gen, N: int, K: int, dtype, device):
    """A symmetric 4-bit weight [N, K], packed for the kernels, of about unit gain."""
    words = torch.randint(-(2**31), 2**31, (N, K // 8), generator=gen, dtype=torch.int64).to(torch.int32)
    scale = (torch.rand(N, K // GROUP, generator=gen) * 0.5 + 0.75) / (4.6 * K**0.5)  # codes - 8 have a deviation of 4.6
    return w4.repack(words.to(device), scale.to(dtype).to(device), None, GROUP, w4.UINT4B8)


def rotate(x: torch.Tensor, position: torch.Tensor, base: float = 10000.0) -> torch.Tensor:
    """Rotary position embedding of x [B, heads, D]: the halves (x1, x2) turned by position * base^(-2 i / D)."""
    half = x.shape[-1] // 2
    rate = base ** (-torch.arange(half, device=x.device, dtype=torch.float32) / half)
    angle = position.float()[:, None, None] * rate
    c, s = torch.cos(angle), torch.sin(angle)
    a, b = x[..., :half].float(), x[..., half:].float()
    return torch.cat([a * c - b * s, b * c + a * s], -1).to(x.dtype)


class DecodeLayer:
    def __init__(self, hidden=4096, heads=32, kv_heads=8, head_dim=128, inner=14336, dtype=torch.bfloat16,
                 kv_kind=w4.KV_INT8, page_size=64, pages=1024, window=0, seed=0, device="cuda:0"):
        gen = torch.Generator()
        gen.manual_seed(seed)
        self.hidden, self.heads, self.kv_heads, self.head_dim, self.inner = hidden, heads, kv_heads, head_dim, inner
        self.dtype, self.kv_kind, self.page_size, self.pages, self.window = dtype, kv_kind, page_size, pages, window
        self.shapes = {"qkv": ((heads + 2 * kv_heads) * head_dim, hidden), "out": (hidden, heads * head_dim),
                       "gate_up": (2 * inner, hidden), "down": (hidden, inner)}
        self.packed = {name: random_weight(gen, N, K, dtype, device) for name, (N, K) in self.shapes.items()}
        self.norms = [(1 + 0.1 * torch.randn(hidden, generator=gen)).to(dtype).to(device) for _ in range(2)]
        self.cache = torch.zeros(w4.kv_cache_size(pages, kv_heads, head_dim, page_size, kv_kind), dtype=torch.uint8,
                                 device=device)
        # one workspace for each kind of call; a layer's calls are ordered on one stream
        self.ws_gemm, self.ws_a8, self.ws_attention = (w4.Workspace(device) for _ in range(3))

    def _gemm(self, x, name):
        N, K = self.shapes[name]
        return w4.gemm(x, self.packed[name], N, K, GROUP, w4.UINT4B8, workspace=self.ws_gemm)

    def _gemm_a8(self, codes, name):
        N, K = self.shapes[name]
        return w4.gemm_w4a8(*codes, self.packed[name], N, K, GROUP, self.dtype, workspace=self.ws_a8)

    def slots(self, table, position):
        """The cache slots of one position per sequence."""
        page = torch.gather(table, 1, (position // self.page_size)[:, None])[:, 0]
        return page.long() * self.page_size + position % self.page_size

    def write(self, k, v, slots):
        w4.kv_write(k, v, slots, self.cache, self.pages, self.page_size, self.kv_kind)

    def step(self, x, residual, table, lengths):
        """One token of every sequence: x [B, hidden] -> the same; ``residual`` is updated in place.
        ``lengths`` [B] int32 counts the new token."""
        B = x.shape[0]
        h = w4.rmsnorm(x, self.norms[0], EPS, residual=residual, residual_out=residual)
        qkv = self._gemm(h, "qkv").view(B, self.heads + 2 * self.kv_heads, self.head_dim)
        position = (lengths - 1).long()
        turned = rotate(qkv[:, : self.heads + self.kv_heads], position)
        q, k, v = turned[:, : self.heads], turned[:, self.heads :], qkv[:, self.heads + self.kv_heads :]
        self.write(k, v, self.slots(table, position))
        o = w4.attention(q, self.cache, table, lengths, self.pages, self.kv_heads, self.page_size, self.kv_kind,
                         window=self.window, workspace=self.ws_attention)
        x = self._gemm(o.view(B, -1), "out")
        codes = w4.rmsnorm_a8(x, self.norms[1], EPS, residual=residual, residual_out=residual)
        codes = w4.silu_mul_a8(self._gemm_a8(codes, "gate_up"))
        return self._gemm_a8(codes, "down")

    def plain_step(self, x, residual, keys, values, lengths):
        """The same step in plain fp32, without 8-bit rounding. ``keys`` and ``values``: per sequence
        [tokens, kv_heads, head_dim] of the tokens before the new one."""
        f = torch.float32
        weight = {n: w4.dequant(self.packed[n], N, K, GROUP, w4.UINT4B8, self.dtype).to(f) for n, (N, K) in self.shapes.items()}

        def norm(h, w):
            return h * torch.rsqrt(h.pow(2).mean(-1, keepdim=True) + EPS) * w.to(f)

        B, group = x.shape[0], self.heads // self.kv_heads
        residual = residual.to(f) + x.to(f)
        qkv = (norm(residual, self.norms[0]) @ weight["qkv"].t().contiguous()).view(B, -1, self.head_dim)
        turned = rotate(qkv[:, : self.heads + self.kv_heads], lengths.long() - 1)
        o = torch.empty(B, self.heads, self.head_dim, device=x.device)
        for b in range(B):
            k = torch.cat([keys[b].to(f), turned[b : b + 1, self.heads :]])
            v = torch.cat([values[b].to(f), qkv[b : b + 1, self.heads + self.kv_heads :]])
            if self.window:
                k, v = k[-self.window :], v[-self.window :]
            for h in range(self.heads):
                p = torch.softmax(k[:, h // group] @ turned[b, h] * self.head_dim**-0.5, 0)
                o[b, h] = p @ v[:, h // group]
        residual = residual + o.view(B, -1) @ weight["out"].t().contiguous()
        g, u = (norm(residual, self.norms[1]) @ weight["gate_up"].t().contiguous()).chunk(2, dim=1)
        return (g * torch.sigmoid(g) * u) @ weight["down"].t().contiguous(), residual


class Batch:
    """Sequences with random prompts of the given lengths in a layer's cache, with room for ``more`` tokens each."""

    def __init__(self, layer: DecodeLayer, prompts: list[int], more: int, seed=1):
        device = layer.cache.device
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        P = layer.page_size
        width = max(-(-(n + more) // P) for n in prompts)
        table = torch.full((len(prompts), width), -1, dtype=torch.int32)
        order = torch.randperm(layer.pages)
        at = 0
        for b, n in enumerate(prompts):
            need = -(-(n + more) // P)
            if at + need > layer.pages:
                raise ValueError(f"the cache's {layer.pages} pages do not hold these sequences")
            table[b, :need] = order[at : at + need].to(torch.int32)
            at += need
        self.table = table.to(device)
        self.lengths = torch.tensor(prompts, dtype=torch.int32, device=device)
        T, H, D = sum(prompts), layer.kv_heads, layer.head_dim
        k = torch.randn(T, H, D, generator=gen, device=device, dtype=torch.float32).to(layer.dtype)
        v = torch.randn(T, H, D, generator=gen, device=device, dtype=torch.float32).to(layer.dtype)
        t = torch.cat([torch.arange(n) for n in prompts])
        row = torch.repeat_interleave(torch.arange(len(prompts)), torch.tensor(prompts))
        slots = table[row, t // P].long() * P + t % P
        layer.write(k, v, slots.to(device))
        self.keys, self.values = k.split(prompts), v.split(prompts)
        self.x = torch.randn(len(prompts), layer.hidden, generator=gen, device=device).to(layer.dtype)
        self.residual = torch.randn(len(prompts), layer.hidden, generator=gen, device=device).to(layer.dtype)


def capture(layer: DecodeLayer, batch: Batch):
    """A graph that adds a token to every sequence and takes it through the layer; returns (graph, output).
    Nothing is run before the capture but one step on copies, which sizes the workspaces."""
    layer.step(batch.x, batch.residual.clone(), batch.table, batch.lengths.clone().add_(1))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        batch.lengths.add_(1)
        y = layer.step(batch.x, batch.residual, batch.table, batch.lengths)
    return graph, y


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--context", type=int, default=2000, help="the longest prompt; others are shorter")
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--kv", choices=["int8", "16bit"], default="int8")
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--check", action="store_true", help="compare the first step with plain fp32")
    a = ap.parse_args()
    prompts = [max(1, a.context * (i + 1) // a.batch) for i in range(a.batch)]
    more = a.steps + 2
    pages = sum(-(-(n + more) // 64) for n in prompts)
    layer = DecodeLayer(kv_kind=w4.KV_INT8 if a.kv == "int8" else w4.KV_ACT, pages=pages, window=a.window)
    batch = Batch(layer, prompts, more)
    if a.check:
        lengths, residual = batch.lengths + 1, batch.residual.clone()
        want, want_r = layer.plain_step(batch.x, batch.residual, batch.keys, batch.values, lengths)
        got = layer.step(batch.x, residual, batch.table, lengths)
        for name, g, w in (("output", got, want), ("residual", residual, want_r)):
            print(f"{name}: relative error {((g.float() - w).norm() / w.norm()).item():.2e} of plain fp32", flush=True)
    graph, _ = capture(layer, batch)
    graph.replay()
    torch.cuda.synchronize()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(end) / a.steps * 1e3
    print(f"{a.batch} sequences, prompts up to {a.context}, {a.kv} cache: {us:.1f} us a layer and step", flush=True)


if __name__ == "__main__":
    main()
