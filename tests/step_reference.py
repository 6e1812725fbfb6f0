"""64-bit definitions of rotation, of what the rows of several new tokens see,
and of sampling, for the tests of the operators for steps of several tokens a
sequence. Written from the formulas in include/w4a16.h; nothing of the library is used."""

from __future__ import annotations

import math

import numpy as np
import torch


def turned(x, positions, rates, interleaved):
    """Rows x [T, heads, D] turned by their positions, in fp64."""
    out = x.double().clone()
    n = rates.numel()
    w = positions.double()[:, None] * rates.double()[None]
    c, s = torch.cos(w)[:, None], torch.sin(w)[:, None]
    lo = slice(0, 2 * n, 2) if interleaved else slice(0, n)
    hi = slice(1, 2 * n, 2) if interleaved else slice(n, 2 * n)
    a, b = x[..., lo].double(), x[..., hi].double()
    out[..., lo], out[..., hi] = a * c - b * s, b * c + a * s
    return out


def spread(x, rates, interleaved):
    """|x| + |y| of each element's pair (0 where nothing is turned): the size of the rounding of a turn."""
    out = torch.zeros(x.shape, dtype=torch.float64)
    n = rates.numel()
    lo = slice(0, 2 * n, 2) if interleaved else slice(0, n)
    hi = slice(1, 2 * n, 2) if interleaved else slice(n, 2 * n)
    out[..., lo] = out[..., hi] = x[..., lo].double().abs() + x[..., hi].double().abs()
    return out


def bits(words, m):
    """Masks [rows, words] int64 as truth values [rows, 64 * words], cut to m."""
    b = np.unpackbits(words.numpy().astype("<i8").view(np.uint8), axis=1, bitorder="little")
    return torch.from_numpy(b[:, :m].astype(bool)), torch.from_numpy(b.sum(1).astype(np.int64))


def rows_see(n, m, window=0, sinks=0, words=None):
    """[m, n]: which of its sequence's n tokens each of the last m sees."""
    t = torch.arange(n)[None]
    past = n - m
    if words is None:
        at = past + torch.arange(m)[:, None]
        seen = t <= at
        return seen & ((t > at - window) | (t < sinks)) if window else seen
    tree, count = bits(words, max(m, 0))
    at = (past + count - 1)[:, None]
    seen = torch.zeros(m, n, dtype=torch.bool)
    if past >= 0:
        old = (t < past).expand(m, n).clone()
        if window:
            old &= (t > at - window) | (t < sinks)
        seen = old & (count > 0)[:, None]
    for j in range(m):
        if 0 <= past + j < n:
            seen[:, past + j] = tree[:, j] if j < tree.shape[1] else False
    return seen


def random_tree(r, m, words):
    """Masks [m, words] of a random tree whose nodes come after their parents."""
    out = np.zeros((m, words), dtype=np.uint64)
    for i in range(m):
        parent = int(r.integers(-1, i))
        if parent >= 0:
            out[i] = out[parent]
        out[i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
    return torch.from_numpy(out.view(np.int64))


def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, probability, distance of u from the nearest border between two tokens) of one row of logits, in fp64."""
    x = x.double().numpy()
    live = np.flatnonzero(~np.isnan(x) & (x != -np.inf))
    if live.size == 0:
        return -1, 0.0, 1.0
    order = live[np.argsort(-x[live], kind="stable")]
    if not temperature > 0:
        return int(order[0]), 1.0, 1.0
    y = x[order]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.exp((y - y[0]) / temperature)
    w = np.where(y == y[0], 1.0, 0.0 if y[0] == np.inf else w)  # below an infinite logit nothing has weight
    n = len(order)
    if top_k > 0:
        n = min(n, top_k)
    if top_p < 1:
        total = math.fsum(w[:n])
        sums = np.cumsum(w[:n])
        n = int(np.searchsorted(sums, top_p * total, side="left")) + 1 if top_p > 0 else 1
        n = min(n, len(sums))
    if min_p > 0:
        n = min(n, int((w >= min(min_p, 1.0)).sum()))
    sums = np.cumsum(w[:n])
    u = 0.0 if not u > 0 else min(u, 1 - 2.0**-24)
    at = min(int(np.searchsorted(sums, u * sums[-1], side="right")), n - 1)
    return int(order[at]), w[at] / sums[-1], float(np.abs(sums / sums[-1] - u).min())
