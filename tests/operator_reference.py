"""64-bit definitions of the operators between a layer's GEMMs, and the places
of a paged cache's elements, for the operator tests. Written from the
formulas in include/w4a16.h; nothing of the library is used."""

from __future__ import annotations

import numpy as np
import torch

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
# half a rounding step, relative, and half the step below the normal range
HALF = {"f16": 2.0**-11, "bf16": 2.0**-8}
TINY = {"f16": 2.0**-25, "bf16": 2.0**-134}
PAIR_ORDER = [0, 4, 1, 5, 2, 6, 3, 7]
KV_ACT, KV_INT8 = 0, 1


def norm(x, weight, eps, residual=None):
    """(y, h) in fp64."""
    h = x.double() if residual is None else x.double() + residual.double()
    return h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * weight.double(), h


def silu_mul(x):
    g, u = x.double().chunk(2, dim=1)
    return g * torch.sigmoid(g) * u


def pair_order(c):
    return c.view(c.shape[0], -1, 8)[..., PAIR_ORDER].reshape(c.shape)


def record_bytes(D, P, kind):
    return 4 * P * D if kind == KV_ACT else 2 * P * D + 8 * P


def places(D, P, kind):
    """Byte offsets in a record: keys [P, D], values [P, D], scales [2, P] (int8, else None)."""
    t, d = np.arange(P)[:, None], np.arange(D)[None, :]
    if kind == KV_ACT:
        k = (t // 16 * (D // 32) + d // 32) * 1024 + (d % 32 // 8 * 16 + t % 16) * 16 + d % 8 * 2
        v = (t // 32 * (D // 16) + d // 16) * 1024 + (t % 16 // 4 * 16 + d % 16) * 16 + (t % 32 // 16 * 4 + t % 4) * 2
        return k, 2 * P * D + v, None
    k = (t // 16 * (D // 64) + d // 64) * 1024 + (d % 32 // 8 * 16 + t % 16) * 16 + d % 64 // 32 * 8 + d % 8
    v = ((t // 32 * (D // 32) + d // 32) * 1024 + (t % 16 // 4 * 16 + d % 16) * 16 + d % 32 // 16 * 8
         + t % 32 // 16 * 4 + t % 4)
    s = 2 * P * D + 4 * (np.arange(2)[:, None] * P + np.arange(P)[None, :])
    return k, P * D + v, s


def gather(cache, slots, H, D, P, kind, dtype):
    """The stored rows of slots from a cache's bytes (numpy uint8): values [T, H, D] twice as raw bits
    (16 bit), or codes and scales (codes [T, H, D] int8 twice, scales [T, H] fp32 twice)."""
    R = record_bytes(D, P, kind)
    rec = cache.reshape(-1, H, R)
    pk, pv, ps = places(D, P, kind)
    page, t = slots // P, slots % P
    rows = rec[page]  # [T, H, R]

    def take(off, n):
        b = np.stack([np.stack([rows[i][:, off[i] + j] for j in range(n)], -1) for i in range(len(slots))])
        return np.ascontiguousarray(b)

    if kind == KV_ACT:
        k = take(pk[t], 2).view(np.int16)[..., 0]
        v = take(pv[t], 2).view(np.int16)[..., 0]
        return k, v
    one = [take(p[t], 1).view(np.int8)[..., 0] for p in (pk, pv)]
    sc = [take(ps[w][t][:, None], 4).view(np.float32)[..., 0, 0] for w in (0, 1)]
    return one[0], one[1], sc[0], sc[1]


def attention(q, k, v, seen, scale):
    """One sequence in fp64: q [Hq, D], k and v [n, H, D] of its tokens, seen [n] bool.
    Returns (out [Hq, D], A [Hq, D] = sum p |v|, S [Hq] = max_t sum_d |q k| * |scale|)."""
    Hq, D = q.shape
    out = torch.zeros(Hq, D, dtype=torch.float64)
    A, S = torch.zeros_like(out), torch.zeros(Hq, dtype=torch.float64)
    k, v = k[seen].double(), v[seen].double()
    if k.shape[0] == 0:
        return out, A, S
    group = Hq // k.shape[1]
    kk, vv = k.permute(1, 0, 2).contiguous(), v.permute(1, 0, 2).contiguous()  # [H, n, D]
    qq = q.double().view(k.shape[1], group, D)
    s = torch.bmm(qq, kk.transpose(1, 2).contiguous()) * scale
    p = torch.softmax(s, -1)
    S = (torch.bmm(qq.abs(), kk.abs().transpose(1, 2).contiguous()).amax(-1) * abs(scale)).reshape(Hq)
    return torch.bmm(p, vv).reshape(Hq, D), torch.bmm(p, vv.abs()).reshape(Hq, D), S


def attention_tolerance(out, A, S, dtype, kind, n):
    """Error bound of one sequence's output [Hq, D], from the roundings made:
    the probability that multiplies a value is rounded to the 16 bits of the
    matrix operand (the act dtype's; fp16's over an int8 cache), the output to
    the act dtype; a score's fp32 sum is off by at most 64 * 2^-24 of the sum
    of its terms' magnitudes, which moves a probability by that much relative,
    and the sums over tokens and exponentials by 2^-17; probabilities below
    2^-38 of the largest may be lost."""
    p_half = HALF["f16"] if kind == KV_INT8 else HALF[dtype]
    delta = 2 * 64 * 2.0**-24 * S[:, None]
    peak = A.amax() if A.numel() else 0.0
    return A * (p_half + delta + 2.0**-17) + HALF[dtype] * out.abs() + n * 2.0**-36 * peak + TINY[dtype]
