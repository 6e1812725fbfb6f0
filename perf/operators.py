"""What is measured of the operators around the W4A16 / W4A8 GEMMs of a decode layer.

Four kinds of case, each one call (or a write and the read that returns it):

- ``norm``: h = x (+ residual), y = h * rsqrt(mean(h^2) + eps) * weight, with
  16-bit output or int8 codes with a scale per row (the input of the W4A8 GEMM);
- ``act``: silu(gate) * up of a fused gate/up product, same two outputs;
- ``cache``: new keys and values written to a paged cache (16 bit, or int8 with
  a scale per token and head) and read back;
- ``attn``: attention of one new token per sequence over such a cache.

``run`` computes them from elementary torch operations in fp32, or, where
``own`` is true, with the library's calls. 8-bit outputs are returned as the
values they stand for, rounded to the activation dtype.
"""

from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # One decoding user: the norm in front of a 4096-wide W4A16 GEMM. Launch latency.
        dict(name="norm_token", op="norm", M=1, K=4096, dtype="f16", out8=False, residual=True),
        # A batch of 64 users whose next GEMM is W4A8: codes and scales in the same pass.
        dict(name="norm_batch_a8", op="norm", M=64, K=4096, dtype="bf16", out8=True, residual=True),
        # Prompts of 8192 tokens in all: the norm as a pure stream.
        dict(name="norm_prompt", op="norm", M=8192, K=4096, dtype="bf16", out8=False, residual=True),
        # An odd width (a row that is no multiple of a 16-byte load) without residual.
        dict(name="norm_odd", op="norm", M=333, K=4099, dtype="f16", out8=False, residual=False),
        # 8 users, the input of a 14336-wide W4A8 down projection.
        dict(name="act_batch_a8", op="act", M=8, K=14336, dtype="f16", out8=True),
        # 2048 prompt tokens in front of the W4A16 down projection.
        dict(name="act_prompt", op="act", M=2048, K=14336, dtype="bf16", out8=False),
        # One decoding step of 48 users (2 of them padding) into an int8 cache.
        dict(name="cache_step_i8", op="cache", T=48, skip=2, H=8, D=128, P=64, pages=2048, dtype="f16", kv8=True),
        # A ragged batch of prompts, 8000 tokens, into a 16-bit cache.
        dict(name="cache_prompt", op="cache", T=8000, skip=0, H=8, D=128, P=64, pages=512, dtype="bf16", kv8=False),
        # One user early in a conversation: latency.
        dict(name="attn_short", op="attn", B=1, Hq=32, H=8, D=128, P=64, len=333, ragged=False, window=0,
             dtype="f16", kv8=False),
        # 64 users of very different lengths (up to 6000, one of them none yet).
        dict(name="attn_ragged", op="attn", B=64, Hq=32, H=8, D=128, P=64, len=6000, ragged=True, window=0,
             dtype="bf16", kv8=False),
        # 32 users over an int8 cache of up to 16 thousand tokens, one query head per kv head of 64, windowed.
        dict(name="attn_window_i8", op="attn", B=32, Hq=16, H=16, D=64, P=32, len=16000, ragged=True, window=4096,
             dtype="f16", kv8=True),
        # One user with a 131 thousand token context, int8: the split over the cache's length.
        dict(name="attn_long_i8", op="attn", B=1, Hq=64, H=8, D=128, P=128, len=131000, ragged=False, window=0,
             dtype="bf16", kv8=True),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges, sizes spread over their logarithm."""
    op = rng.choice(["norm", "act", "cache", "attn", "attn"])
    dtype = rng.choice(["f16", "bf16"])
    if op in ("norm", "act"):
        out8 = rng.random() < 0.5
        K = _logint(rng, 256, 16384)
        if out8:
            K = max(8, K // 8 * 8)
        M = _logint(rng, 1, max(1, min(8192, (1 << 25) // K)))
        case = dict(op=op, M=M, K=K, dtype=dtype, out8=out8)
        if op == "norm":
            case["residual"] = rng.random() < 0.7
        return case
    D = rng.choice([64, 128, 128, 192, 256])
    P = rng.choice([32, 64, 128, 256])
    kv8 = rng.random() < 0.5
    if op == "cache":
        H = rng.choice([1, 2, 4, 8, 16])
        T = _logint(rng, 1, min(16384, (1 << 23) // (H * D)))
        return dict(op=op, T=T, skip=T // 16, H=H, D=D, P=P, pages=2 * (-(-T // P)) + 8, dtype=dtype, kv8=kv8)
    H, group = rng.choice([(1, 16), (2, 8), (4, 7), (8, 4), (8, 8), (8, 5), (16, 1), (16, 2), (32, 1), (1, 32)])
    # at most the largest listed case's cache values (131 thousand tokens of 8 heads of 128)
    total = _logint(rng, 64, 131000 * 8 * 128 // (H * D))
    B = _logint(rng, 1, max(1, min(256, total // 16)))
    ragged = B > 1 and rng.random() < 0.7
    length = max(1, min(131000, int(total / B * (2.5 if ragged else 1))))
    window = _logint(rng, 1, max(2, length)) if rng.random() < 0.25 else 0
    return dict(op=op, B=B, Hq=H * group, H=H, D=D, P=P, len=length, ragged=ragged, window=window, dtype=dtype, kv8=kv8)


def _lengths(case):
    """The batch's cache lengths: equal, or from none to the longest along a square."""
    B, n = case["B"], case["len"]
    if not case["ragged"]:
        return [n] * B
    lens = [max(1, int(n * ((i + 1) / B) ** 2)) for i in range(B)]
    if B >= 8:
        lens[0] = 0
    return lens


def work(case):
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        n = M * K * (2 + (1 if case["out8"] else 2) + (4 if case["residual"] else 0)) + 2 * K + (4 * M if case["out8"] else 0)
        return {"bytes": n, "flops": 6 * M * K}
    if case["op"] == "act":
        M, K = case["M"], case["K"]
        return {"bytes": M * K * (4 + (1 if case["out8"] else 2)) + (4 * M if case["out8"] else 0), "flops": 6 * M * K}
    H, D = case["H"], case["D"]
    row = H * (2 * D + 8) if case["kv8"] else H * 4 * D  # one token's keys and values in the cache
    if case["op"] == "cache":
        T = case["T"]
        return {"bytes": T * (2 * H * 4 * D + 2 * row + 16), "flops": 8 * T * H * D}
    seen = [min(n, case["window"]) if case["window"] else n for n in _lengths(case)]
    n = sum(seen)
    return {"bytes": n * row + case["B"] * case["Hq"] * D * 4 + 4 * case["B"] + 4 * sum(-(-s // case["P"]) for s in seen),
            "flops": 4 * n * case["Hq"] * D}


# ---------------------------------------------------------------- the cache's layout
# A page holds one record for each kv head, keys first, then values, each in
# tiles of 1024 bytes, then (int8) the page's key scales and value scales.


def _head_bytes(case):
    P, D = case["P"], case["D"]
    return 2 * P * D + 8 * P if case["kv8"] else 4 * P * D


def _regions(cache, case):
    """The cache's bytes as four views indexed by (page, token parts, head, ...):
    keys [n, P/16, 16, H, ...dims], values [n, P/32, 2, 4, 4, H, ...dims], scales [n, P, H] twice."""
    H, D, P = case["H"], case["D"], case["P"]
    n = cache.numel() // (H * _head_bytes(case))
    rec = cache.view(n, H, _head_bytes(case))
    if case["kv8"]:
        codes = rec.view(torch.int8)
        k = codes[..., : P * D].view(n, H, P // 16, D // 64, 4, 16, 2, 8).permute(0, 2, 5, 1, 3, 6, 4, 7)
        v = codes[..., P * D : 2 * P * D].view(n, H, P // 32, D // 32, 4, 16, 2, 2, 4).permute(0, 2, 7, 4, 8, 1, 3, 6, 5)
        s = rec.view(torch.float32)[..., P * D // 2 :]
        return k, v, s[..., :P].permute(0, 2, 1), s[..., P:].permute(0, 2, 1)
    vals = rec.view(DTYPES[case["dtype"]])
    k = vals[..., : P * D].view(n, H, P // 16, D // 32, 4, 16, 8).permute(0, 2, 5, 1, 3, 4, 6)
    v = vals[..., P * D :].view(n, H, P // 32, D // 16, 4, 16, 2, 4).permute(0, 2, 6, 4, 7, 1, 3, 5)
    return k, v, None, None


def _quantise(x):
    """Codes and scales of rows [..., D]: scale max|x| / 127, code round-half-even(x / scale)."""
    x = x.float()
    s = x.abs().amax(-1) / 127
    c = torch.where(s[..., None] > 0, torch.round(x / s[..., None]), torch.zeros_like(x))
    return c.to(torch.int8), s


def _store(cache, case, page, off, k, v):
    """Rows k, v [T, H, D] to (page, offset)."""
    kr, vr, ks, vs = _regions(cache, case)
    if case["kv8"]:
        (k, ksc), (v, vsc) = _quantise(k), _quantise(v)
        ks[page, off], vs[page, off] = ksc, vsc
    kr[page, off // 16, off % 16] = k.view(k.shape[:2] + kr.shape[4:])
    o = off % 32
    vr[page, off // 32, o // 16, o % 16 // 4, o % 4] = v.view(v.shape[:2] + vr.shape[6:])


def _load(cache, case, page, off):
    """Rows k, v [T, H, D] in fp32 from (page, offset)."""
    kr, vr, ks, vs = _regions(cache, case)
    T, H, D = page.numel(), case["H"], case["D"]
    o = off % 32
    k = kr[page, off // 16, off % 16].reshape(T, H, D).float()
    v = vr[page, off // 32, o // 16, o % 16 // 4, o % 4].reshape(T, H, D).float()
    if case["kv8"]:
        k, v = k * ks[page, off][..., None], v * vs[page, off][..., None]
    return k, v


# ---------------------------------------------------------------- inputs


def _randn(gen, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 7919 + 17)
    dt = DTYPES[case["dtype"]]
    st = {"case": case}
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        # a hidden state has a few channels far larger than the rest
        big = torch.where(torch.rand(K, generator=gen, device=DEV) < 0.01, 8.0, 1.0)
        st["x"] = (_randn(gen, M, K) * big).to(dt)
        st["weight"] = (1 + _randn(gen, K, std=0.2)).to(dt)
        st["residual"] = (_randn(gen, M, K, std=2.0) * big).to(dt) if case["residual"] else None
        st["residual_out"] = torch.empty(M, K, dtype=dt, device=DEV) if case["residual"] else None
        return st
    if case["op"] == "act":
        st["x"] = _randn(gen, case["M"], 2 * case["K"], dtype=dt, std=2.0)
        return st
    H, D, P = case["H"], case["D"], case["P"]
    if case["op"] == "cache":
        T, pages = case["T"], case["pages"]
        st["k"] = _randn(gen, T, H, D, dtype=dt, std=1.5)
        st["v"] = _randn(gen, T, H, D, dtype=dt)
        if T * 4 > pages * P:  # prompts: whole pages in any order, filled in order, the last one in part
            need = -(-T // P)
            page = torch.randperm(pages, generator=gen, device=DEV)[:need]
            t = torch.arange(T, device=DEV)
            slots = page[t // P] * P + t % P
        else:  # one token each of many sequences
            slots = torch.randperm(pages * P, generator=gen, device=DEV)[:T]
        if case["skip"]:
            slots[torch.randperm(T, generator=gen, device=DEV)[: case["skip"]]] = -1
        st["slots"] = slots
        st["cache"] = torch.zeros(pages * H * _head_bytes(case), dtype=torch.uint8, device=DEV)
        return st
    B = case["B"]
    lens = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)[torch.randperm(B, generator=gen, device=DEV)]
    width = -(-case["len"] // P)
    used = torch.arange(width, device=DEV)[None] * P < lens[:, None]
    need = sum(-(-n // P) for n in _lengths(case))
    pages = need + 3
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    table[used] = torch.randperm(pages, generator=gen, device=DEV)[:need].to(torch.int32)
    k = _randn(gen, pages * P, H, D, dtype=dt) + _randn(gen, 1, H, D, dtype=dt)
    v = _randn(gen, pages * P, H, D, dtype=dt)
    st["cache"] = torch.empty(pages * H * _head_bytes(case), dtype=torch.uint8, device=DEV)
    slot = torch.arange(pages * P, device=DEV)
    _store(st["cache"], case, slot // P, slot % P, k, v)
    st["q"] = _randn(gen, B, case["Hq"], D, dtype=dt, std=1.5)
    st["table"], st["lengths"], st["pages"] = table, lens, pages
    return st


# ---------------------------------------------------------------- one pass


def _pair_order(x):
    """Columns in the stored order of 8-bit activations: 0, 4, 1, 5, 2, 6, 3, 7 of each 8."""
    return x.view(x.shape[0], -1, 2, 4).transpose(2, 3).reshape(x.shape)


def _plain_out(y, dt, out8):
    if not out8:
        return y.to(dt)
    c, s = _quantise(y)
    return (_pair_order(c).float() * s[:, None]).to(dt)


def _plain(st):
    case = st["case"]
    dt = DTYPES[case["dtype"]]
    if case["op"] == "norm":
        h = st["x"].float()
        if case["residual"]:
            h = h + st["residual"].float()
        y = h * torch.rsqrt(h.pow(2).mean(-1, keepdim=True) + EPS) * st["weight"].float()
        y = _plain_out(y, dt, case["out8"])
        return (y, h.to(dt)) if case["residual"] else y
    if case["op"] == "act":
        g, u = st["x"].float().split(case["K"], dim=1)
        return _plain_out(g / (1 + torch.exp(-g)) * u, dt, case["out8"])
    P = case["P"]
    if case["op"] == "cache":
        slots, k, v = st["slots"], st["k"], st["v"]
        if case["skip"]:
            keep = slots >= 0
            _store(st["cache"], case, slots[keep] // P, slots[keep] % P, k[keep], v[keep])
        else:
            _store(st["cache"], case, slots // P, slots % P, k, v)
        s = slots.clamp(min=0)
        k, v = _load(st["cache"], case, s // P, s % P)
        keep = (slots >= 0)[:, None, None]
        return torch.where(keep, k, 0.0).to(dt), torch.where(keep, v, 0.0).to(dt)
    B, H, D, Hq = case["B"], case["H"], case["D"], case["Hq"]
    # all sequences padded to the longest (or to the longest window)
    n = case["len"] if not case["window"] else min(case["len"], case["window"])
    lens = st["lengths"].long()[:, None]
    t = torch.arange(n, device=DEV)[None] + ((lens - n).clamp(min=0) if case["window"] else 0 * lens)
    page = torch.gather(st["table"].long(), 1, t // P)
    seen = (t < lens) & (page >= 0)
    k, v = _load(st["cache"], case, page.clamp(min=0).reshape(-1), (t % P).reshape(-1))
    v = torch.where(seen.reshape(-1, 1, 1), v, 0.0).view(B, n, H, D).transpose(1, 2).contiguous()
    k = k.view(B, n, H, D).permute(0, 2, 3, 1).contiguous()
    s = torch.matmul(st["q"].float().view(B, H, Hq // H, D), k) * D**-0.5
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return o.view(B, Hq, D).to(dt)


def _own(st):
    import mixed_precision_w4a16_repack_amd as w4

    case = st["case"]
    dt = DTYPES[case["dtype"]]
    if case["op"] in ("norm", "act"):
        if case["op"] == "norm":
            args = dict(eps=EPS, residual=st["residual"], residual_out=st["residual_out"])
            y = (w4.rmsnorm_a8 if case["out8"] else w4.rmsnorm)(st["x"], st["weight"], **args)
        else:
            y = (w4.silu_mul_a8 if case["out8"] else w4.silu_mul)(st["x"])
        if case["out8"]:
            codes, scales = y
            y = torch.mul(codes, scales[:, None], out=torch.empty(codes.shape, dtype=dt, device=DEV))
        return (y, st["residual_out"]) if case.get("residual") else y
    kind = w4.KV_INT8 if case["kv8"] else w4.KV_ACT
    if case["op"] == "cache":
        w4.kv_write(st["k"], st["v"], st["slots"], st["cache"], case["pages"], case["P"], kind)
        return w4.kv_read(st["slots"], st["cache"], case["pages"], case["H"], case["D"], case["P"], kind, dt)
    return w4.attention(st["q"], st["cache"], st["table"], st["lengths"], st["pages"], case["H"], case["P"], kind,
                        window=case["window"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64-bit definitions


def _exact_codes(x):
    s = x.abs().max(-1, keepdim=True).values / 127.0
    return torch.round(x / s.masked_fill(s == 0, 1.0)) * s


def _exact_out(y, out8):
    if not out8:
        return y
    order = torch.tensor([0, 4, 1, 5, 2, 6, 3, 7], device=y.device)
    cols = (torch.arange(0, y.shape[1], 8, device=y.device)[:, None] + order).reshape(-1)
    return _exact_codes(y)[:, cols]


def _exact_row(st, slots):
    """The cache's rows of some slots, by the place of each element: element
    (t, d) of a record's keys lies in tile (t / 16, d / 32 or 64), of its
    values in tile (t / 32, d / 16 or 32)."""
    case = st["case"]
    H, D, P = case["H"], case["D"], case["P"]
    hb = _head_bytes(case)
    d = torch.arange(D, device=DEV)[None, None]
    h = torch.arange(H, device=DEV)[None, :, None]
    page, t = (slots // P)[:, None, None], (slots % P)[:, None, None]
    base = (page * H + h) * hb
    place = (t % 16 // 4) * (128 if not case["kv8"] else 256)  # lane group of a token in a value tile
    pos = t % 4 + 4 * (t % 32 // 16)
    if case["kv8"]:
        b = st["cache"].view(torch.int8)
        f = st["cache"].view(torch.float32)
        k = b[base + (t // 16 * (D // 64) + d // 64) * 1024 + d % 32 // 8 * 256 + t % 16 * 16 + d % 64 // 32 * 8 + d % 8]
        v = b[base + P * D + (t // 32 * (D // 32) + d // 32) * 1024 + place + d % 16 * 16 + d % 32 // 16 * 8 + pos]
        sk = f[(base + 2 * P * D) // 4 + t].double()
        sv = f[(base + 2 * P * D) // 4 + P + t].double()
        return k.double() * sk, v.double() * sv
    b = st["cache"].view(DTYPES[case["dtype"]])
    k = b[base // 2 + (t // 16 * (D // 32) + d // 32) * 512 + d % 32 // 8 * 128 + t % 16 * 8 + d % 8]
    v = b[base // 2 + P * D + (t // 32 * (D // 16) + d // 16) * 512 + place + d % 16 * 8 + pos]
    return k.double(), v.double()


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        h = st["x"].double()
        if case["residual"]:
            h = h + st["residual"].double()
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["K"] + EPS) * st["weight"].double()
        y = _exact_out(y, case["out8"])
        return (y, h) if case["residual"] else y
    if case["op"] == "act":
        x = st["x"].double()
        g, u = x[:, : case["K"]], x[:, case["K"] :]
        return _exact_out(g * torch.sigmoid(g) * u, case["out8"])
    if case["op"] == "cache":
        keep = (st["slots"] >= 0).double()[:, None, None]
        k, v = st["k"].double(), st["v"].double()
        if case["kv8"]:
            k, v = _exact_codes(k), _exact_codes(v)
        return k * keep, v * keep
    B, H, D, P = case["B"], case["H"], case["D"], case["P"]
    out = torch.zeros(B, case["Hq"], D, dtype=torch.float64, device=DEV)
    for b, n in enumerate(st["lengths"].tolist()):
        first = max(0, n - case["window"]) if case["window"] else 0
        if n == first:
            continue
        t = torch.arange(first, n, device=DEV)
        k, v = _exact_row(st, st["table"][b].long()[t // P] * P + t % P)
        q = st["q"][b].double().view(H, case["Hq"] // H, D)
        s = torch.bmm(q, k.permute(1, 2, 0).contiguous()) / math.sqrt(D)
        p = torch.softmax(s, -1)
        out[b] = torch.bmm(p, v.permute(1, 0, 2).contiguous()).reshape(case["Hq"], D)
    return out
