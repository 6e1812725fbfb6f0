"""What is measured of the operators for steps of several tokens a sequence, and of what follows the logits.

Four kinds of case, each one call (int8 caches: and the read that returns what was written):

- ``append``: queries and keys turned by their positions, keys and values written to a paged cache;
- ``sinks``: attention of one new token per sequence that sees a window and the first tokens;
- ``tokens``: attention of several new tokens per sequence over the cache: prompts (causal, with or without a window
  and first tokens) and trees of drafted tokens;
- ``sample``: a token from each row of logits with temperature, top-k, top-p and min-p, from given random numbers.

``run`` computes them from elementary torch operations, or, where ``own`` is true, with the library's calls.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # One decoding step of 8 users, two of them padding, far into long contexts, int8 cache: latency.
        dict(name="append_step_i8", op="append", B=8, m=1, skip=2, Hq=32, H=8, D=128, P=64, pairs=64, turn="half",
             far=131000, dtype="f16", kv8=True),
        # 16 users with 24 drafted tokens each; half of each head turned, pairs of neighbours.
        dict(name="append_drafts", op="append", B=16, m=24, skip=0, Hq=32, H=8, D=128, P=64, pairs=32, turn="pairs",
             far=6000, dtype="bf16", kv8=False),
        # Prompts, 8000 tokens in all, that go on where earlier ones ended: a stream.
        dict(name="append_prompt", op="append", B=4, m=2000, skip=0, Hq=32, H=8, D=128, P=64, pairs=64, turn="half",
             far=1000, dtype="bf16", kv8=False),
        # One user in a long conversation held to a window and its first 4 tokens: latency.
        dict(name="sinks_one", op="sinks", B=1, Hq=32, H=8, D=128, P=64, len=9001, ragged=False, window=1024, sinks=4,
             dtype="f16", kv8=False),
        # 48 users of very different lengths, int8, head size 64, no shared heads.
        dict(name="sinks_batch_i8", op="sinks", B=48, Hq=16, H=16, D=64, P=32, len=20000, ragged=True, window=4096,
             sinks=70, dtype="f16", kv8=True),
        # Ragged prompts under a window with first tokens.
        dict(name="prompt_sinks", op="tokens", B=6, m=2500, Hq=16, H=4, D=128, P=64, len=2500, ragged=True, tree=False,
             window=700, sinks=5, dtype="bf16", kv8=False),
        # One user with 16 drafted tokens: latency.
        dict(name="tree_one", op="tokens", B=1, m=16, Hq=32, H=8, D=128, P=64, len=700, ragged=False, tree=True,
             window=0, sinks=0, dtype="f16", kv8=False),
        # 24 users with trees of 32 tokens over ragged contexts.
        dict(name="tree_batch", op="tokens", B=24, m=32, Hq=32, H=8, D=128, P=64, len=6000, ragged=True, tree=True,
             window=0, sinks=0, dtype="bf16", kv8=False),
        # Two users with trees of 80 tokens over long int8 contexts, 8 query heads a kv head.
        dict(name="tree_long_i8", op="tokens", B=2, m=80, Hq=64, H=8, D=128, P=128, len=50000, ragged=False, tree=True,
             window=0, sinks=0, dtype="bf16", kv8=True),
        # Four prompts up to 2048 tokens: the matrix products.
        dict(name="prompt", op="tokens", B=4, m=2048, Hq=32, H=8, D=128, P=64, len=2048, ragged=False, tree=False,
             window=0, sinks=0, dtype="bf16", kv8=False),
        # One user's next token, an odd vocabulary.
        dict(name="sample_one", op="sample", B=1, V=32003, dtype="bf16", top_k=True, top_p=True, min_p=True, masked=False),
        # 64 users, each with settings of its own; some rows with most tokens forbidden, one with all.
        dict(name="sample_batch", op="sample", B=64, V=128000, dtype="f16", top_k=True, top_p=True, min_p=True, masked=True),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges, sizes spread over their logarithm."""
    op = rng.choice(["append", "sinks", "tokens", "tokens", "sample"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "sample":
        V = _logint(rng, 1000, 200000)
        B = _logint(rng, 1, max(1, min(512, 64 * 128000 // V)))
        return dict(op=op, B=B, V=V, dtype=dtype, top_k=rng.random() < 0.6, top_p=rng.random() < 0.6,
                    min_p=rng.random() < 0.4, masked=rng.random() < 0.3)
    D = rng.choice([64, 128, 128, 192, 256])
    P = rng.choice([32, 64, 128, 256])
    kv8 = rng.random() < 0.5
    if op == "append":
        H, group = rng.choice([(1, 8), (2, 8), (4, 4), (8, 4), (8, 8), (8, 1)])
        T = _logint(rng, 1, 8000 * 8 * 128 * 5 // (H * D * (group + 2)))
        B = _logint(rng, 1, min(T, 64))
        pairs = rng.choice([D // 2, D // 2, D // 4, 8])
        return dict(op=op, B=B, m=max(1, T // B), skip=rng.choice([0, 0, B * max(1, T // B) // 10]), Hq=H * group, H=H, D=D,
                    P=P, pairs=pairs, turn=rng.choice(["half", "half", "pairs"]), far=_logint(rng, 100, 1000000),
                    dtype=dtype, kv8=kv8)
    H, group = rng.choice([(1, 16), (2, 8), (4, 7), (8, 4), (8, 8), (8, 5), (16, 1), (16, 2)])
    if op == "sinks":
        window = _logint(rng, 16, 16000)
        sinks = _logint(rng, 1, 128)
        # at most as many values seen, and as many cached, as in the largest listed case
        B = _logint(rng, 1, max(1, min(128, 4166 * 16 * 64 * 32 // (H * D * (window + sinks)))))
        length = _logint(rng, max(16, window // 4), max(32, window // 4, min(60000, 20000 * 16 * 64 * 16 // (B * H * D))))
        return dict(op=op, B=B, Hq=H * group, H=H, D=D, P=P, len=length, ragged=B > 1 and rng.random() < 0.7, window=window,
                    sinks=sinks, dtype=dtype, kv8=kv8)
    tree = rng.random() < 0.5
    # at most as many scores as the largest listed case
    most = 4 * 32 * 2048 * 2048 * 128 // (H * group * D)
    if tree:
        m = _logint(rng, 2, 128)
        B = _logint(rng, 1, max(1, min(64, most // (m * 4 * m))))
        length = _logint(rng, m + 1, max(m + 2, min(50000, most // (B * m), (1 << 27) // (B * H * D))))
    else:
        length = _logint(rng, 3, int(math.sqrt(most)))
        B = _logint(rng, 1, max(1, min(64, most // (length * length))))
        m = length if rng.random() < 0.7 else _logint(rng, 1, length)
    windowed = rng.random() < 0.4
    return dict(op=op, B=B, m=m, Hq=H * group, H=H, D=D, P=P, len=length, ragged=B > 1 and rng.random() < 0.7, tree=tree,
                window=_logint(rng, max(1, m if tree else 1), max(2, m, length)) if windowed else 0,
                sinks=_logint(rng, 1, 64) if windowed and rng.random() < 0.7 else 0, dtype=dtype, kv8=kv8)


def _lengths(case):
    """The batch's cache lengths: equal, or from none to the longest along a square."""
    B, n = case["B"], case["len"]
    if not case["ragged"]:
        return [n] * B
    lens = [max(1, int(n * ((i + 1) / B) ** 2)) for i in range(B)]
    if B >= 8:
        lens[0] = 0
    return lens


def _spans(case):
    """Of each sequence (tokens any of its new ones sees, tokens seen by all new ones together)."""
    w, s = case["window"], case["sinks"]
    out = []
    for n in _lengths(case):
        m = min(case.get("m", 1), n)
        if case.get("tree"):
            past = n - m
            out.append(((min(past, w + s) if w else past) + m, m * ((min(past, w + s) if w else past) + 1)))
            continue
        at = np.arange(n - m + 1, n + 1)  # tokens up to the new one
        seen = at if not w else np.minimum(at, w) + np.minimum(s, np.maximum(at - w, 0))
        low = max(0, n - m + 1 - w) if w else 0
        out.append((n - low + min(s, low) if n else 0, int(seen.sum())))
    return out


def work(case):
    if case["op"] == "sample":
        return {"bytes": case["B"] * case["V"] * 2 + 32 * case["B"], "flops": case["B"] * case["V"]}
    H, D, Hq = case["H"], case["D"], case["Hq"]
    row = H * (2 * D + 8) if case["kv8"] else H * 4 * D  # one token's keys and values in the cache
    if case["op"] == "append":
        T = case["B"] * case["m"]
        read = T * row if case["kv8"] else 0  # what comes back of an int8 cache
        return {"bytes": T * (4 * Hq * D + 4 * H * D + row + 12) + read + (T * 4 * H * D if case["kv8"] else 0),
                "flops": 6 * T * (Hq + H) * case["pairs"]}
    spans = _spans(case)
    T = sum(min(case.get("m", 1), n) for n in _lengths(case)) if case["op"] == "tokens" else case["B"]
    return {"bytes": sum(t for t, _ in spans) * row + T * Hq * D * 4 + (8 * T if case.get("tree") else 0),
            "flops": 4 * D * Hq * sum(s for _, s in spans)}


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
    s = x.abs().amax(-1) / 127
    c = torch.where(s[..., None] > 0, torch.round(x / s[..., None]), torch.zeros_like(x))
    return c.to(torch.int8), s


def _store(cache, case, page, off, k, v):
    """Rows k, v [T, H, D] in fp32 to (page, offset)."""
    kr, vr, ks, vs = _regions(cache, case)
    if case["kv8"]:
        (k, ksc), (v, vsc) = _quantise(k), _quantise(v)
        ks[page, off], vs[page, off] = ksc, vsc
    else:
        k, v = k.to(kr.dtype), v.to(vr.dtype)
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


def _rates(case):
    return (500000.0 ** (-torch.arange(case["pairs"], device=DEV, dtype=torch.float64) / case["pairs"])).float()


def _trees(gen, counts, most):
    """Masks [rows, words] of random trees: row i sees its ancestors and itself; every parent comes before its children."""
    B, words = len(counts), -(-most // 64)
    parent = (torch.rand(B, most, generator=gen, device=DEV).cpu() * (torch.arange(most) + 1)).long() - 1
    mask = torch.zeros(B, most + 1, words, dtype=torch.int64)  # row 0: no parent
    for i in range(most):
        mask[:, i + 1] = mask[torch.arange(B), parent[:, i] + 1]
        mask[:, i + 1, i // 64] |= (1 << (i % 64)) - (1 << 64 if i % 64 == 63 else 0)
    return torch.cat([mask[b, 1 : c + 1] for b, c in enumerate(counts)]).to(DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 7919 + 17)
    dt = DTYPES[case["dtype"]]
    st = {"case": case}
    if case["op"] == "sample":
        B, V = case["B"], case["V"]
        # most logits in a bulk, a few well above it
        x = _randn(gen, B, V, std=2.0) + 6 * torch.relu(_randn(gen, B, V) - 2.5)
        pick = lambda *of: torch.tensor(of, device=DEV)[torch.randint(len(of), (B,), generator=gen, device=DEV)]  # noqa: E731
        if case["masked"]:
            allowed = pick(1.0, 1.0, 0.5, 50.0 / V)[:, None]
            x = torch.where(torch.rand(B, V, generator=gen, device=DEV) < allowed, x, -math.inf)
            x[B - 1] = -math.inf if B > 1 else x[B - 1]
        st["logits"] = x.to(dt)
        st["u"] = torch.rand(B, generator=gen, device=DEV)
        st["temperature"] = pick(0.0, 0.6, 0.8, 1.0, 1.3)
        st["top_k"] = pick(0, 1, 40, 1000).int() if case["top_k"] else None
        st["top_p"] = pick(1.0, 0.95, 0.9, 0.5) if case["top_p"] else None
        st["min_p"] = pick(0.0, 0.02, 0.1) if case["min_p"] else None
        return st
    H, D, P, B = case["H"], case["D"], case["P"], case["B"]
    if case["op"] == "append":
        m = case["m"]
        T = B * m
        # the queries, keys and values are columns of one product's rows
        qkv = _randn(gen, T, case["Hq"] + 2 * H, D, dtype=dt, std=1.5)
        st["q"], st["k"], st["v"] = qkv.split([case["Hq"], H, H], dim=1)
        first = torch.randint(case["far"], (B,), generator=gen, device=DEV)
        pos = first[:, None] + torch.arange(m, device=DEV)
        st["positions"] = pos.reshape(-1).int()
        each = -(-m // P) + 1  # pages a sequence's new tokens may touch
        pages = B * each + 3
        table = torch.randperm(pages, generator=gen, device=DEV)[: B * each].view(B, each)
        slots = (torch.gather(table, 1, pos // P - (first // P)[:, None]) * P + pos % P).reshape(-1)
        if case["skip"]:
            slots[torch.randperm(T, generator=gen, device=DEV)[: case["skip"]]] = -1
        st["slots"], st["pages"], st["rates"] = slots, pages, _rates(case)
        st["cache"] = torch.zeros(pages * H * _head_bytes(case), dtype=torch.uint8, device=DEV)
        return st
    lens = [_lengths(case)[i] for i in torch.randperm(B, generator=gen, device=DEV).tolist()]
    st["lengths"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    width = -(-case["len"] // P)
    used = torch.arange(width, device=DEV)[None] * P < st["lengths"][:, None]
    need = sum(-(-n // P) for n in lens)
    pages = need + 3
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    table[used] = torch.randperm(pages, generator=gen, device=DEV)[:need].to(torch.int32)
    k = _randn(gen, pages * P, H, D, dtype=dt) + _randn(gen, 1, H, D, dtype=dt)
    v = _randn(gen, pages * P, H, D, dtype=dt)
    st["cache"] = torch.empty(pages * H * _head_bytes(case), dtype=torch.uint8, device=DEV)
    slot = torch.arange(pages * P, device=DEV)
    _store(st["cache"], case, slot // P, slot % P, k.float(), v.float())
    st["table"], st["pages"] = table, pages
    if case["op"] == "sinks":
        st["q"] = _randn(gen, B, case["Hq"], D, dtype=dt, std=1.5)
        return st
    counts = [min(case["m"], n) for n in lens]
    st["starts"] = torch.tensor([0] + counts, device=DEV).cumsum(0).int()
    st["q"] = _randn(gen, sum(counts), case["Hq"], D, dtype=dt, std=1.5)
    st["tree"] = _trees(gen, counts, case["m"]) if case["tree"] else None
    return st


# ---------------------------------------------------------------- one pass


def _turned(x, positions, case, rates):
    """Rows x [T, heads, D] in fp32, turned by their positions; angles in 64 bits."""
    angle = positions.double()[:, None] * rates.double()
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    x, n = x.float(), case["pairs"]
    if case["turn"] == "half":
        a, b = x[..., :n], x[..., n : 2 * n]
        return torch.cat([a * c - b * s, b * c + a * s, x[..., 2 * n :]], -1)
    a, b = x[..., 0 : 2 * n : 2], x[..., 1 : 2 * n : 2]
    return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), x[..., 2 * n :]], -1)


def _plain_append(st):
    case = st["case"]
    dt, P, slots = DTYPES[case["dtype"]], case["P"], st["slots"]
    q = _turned(st["q"], st["positions"], case, st["rates"]).to(dt)
    k, v = _turned(st["k"], st["positions"], case, st["rates"]), st["v"].float()
    keep = slots >= 0
    to = slots[keep] if case["skip"] else slots
    _store(st["cache"], case, to // P, to % P, k[keep] if case["skip"] else k, v[keep] if case["skip"] else v)
    if not case["kv8"]:
        return q, st["cache"].view(dt)
    s = slots.clamp(min=0)
    k, v = _load(st["cache"], case, s // P, s % P)
    keep = keep[:, None, None]
    return q, torch.where(keep, k, 0.0).to(dt), torch.where(keep, v, 0.0).to(dt)


def _softmax_rows(s, seen, v):
    """softmax over the seen scores, times v; zeros where nothing is seen."""
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, 1.0, total)


def _plain_sinks(st):
    case = st["case"]
    P, B, H, D, Hq = case["P"], case["B"], case["H"], case["D"], case["Hq"]
    # the first tokens, then the longest window's
    n = min(case["len"], case["window"])
    lens = st["lengths"].long()[:, None]
    low = (lens - n).clamp(min=0)
    first = torch.arange(min(case["sinks"], case["len"]), device=DEV)[None].expand(B, -1)
    t = torch.cat([first, torch.arange(n, device=DEV)[None] + low], 1)
    seen = t < lens
    seen[:, : first.shape[1]] &= first < low
    page = torch.gather(st["table"].long(), 1, t.clamp(max=case["len"] - 1) // P)
    k, v = _load(st["cache"], case, page.clamp(min=0).reshape(-1), (t % P).reshape(-1))
    v = torch.where(seen.reshape(-1, 1, 1), v, 0.0).view(B, -1, H, D).transpose(1, 2).contiguous()
    k = k.view(B, -1, H, D).permute(0, 2, 3, 1).contiguous()
    s = torch.matmul(st["q"].float().view(B, H, Hq // H, D), k) * D**-0.5
    return _softmax_rows(s, seen[:, None, None], v).view(B, Hq, D).to(DTYPES[case["dtype"]])


def _plain_tokens(st):
    case = st["case"]
    P, B, H, D, Hq, m, n = (case[x] for x in ("P", "B", "H", "D", "Hq", "m", "len"))
    starts, T = st["starts"].long(), st["q"].shape[0]
    row = torch.arange(T, device=DEV)
    b = torch.searchsorted(starts[1:].contiguous(), row, right=True)
    i = row - starts[b]
    lens = st["lengths"].long()[:, None]
    past = lens - (starts[1:] - starts[:-1])[:, None]
    # all sequences padded to the longest, all their new tokens to the most
    q = torch.zeros(B, m, Hq, D, device=DEV)
    q[b, i] = st["q"].float()
    q = q.view(B, m, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(B, H, Hq // H * m, D)
    t = torch.arange(n, device=DEV)
    page = torch.gather(st["table"].long(), 1, (t // P)[None].expand(B, -1))
    k, v = _load(st["cache"], case, page.clamp(min=0).reshape(-1), (t % P)[None].expand(B, -1).reshape(-1))
    v = torch.where((t < lens).reshape(-1, 1, 1), v, 0.0).view(B, n, H, D).transpose(1, 2).contiguous()
    k = k.view(B, n, H, D).permute(0, 2, 3, 1).contiguous()
    if case["tree"]:
        words = torch.zeros(B, m, st["tree"].shape[1], dtype=torch.int64, device=DEV)
        words[b, i] = st["tree"]
        new = (t - past)[:, None]  # [B, 1, n]
        bits = torch.gather(words, 2, (new // 64).clamp(0, words.shape[2] - 1).expand(-1, m, -1)) >> (new % 64) & 1
        every = words[..., None] >> torch.arange(64, device=DEV) & 1
        at = past + every.sum((2, 3)) - 1  # a drafted token's position: its depth behind the past
        seen = (new < 0) | ((bits == 1) & (new >= 0))
        past_only = new < 0
    else:
        at = past + torch.arange(m, device=DEV)
        seen = t <= at[..., None]
        past_only = torch.ones_like(seen)
    if case["window"]:
        seen &= (t > at[..., None] - case["window"]) | (t < case["sinks"]) | ~past_only
    seen &= (t < lens)[:, None]
    s = torch.matmul(q, k) * D**-0.5
    s = s.view(B, H, Hq // H, m, n)
    o = _softmax_rows(s, seen[:, None, None], v[:, :, None])
    return o.permute(0, 3, 1, 2, 4)[b, i].reshape(T, Hq, D).to(DTYPES[case["dtype"]])


def _plain_sample(st):
    x = st["logits"].double()
    V = x.shape[1]
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    t = st["temperature"].double()[:, None]
    top = x[:, :1]
    w = torch.exp((x - top) / torch.where(t > 0, t, 1.0))
    w = torch.where(x == top, 1.0, torch.where(t > 0, w, 0.0))
    w = torch.where(x == -math.inf, 0.0, w)  # forbidden tokens
    j = torch.arange(V, device=DEV)[None]
    w = torch.where((t > 0) | (j == 0), w, 0.0)  # temperature 0: the first of the largest
    if st["top_k"] is not None:
        k = st["top_k"][:, None]
        w = torch.where((k <= 0) | (j < k), w, 0.0)
    total = w.cumsum(1)
    keep = w > 0
    if st["top_p"] is not None:
        p = st["top_p"].double()[:, None]
        keep &= (p >= 1) | (j == 0) | (total - w < p * total[:, -1:])
    if st["min_p"] is not None:
        keep &= w >= st["min_p"].double()[:, None]
    total = torch.where(keep, w, 0.0).cumsum(1)
    last = keep.sum(1, keepdim=True) - 1
    at = (total <= st["u"].double()[:, None] * total[:, -1:]).sum(1, keepdim=True)
    at = torch.minimum(at, last)
    none = at < 0
    at = at.clamp(min=0)
    token = torch.where(none, -1, torch.gather(order, 1, at))[:, 0]
    prob = torch.where(none, 0.0, torch.gather(w, 1, at) / torch.where(none, 1.0, total[:, -1:]))[:, 0]
    return token, prob.float()


def _plain(st):
    return {"append": _plain_append, "sinks": _plain_sinks, "tokens": _plain_tokens, "sample": _plain_sample}[st["case"]["op"]](st)


def _own(st):
    import mixed_precision_w4a16_repack_amd as w4

    case = st["case"]
    if case["op"] == "sample":
        prob = torch.empty(case["B"], device=DEV)
        token = w4.sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                          min_p=st["min_p"], probs=prob)
        return token, prob
    kind = w4.KV_INT8 if case["kv8"] else w4.KV_ACT
    dt = DTYPES[case["dtype"]]
    if case["op"] == "append":
        q = w4.kv_append(st["q"], st["k"], st["v"], st["positions"], st["rates"], st["slots"], st["cache"], st["pages"],
                         case["P"], kind, interleaved=case["turn"] == "pairs")
        if not case["kv8"]:
            return q, st["cache"].view(dt)
        return (q, *w4.kv_read(st["slots"], st["cache"], st["pages"], case["H"], case["D"], case["P"], kind, dt))
    if case["op"] == "sinks":
        return w4.attention(st["q"], st["cache"], st["table"], st["lengths"], st["pages"], case["H"], case["P"], kind,
                            window=case["window"], sinks=case["sinks"])
    return w4.attention_tokens(st["q"], st["starts"], st["cache"], st["table"], st["lengths"], st["pages"], case["H"],
                               case["P"], kind, tree=st["tree"], window=case["window"], sinks=case["sinks"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64-bit definitions


def _places(case, slots):
    """Byte offsets [T, H, D] of the keys and of the values of slots, and of their scales [T, H] (int8), by the place of
    each element: (t, d) of a record's keys lies in tile (t / 16, d / 32 or 64), of its values in tile (t / 32, d / 16 or 32)."""
    H, D, P = case["H"], case["D"], case["P"]
    d = torch.arange(D, device=DEV)[None, None]
    h = torch.arange(H, device=DEV)[None, :, None]
    page, t = (slots // P)[:, None, None], (slots % P)[:, None, None]
    base = (page * H + h) * _head_bytes(case)
    lane, pos = t % 16 // 4 * 256, t % 4 + 4 * (t % 32 // 16)
    if case["kv8"]:
        k = base + (t // 16 * (D // 64) + d // 64) * 1024 + d % 32 // 8 * 256 + t % 16 * 16 + d % 64 // 32 * 8 + d % 8
        v = base + P * D + (t // 32 * (D // 32) + d // 32) * 1024 + lane + d % 16 * 16 + d % 32 // 16 * 8 + pos
        s = (base + 2 * P * D + 4 * t)[..., 0]
        return k, v, s, s + 4 * P
    k = base + (t // 16 * (D // 32) + d // 32) * 1024 + d % 32 // 8 * 256 + t % 16 * 16 + d % 8 * 2
    v = base + 2 * P * D + (t // 32 * (D // 16) + d // 16) * 1024 + lane + d % 16 * 16 + pos * 2
    return k, v, None, None


def _exact_rows(st, slots):
    case = st["case"]
    k, v, ks, vs = _places(case, slots)
    if not case["kv8"]:
        b = st["cache"].view(DTYPES[case["dtype"]])
        return b[k // 2].double(), b[v // 2].double()
    b, f = st["cache"].view(torch.int8), st["cache"].view(torch.float32)
    return b[k].double() * f[ks // 4].double()[..., None], b[v].double() * f[vs // 4].double()[..., None]


def _exact_codes(x):
    s = x.abs().max(-1, keepdim=True).values / 127.0
    return torch.round(x / s.masked_fill(s == 0, 1.0)) * s


def _exact_turn(x, st):
    """Pairs as complex numbers, times exp(i position rate)."""
    case, n = st["case"], st["case"]["pairs"]
    x = x.double().clone()
    lo = torch.arange(n, device=DEV) if case["turn"] == "half" else torch.arange(n, device=DEV) * 2
    hi = lo + (n if case["turn"] == "half" else 1)
    angle = st["positions"].double()[:, None] * st["rates"].double()[None]
    z = torch.complex(x[..., lo], x[..., hi]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    x[..., lo], x[..., hi] = z.real, z.imag
    return x


def _exact_append(st):
    case, slots = st["case"], st["slots"]
    q, k, v = _exact_turn(st["q"], st), _exact_turn(st["k"], st), st["v"].double()
    keep = slots >= 0
    if case["kv8"]:
        here = keep.double()[:, None, None]
        return q, _exact_codes(k) * here, _exact_codes(v) * here
    cache = torch.zeros(st["cache"].numel() // 2, dtype=torch.float64, device=DEV)
    pk, pv, _, _ = _places(case, slots[keep])
    cache[pk // 2], cache[pv // 2] = k[keep], v[keep]
    return q, cache


def _exact_attention(st):
    case = st["case"]
    H, D, P, group = case["H"], case["D"], case["P"], case["Hq"] // case["H"]
    w, sinks = case["window"], case["sinks"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    starts = st["starts"].tolist() if "starts" in st else list(range(case["B"] + 1))
    for b, n in enumerate(st["lengths"].tolist()):
        m = starts[b + 1] - starts[b]
        if n == 0 or m == 0:
            continue
        t = torch.arange(n, device=DEV)
        k, v = _exact_rows(st, st["table"][b].long()[t // P] * P + t % P)
        at = torch.arange(n - m, n, device=DEV)
        if st.get("tree") is not None:
            words = st["tree"][starts[b] : starts[b + 1]].cpu().numpy().astype("<i8")
            bits = np.unpackbits(np.ascontiguousarray(words).view(np.uint8), axis=1, bitorder="little")
            bits = torch.from_numpy(bits).to(DEV).bool()
            depth = bits.sum(1)
            hidden = torch.ones(m, n, dtype=torch.bool, device=DEV)
            hidden[:, n - m :] = ~bits[:, :m]
            hidden[:, : n - m] = False
            if w:
                old = t[None, : n - m] + w < (n - m + depth)[:, None]
                hidden[:, : n - m] = old & (t[None, : n - m] >= sinks)
        else:
            hidden = t[None] > at[:, None]
            if w:
                hidden |= (t[None] + w <= at[:, None]) & (t[None] >= sinks)
        for h in range(H):
            q = st["q"][starts[b] : starts[b + 1], h * group : (h + 1) * group].double().reshape(m * group, D)
            s = torch.mm(q, k[:, h].t().contiguous()) / math.sqrt(D)
            s = s.view(m, group, n).masked_fill(hidden[:, None], -math.inf).view(m * group, n)
            p = torch.softmax(s, -1).nan_to_num(0.0)
            out[starts[b] : starts[b + 1], h * group : (h + 1) * group] = torch.mm(p, v[:, h].contiguous()).view(m, group, D)
    return out


def _exact_sample(st):
    """Row by row on the host, by ranks in a sorted list."""
    got = []
    logits = st["logits"].double().cpu().numpy()
    of = lambda name, off: np.full(len(logits), off) if st[name] is None else st[name].double().cpu().numpy()  # noqa: E731
    u, temperature, top_k, top_p, min_p = st["u"].double().cpu().numpy(), of("temperature", 1), of("top_k", 0), of("top_p", 1), of("min_p", 0)
    for r, x in enumerate(logits):
        order = np.argsort(-x, kind="stable")
        y = x[order][: np.isfinite(x).sum()]
        if y.size == 0:
            got.append(0.0)
            continue
        if temperature[r] == 0:
            got.append(1.0)
            continue
        y = y[: int(top_k[r])] if top_k[r] > 0 else y
        p = np.exp((y - y[0]) / temperature[r])
        n = p.size
        if top_p[r] < 1:
            n = min(n, int(np.searchsorted(np.cumsum(p), top_p[r] * p.sum(), side="left")) + 1)
        p = p[:n]
        p = p[p >= min_p[r]]
        sums = np.cumsum(p)
        got.append(p[min(p.size - 1, int(np.searchsorted(sums, u[r] * sums[-1], side="right")))] / sums[-1])
    return [None, torch.tensor(got, dtype=torch.float64)]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    return _exact_sample(st) if case["op"] == "sample" else _exact_attention(st)
