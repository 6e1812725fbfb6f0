"""GPU tests of the operators between a layer's GEMMs against 64-bit plain
forms (tests/operator_reference.py). Tolerances count the roundings each
kernel makes (see each check); inputs are seeded."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import mixed_precision_w4a16_repack_amd as w4
from tests import operator_reference as ref
from tests.operator_reference import DTYPES, HALF, TINY

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BOTH = ["f16", "bf16"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    w4.load_library()
    yield
    torch.cuda.synchronize()


def gen(*key):
    g = torch.Generator()
    g.manual_seed(sum(ord(c) * (i + 1) for i, c in enumerate(repr(key))))
    return g


def randn(g, *shape, dtype, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def within(got, want, tol, what=""):
    err = (got.double() - want).abs() - tol
    worst = err.max().item() if err.numel() else -1.0
    assert worst <= 0, f"{what}: over the bound by {worst:.3e} at {int(err.argmax())}"


# ---------------------------------------------------------------- norm

# The sum of squares, its root and the two products lose at most 2^-18
# relative in fp32 (up to 64 serial additions a thread, then a tree), the
# output half a step.
REL = 2.0**-18
WIDTHS = [(1, 1), (3, 7), (1, 8), (2, 250), (5, 513), (4, 1024), (9, 1031), (2, 2056), (7, 4099), (3, 8192),
          (2, 14336), (2, 16385), (1, 40001)]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("M,K", WIDTHS)
@pytest.mark.parametrize("with_res", [False, True])
def test_rmsnorm(M, K, dtype, with_res):
    g = gen("norm", M, K, dtype, with_res)
    dt = DTYPES[dtype]
    x, w = randn(g, M, K, dtype=dt, std=3.0), randn(g, K, dtype=dt)
    r = randn(g, M, K, dtype=dt, std=2.0) if with_res else None
    y_ref, h_ref = ref.norm(x, w, 1e-5, r)
    rd = None if r is None else r.to(DEV)
    ro = torch.full((M, K), 9.0, dtype=dt, device=DEV)
    y = w4.rmsnorm(x.to(DEV), w.to(DEV), eps=1e-5, residual=rd, residual_out=ro)
    within(y.cpu(), y_ref, y_ref.abs() * (HALF[dtype] + REL) + TINY[dtype], "y")
    within(ro.cpu(), h_ref, h_ref.abs() * (HALF[dtype] + 2.0**-23) + TINY[dtype], "residual_out")


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("K", [24, 4099, 16400])
def test_rmsnorm_strided_unaligned_and_in_place(dtype, K):
    g = gen("norm strided", K, dtype)
    dt = DTYPES[dtype]
    M = 5
    base = randn(g, M, K + 7, dtype=dt).to(DEV)
    x = base[:, 3 : 3 + K]  # rows at odd 2-byte addresses
    w = randn(g, K, dtype=dt).to(DEV)
    res = randn(g, M, K + 3, dtype=dt).to(DEV)
    r = res[:, 1 : 1 + K]
    y_ref, h_ref = ref.norm(x.cpu(), w.cpu(), 0.0, r.cpu())
    out = torch.full((M, K + 5), 7.0, dtype=dt, device=DEV)
    before, edges = base.clone(), res.clone()
    w4.rmsnorm(x, w, eps=0.0, residual=r, residual_out=r, out=out[:, 2 : 2 + K])
    within(out[:, 2 : 2 + K].cpu(), y_ref, y_ref.abs() * (HALF[dtype] + REL) + TINY[dtype], "y")
    within(r.cpu(), h_ref, h_ref.abs() * (HALF[dtype] + 2.0**-23) + TINY[dtype], "residual in place")
    assert torch.equal(base, before)
    assert torch.equal(res[:, :1], edges[:, :1]) and torch.equal(res[:, 1 + K :], edges[:, 1 + K :])
    assert bool((out[:, :2] == 7).all()) and bool((out[:, 2 + K :] == 7).all())
    # y over x
    y2_ref, _ = ref.norm(x.cpu(), w.cpu(), 1e-6)
    w4.rmsnorm(x, w, eps=1e-6, out=x)
    within(x.cpu(), y2_ref, y2_ref.abs() * (HALF[dtype] + REL) + TINY[dtype], "y over x")


def check_codes(qa, xs, y_ref, rel):
    """Codes and scales of y (fp64) known to `rel` relative of each row's largest magnitude."""
    amax = y_ref.abs().amax(1)
    s = amax / 127
    assert bool(((xs.double() - s).abs() <= s * rel).all()), "scales"
    q = torch.where(s[:, None] > 0, y_ref / s[:, None].clamp(min=1e-300), torch.zeros_like(y_ref))
    # the quotient is known to 2 * rel of its size (127 at most)
    err = (qa.double() - ref.pair_order(q)).abs() - (0.5 + 2 * 127 * rel)
    assert err.max().item() <= 0, f"codes: over the bound by {err.max().item():.3e}"
    assert bool(((qa.double().abs().amax(1) == 127) | (amax == 0)).all()), "the largest value has code 127"


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("M,K", [(1, 8), (3, 40), (5, 512), (4, 1024), (2, 2048), (64, 4096), (3, 8200), (2, 16384),
                                 (2, 28672)])
def test_rmsnorm_a8(M, K, dtype):
    g = gen("norm a8", M, K, dtype)
    dt = DTYPES[dtype]
    x, w, r = randn(g, M, K, dtype=dt, std=3.0), randn(g, K, dtype=dt), randn(g, M, K, dtype=dt)
    if M > 1:
        x[1] = 0
        r[1] = 0
    y_ref, h_ref = ref.norm(x, w, 1e-5, r)
    ro = torch.empty(M, K, dtype=dt, device=DEV)
    qa, xs = w4.rmsnorm_a8(x.to(DEV), w.to(DEV), eps=1e-5, residual=r.to(DEV), residual_out=ro)
    within(ro.cpu(), h_ref, h_ref.abs() * (HALF[dtype] + 2.0**-23) + TINY[dtype], "residual_out")
    check_codes(qa.cpu(), xs.cpu(), y_ref, REL)
    if M > 1:
        assert xs[1].item() == 0 and not bool(qa[1].any())


def test_a8_codes_of_tiny_and_huge_rows():
    # bf16 rows far below and above fp32's comfortable range of 127 / max
    x = torch.ones(4, 64, dtype=torch.bfloat16)
    x[:, 1::3] = -0.25
    gate = torch.full((4, 64), 40.0, dtype=torch.bfloat16)  # silu(40) = 40 up to fp32
    scale = torch.tensor([1e-38, 1e-30, 1e30, 3e36], dtype=torch.float64)
    up = (x.double() * scale[:, None]).to(torch.bfloat16)
    qa, xs = w4.silu_mul_a8(torch.cat([gate, up], 1).to(DEV))
    check_codes(qa.cpu(), xs.cpu(), ref.silu_mul(torch.cat([gate, up], 1)), 2.0**-16)


@pytest.mark.parametrize("dtype", BOTH)
def test_silu_mul_a8_of_large_gates(dtype):
    """Gates from -80 to 80: the scale and the codes stay within 2^-20 of the definition at any of them (the codes'
    quotient: 7 roundings of 2^-24 each in the value and in the maximum, and two)."""
    g = gen("gate a8 large", dtype)
    K = 4096
    gate = (torch.linspace(-80, 80, K) + randn(g, 40, K, dtype=torch.float32, std=0.1)).to(DTYPES[dtype])
    gate[::2] = -gate[::2].abs()  # rows of small results only
    x = torch.cat([gate, randn(g, 40, K, dtype=DTYPES[dtype])], 1)
    qa, xs = w4.silu_mul_a8(x.to(DEV))
    check_codes(qa.cpu(), xs.cpu(), ref.silu_mul(x), 2.0**-20)


def test_a8_rows_with_a_nan_keep_it():
    x = torch.ones(3, 512, dtype=torch.float16)
    x[1, 77] = float("nan")
    w = torch.ones(512, dtype=torch.float16)
    _, xs = w4.rmsnorm_a8(x.to(DEV), w.to(DEV))
    _, gs = w4.silu_mul_a8(x.to(DEV))
    for s in (xs, gs):
        assert s.isnan().tolist() == [False, True, False]


@pytest.mark.parametrize("dtype", BOTH)
def test_norm_codes_feed_the_w4a8_gemm(dtype):
    """rmsnorm_a8 + gemm_w4a8 against rmsnorm + quantize_a8 + gemm_w4a8: the codes differ by the rounding
    of y to 16 bits that the second one makes in between."""
    import w4a16_inputs as wi

    dt = DTYPES[dtype]
    M, N, K, G = 24, 512, 1024, 128
    case = wi.make_case(5, M, N, K, G, wi.UINT4B8, dtype)
    packed = w4.repack(torch.from_numpy(case.weight_packed).to(DEV), case.weight_scale.to(DEV), None, G, w4.UINT4B8)
    g = gen("chain", dtype)
    x, w = randn(g, M, K, dtype=dt).to(DEV), randn(g, K, dtype=dt).to(DEV)
    qa, xs = w4.rmsnorm_a8(x, w)
    a = w4.gemm_w4a8(qa, xs, packed, N, K, G, dt).double()
    qb, ys = w4.quantize_a8(w4.rmsnorm(x, w))
    b = w4.gemm_w4a8(qb, ys, packed, N, K, G, dt).double()
    # a code moves by at most 1 where y's rounding (HALF) moves the quotient over a tie
    assert (qa.int() - qb.int()).abs().max().item() <= 1
    assert ((a - b).norm() / b.norm()).item() <= 2.0**-6


# ---------------------------------------------------------------- gate


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("M,K", [(1, 1), (1, 8), (3, 13), (5, 2047), (2, 4099), (4, 14336), (300, 512)])
def test_silu_mul(M, K, dtype):
    g = gen("gate", M, K, dtype)
    dt = DTYPES[dtype]
    x = randn(g, M, 2 * K, dtype=dt, std=4.0)
    want = ref.silu_mul(x)
    y = w4.silu_mul(x.to(DEV))
    # exp's argument g * log2(e) is rounded: up to 24 * 1.45 * 2^-24 of exp; two roundings more
    within(y.cpu(), want, want.abs() * (HALF[dtype] + 2.0**-17) + TINY[dtype] + 1e-36, "y")


@pytest.mark.parametrize("dtype", BOTH)
def test_silu_mul_extremes_and_strides(dtype):
    dt = DTYPES[dtype]
    g = torch.tensor([0.0, -0.0, 30.0, -30.0, -100.0, 100.0, -60000.0, 60000.0, float("inf")], dtype=dt)
    u = torch.tensor([1.0, 2.0, -3.0, 4.0, 5.0, 0.5, 1.0, 1.0, 1.0], dtype=dt)
    wide = torch.zeros(3, 25, dtype=dt)
    wide[:, 5:23] = torch.cat([g, u])
    want = ref.silu_mul(wide[:, 5:23])
    out = torch.full((3, 12), 7.0, dtype=dt, device=DEV)
    w4.silu_mul(wide.to(DEV)[:, 5:23], out=out[:, 1:10])
    got = out[:, 1:10].cpu().double()
    assert bool((got[:, 8] == float("inf")).all())
    want, got = want[:, :8], got[:, :8]
    # exp(30) carries 30 * 1.45 * 2^-24; beyond |g| = 88 the result underflows or is g itself
    within(got, want, want.abs() * (HALF[dtype] + 2.0**-17) + TINY[dtype] + 1e-30, "y")
    assert bool((out[:, 0] == 7).all()) and bool((out[:, 10:] == 7).all())


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("M,K", [(1, 8), (5, 504), (3, 1024), (64, 2048), (8, 14336), (2, 16392), (1, 53248)])
def test_silu_mul_a8(M, K, dtype):
    g = gen("gate a8", M, K, dtype)
    x = randn(g, M, 2 * K, dtype=DTYPES[dtype], std=3.0)
    if M > 1:
        x[1, K:] = 0
    qa, xs = w4.silu_mul_a8(x.to(DEV))
    check_codes(qa.cpu(), xs.cpu(), ref.silu_mul(x), 2.0**-17)


# ---------------------------------------------------------------- cache


def stored(cache, slots, H, D, P, kind):
    return ref.gather(cache.cpu().numpy(), np.asarray(slots), H, D, P, kind, None)


def quantised(x):
    """fp32 scale and the fp64 quotients of rows [..., D]."""
    s = (x.float().abs().amax(-1) / 127).numpy()
    q = np.where(s[..., None] > 0, x.double().numpy() / np.maximum(s[..., None].astype(np.float64), 1e-300), 0.0)
    return s, q


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("kind", [ref.KV_ACT, ref.KV_INT8])
@pytest.mark.parametrize("H,D,P,T,order", [
    (1, 64, 32, 1, "random"), (2, 128, 32, 33, "random"), (3, 192, 96, 100, "runs"), (8, 128, 64, 130, "runs"),
    (1, 256, 256, 515, "runs"), (5, 64, 32, 64, "prompt"), (2, 128, 128, 257, "prompt"), (2, 256, 64, 200, "prompt"),
    (4, 128, 64, 77, "backwards"),
])
def test_cache_write_places_and_read(H, D, P, T, order, kind, dtype):
    g = gen("cache", H, D, P, T, order, kind, dtype)
    dt = DTYPES[dtype]
    pages = -(-T // P) + 3
    if order == "random":
        slots = torch.randperm(pages * P, generator=g)[:T]
    elif order == "prompt":  # whole pages in any order, filled from their start
        page = torch.randperm(pages, generator=g)[: -(-T // P)]
        t = torch.arange(T)
        slots = page[t // P] * P + t % P
    elif order == "runs":  # from the middle of a page, with a gap
        slots = torch.arange(T) + 7
        slots[T // 2 :] += 13
    else:
        slots = torch.arange(T).flip(0) + 5
    skip = torch.randperm(T, generator=g)[: T // 9]
    slots[skip] = torch.where(torch.arange(len(skip)) % 2 == 0, -1, pages * P + 5)
    qkv = randn(g, T, 3 * H, D + 8, dtype=dt, std=2.0)
    k, v = qkv[:, :H, 8:], qkv[:, 2 * H :, :D]  # strided views of one tensor
    if T > 3:
        qkv[3] = 0  # a token of zeros
    nbytes = w4.kv_cache_size(pages, H, D, P, kind)
    fill = torch.randint(0, 256, (nbytes,), generator=g, dtype=torch.uint8)
    cache = fill.to(DEV)
    dqkv = qkv.to(DEV)
    w4.kv_write(dqkv[:, :H, 8:], dqkv[:, 2 * H :, :D], slots.to(DEV), cache, pages, P, kind)
    keep = (slots >= 0) & (slots < pages * P)
    ks, vs = k[keep], v[keep]
    got = stored(cache, slots[keep].numpy(), H, D, P, kind)
    if kind == ref.KV_ACT:
        assert np.array_equal(got[0], ks.contiguous().view(torch.int16).numpy())
        assert np.array_equal(got[1], vs.contiguous().view(torch.int16).numpy())
    else:
        for codes, scales, x in ((got[0], got[2], ks), (got[1], got[3], vs)):
            s, q = quantised(x)
            assert np.allclose(scales, s, rtol=2.0**-23, atol=0)
            # the quotient may be computed with three fp32 roundings
            assert np.abs(codes - q).max() <= 0.5 + 127 * 2.0**-22
    # every other byte is as before
    after = cache.cpu().numpy().reshape(pages, H, -1).copy()
    was = fill.numpy().reshape(pages, H, -1)
    pk, pv, psc = ref.places(D, P, kind)
    width = 2 if kind == ref.KV_ACT else 1
    for s in slots[keep].tolist():
        page, t = s // P, s % P
        for p in (pk, pv):
            for j in range(width):
                after[page][:, p[t] + j] = was[page][:, p[t] + j]
        if psc is not None:
            for w_ in range(2):
                for j in range(4):
                    after[page][:, psc[w_][t] + j] = was[page][:, psc[w_][t] + j]
    assert np.array_equal(after, was), "a byte of another slot changed"
    # reading: the stored values, zeros where there is no slot
    out = torch.full((T, 2 * H, D), 5.0, dtype=dt, device=DEV)
    rk, rv = w4.kv_read(slots.to(DEV), cache, pages, H, D, P, kind, dt, out=(out[:, :H], out[:, H:]))
    assert not bool(rk.cpu()[~keep].any()) and not bool(rv.cpu()[~keep].any())
    if kind == ref.KV_ACT:
        want_k, want_v = ks, vs
    else:
        want_k = (torch.from_numpy(got[0]).float() * torch.from_numpy(got[2].copy())[..., None]).to(dt)
        want_v = (torch.from_numpy(got[1]).float() * torch.from_numpy(got[3].copy())[..., None]).to(dt)
    assert torch.equal(rk.cpu()[keep], want_k) and torch.equal(rv.cpu()[keep], want_v)


@pytest.mark.parametrize("T", [3, 200])
def test_cache_int8_rows_with_a_nan_keep_it(T):
    H, D, P, dt = 2, 64, 32, torch.bfloat16
    g = gen("cache nan", T)
    k, v = randn(g, T, H, D, dtype=dt), randn(g, T, H, D, dtype=dt)
    k[1, 0, 7] = float("nan")
    v[2, 1, 63] = float("nan")
    pages = -(-T // P)
    cache = torch.zeros(w4.kv_cache_size(pages, H, D, P, ref.KV_INT8), dtype=torch.uint8, device=DEV)
    slots = torch.arange(T, device=DEV)
    w4.kv_write(k.to(DEV), v.to(DEV), slots, cache, pages, P, ref.KV_INT8)
    rk, rv = w4.kv_read(slots, cache, pages, H, D, P, ref.KV_INT8, dt)
    for got, x in ((rk.cpu(), k), (rv.cpu(), v)):
        assert torch.equal(got.isnan().all(-1), x.isnan().any(-1)) and torch.equal(got.isnan().any(-1), x.isnan().any(-1))


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("T", [40, 520])
def test_cache_int8_codes_are_exact_at_ties_and_at_the_range_ends(T, dtype):
    """code = 127 x / max rounded half to even, in integers: rows of small integers (many quotients are ties)
    times a power of two from far below to far above 1."""
    H, D, P, dt = 8, 64, 32, DTYPES[dtype]
    g = gen("cache ties", T, dtype)
    top = torch.randint(1, 128, (T, H, 1), generator=g)
    n = torch.minimum(torch.maximum(torch.randint(-127, 128, (T, H, D), generator=g), -top), top)
    n[:, :, :1] = top
    n[:, 0] = torch.where(torch.arange(D) % 2 == 0, 2 * top[:, 0], top[:, 0])  # max / 2: 63.5
    span = 110 if dtype == "bf16" else 7
    x = (n.double() * 2.0 ** torch.randint(-span, span, (T, H, 1), generator=g).double()).to(dt)
    amax = n.abs().amax(-1, keepdim=True)
    twice, whole = 254 * n, 2 * amax  # 127 n / amax + 1/2 = (254 n + amax) / (2 amax)
    up = torch.div(twice + amax, whole, rounding_mode="floor")
    tie = (twice + amax) % whole == 0
    want = torch.where(tie & (up % 2 != 0), up - 1, up)
    pages = -(-T // P)
    cache = torch.zeros(w4.kv_cache_size(pages, H, D, P, ref.KV_INT8), dtype=torch.uint8, device=DEV)
    slots = torch.arange(T)
    w4.kv_write(x.to(DEV), x.flip(0).to(DEV), slots.to(DEV), cache, pages, P, ref.KV_INT8)
    kc, vc, _, _ = stored(cache, slots.numpy(), H, D, P, ref.KV_INT8)
    assert bool(tie.any())
    assert np.array_equal(kc, want.numpy()) and np.array_equal(vc, want.flip(0).numpy())


@pytest.mark.parametrize("kind", [ref.KV_ACT, ref.KV_INT8])
@pytest.mark.parametrize("start", [0, 1, 2, 3, 4, 30, 64])
def test_cache_prompts_that_start_inside_a_tile(start, kind):
    """A ragged batch of prompts in one call: runs that begin anywhere in a tile and end inside a group of 32 tokens."""
    H, D, P, dt = 3, 128, 64, torch.float16
    lens = [33, 100, 5, 64, 31, 200]
    g = gen("ragged prompts", start, kind)
    T = sum(lens)
    pages = sum(-(-(n + start) // P) for n in lens) + 1
    order, slots, at = torch.randperm(pages, generator=g), [], 0
    for n in lens:
        t = torch.arange(n) + start
        slots.append(order[at + t // P] * P + t % P)
        at += -(-(n + start) // P)
    slots = torch.cat(slots)
    k, v = randn(g, T, H, D, dtype=dt), randn(g, T, H, D, dtype=dt)
    fill = torch.randint(0, 256, (w4.kv_cache_size(pages, H, D, P, kind),), generator=g, dtype=torch.uint8)
    cache, whole = fill.to(DEV), fill.to(DEV)
    w4.kv_write(k.to(DEV), v.to(DEV), slots.to(DEV), cache, pages, P, kind)
    for i in range(0, T, 50):  # the same by few tokens at a time
        w4.kv_write(k[i : i + 50].to(DEV), v[i : i + 50].to(DEV), slots[i : i + 50].to(DEV), whole, pages, P, kind)
    assert torch.equal(cache, whole)
    rk, rv = w4.kv_read(slots.to(DEV), cache, pages, H, D, P, kind, dt)
    sk, sv = zip(*(w4.kv_read(slots[i : i + 50].to(DEV), cache, pages, H, D, P, kind, dt) for i in range(0, T, 50)))
    assert torch.equal(rk, torch.cat(sk)) and torch.equal(rv, torch.cat(sv))
    if kind == ref.KV_ACT:
        assert torch.equal(rk.cpu(), k) and torch.equal(rv.cpu(), v)


def test_cache_offsets_past_32_bits():
    """A cache of more than 4 GiB: slots at its end are written, read and attended."""
    H, D, P, kind, dt = 8, 128, 64, ref.KV_ACT, torch.float16
    pages = 18000  # 4.7 GB
    cache = torch.empty(w4.kv_cache_size(pages, H, D, P, kind), dtype=torch.uint8, device=DEV)
    assert cache.numel() > 1 << 32
    g = gen("big cache")
    k, v = randn(g, P, H, D, dtype=dt), randn(g, P, H, D, dtype=dt)
    slots = torch.arange(P) + (pages - 1) * P
    w4.kv_write(k.to(DEV), v.to(DEV), slots.to(DEV), cache, pages, P, kind)
    rk, rv = w4.kv_read(slots.to(DEV), cache, pages, H, D, P, kind, dt)
    assert torch.equal(rk.cpu(), k) and torch.equal(rv.cpu(), v)
    q = randn(g, 1, 2 * H, D, dtype=dt)
    o = w4.attention(q.to(DEV), cache, torch.tensor([[pages - 1]], dtype=torch.int32, device=DEV),
                     torch.tensor([P], dtype=torch.int32, device=DEV), pages, H, P, kind)
    want, A, S = ref.attention(q[0], k, v, torch.ones(P, dtype=torch.bool), D**-0.5)
    within(o[0].cpu(), want, ref.attention_tolerance(want, A, S, "f16", kind, P))


# ---------------------------------------------------------------- attention


class Batch:
    """Sequences over a poisoned cache: everything outside their tokens is 0xFF bytes (NaN values and scales)."""

    def __init__(self, key, lens, H, D, P, kind, dtype, k_std=1.0, holes=()):
        g = gen("attention", key, tuple(lens), H, D, P, kind, dtype)
        self.g, self.dt, self.kind, self.P, self.H, self.D = g, DTYPES[dtype], kind, P, H, D
        self.dtype, self.lens = dtype, list(lens)
        B = len(lens)
        width = max(1, max(-(-n // P) for n in lens)) + 1
        need = sum(-(-n // P) for n in lens)
        self.pages = need + 2
        order = torch.randperm(self.pages, generator=g)
        self.table = torch.full((B, width), -1, dtype=torch.int32)
        self.cache = torch.full((w4.kv_cache_size(self.pages, H, D, P, kind),), 255, dtype=torch.uint8, device=DEV)
        self.k, self.v, at = [], [], 0
        for b, n in enumerate(lens):
            used = -(-n // P)
            self.table[b, :used] = order[at : at + used].to(torch.int32)
            at += used
            k = randn(g, n, H, D, dtype=self.dt, std=k_std)
            v = randn(g, n, H, D, dtype=self.dt) + randn(g, 1, H, D, dtype=self.dt)
            t = torch.arange(n)
            slots = self.table[b].long()[t // P] * P + t % P
            w4.kv_write(k.to(DEV), v.to(DEV), slots.to(DEV), self.cache, self.pages, P, kind)
            if kind == ref.KV_INT8 and n:  # what the cache holds, as values
                c = stored(self.cache, slots.numpy(), H, D, P, kind)
                k = torch.from_numpy(c[0]).double() * torch.from_numpy(c[2].copy()).double()[..., None]
                v = torch.from_numpy(c[1]).double() * torch.from_numpy(c[3].copy()).double()[..., None]
            self.k.append(k)
            self.v.append(v)
        # pages past the sequences' last ones hold any number; some of their own are missing
        self.table[:, -1] = self.pages + 7
        for b, page, value in holes:
            self.table[b, page] = value
        self.dev_table = self.table.to(DEV)
        self.lengths = torch.tensor(lens, dtype=torch.int32, device=DEV)

    def seen(self, b, window):
        n = self.lens[b]
        t = torch.arange(n)
        page = self.table[b].long()[t // self.P]
        ok = (page >= 0) & (page < self.pages)
        return ok & (t >= n - window) if window else ok

    def check(self, Hq, window=0, scale=None, q_std=1.5, q=None, **kw):
        if q is None:
            q = randn(self.g, len(self.lens), Hq, self.D, dtype=self.dt, std=q_std)
        o = w4.attention(q.to(DEV), self.cache, self.dev_table, self.lengths, self.pages, self.H, self.P, self.kind,
                         window=window, scale=scale, **kw)
        got = o.cpu()
        for b, n in enumerate(self.lens):
            want, A, S = ref.attention(q[b], self.k[b], self.v[b], self.seen(b, window),
                                       self.D**-0.5 if scale is None else scale)
            within(got[b], want, ref.attention_tolerance(want, A, S, self.dtype, self.kind, n), f"sequence {b} ({n} tokens)")
            if not bool(self.seen(b, window).any()):
                assert not bool(got[b].any()), f"sequence {b} sees nothing"
        return o


KINDS = [ref.KV_ACT, ref.KV_INT8]
SHORT = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 129]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,H,D,P", [(1, 1, 64, 32), (32, 8, 128, 64), (16, 16, 64, 32), (28, 4, 128, 96),
                                      (40, 8, 192, 64), (16, 1, 256, 128), (32, 1, 128, 32), (64, 1, 64, 64),
                                      (34, 2, 256, 32), (48, 1, 192, 256)])
def test_attention_short(Hq, H, D, P, kind, dtype):
    Batch("short", SHORT, H, D, P, kind, dtype).check(Hq)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,H,D,P,lens", [
    (32, 8, 128, 64, [333]), (8, 8, 128, 32, [1000, 3, 4097]), (16, 2, 64, 256, [5000, 1]),
    (7, 1, 128, 64, [20001]), (10, 2, 256, 64, [3001, 2048]), (6, 3, 192, 32, [1537]),
])
def test_attention_long(Hq, H, D, P, lens, kind, dtype):
    batch = Batch("long", lens, H, D, P, kind, dtype)
    first = batch.check(Hq)
    assert first.shape == (len(lens), Hq, D)


@pytest.mark.parametrize("kind,D,n", [(ref.KV_ACT, 64, 140000), (ref.KV_ACT, 64, 500000), (ref.KV_ACT, 256, 8200),
                                      (ref.KV_INT8, 64, 140000), (ref.KV_INT8, 128, 8200)])
def test_attention_one_head_joined_over_levels(kind, D, n):
    Batch("levels", [n], 1, D, 32, kind, "f16").check(3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,most,zeros", [(64, 1500, 3), (96, 2000, 4), (200, 300, 2), (700, 40, 2), (130, 5000, 60)])
def test_attention_many_sequences(B, most, zeros, kind):
    """Lengths from a square law, most of them cut by the division of work; every `zeros`-th is empty, with runs of
    empty ones longer than a block of 64 in the last case."""
    r = np.random.default_rng(B)
    lens = (most * r.random(B) ** 2).astype(int) + 1
    lens[::zeros] = 0
    if zeros == 60:
        lens[5:125] = 0
    Batch("many", lens.tolist(), 2, 64, 32, kind, "bf16").check(8)


@pytest.mark.parametrize("kind,most,window", [(ref.KV_ACT, 16000, 0), (ref.KV_ACT, 20000, 9001), (ref.KV_INT8, 34000, 0)])
def test_attention_few_heads_cut_evenly(kind, most, window):
    """Fewer heads than workgroups and more tiles than the smallest parts would cover: cut into equal larger parts."""
    r = np.random.default_rng(7)
    lens = r.integers(most // 3, most, 20)
    lens[3], lens[11] = 0, 40
    Batch("even", lens.tolist(), 1, 64, 32, kind, "f16").check(20, window=window)


@pytest.mark.parametrize("kind", KINDS)
def test_attention_split_windows_and_wide_groups(kind):
    """Heads shared by workgroups with a window that starts inside a tile, and more query heads than one operand."""
    Batch("split window", [9000, 4000, 0, 7777, 12345], 2, 128, 64, kind, "f16").check(40, window=5001)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 100, 1000, 100000])
def test_attention_window(window, kind):
    Batch("window", [0, 1, 31, 40, 64, 333, 2500], 2, 128, 64, kind, "f16").check(8, window=window)


@pytest.mark.parametrize("kind", KINDS)
def test_attention_missing_pages_are_not_seen(kind):
    # holes in the middle, at the start, and a sequence whose pages are all missing
    holes = [(0, 1, -1), (0, 3, 10**9), (1, 0, -5), (2, 0, -1), (2, 1, 2**31 - 1)]
    Batch("holes", [300, 65, 100], 2, 64, 64, kind, "bf16", holes=holes).check(8)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", BOTH)
def test_attention_peaked_and_flat_scores(kind, dtype):
    batch = Batch("peaked", [700, 64, 5], 2, 128, 32, kind, dtype, k_std=4.0)
    batch.check(6, q_std=30.0)  # scores in the thousands: one token takes all
    batch.check(6, scale=0.0)  # the plain mean
    batch.check(6, scale=-0.2)  # a negative scale


def test_attention_one_outlier_over_a_long_tail():
    """One token 2^12 times as likely as each of the 60000 others, which together still outweigh it: the
    tail's small probabilities have to count in full."""
    n, H, D, P = 60000, 1, 64, 64
    for kind in KINDS:
        for dtype in BOTH:
            batch = Batch("tail", [n], H, D, P, kind, dtype, k_std=0.0)
            dt = batch.dt
            k = torch.zeros(n, H, D, dtype=dt)
            k[1234, 0, 0] = 8.0
            v = randn(batch.g, n, H, D, dtype=dt, std=0.02) + 1.0
            v[1234] = -3.0
            t = torch.arange(n)
            slots = batch.table[0].long()[t // P] * P + t % P
            w4.kv_write(k.to(DEV), v.to(DEV), slots.to(DEV), batch.cache, batch.pages, P, kind)
            rk, rv = w4.kv_read(slots.to(DEV), batch.cache, batch.pages, H, D, P, kind, dt)
            if kind == ref.KV_INT8:
                page, off = slots // P, slots % P
                rec = batch.cache.cpu().view(batch.pages, -1)
                sc = rec[:, 2 * P * D :].contiguous().view(torch.float32).view(batch.pages, 2, P)
                _, pv, _ = ref.places(D, P, kind)
                codes = rec[page[:, None], torch.from_numpy(pv)[off]].view(torch.int8)
                batch.v = [(codes.double() * sc[page, 1, off][:, None].double())[:, None]]
                batch.k = [k.double()]
            else:
                batch.k, batch.v = [k], [v]
            q = torch.zeros(1, 1, D, dtype=dt)
            q[0, 0, 0] = 8.0
            batch.check(1, scale=float(np.log(2.0**12) / 64.0), q=q)


def test_attention_int8_scales_of_any_size():
    """Values whose scales differ by many orders between tokens, zero rows among them."""
    H, D, P, n = 2, 128, 64, 500
    for dtype, span in (("bf16", 30.0), ("f16", 4.0)):
        batch = Batch("scales", [n], H, D, P, ref.KV_INT8, dtype)
        dt = batch.dt
        mag = 10.0 ** (torch.rand(n, H, 1, generator=batch.g) * 2 * span - span).double()
        v = (randn(batch.g, n, H, D, dtype=torch.float64) * mag).to(dt)
        v[::7] = 0
        t = torch.arange(n)
        slots = batch.table[0].long()[t // P] * P + t % P
        k = batch.k[0].to(dt)
        w4.kv_write(k.to(DEV), v.to(DEV), slots.to(DEV), batch.cache, batch.pages, P, ref.KV_INT8)
        c = stored(batch.cache, slots.numpy(), H, D, P, ref.KV_INT8)
        batch.k = [torch.from_numpy(c[0]).double() * torch.from_numpy(c[2].copy()).double()[..., None]]
        batch.v = [torch.from_numpy(c[1]).double() * torch.from_numpy(c[3].copy()).double()[..., None]]
        batch.check(8)


def test_attention_query_of_any_size_over_int8():
    batch = Batch("query", [200, 1], 2, 64, 32, ref.KV_INT8, "bf16")
    for q_std, scale in ((1e30, 1e-30), (1e-30, 1e30), (1e6, 1e-6)):
        batch.check(4, q_std=q_std, scale=scale)


def test_attention_infinite_and_lowest_keys():
    """Keys of the type's lowest value mask a token by its score; a score of -infinity drops it."""
    H, D, P, n = 1, 64, 32, 70
    for dtype in BOTH:
        batch = Batch("lowest", [n, 40], H, D, P, ref.KV_ACT, dtype)
        dt = batch.dt
        k = batch.k[0].clone()
        k[:, :, 0] = 0
        k[5:60, 0, 0] = torch.finfo(dt).min
        k[60:, 0, 0] = -float("inf")
        k2 = batch.k[1].clone()
        k2[:, 0, 0] = -float("inf")  # every score of this sequence
        for b, kk in ((0, k), (1, k2)):
            t = torch.arange(len(kk))
            slots = batch.table[b].long()[t // P] * P + t % P
            w4.kv_write(kk.to(DEV), batch.v[b].to(DEV), slots.to(DEV), batch.cache, batch.pages, P, ref.KV_ACT)
        q = randn(batch.g, 2, 4, D, dtype=dt).abs() + 0.5
        o = w4.attention(q.to(DEV), batch.cache, batch.dev_table, batch.lengths, batch.pages, H, P, ref.KV_ACT).cpu()
        seen = torch.arange(n) < 5
        want, A, S = ref.attention(q[0], k, batch.v[0], seen, D**-0.5)
        within(o[0], want, ref.attention_tolerance(want, A, S, dtype, ref.KV_ACT, n))
        assert not bool(o[1].any())


def test_attention_nan_in_a_seen_token_shows():
    batch = Batch("nan", [40, 40], 1, 64, 32, ref.KV_ACT, "f16")
    v = batch.v[0].clone()
    v[33, 0, 5] = float("nan")
    slots = batch.table[0].long()[torch.arange(40) // 32] * 32 + torch.arange(40) % 32
    w4.kv_write(batch.k[0].to(DEV), v.to(DEV), slots.to(DEV), batch.cache, batch.pages, 32, ref.KV_ACT)
    q = randn(batch.g, 2, 2, 64, dtype=torch.float16)
    o = w4.attention(q.to(DEV), batch.cache, batch.dev_table, batch.lengths, batch.pages, 1, 32, ref.KV_ACT).cpu()
    assert bool(o[0, :, 5].isnan().all()) and not bool(o[0, :, :5].isnan().any()) and not bool(o[1].isnan().any())


def test_attention_strided_query_output_and_table():
    batch = Batch("strides", [100, 257, 3], 2, 128, 64, ref.KV_ACT, "bf16")
    Hq, D = 8, 128
    qkv = randn(batch.g, 3, (Hq + 4) * D + 3, dtype=torch.bfloat16).to(DEV)
    q = qkv[:, 3 : 3 + Hq * D].view(3, Hq, D)  # odd addresses, a fused product's stride
    wide = torch.full((3, batch.table.shape[1] + 5), 3, dtype=torch.int32, device=DEV)
    wide[:, 1 : 1 + batch.table.shape[1]] = batch.dev_table
    out = torch.full((3, Hq + 1, D + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    batch.dev_table = wide[:, 1 : 1 + batch.table.shape[1]]
    batch.check(Hq, q=q.cpu(), out=out[:, 1:, 8:])
    assert bool((out[:, 0] == 7).all()) and bool((out[:, :, :8] == 7).all())
    got = w4.attention(q, batch.cache, batch.dev_table, batch.lengths, batch.pages, 2, 64, ref.KV_ACT)
    assert torch.equal(got, out[:, 1:, 8:])


def test_attention_lengths_are_clamped_to_the_table():
    batch = Batch("clamp", [128, 128], 1, 64, 64, ref.KV_INT8, "f16")
    batch.dev_table = batch.dev_table[:, :2].contiguous()
    batch.table = batch.table[:, :2]
    batch.lengths = torch.tensor([5000, -3], dtype=torch.int32, device=DEV)
    q = randn(batch.g, 2, 4, 64, dtype=torch.float16)
    o = w4.attention(q.to(DEV), batch.cache, batch.dev_table, batch.lengths, batch.pages, 1, 64, ref.KV_INT8).cpu()
    want, A, S = ref.attention(q[0], batch.k[0], batch.v[0], torch.ones(128, dtype=torch.bool), 64**-0.5)
    within(o[0], want, ref.attention_tolerance(want, A, S, "f16", ref.KV_INT8, 128))
    assert not bool(o[1].any())
    none = w4.attention(q.to(DEV), batch.cache, batch.dev_table[:, :0], batch.lengths, batch.pages, 1, 64, ref.KV_INT8)
    assert not bool(none.any())


@pytest.mark.parametrize("kind", KINDS)
def test_attention_repeats_bit_for_bit_and_on_another_stream(kind):
    batch = Batch("repeat", [3000, 17, 900], 4, 128, 64, kind, "f16")
    q = randn(batch.g, 3, 16, 128, dtype=torch.float16).to(DEV)

    def run(**kw):
        return w4.attention(q, batch.cache, batch.dev_table, batch.lengths, batch.pages, 4, 64, kind, **kw)

    first = run()
    other = Batch("repeat other", [1], 4, 128, 64, kind, "f16")
    other.check(16)  # another shape on the same workspace
    assert torch.equal(run(), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = run()
    torch.cuda.current_stream().wait_stream(side)
    there.record_stream(torch.cuda.current_stream())
    assert torch.equal(there, first)
    ws = w4.Workspace(DEV)
    assert torch.equal(run(workspace=ws), first) and torch.equal(run(workspace=ws), first)


@pytest.mark.parametrize("kind", KINDS)
def test_decode_operators_in_a_graph(kind):
    """Norm, cache write and attention captured together; replays follow the inputs, with eager work between."""
    B, Hq, H, D, P = 3, 8, 2, 128, 64
    batch = Batch("graph", [1500, 40, 64], H, D, P, kind, "bf16")
    g, dt = batch.g, torch.bfloat16
    x = randn(g, B, Hq * D, dtype=dt).to(DEV)
    w = randn(g, Hq * D, dtype=dt).to(DEV)
    kv = randn(g, B, 2 * H, D, dtype=dt).to(DEV)
    lens = torch.tensor([1400, 33, 60], dtype=torch.int32, device=DEV)

    def step(x, kv, lens, ws):
        q = w4.rmsnorm(x, w).view(B, Hq, D)
        at = (lens - 1).long()
        page = torch.gather(batch.dev_table.long(), 1, (at // P)[:, None])[:, 0]
        w4.kv_write(kv[:, :H], kv[:, H:], page * P + at % P, batch.cache, batch.pages, P, kind)
        o = w4.attention(q, batch.cache, batch.dev_table, lens, batch.pages, H, P, kind, workspace=ws)
        return w4.silu_mul(o.reshape(B, Hq * D))

    ws = w4.Workspace(DEV)
    step(x, kv, lens, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(x, kv, lens, ws)
    for rep in range(4):
        lens.add_(1)
        kv.copy_(randn(g, B, 2 * H, D, dtype=dt).to(DEV))
        x.copy_(randn(g, B, Hq * D, dtype=dt).to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(step(x, kv, lens, ws), got), f"replay {rep}"
