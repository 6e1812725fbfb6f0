"""GPU tests of kv_append against the 64-bit definition: turned queries, the
cache's bytes, and that nothing else changes."""

from __future__ import annotations

import pytest
import torch

import mixed_precision_w4a16_repack_amd as w4
from tests import operator_reference as ref
from tests import step_reference as step
from tests.operator_reference import DTYPES, HALF, TINY
from tests.test_gpu_operators import BOTH, DEV, KINDS, gen, randn, within

pytestmark = pytest.mark.gpu

# A turn in fp32: sine and cosine are off by 2^-23 at most (the angle's part of
# a turn is rounded to fp32, then sums of a few roundings of their terms), two products and
# a sum round once each: 4 * 2^-23 of |x| + |y| is more than all of them.
TURN = 2.0**-21


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    w4.load_library()
    yield
    torch.cuda.synchronize()


def rates_of(pairs, base=10000.0):
    return (base ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float()


def slots_of(g, T, pages, P, order):
    if order == "run":
        return torch.arange(T) + int(torch.randint(0, pages * P - T + 1, (1,), generator=g))
    s = torch.randperm(pages * P, generator=g)[:T]
    s[torch.rand(T, generator=g) < 0.15] = -1
    if T > 3:
        s[1] = pages * P + 5
    return s


def check_keys(stored, k, rates, positions, interleaved, kind, dtype):
    want = step.turned(k, positions, rates, interleaved)
    slack = step.spread(k, rates, interleaved) * TURN
    if kind == ref.KV_ACT:
        got = torch.from_numpy(stored[0]).view(DTYPES[dtype])
        within(got, want, want.abs() * HALF[dtype] + slack + TINY[dtype], "keys")
        return
    codes, scale = torch.from_numpy(stored[0]), torch.from_numpy(stored[2].copy()).double()
    amax = want.abs().amax(-1)
    off = slack.amax(-1) + amax * 2.0**-23
    assert bool(((scale - amax / 127).abs() <= off / 127 + amax * 2.0**-30).all()), "scales"
    q = torch.where(amax[..., None] > 0, 127 * want / amax[..., None].clamp(min=1e-300), torch.zeros_like(want))
    # the element and the row's largest are each known to `off`
    within(codes, q, 0.5 + 2 * 127 * (off / amax.clamp(min=1e-300))[..., None] + 1e-5, "codes")


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,H,D,P,T,pairs,order", [
    (4, 1, 64, 32, 1, 32, "any"), (3, 2, 64, 32, 5, 8, "any"), (8, 2, 128, 64, 33, 64, "run"),
    (2, 1, 192, 96, 70, 40, "any"), (5, 1, 256, 32, 40, 128, "run"), (1, 3, 256, 64, 3, 16, "any"),
    # more than a wave for each row of
    (32, 8, 128, 64, 400, 64, "run"), (32, 8, 128, 64, 300, 32, "any"), (64, 16, 64, 32, 131, 24, "run"),
    (20, 10, 192, 32, 333, 96, "any"), (24, 12, 256, 64, 200, 128, "run"), (0, 40, 128, 64, 130, 48, "any"),
])
def test_append(Hq, H, D, P, T, pairs, order, interleaved, kind, dtype):
    g = gen("append", Hq, H, D, P, T, pairs, order, interleaved, kind, dtype)
    dt = DTYPES[dtype]
    pages = -(-T // P) + 3
    q, k, v = (randn(g, T, h, D, dtype=dt, std=2.0) for h in (max(Hq, 1), H, H))
    positions = torch.randint(0, 200000, (T,), generator=g, dtype=torch.int32)
    rates = rates_of(pairs)
    slots = slots_of(g, T, pages, P, order)
    before = torch.randint(0, 256, (w4.kv_cache_size(pages, H, D, P, kind),), generator=g, dtype=torch.uint8)
    cache, plain = before.to(DEV), before.to(DEV)
    got = w4.kv_append(q.to(DEV) if Hq else None, k.to(DEV), v.to(DEV), positions.to(DEV), rates.to(DEV),
                       slots.to(DEV), cache, pages, P, kind, interleaved=interleaved)
    if Hq:
        want = step.turned(q, positions, rates, interleaved)
        within(got.cpu(), want, want.abs() * HALF[dtype] + step.spread(q, rates, interleaved) * TURN + TINY[dtype], "queries")
        assert torch.equal(got[..., 2 * pairs :].cpu(), q[..., 2 * pairs :]), "what is not turned stays"
    else:
        assert got is None
    here = (slots >= 0) & (slots < pages * P)
    stored = ref.gather(cache.cpu().numpy(), slots[here].numpy(), H, D, P, kind, dtype)
    check_keys(stored, k[here], rates, positions[here], interleaved, kind, dtype)
    # Values as kv_write stores them, and every other byte as it was: the keys' bytes of the two caches are made alike.
    w4.kv_write(k.to(DEV), v.to(DEV), slots.to(DEV), plain, pages, P, kind)
    a, b = (c.view(pages, H, -1).cpu().numpy().copy() for c in (cache, plain))
    pk, _, ps = ref.places(D, P, kind)
    for s in slots[here].tolist():
        off = (pk[s % P][:, None] + (range(2) if kind == ref.KV_ACT else range(1))).ravel()
        b[s // P][:, off] = a[s // P][:, off]
        if ps is not None:
            off = ps[0][s % P] + torch.arange(4).numpy()
            b[s // P][:, off] = a[s // P][:, off]
    assert (a == b).all()


@pytest.mark.parametrize("T", [6, 150])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_of_far_negative_and_zero_positions(T, interleaved):
    g = gen("far", T, interleaved)
    H, D, P, dtype = 16, 128, 64, "f16"
    k, v, q = (randn(g, T, H, D, dtype=torch.float16) for _ in range(3))
    positions = torch.tensor([0, 2**31 - 1, -1, -(2**31), 1, 1 << 24], dtype=torch.int32).repeat(T // 6)
    T = positions.numel()
    rates = rates_of(64, 500000.0)
    rates[3], rates[5] = 0.0, -1.0
    cache = torch.zeros(w4.kv_cache_size(4, H, D, P, ref.KV_ACT), dtype=torch.uint8, device=DEV)
    got = w4.kv_append(q[:T].to(DEV), k[:T].to(DEV), v[:T].to(DEV), positions.to(DEV), rates.to(DEV),
                       torch.arange(T).to(DEV), cache, 4, P, ref.KV_ACT, interleaved=interleaved).cpu()
    want = step.turned(q[:T], positions, rates, interleaved)
    # fp64's own rounding of angles of 2^31: 2^-22 in the reference as in the kernel
    slack = step.spread(q[:T], rates, interleaved) * (TURN + 2 * 2.0**-22)
    within(got, want, want.abs() * HALF[dtype] + slack + TINY[dtype])
    zero = positions == 0
    assert torch.equal(got[zero], q[:T][zero]), "position 0 turns nothing"


@pytest.mark.parametrize("T", [4, 120])
def test_append_of_columns_of_one_product_in_place(T):
    """q, k and v as strided columns at odd addresses; the queries are turned in place, the rest stays as it is."""
    g = gen("columns", T)
    Hq, H, D, P, dt = 32, 8, 128, 64, torch.bfloat16
    wide = randn(g, T, (Hq + 2 * H) * D + 7, dtype=dt)
    dev = wide.to(DEV)
    q, k, v = wide[:, 3 : 3 + (Hq + 2 * H) * D].view(T, Hq + 2 * H, D).split([Hq, H, H], dim=1)
    dq, dk, dv = dev[:, 3 : 3 + (Hq + 2 * H) * D].view(T, Hq + 2 * H, D).split([Hq, H, H], dim=1)
    positions, rates = torch.arange(T, dtype=torch.int32) + 77, rates_of(64)
    pages = T // P + 2
    for kind in KINDS:
        cache = torch.zeros(w4.kv_cache_size(pages, H, D, P, kind), dtype=torch.uint8, device=DEV)
        apart = w4.kv_append(dq, dk, dv, positions.to(DEV), rates.to(DEV), torch.arange(T).to(DEV), cache, pages, P, kind)
        want = step.turned(q, positions, rates, False)
        within(apart.cpu(), want, want.abs() * HALF["bf16"] + step.spread(q, rates, False) * TURN + TINY["bf16"])
        check_keys(ref.gather(cache.cpu().numpy(), torch.arange(T).numpy(), H, D, P, kind, "bf16"), k, rates, positions,
                   False, kind, "bf16")
    w4.kv_append(dq, dk, dv, positions.to(DEV), rates.to(DEV), torch.arange(T).to(DEV), cache, pages, P, kind, out=dq)
    assert torch.equal(dq, apart)
    after = dev.cpu()
    after[:, 3 : 3 + Hq * D] = wide[:, 3 : 3 + Hq * D]
    assert torch.equal(after, wide)


@pytest.mark.parametrize("T", [3, 200])
def test_append_int8_rows_with_a_nan_or_of_zeros(T):
    g = gen("nan rows", T)
    H, D, P = 16, 64, 32
    k, v = (randn(g, T, H, D, dtype=torch.float16) for _ in range(2))
    k[1, 0, 5] = float("nan")
    k[2, 1], v[2, 1] = 0, 0
    pages = T // P + 1
    cache = torch.zeros(w4.kv_cache_size(pages, H, D, P, ref.KV_INT8), dtype=torch.uint8, device=DEV)
    w4.kv_append(None, k.to(DEV), v.to(DEV), torch.arange(T, dtype=torch.int32, device=DEV), rates_of(32).to(DEV),
                 torch.arange(T).to(DEV), cache, pages, P, ref.KV_INT8)
    kc, vc, ks, vs = ref.gather(cache.cpu().numpy(), torch.arange(T).numpy(), H, D, P, ref.KV_INT8, "f16")
    assert ks[1, 0] != ks[1, 0] and not (ks[1, 1:] != ks[1, 1:]).any()
    assert ks[2, 1] == 0 and vs[2, 1] == 0 and not kc[2, 1].any() and not vc[2, 1].any()


def test_append_of_no_tokens_and_into_no_pages():
    H, D, P = 2, 64, 32
    empty = torch.empty(0, H, D, dtype=torch.float16, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    cache = torch.zeros(w4.kv_cache_size(1, H, D, P, 0), dtype=torch.uint8, device=DEV)
    got = w4.kv_append(empty, empty, empty, none, rates_of(32).to(DEV), none.long(), cache, 1, P, 0)
    assert got.shape == (0, H, D)
    x = torch.ones(2, H, D, dtype=torch.float16, device=DEV)
    slots = torch.tensor([0, 1], device=DEV)
    got = w4.kv_append(x, x, x, torch.zeros(2, dtype=torch.int32, device=DEV), rates_of(32).to(DEV), slots, cache[:0], 0, P, 0)
    assert torch.equal(got, x) and not bool(cache.any())
