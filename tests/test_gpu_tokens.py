"""GPU tests of attention with first tokens that stay visible, and of several
new tokens per sequence (prompts, parts of them, trees of drafted tokens),
against 64-bit plain forms. Tolerances: tests/operator_reference.py's, which count
the roundings (the sums here have no other ones)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import mixed_precision_w4a16_repack_amd as w4
from tests import operator_reference as ref
from tests import step_reference as step
from tests.test_gpu_operators import BOTH, DEV, KINDS, Batch, gen, randn, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    w4.load_library()
    yield
    torch.cuda.synchronize()


# ---------------------------------------------------------------- first tokens and a window, one new token


class Sinks(Batch):
    sinks = 0

    def seen(self, b, window):
        n = self.lens[b]
        t = torch.arange(n)
        whole = super().seen(b, 0)
        return whole & ((t >= n - window) | (t < self.sinks)) if window else whole


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 31, 32, 100, 1000])
@pytest.mark.parametrize("sinks", [1, 4, 32, 33, 200, 100000])
def test_sinks(sinks, window, kind):
    batch = Sinks("sinks", [0, 1, 5, 31, 40, 64, 130, 333, 2500], 2, 128, 64, kind, "f16")
    batch.sinks = sinks
    batch.check(8, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,H,D,P,lens,window,sinks", [
    (16, 16, 64, 32, [700, 90, 1], 64, 5), (28, 4, 192, 96, [500, 1000], 300, 70), (34, 2, 256, 64, [900, 30], 100, 33),
    (40, 2, 128, 64, [9000, 4000, 0, 7777], 5001, 40), (5, 1, 128, 128, [20001], 9000, 1000),
])
def test_sinks_shapes(Hq, H, D, P, lens, window, sinks, kind, dtype):
    batch = Sinks("sinks shapes", lens, H, D, P, kind, dtype)
    batch.sinks = sinks
    batch.check(Hq, window=window, sinks=sinks)


@pytest.mark.parametrize("kind", KINDS)
def test_sinks_with_missing_pages(kind):
    """A window's tokens whose first page is gone, and first tokens that are."""
    batch = Sinks("sinks holes", [300, 300], 2, 64, 32, kind, "bf16", holes=[(0, 2, -1), (0, 3, -1), (1, 0, -1)])
    batch.sinks = 10
    batch.check(8, window=100, sinks=10)


@pytest.mark.parametrize("kind", KINDS)
def test_sinks_without_a_window_or_without_sinks_are_the_plain_call(kind):
    batch = Batch("plain call", [500, 33], 2, 64, 32, kind, "f16")
    q = randn(batch.g, 2, 8, 64, dtype=torch.float16).to(DEV)

    def run(**kw):
        return w4.attention(q, batch.cache, batch.dev_table, batch.lengths, batch.pages, 2, 32, kind, **kw)

    assert torch.equal(run(), run(sinks=7))
    assert torch.equal(run(window=64), run(window=64, sinks=0))


@pytest.mark.parametrize("kind", KINDS)
def test_sinks_many_sequences(kind):
    r = np.random.default_rng(5)
    lens = (3000 * r.random(90) ** 2).astype(int)
    batch = Sinks("sinks many", lens.tolist(), 2, 64, 32, kind, "bf16")
    batch.sinks = 4
    batch.check(8, window=512, sinks=4)


# ---------------------------------------------------------------- several new tokens


def tokens(batch, news, Hq, tree=None, window=0, sinks=0, q=None, spare=3, scale=None, **kw):
    """Runs the call for the last news[b] tokens of each sequence and checks it row by row; rows behind the last one stay."""
    starts = np.concatenate([[0], np.cumsum(news)])
    T = int(starts[-1]) + spare
    if q is None:
        q = randn(batch.g, T, Hq, batch.D, dtype=batch.dt, std=1.5)
    words = None
    if tree is not None:
        words = torch.cat([*tree, torch.full((spare, tree[0].shape[1]), -1)])
    out = torch.full((T, Hq, batch.D), 7.0, dtype=batch.dt, device=DEV)
    got = w4.attention_tokens(q.to(DEV), torch.tensor(starts, dtype=torch.int32, device=DEV), batch.cache, batch.dev_table,
                              batch.lengths, batch.pages, batch.H, batch.P, batch.kind,
                              tree=None if words is None else words.to(DEV), window=window, sinks=sinks, scale=scale, out=out, **kw)
    assert got is out
    o = out.cpu()
    assert bool((o[T - spare :] == 7).all()), "rows of no sequence"
    for b, (n, m) in enumerate(zip(batch.lens, news)):
        sees = step.rows_see(n, m, window, sinks, None if tree is None else tree[b]) & batch.seen(b, 0)[None]
        rows = range(m) if m <= 80 else sorted({0, 1, m // 3, m // 2, m - 2, m - 1, *np.random.default_rng(m).integers(0, m, 40)})
        for i in rows:
            row = int(starts[b]) + i
            want, A, S = ref.attention(q[row], batch.k[b], batch.v[b], sees[i], batch.D**-0.5 if scale is None else scale)
            within(o[row], want, ref.attention_tolerance(want, A, S, batch.dtype, batch.kind, n), f"sequence {b}, token {i} of {m} ({n})")
            if not bool(sees[i].any()):
                assert not bool(o[row].any()), f"sequence {b}, token {i} sees nothing"
    return out


SHAPES = [(1, 1, 64, 32), (32, 8, 128, 64), (16, 16, 64, 32), (28, 4, 128, 96), (20, 4, 192, 64), (8, 1, 256, 128)]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,H,D,P", SHAPES)
def test_tokens_short(Hq, H, D, P, kind, dtype):
    """Whole prompts, parts of them and single tokens, none among them, around the tiles' borders."""
    lens = [0, 1, 2, 17, 32, 33, 64, 100, 70, 129]
    news = [0, 1, 1, 17, 32, 5, 1, 33, 0, 16]
    tokens(Batch("tokens short", lens, H, D, P, kind, dtype), news, Hq)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,H,D,P,lens,news", [
    (32, 8, 128, 64, [333], [16]), (8, 8, 128, 32, [1000, 3, 4097], [200, 3, 64]), (16, 2, 64, 256, [5000, 1], [7, 1]),
    (7, 1, 128, 64, [20001], [31]), (10, 2, 256, 64, [1001, 700], [1001, 1]), (6, 3, 192, 32, [1537], [900]),
    (12, 3, 128, 64, [2048, 300], [2048, 300]),
])
def test_tokens_long(Hq, H, D, P, lens, news, kind, dtype):
    tokens(Batch("tokens long", lens, H, D, P, kind, dtype), news, Hq)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (32, 0), (33, 5), (100, 40), (500, 1), (10000, 7)])
def test_tokens_window_and_sinks(window, sinks, kind):
    lens, news = [0, 1, 40, 64, 333, 1200, 900], [0, 1, 40, 5, 333, 70, 400]
    tokens(Batch("tokens window", lens, 2, 128, 64, kind, "f16"), news, 8, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,H,D,P", SHAPES)
def test_tree_short(Hq, H, D, P, kind, dtype):
    r = np.random.default_rng(3)
    lens = [0, 1, 8, 40, 64, 100, 131, 257]
    news = [0, 1, 8, 16, 33, 64, 3, 31]
    tree = [step.random_tree(r, m, 1) for m in news]
    tokens(Batch("tree short", lens, H, D, P, kind, dtype), news, Hq, tree=tree)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (64, 0), (100, 5), (1000, 40)])
def test_tree_of_several_words(window, sinks, kind):
    """Masks of 1 to 200 drafted tokens; a tile may hold bits of two words, or tokens before and in the tree."""
    r = np.random.default_rng(4)
    lens, news = [200, 777, 300, 1500, 64], [200, 130, 65, 97, 64]
    tree = [step.random_tree(r, m, 4) for m in news]
    tokens(Batch("tree words", lens, 2, 128, 64, kind, "bf16"), news, 8, tree=tree, window=window, sinks=sinks)


@pytest.mark.parametrize("kind", KINDS)
def test_tree_rows_without_bits_and_bits_past_the_tree(kind):
    lens, news = [40, 5, 300], [8, 5, 8]
    tree = [torch.zeros(m, 1, dtype=torch.int64) for m in news]
    tree[0][2] = -1  # sees all drafted tokens; bits past the last do not count, but move its position
    tree[0][5] = 1 << 40  # only such a bit: the past
    tree[1][4] = 1
    tree[2][:] = (1 << torch.arange(8))[:, None]
    tokens(Batch("tree empty", lens, 2, 64, 32, kind, "f16"), news, 8, tree=tree)


def test_tree_of_any_mask():
    """Masks need not be trees."""
    g = gen("any mask")
    lens, news = [90, 128, 33], [64, 50, 33]
    tree = [torch.randint(-(2**63), 2**63 - 1, (m, 1), generator=g) for m in news]
    tokens(Batch("any mask", lens, 2, 64, 32, ref.KV_ACT, "f16"), news, 6, tree=tree)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("B,most,m", [(70, 300, 3), (130, 700, 9), (300, 40, 2), (65, 150, 150)])
def test_tokens_many_sequences(B, most, m, tree, kind):
    r = np.random.default_rng(B)
    lens = (most * r.random(B) ** 2).astype(int) + 1
    lens[::5] = 0
    news = np.minimum(lens, r.integers(0, m + 1, B))
    if B == 300:
        news[10:200] = 0
    masks = [step.random_tree(r, int(x), 3) for x in news] if tree else None
    tokens(Batch("tokens many", lens.tolist(), 2, 64, 32, kind, "bf16"), news.tolist(), 8, tree=masks)


@pytest.mark.parametrize("kind", KINDS)
def test_tokens_missing_pages_are_not_seen(kind):
    holes = [(0, 1, -1), (0, 3, 10**9), (1, 0, -5), (2, 0, -1), (2, 1, 2**31 - 1)]
    batch = Batch("tokens holes", [300, 65, 100], 2, 64, 64, kind, "bf16", holes=holes)
    tokens(batch, [70, 65, 20], 8)
    tokens(batch, [3, 1, 0], 8)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", BOTH)
def test_tokens_peaked_and_flat_scores(kind, dtype):
    tokens(Batch("peaked", [400, 70], 2, 64, 32, kind, dtype, k_std=6.0), [50, 70], 8, scale=1.0)
    tokens(Batch("flat", [400, 70], 2, 64, 32, kind, dtype), [50, 70], 8, scale=0.0)
    tokens(Batch("negative", [400, 70], 2, 64, 32, kind, dtype), [50, 70], 8, scale=-0.2)


def write(batch, b, k, v):
    t = torch.arange(len(k))
    slots = batch.table[b].long()[t // batch.P] * batch.P + t % batch.P
    w4.kv_write(k.to(DEV), v.to(DEV), slots.to(DEV), batch.cache, batch.pages, batch.P, batch.kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_tokens_values_that_are_not_finite_reach_only_the_rows_that_see_them(bad, kind):
    n, m, at = 150, 60, 110  # token 110 is new: rows 20 .. see it
    batch = Batch("bad values", [n, 40], 1, 64, 32, kind, "bf16")
    q = randn(batch.g, m + 40 + 3, 4, 64, dtype=torch.bfloat16)
    clean = tokens(batch, [m, 40], 4, q=q).cpu()
    k, v = randn(batch.g, n, 1, 64, dtype=torch.bfloat16), randn(batch.g, n, 1, 64, dtype=torch.bfloat16)
    write(batch, 0, k, v)
    args = (q.to(DEV), torch.tensor([0, m, m + 40], dtype=torch.int32, device=DEV), batch.cache, batch.dev_table, batch.lengths,
            batch.pages, 1, 32, kind)
    before = w4.attention_tokens(*args).cpu()
    v[at, 0, 7] = bad
    write(batch, 0, k, v)
    got = w4.attention_tokens(*args).cpu()
    first = at - (n - m)
    assert torch.equal(got[:first], before[:first]) and torch.equal(got[m : m + 40], clean[m : m + 40])
    assert not bool(got[first:m, :, 7].isfinite().any())
    if kind == ref.KV_ACT:
        others = [d for d in range(64) if d != 7]
        assert torch.equal(got[first:m][..., others], before[first:m][..., others])
    v[at, 0, 7] = 0.0
    k[at, 0, 3] = float("nan")
    write(batch, 0, k, v)
    got = w4.attention_tokens(*args).cpu()
    assert torch.equal(got[:first], before[:first]) and bool(got[first:m].isnan().all())


def test_tokens_infinite_and_lowest_keys():
    for dtype in BOTH:
        n = 70
        batch = Batch("tokens lowest", [n, 40], 1, 64, 32, ref.KV_ACT, dtype)
        k = batch.k[0].clone()
        k[:, :, 0] = 0
        k[5:60, 0, 0] = torch.finfo(batch.dt).min
        k[60:, 0, 0] = -float("inf")
        k2 = batch.k[1].clone()
        k2[:, 0, 0] = -float("inf")
        write(batch, 0, k, batch.v[0])
        write(batch, 1, k2, batch.v[1])
        q = randn(batch.g, 50, 4, 64, dtype=batch.dt).abs() + 0.5
        o = w4.attention_tokens(q.to(DEV), torch.tensor([0, 10, 50], dtype=torch.int32, device=DEV), batch.cache, batch.dev_table,
                                batch.lengths, batch.pages, 1, 32, ref.KV_ACT).cpu()
        for i in range(10):
            want, A, S = ref.attention(q[i], k, batch.v[0], torch.arange(n) < 5, 64**-0.5)
            within(o[i], want, ref.attention_tolerance(want, A, S, dtype, ref.KV_ACT, n))
        assert not bool(o[10:].any())


def test_tokens_int8_scales_of_any_size():
    """Rows of very different magnitude: the value scales' range passes fp16's."""
    batch = Batch("tokens scales", [200], 1, 64, 32, ref.KV_INT8, "bf16")
    v = batch.v[0].to(torch.bfloat16) * (10.0 ** torch.linspace(-12, 12, 200))[torch.randperm(200, generator=batch.g)][:, None, None].to(torch.bfloat16)
    k = randn(batch.g, 200, 1, 64, dtype=torch.bfloat16)
    write(batch, 0, k, v)
    t = torch.arange(200)
    slots = batch.table[0].long()[t // 32] * 32 + t % 32
    rk, rv = w4.kv_read(slots.to(DEV), batch.cache, batch.pages, 1, 64, 32, ref.KV_INT8, torch.bfloat16)
    c = ref.gather(batch.cache.cpu().numpy(), slots.numpy(), 1, 64, 32, ref.KV_INT8, "bf16")
    batch.k[0] = torch.from_numpy(c[0]).double() * torch.from_numpy(c[2].copy()).double()[..., None]
    batch.v[0] = torch.from_numpy(c[1]).double() * torch.from_numpy(c[3].copy()).double()[..., None]
    tokens(batch, [60], 4)


def test_tokens_strided_rows_output_table_and_masks():
    r = np.random.default_rng(9)
    lens, news, Hq, D = [100, 257, 3], [20, 40, 3], 8, 128
    batch = Batch("tokens strides", lens, 2, D, 64, ref.KV_ACT, "bf16")
    T = sum(news)
    qkv = randn(batch.g, T, (Hq + 4) * D + 3, dtype=torch.bfloat16).to(DEV)
    q = qkv[:, 3 : 3 + Hq * D].view(T, Hq, D)
    wide = torch.full((3, batch.table.shape[1] + 5), 3, dtype=torch.int32, device=DEV)
    wide[:, 1 : 1 + batch.table.shape[1]] = batch.dev_table
    words = torch.full((T, 5), -1, device=DEV)
    tree = [step.random_tree(r, m, 2) for m in news]
    words[:, 2:4] = torch.cat(tree).to(DEV)
    starts = torch.tensor([0, 20, 60, 63], dtype=torch.int32, device=DEV)
    for mask, masks in ((None, None), (words[:, 2:4], tree)):
        out = torch.full((T, Hq + 1, D + 8), 7.0, dtype=torch.bfloat16, device=DEV)
        w4.attention_tokens(q, starts, batch.cache, wide[:, 1 : 1 + batch.table.shape[1]], batch.lengths, batch.pages, 2, 64,
                            ref.KV_ACT, tree=mask, out=out[:, 1:, 8:])
        assert bool((out[:, 0] == 7).all()) and bool((out[:, :, :8] == 7).all())
        plain = tokens(batch, news, Hq, q=q.cpu(), tree=masks, spare=0)
        assert torch.equal(out[:, 1:, 8:], plain)


def test_tokens_starts_and_lengths_out_of_range():
    """Starts are cut to the rows, lengths to the table; more new tokens than cached ones: the first see nothing."""
    batch = Batch("tokens clamp", [64, 64, 64], 1, 64, 32, ref.KV_ACT, "f16")
    batch.dev_table, batch.table = batch.dev_table[:, :2].contiguous(), batch.table[:, :2]
    batch.lengths = torch.tensor([5000, 3, -7], dtype=torch.int32, device=DEV)
    q = randn(batch.g, 20, 4, 64, dtype=torch.float16)

    def run(starts, tree=None):
        out = torch.full((20, 4, 64), 7.0, dtype=torch.float16, device=DEV)
        w4.attention_tokens(q.to(DEV), torch.tensor(starts, dtype=torch.int32, device=DEV), batch.cache, batch.dev_table, batch.lengths,
                            batch.pages, 1, 32, ref.KV_ACT, tree=tree, out=out)
        return out.cpu()

    def check(o, row, b, count):
        want, A, S = ref.attention(q[row], batch.k[b], batch.v[b], torch.arange(64) < count, 64**-0.5)
        within(o[row], want, ref.attention_tolerance(want, A, S, "f16", ref.KV_ACT, 64))

    full = torch.full((20, 1), -1, device=DEV)
    for tree in (None, full):
        o = run([-5, 4, 12, 100], tree)
        for i in range(4):  # rows 0 .. 3 are tokens 60 .. 63
            check(o, i, 0, 64 if tree is not None else 61 + i)
        for i in range(5, 8) if tree is None else []:
            check(o, 4 + i, 1, i - 4)
        if tree is None:
            assert not bool(o[4:9].any())
        else:
            for i in range(8):
                check(o, 4 + i, 1, 3)
        assert not bool(o[12:].any())
        o = run([2, 2, 1, 1], tree)  # none, and one that ends before it begins
        assert bool((o == 7).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tree", [False, True])
def test_tokens_repeat_bit_for_bit_and_on_another_stream(tree, kind):
    r = np.random.default_rng(1)
    news = [40, 17, 33]
    batch = Batch("tokens repeat", [3000, 17, 900], 4, 128, 64, kind, "f16")
    q = randn(batch.g, sum(news), 16, 128, dtype=torch.float16).to(DEV)
    masks = torch.cat([step.random_tree(r, m, 1) for m in news]).to(DEV) if tree else None
    starts = torch.tensor([0, 40, 57, 90], dtype=torch.int32, device=DEV)

    def run(**kw):
        return w4.attention_tokens(q, starts, batch.cache, batch.dev_table, batch.lengths, batch.pages, 4, 64, kind, tree=masks, **kw)

    first = run()
    tokens(Batch("tokens other", [70], 4, 128, 64, kind, "f16"), [70], 16)
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
    ws.buf.fill_(255)  # the workspace's contents do not matter
    assert torch.equal(run(workspace=ws), first)


def test_tokens_of_one_new_token_agree_with_attention():
    batch = Batch("one token", [500, 33, 1, 64], 2, 128, 64, ref.KV_ACT, "f16")
    q = randn(batch.g, 4, 8, 128, dtype=torch.float16)
    starts = torch.arange(5, dtype=torch.int32, device=DEV)
    got = tokens(batch, [1, 1, 1, 1], 8, q=q, spare=0)
    one = w4.attention(q.to(DEV), batch.cache, batch.dev_table, batch.lengths, batch.pages, 2, 64, ref.KV_ACT)
    # each within its own bound of the exact result: half a step and the sums' 2^-17 or so
    assert bool(((got.float() - one.float()).abs() <= 2 * 2.0**-11 * one.float().abs() + 2.0**-14).all())
    assert starts.numel() == 5


def test_tokens_cache_offsets_past_32_bits():
    H, D, P, kind = 8, 128, 64, ref.KV_ACT
    pages = 18000  # 4.7 GB
    cache = torch.empty(w4.kv_cache_size(pages, H, D, P, kind), dtype=torch.uint8, device=DEV)
    g = gen("big cache tokens")
    k, v, q = (randn(g, P, h, D, dtype=torch.float16) for h in (H, H, 2 * H))
    slots = torch.arange(P) + (pages - 1) * P
    rates = torch.zeros(64, device=DEV)
    turned = w4.kv_append(q.to(DEV), k.to(DEV), v.to(DEV), torch.arange(P, dtype=torch.int32, device=DEV), rates, slots.to(DEV), cache,
                          pages, P, kind)
    assert torch.equal(turned.cpu(), q), "rates of 0 turn nothing"
    o = w4.attention_tokens(turned, torch.tensor([0, P], dtype=torch.int32, device=DEV), cache,
                            torch.tensor([[pages - 1]], dtype=torch.int32, device=DEV), torch.tensor([P], dtype=torch.int32, device=DEV),
                            pages, H, P, kind).cpu()
    for i in (0, 31, 63):
        want, A, S = ref.attention(q[i], k, v, torch.arange(P) <= i, D**-0.5)
        within(o[i], want, ref.attention_tolerance(want, A, S, "f16", kind, P))


def test_tokens_of_nothing():
    batch = Batch("nothing", [40], 1, 64, 32, ref.KV_ACT, "f16")
    empty = torch.empty(0, 4, 64, dtype=torch.float16, device=DEV)
    o = w4.attention_tokens(empty, torch.tensor([0, 0], dtype=torch.int32, device=DEV), batch.cache, batch.dev_table, batch.lengths,
                            batch.pages, 1, 32, ref.KV_ACT)
    assert o.shape == (0, 4, 64)
    q = torch.ones(2, 4, 64, dtype=torch.float16, device=DEV)
    out = torch.full_like(q, 7)
    w4.attention_tokens(q, torch.tensor([0], dtype=torch.int32, device=DEV), batch.cache, batch.dev_table[:0], batch.lengths[:0],
                        batch.pages, 1, 32, ref.KV_ACT, out=out)
    assert bool((out == 7).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,H,D", [(6, 2, 192), (4, 2, 256), (16, 2, 192), (16, 2, 64)])
def test_tokens_several_blocks_a_workgroup(Hq, H, D, kind):
    """More blocks than workgroups: each goes from one to the next, and blocks begin and end in different ones."""
    r = np.random.default_rng(D + Hq)
    news = r.integers(100, 330, 40)
    lens = news + (r.random(40) < 0.5) * r.integers(0, 200, 40)
    tokens(Batch("tokens blocks", lens.tolist(), H, D, 32, kind, "bf16"), news.tolist(), Hq)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 192, 256])
def test_tree_values_that_are_not_finite_in_the_tree(D, kind):
    """A drafted token's value that is not finite reaches its descendants only."""
    past, m, bad = 40, 30, 4
    r = np.random.default_rng(D)
    words = step.random_tree(r, m, 1)
    sees, _ = step.bits(words, m)
    batch = Batch("tree bad", [past + m], 1, D, 32, kind, "f16")
    n = past + m
    q = randn(batch.g, m, 4, D, dtype=torch.float16)
    k, v = randn(batch.g, n, 1, D, dtype=torch.float16), randn(batch.g, n, 1, D, dtype=torch.float16)
    args = (q.to(DEV), torch.tensor([0, m], dtype=torch.int32, device=DEV), batch.cache, batch.dev_table, batch.lengths,
            batch.pages, 1, 32, kind)
    write(batch, 0, k, v)
    before = w4.attention_tokens(*args, tree=words.to(DEV)).cpu()
    v[past + bad, 0, 3] = float("inf")
    write(batch, 0, k, v)
    got = w4.attention_tokens(*args, tree=words.to(DEV)).cpu()
    below = sees[:, bad]
    assert bool(below.any()) and not bool(below.all())
    assert torch.equal(got[~below], before[~below]) and not bool(got[below][..., 3].isfinite().any())


@pytest.mark.parametrize("tree", [False, True])
def test_tokens_windows_near_2_63(tree):
    """As without a window, also at positions below 0 (more tokens new than cached), and with an empty table."""
    batch = Batch("huge window", [64, 3], 1, 64, 32, ref.KV_ACT, "f16")
    q = randn(batch.g, 130, 4, 64, dtype=torch.float16).to(DEV)
    starts = torch.tensor([0, 30, 130], dtype=torch.int32, device=DEV)
    words = torch.randint(-(2**63), 2**63 - 1, (130, 2), generator=batch.g).to(DEV) if tree else None

    def run(table, **kw):
        return w4.attention_tokens(q, starts, batch.cache, table, batch.lengths, batch.pages, 1, 32, ref.KV_ACT, tree=words, **kw)

    want = run(batch.dev_table)
    for window in (1 << 32, 1 << 62, 2**63 - 100, 2**63 - 4, 2**63 - 1):
        for sinks in (0, 4, 2**63 - 1):
            assert torch.equal(run(batch.dev_table, window=window, sinks=sinks), want)
            assert not bool(run(batch.dev_table[:, :0], window=window, sinks=sinks).any())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 0), (40, 3), (100, 0), (300, 40)])
def test_tree_bits_past_the_new_tokens_change_nothing(window, sinks, kind):
    """Words padded with ones, or with any bits, behind a sequence's new tokens: neither the tokens that a row sees nor
    its position in a window depend on them."""
    r = np.random.default_rng(6)
    lens, news, words = [200, 333, 64, 700, 65], [5, 40, 64, 130, 65], 3
    tree = [step.random_tree(r, m, words) for m in news]
    batch = Batch("tree padding", lens, 2, 128, 64, kind, "bf16")
    q = randn(batch.g, sum(news), 8, 128, dtype=torch.bfloat16)
    clean = tokens(batch, news, 8, tree=tree, window=window, sinks=sinks, q=q, spare=0)
    starts = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device=DEV)
    for fill in ("ones", "any"):
        padded = []
        for m, t in zip(news, tree):
            past = torch.zeros(words, 64, dtype=torch.bool)
            past.view(-1)[m:] = True
            mask = torch.from_numpy(np.packbits(past.numpy(), axis=1, bitorder="little").view("<i8")[:, 0].copy())
            some = -1 if fill == "ones" else torch.from_numpy(r.integers(-(2**63), 2**63 - 1, t.shape))
            padded.append(t | (mask & some))
        assert any(bool((p != t).any()) for p, t in zip(padded, tree))
        got = w4.attention_tokens(q.to(DEV), starts, batch.cache, batch.dev_table, batch.lengths, batch.pages, 2, 64, kind,
                                  tree=torch.cat(padded).to(DEV), window=window, sinks=sinks)
        assert torch.equal(got, clean)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (7, 0), (40, 3), (64, 0)])
def test_tree_rows_of_bits_past_the_new_tokens_only(window, sinks, kind):
    """They see what lies before the new tokens, as at the first new one's position; a row of zeros sees nothing."""
    lens, news, Hq = [90, 129], [6, 33], 4
    batch = Batch("tree past only", lens, 2, 64, 32, kind, "f16")
    q = randn(batch.g, sum(news), Hq, 64, dtype=torch.float16)
    tree = torch.zeros(sum(news), 2, dtype=torch.int64)
    for row, words in ((1, [1 << 6, 0]), (2, [-64, -1]), (4, [0, 1]), (8, [1 << 33, 0]), (30, [0, -1])):
        tree[row] = torch.tensor(words)
    starts = torch.tensor([0, 6, 39], dtype=torch.int32, device=DEV)
    o = w4.attention_tokens(q.to(DEV), starts, batch.cache, batch.dev_table, batch.lengths, batch.pages, 2, 32, kind,
                            tree=tree.to(DEV), window=window, sinks=sinks).cpu()
    for row in range(sum(news)):
        b = int(row >= 6)
        n, past = lens[b], lens[b] - news[b]
        t = torch.arange(n)
        seen = (t < past) & ((t > past - window) | (t < sinks) | (window == 0)) & bool(tree[row].any())
        want, A, S = ref.attention(q[row], batch.k[b], batch.v[b], seen, 64**-0.5)
        within(o[row], want, ref.attention_tolerance(want, A, S, "f16", kind, n), f"row {row}")



def test_tokens_int8_tiny_scales_of_queries_and_scores():
    """A factor on the scores below fp32's range, from the scale or the queries: unseen tokens stay unseen."""
    batch = Batch("tiny factor", [100, 40], 2, 64, 32, ref.KV_INT8, "bf16")
    tokens(batch, [70, 40], 8, scale=1e-42)
    tokens(batch, [70, 40], 8, scale=-1e-40, window=20, sinks=2)
    q = (randn(batch.g, 113, 8, 64, dtype=torch.bfloat16).float() * 2.0**-129).to(torch.bfloat16)
    assert bool((q != 0).any())
    tokens(batch, [70, 40], 8, q=q, scale=1e-4)



def test_tokens_int8_sums_over_2_28_tokens_of_tiny_values():
    """Values with scales far below the others' range, one page 2^20 times: the sum of the probabilities, which are
    relative to a low reference then, stays within fp32."""
    P, pages = 256, 1 << 20
    n = P * pages
    cache = torch.zeros(w4.kv_cache_size(1, 1, 64, P, ref.KV_INT8), dtype=torch.uint8, device=DEV)
    g = gen("tiny values")
    k = randn(g, P, 1, 64, dtype=torch.bfloat16).to(DEV)
    v = torch.full((P, 1, 64), 2.0**-103, dtype=torch.bfloat16, device=DEV)
    w4.kv_write(k, v, torch.arange(P, device=DEV), cache, 1, P, ref.KV_INT8)
    q = torch.zeros(2, 1, 64, dtype=torch.bfloat16, device=DEV)
    o = w4.attention_tokens(q, torch.tensor([0, 2], dtype=torch.int32, device=DEV), cache,
                            torch.zeros(1, pages, dtype=torch.int32, device=DEV), torch.tensor([n], dtype=torch.int32, device=DEV),
                            1, 1, P, ref.KV_INT8)
    # Scores of 0: every probability is 1 / n, and the mean of equal values is that value. A probability's operand is
    # rounded by 2^-11, a workgroup's fp32 sums of 2^28 / 32 / 512 = 2^14 tiles by 2^-23 each at most, the join's of 512
    # by less than 2^-13, the output by 2^-8.
    within(o.cpu(), torch.full(o.shape, 2.0**-103, dtype=torch.float64),
           2.0**-103 * (2.0**-8 + 2.0**-9 + 2.0**-11 + 2.0**-13 + 2.0**-23))
