"""GPU tests of the operators between a layer's GEMMs at the ends of their
ranges: gates past exp's range, rows whose products leave fp32's, wide rows
in place, workspaces under capture. References in 64 bits
(tests/operator_reference.py); tolerances count the roundings made."""

from __future__ import annotations

import math

import pytest
import torch

import mixed_precision_w4a16_repack_amd as w4
from tests import operator_reference as ref
from tests.operator_reference import DTYPES, HALF, TINY
from tests.test_gpu_operators import BOTH, DEV, REL, Batch, check_codes, gen, randn, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    w4.load_library()
    yield
    torch.cuda.synchronize()


def finite_values(dtype):
    """Every finite value of a 16-bit type."""
    v = torch.arange(-(2**15), 2**15, dtype=torch.int32).to(torch.int16).view(DTYPES[dtype])
    return v[v.isfinite()]


# ---------------------------------------------------------------- norm


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("K", [64, 1000, 4096, 40000])
def test_rmsnorm_a8_row_of_zeros_without_eps(K, dtype):
    """eps = 0: a row of zeros (given so, or where the residual cancels x) has scale 0 and codes 0."""
    g = gen("norm a8 zeros", K, dtype)
    dt = DTYPES[dtype]
    x, w, r = randn(g, 4, K, dtype=dt, std=3.0), randn(g, K, dtype=dt), randn(g, 4, K, dtype=dt)
    x[1], r[1] = 0, 0
    r[2] = -x[2]
    qa, xs = w4.rmsnorm_a8(x.to(DEV), w.to(DEV), eps=0.0, residual=r.to(DEV))
    assert xs[1:3].tolist() == [0.0, 0.0] and not bool(qa[1:3].any())
    keep = [0, 3]
    check_codes(qa.cpu()[keep], xs.cpu()[keep], ref.norm(x[keep], w, 0.0, r[keep])[0], REL)


@pytest.mark.parametrize("K", [64, 4099])
def test_rmsnorm_of_small_rows_without_eps(K):
    """Down to a mean square of 2^-100: squares of elements that leave fp32's range do not count there."""
    g = gen("norm small", K)
    x, w = randn(g, 3, K, dtype=torch.bfloat16, std=2e-15), randn(g, K, dtype=torch.bfloat16)
    want, _ = ref.norm(x, w, 0.0)
    assert (x.double() ** 2).mean(1).min().item() > 2.0**-100
    y = w4.rmsnorm(x.to(DEV), w.to(DEV), eps=0.0)
    within(y.cpu(), want, want.abs() * (HALF["bf16"] + REL) + TINY["bf16"], "y")


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("K", [32769, 33000, 40001, 70000])
def test_rmsnorm_of_wide_rows_in_place(K, dtype):
    """Rows that are read twice (above 32768 columns), with an output over an input: bit for bit as beside it."""
    g = gen("norm wide in place", K, dtype)
    dt = DTYPES[dtype]
    x, w, r = (randn(g, *s, dtype=dt).to(DEV) for s in ((3, K), (K,), (3, K)))
    h = torch.empty_like(x)
    y = w4.rmsnorm(x, w, residual=r, residual_out=h)
    want, want_h = ref.norm(x.cpu(), w.cpu(), 1e-5, r.cpu())
    within(y.cpu(), want, want.abs() * (HALF[dtype] + REL) + TINY[dtype], "y")
    within(h.cpu(), want_h, want_h.abs() * (HALF[dtype] + 2.0**-23) + TINY[dtype], "residual_out")
    r2 = r.clone()
    assert torch.equal(w4.rmsnorm(x, w, residual=r2, residual_out=r2), y) and torch.equal(r2, h)
    x2 = x.clone()
    assert torch.equal(w4.rmsnorm(x2, w, residual=r, residual_out=x2), y) and torch.equal(x2, h)
    x2 = x.clone()
    assert torch.equal(w4.rmsnorm(x2, w, residual=r, out=x2), y) and torch.equal(x2, y)
    if K % 8 == 0:
        qa, xs = w4.rmsnorm_a8(x, w, residual=r)
        r2 = r.clone()
        qb, ys = w4.rmsnorm_a8(x, w, residual=r2, residual_out=r2)
        assert torch.equal(qa, qb) and torch.equal(xs, ys) and torch.equal(r2, h)


# ---------------------------------------------------------------- gate


@pytest.mark.parametrize("dtype", BOTH)
def test_silu_mul_a8_of_gates_past_exps_range(dtype):
    """Every finite gate of -80 and below, the type's lowest among them: exp(-g) passes fp32's range at -88.7,
    where silu is 0. Each row holds ordinary gates too, whose codes have to be right beside them."""
    low = finite_values(dtype)
    low = low[low <= -80]
    low = torch.cat([low, torch.tensor([-88.75, -95.0, -110.0, -500.0, -60000.0]).to(DTYPES[dtype])])
    n = 64
    rows = low[: low.numel() // n * n].view(-1, n)
    rows = torch.cat([rows, low[-n:][None]])
    g = gen("gate a8 low", dtype)
    gate = torch.stack([rows, randn(g, *rows.shape, dtype=DTYPES[dtype], std=3.0)], -1).flatten(1)
    x = torch.cat([gate, randn(g, *gate.shape, dtype=DTYPES[dtype])], 1)
    qa, xs = w4.silu_mul_a8(x.to(DEV))
    assert bool(xs.isfinite().all()), f"{int((~xs.isfinite()).sum())} of {len(xs)} rows have no finite scale"
    check_codes(qa.cpu(), xs.cpu(), ref.silu_mul(x), 2.0**-17)


@pytest.mark.parametrize("dtype", BOTH)
def test_silu_mul_a8_of_only_low_gates_is_a_row_of_zeros(dtype):
    x = torch.ones(3, 128, dtype=DTYPES[dtype])
    x[:, :64] = torch.tensor([-100.0, -110.0, torch.finfo(DTYPES[dtype]).min]).to(DTYPES[dtype])[:, None]
    qa, xs = w4.silu_mul_a8(x.to(DEV))
    assert not bool(xs.any()) and not bool(qa.any())


@pytest.mark.parametrize("dtype", BOTH)
def test_silu_mul_a8_of_large_positive_gates(dtype):
    """Gates up to the type's largest, where the argument of exp passes fp32's range: silu(g) is g itself."""
    high = finite_values(dtype)
    high = high[high >= 1000]
    x = torch.zeros(high.numel(), 32, dtype=DTYPES[dtype])
    x[:, :16] = high[:, None]
    x[:, 16:] = torch.linspace(-1, 1, 16).to(DTYPES[dtype])
    qa, xs = w4.silu_mul_a8(x.to(DEV))
    check_codes(qa.cpu(), xs.cpu(), ref.silu_mul(x), 2.0**-20)


@pytest.mark.parametrize("dtype", BOTH)
def test_silu_mul_a8_of_an_infinite_gate(dtype):
    """An infinite gate gives an infinite scale, as an infinite value does, and leaves the other rows alone."""
    x = torch.ones(3, 128, dtype=DTYPES[dtype])
    x[1, 7] = float("inf")
    _, xs = w4.silu_mul_a8(x.to(DEV))
    assert xs[1].item() == float("inf") and bool(xs[[0, 2]].isfinite().all())


# ---------------------------------------------------------------- attention: the probabilities' bits


def two_part_tolerance(out, A, S, dtype, n):
    """ref.attention_tolerance with the probability in two parts: they leave a half step of a half step (fp16,
    cut instead of rounded: a step of a step)."""
    delta = 2 * 64 * 2.0**-24 * S[:, None]
    part = (HALF[dtype] if dtype == "bf16" else 2 * HALF[dtype]) ** 2
    return A * (part + delta + 2.0**-17) + HALF[dtype] * out.abs() + n * 2.0**-36 * A.amax() + TINY[dtype]


@pytest.mark.parametrize("dtype", BOTH)
def test_attention_equal_probabilities_between_two_steps(dtype):
    """All but the first tokens have one probability, almost half a step above a 16-bit number relative to the
    first ones': rounded alone it would move every result the same way, by as much as the result's own rounding."""
    H, D, P, n = 1, 64, 32, 512
    batch = Batch("between", [n], H, D, P, ref.KV_ACT, dtype)
    k = torch.zeros(n, H, D, dtype=batch.dt)
    k[128:, 0, 0] = 1.0
    v = (torch.rand(n, H, D, generator=batch.g) + 1.0).to(batch.dt)
    t = torch.arange(n)
    slots = batch.table[0].long()[t // P] * P + t % P
    w4.kv_write(k.to(DEV), v.to(DEV), slots.to(DEV), batch.cache, batch.pages, P, ref.KV_ACT)
    q = torch.zeros(1, 3, D, dtype=batch.dt)
    q[:, :, 0] = 1.0
    scale = math.log(2 * (1 + 0.95 * HALF[dtype]))
    o = w4.attention(q.to(DEV), batch.cache, batch.dev_table, batch.lengths, batch.pages, H, P, ref.KV_ACT, scale=scale)
    want, A, S = ref.attention(q[0], k, v, torch.ones(n, dtype=torch.bool), scale)
    within(o[0].cpu(), want, two_part_tolerance(want, A, S, dtype, n))


@pytest.mark.parametrize("dtype,kind", [("f16", ref.KV_ACT), ("bf16", ref.KV_ACT), ("f16", ref.KV_INT8)])
@pytest.mark.parametrize("Hq,H,D,P,lens,window", [
    (32, 8, 128, 64, [0, 1, 33, 333, 2000], 0), (16, 16, 64, 32, [700, 5000], 300), (34, 2, 256, 32, [1000, 77], 0),
    (40, 8, 192, 64, [129, 2500], 0), (32, 1, 128, 32, [9000], 0),
])
def test_attention_probabilities_in_two_parts(Hq, H, D, P, lens, window, dtype, kind):
    batch = Batch("two parts", lens, H, D, P, kind, dtype)
    q = randn(batch.g, len(lens), Hq, D, dtype=batch.dt)
    o = w4.attention(q.to(DEV), batch.cache, batch.dev_table, batch.lengths, batch.pages, H, P, kind,
                     window=window).cpu()
    for b, n in enumerate(lens):
        want, A, S = ref.attention(q[b], batch.k[b], batch.v[b], batch.seen(b, window), D**-0.5)
        within(o[b], want, two_part_tolerance(want, A, S, dtype, n), f"sequence {b} ({n} tokens)")


# ---------------------------------------------------------------- workspaces and graphs


def split_attention(n, kind, seed):
    """An attention call on one long sequence, whose heads many workgroups share: (call, eager result)."""
    H, D, P, Hq = 1, 64, 32, 8
    g = gen("split attention", n, kind, seed)
    pages = -(-n // P)
    cache = torch.zeros(w4.kv_cache_size(pages, H, D, P, kind), dtype=torch.uint8, device=DEV)
    k, v = (randn(g, n, H, D, dtype=torch.float16).to(DEV) for _ in range(2))
    w4.kv_write(k, v, torch.arange(n, device=DEV), cache, pages, P, kind)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    lengths = torch.tensor([n], dtype=torch.int32, device=DEV)
    q = randn(g, 1, Hq, D, dtype=torch.float16).to(DEV)

    def call(**kw):
        return w4.attention(q, cache, table, lengths, pages, H, P, kind, **kw)

    return call, call()


@pytest.mark.parametrize("kind", [w4.KV_ACT, w4.KV_INT8])
def test_graphs_captured_without_a_workspace_replay_in_any_order(kind):
    calls = [split_attention(n, kind, i) for i, n in enumerate((20000, 15000))]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for call, _ in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call())
        graphs.append(graph)
    for i in (1, 0, 1, 1, 0):
        outs[i].fill_(7.0)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], calls[i][1]), f"graph {i}"
        for call, want in calls:
            assert torch.equal(call(), want)


def test_products_captured_without_a_workspace_replay_in_any_order():
    """Split-K products: their arrival counters live in the workspace too."""
    import w4a16_inputs as wi
    from tests.gpu_cases import repack

    graphs, outs, wants = [], [], []
    for seed, (M, N, K, G) in enumerate([(16, 4096, 14336, 128), (5, 1024, 4096, 64)]):
        assert w4.workspace_size(M, N, K, G) > 0
        case = wi.make_case(70 + seed, M, N, K, G, wi.UINT4B8, "f16")
        packed, A = repack(case), case.A.to(DEV)
        wants.append(w4.gemm(A, packed, N, K, G, wi.UINT4B8))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(w4.gemm(A, packed, N, K, G, wi.UINT4B8))
        graphs.append((graph, packed, A))
    for i in (1, 0, 1, 0):
        outs[i].fill_(7.0)
        graphs[i][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], wants[i]), f"graph {i}"


def test_a_larger_eager_call_between_replays_leaves_the_graph_its_workspace():
    small, want = split_attention(600, w4.KV_ACT, 0)
    large, want_large = split_attention(30000, w4.KV_ACT, 1)
    ws = w4.Workspace(DEV)
    assert torch.equal(small(workspace=ws), want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = small(workspace=ws)
    before = ws.buf.numel()
    for rep in range(4):
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {rep}"
        assert torch.equal(large(workspace=ws), want_large)
        assert ws.buf.numel() > before
        # memory that the allocator hands out now is not the graph's
        other = [torch.full((before,), 0x5A, dtype=torch.uint8, device=DEV) for _ in range(4)]
        graph.replay()
        torch.cuda.synchronize()
        assert all(bool((t == 0x5A).all()) for t in other)
        assert torch.equal(out, want)


def test_a_workspace_first_used_in_a_capture_serves_eager_calls_before_the_replay():
    call, want = split_attention(9000, w4.KV_INT8, 0)
    ws = w4.Workspace(DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(workspace=ws)
    for rep in range(3):
        assert torch.equal(call(workspace=ws), want)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {rep}"
