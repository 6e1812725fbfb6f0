"""GPU tests of the operators for steps of several tokens as they are used
together: prompts in parts, drafted trees against their paths, a chain from a
norm to a sampled token, captured and eager."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import mixed_precision_w4a16_repack_amd as w4
from examples.decode_layer import EPS, GROUP, random_weight
from tests import operator_reference as ref
from tests import step_reference as step
from tests.test_gpu_operators import DEV, KINDS, gen, randn, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    w4.load_library()
    yield
    torch.cuda.synchronize()


# Two calls' errors; and 1 %, as an int8 cache's keys and values are known here as
# they are read, rounded by 2^-8 at most, which moves the bound itself by no more than that.
BOTH_CALLS = 2.02


def int32(values):
    return torch.as_tensor(values, dtype=torch.int32, device=DEV)


def rates(n):
    return (10000.0 ** (-torch.arange(n, dtype=torch.float32) / n)).to(DEV)


class Cache:
    """A cache with one sequence a row of its table, pages in shuffled order."""

    def __init__(self, B, width, H, D, P, kind):
        self.H, self.D, self.P, self.kind, self.pages = H, D, P, kind, B * width + 2
        self.data = torch.zeros(w4.kv_cache_size(self.pages, H, D, P, kind), dtype=torch.uint8, device=DEV)
        self.table = torch.randperm(self.pages, generator=gen("cache"))[: B * width].view(B, width).to(torch.int32)
        self.dev_table = self.table.to(DEV)

    def slots(self, b, t):
        t = torch.as_tensor(t)
        return (self.table[b].long()[t // self.P] * self.P + t % self.P).to(DEV)

    def append(self, b, t, positions, q, k, v, rate):
        return w4.kv_append(q, k, v, int32(positions), rate, self.slots(b, t), self.data, self.pages, self.P, self.kind)

    def read(self, b, n, dtype):
        return w4.kv_read(self.slots(b, torch.arange(n)), self.data, self.pages, self.H, self.D, self.P, self.kind, dtype)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("parts", [[700], [1, 699], [300, 33, 1, 366], [64] * 10 + [60]])
def test_a_prompt_in_parts_is_the_whole_prompt(parts, kind):
    """Cache and queries bit by bit, the attention within both calls' roundings; parts of one token by both calls."""
    n, Hq, H, D, dt = 700, 8, 2, 128, torch.bfloat16
    g = gen("prompt in parts")
    q, k, v = (randn(g, n, heads, D, dtype=dt).to(DEV) for heads in (Hq, H, H))
    whole, pieces = Cache(1, 11, H, D, 64, kind), Cache(1, 11, H, D, 64, kind)
    rate = rates(D // 2)
    turned = whole.append(0, torch.arange(n), torch.arange(n), q, k, v, rate)
    want = w4.attention_tokens(turned, int32([0, n]), whole.data, whole.dev_table, int32([n]), whole.pages, H, 64, kind)
    rk, rv = (x.cpu() for x in whole.read(0, n, dt))
    at = 0
    for m in parts:
        rows = slice(at, at + m)
        t = torch.arange(at, at + m)
        tq = pieces.append(0, t, t, q[rows], k[rows], v[rows], rate)
        assert torch.equal(tq, turned[rows])
        args = (pieces.data, pieces.dev_table, int32([at + m]), pieces.pages, H, 64, kind)
        got = w4.attention_tokens(tq, int32([0, m]), *args).cpu()
        for i in sorted({0, m // 2, m - 1}):
            o, A, S = ref.attention(tq[i].cpu(), rk, rv, torch.arange(n) <= at + i, D**-0.5)
            tolerance = BOTH_CALLS * ref.attention_tolerance(o, A, S, "bf16", kind, n)
            within(got[i], want[at + i].cpu().double(), tolerance, f"token {at + i}")
            if m == 1:
                within(w4.attention(tq, *args).cpu()[0], want[at].cpu().double(), tolerance, f"step at {at}")
        at += m
    assert torch.equal(pieces.data, whole.data)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("past,m,window,sinks", [(0, 20, 0, 0), (77, 64, 0, 0), (500, 90, 0, 0), (500, 40, 200, 4)])
def test_a_drafted_token_sees_what_its_path_sees(past, m, window, sinks, kind):
    """A node of a tree against a sequence that holds only the node's path, whose last token it is."""
    Hq, H, D, dt = 8, 2, 64, torch.float16
    g, r = gen("paths"), np.random.default_rng(past + m)
    words = step.random_tree(r, m, 2)
    sees, depth = step.bits(words, m)
    n = past + m
    q, k, v = (randn(g, n, heads, D, dtype=dt).to(DEV) for heads in (Hq, H, H))
    positions = torch.cat([torch.arange(past), past + depth - 1])
    cache, rate = Cache(2, -(-n // 32), H, D, 32, kind), rates(D // 2)
    tq = cache.append(0, torch.arange(n), positions, q, k, v, rate)
    got = w4.attention_tokens(tq[past:], int32([0, m]), cache.data, cache.dev_table[:1], int32([n]), cache.pages, H, 32, kind,
                              tree=words.to(DEV), window=window, sinks=sinks).cpu()
    for i in sorted({0, 1, m // 2, m - 1}):
        rows = torch.cat([torch.arange(past), past + torch.nonzero(sees[i])[:, 0]])
        assert len(rows) == past + int(depth[i])
        one = cache.append(1, torch.arange(len(rows)), positions[rows], q[rows.to(DEV)], k[rows.to(DEV)], v[rows.to(DEV)], rate)
        assert torch.equal(one[-1], tq[past + i])
        want = w4.attention(one[-1:], cache.data, cache.dev_table[1:], int32([len(rows)]), cache.pages, H, 32, kind,
                            window=window, sinks=sinks).cpu()[0]
        rk, rv = (x.cpu() for x in cache.read(1, len(rows), dt))
        t, at = torch.arange(len(rows)), len(rows) - 1
        o, A, S = ref.attention(one[-1].cpu(), rk, rv, (t > at - window) | (t < sinks) if window else t >= 0, D**-0.5)
        within(got[i], want.double(), BOTH_CALLS * ref.attention_tolerance(o, A, S, "f16", kind, len(rows)), f"node {i}")


class Chain:
    """A norm, products, rotation with the cache write, attention of drafted trees, logits and a token for each row."""

    hidden, Hq, H, D, V, P = 512, 8, 2, 64, 1600, 32

    def __init__(self, past, drafts, kind, seed):
        g = torch.Generator()
        g.manual_seed(seed)
        dt = torch.bfloat16
        self.shapes = {"qkv": ((self.Hq + 2 * self.H) * self.D, self.hidden), "out": (self.hidden, self.Hq * self.D), "logits": (self.V, self.hidden)}
        self.packed = {name: random_weight(g, N, K, dt, DEV) for name, (N, K) in self.shapes.items()}
        self.norm = (1 + 0.1 * torch.randn(self.hidden, generator=g)).to(dt).to(DEV)
        self.rates = rates(self.D // 2)
        B, T = len(past), sum(drafts)
        self.cache = Cache(B, max(-(-(p + 3 * m) // self.P) for p, m in zip(past, drafts)), self.H, self.D, self.P, kind)
        for b, p in enumerate(past):
            if p:
                k, v = (torch.randn(p, self.H, self.D, generator=g).to(dt).to(DEV) for _ in range(2))
                self.cache.append(b, torch.arange(p), torch.arange(p), None, k, v, self.rates)
        r = np.random.default_rng(seed)
        trees = [step.random_tree(r, m, 1) for m in drafts]
        depth = [step.bits(x, m)[1] for x, m in zip(trees, drafts)]
        self.tree = torch.cat(trees).to(DEV)
        self.starts = int32(np.concatenate([[0], np.cumsum(drafts)]))
        self.news = int32(drafts)
        self.lengths = int32([p + m for p, m in zip(past, drafts)])
        self.positions = int32(torch.cat([p + d - 1 for p, d in zip(past, depth)]))
        row = torch.repeat_interleave(torch.arange(B), torch.tensor(drafts))
        self.row = row.to(DEV)
        self.at = int32(torch.cat([p + torch.arange(m) for p, m in zip(past, drafts)]))
        self.x = torch.randn(T, self.hidden, generator=g).to(dt).to(DEV)
        self.u = torch.rand(T, generator=g).to(DEV)
        self.top_p = torch.full((T,), 0.9, device=DEV)
        self.ws = {}

    def product(self, x, name):
        N, K = self.shapes[name]
        return w4.gemm(x, self.packed[name], N, K, GROUP, w4.UINT4B8, workspace=self.ws.get("gemm"))

    def step(self):
        """One step of all drafted tokens; the next one follows it in the cache."""
        T, c = self.x.shape[0], self.cache
        page = c.dev_table[self.row, (self.at // self.P).long()].long()
        slots = page * self.P + self.at % self.P
        qkv = self.product(w4.rmsnorm(self.x, self.norm, EPS), "qkv").view(T, -1, self.D)
        q, k, v = qkv.split([self.Hq, self.H, self.H], 1)
        q = w4.kv_append(q, k, v, self.positions, self.rates, slots, c.data, c.pages, self.P, c.kind)
        o = w4.attention_tokens(q, self.starts, c.data, c.dev_table, self.lengths, c.pages, self.H, self.P, c.kind, tree=self.tree,
                                workspace=self.ws.get("attention"))
        logits = self.product(self.product(o.view(T, -1), "out"), "logits")
        token = w4.sample(logits, self.u, top_p=self.top_p)
        self.at.add_(self.news[self.row])
        self.positions.add_(self.news[self.row])
        self.lengths.add_(self.news)
        return token, o, logits, q

    def feed(self, token):
        """Inputs of the next step that depend on this one's tokens."""
        self.x.copy_(torch.roll(self.x, 1, 0) + (token % 7)[:, None].to(self.x.dtype) * 0.125)
        self.u.copy_((self.u + 0.37) % 1.0)


PAST, DRAFTS = [130, 0, 33, 500], [16, 3, 1, 40]


@pytest.mark.parametrize("kind", KINDS)
def test_chain_against_its_definition(kind):
    """Attention and token of every drafted token from the chain's own queries, cache and logits."""
    chain = Chain(PAST, DRAFTS, kind, 1)
    u = chain.u.cpu()
    lengths, starts, tree = chain.lengths.tolist(), chain.starts.tolist(), chain.tree.cpu()
    token, o, logits, q = (t.cpu() for t in chain.step())
    for b, (n, m) in enumerate(zip(lengths, DRAFTS)):
        k, v = (t.cpu() for t in chain.cache.read(b, n, torch.bfloat16))
        sees = step.rows_see(n, m, words=tree[starts[b] : starts[b + 1]])
        for i in range(m):
            row = starts[b] + i
            # int8: the reference's keys and values are rounded to 16 bits as they are
            # read, by 2^-8 of each at most: of a score's terms, and so twice that of a
            # probability relative to the others, and of the values.
            want, A, S = ref.attention(q[row], k, v, sees[i], chain.D**-0.5)
            tolerance = ref.attention_tolerance(want, A, S, "bf16", kind, n)
            if kind == ref.KV_INT8:
                tolerance = tolerance + 2.0**-8 * (A + 2 * S[:, None] * A)
            within(o[row], want, tolerance, f"sequence {b}, token {i}")
    for row in range(len(u)):
        want, p, border = step.sample(logits[row], u[row].item(), top_p=float(np.float32(0.9)))
        assert token[row].item() == want or border < 2.0**-38


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_captured_chains_equal_eager_ones(kind, own):
    """Two chains' graphs, replayed in turn with eager work between; own: workspaces that both share."""
    chains = [Chain(PAST, DRAFTS, kind, 2), Chain([64, 900], [32, 5], kind, 3)]
    twins = [Chain(PAST, DRAFTS, kind, 2), Chain([64, 900], [32, 5], kind, 3)]
    if own:
        shared = {"gemm": w4.Workspace(DEV), "attention": w4.Workspace(DEV)}
        for chain in chains:
            chain.ws = shared
    state = [[t.clone() for t in (c.cache.data, c.at, c.positions, c.lengths)] for c in chains]
    for chain, kept in zip(chains, state):  # sizes the workspaces; taken back
        chain.step()
        for t, was in zip((chain.cache.data, chain.at, chain.positions, chain.lengths), kept):
            t.copy_(was)
    torch.cuda.synchronize()
    graphs, results = [], []
    for chain in chains:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(chain.step())
        graphs.append(graph)
    for turn in range(3):
        for chain, twin, graph, result in zip(chains, twins, graphs, results):
            graph.replay()
            want = twin.step()
            torch.cuda.synchronize()
            for name, got, expect in zip(("token", "attention", "logits", "queries"), result, want):
                assert torch.equal(got, expect), f"{name} at replay {turn}"
            assert torch.equal(chain.cache.data, twin.cache.data) and torch.equal(chain.lengths, twin.lengths)
            for c in (chain, twin):
                c.feed(want[0])


def test_calls_with_another_current_device(monkeypatch):
    """With the wrong device current a call makes its tensors' device current; one card shows it by a wrong answer about it."""
    chain, twin = Chain(PAST, DRAFTS, ref.KV_INT8, 4), Chain(PAST, DRAFTS, ref.KV_INT8, 4)
    want = chain.step()
    monkeypatch.setattr(w4, "_current_device", lambda: 1)
    got = twin.step()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_two_streams_at_once():
    """The same calls on two streams: each stream has its own default workspaces."""
    chains = [Chain([3000, 900], [60, 40], ref.KV_ACT, 5) for _ in range(3)]
    want = chains[2].step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for chain, stream in zip(chains, streams):
        with torch.cuda.stream(stream):
            got.append(chain.step())
    torch.cuda.synchronize()
    for result in got:
        assert all(torch.equal(x, y) for x, y in zip(result, want))


@pytest.mark.parametrize("kind", KINDS)
def test_one_workspace_for_all_calls(kind):
    """Products and both attentions share one: none leaves the others' counters changed."""
    chain, twin = Chain([3000, 900], [60, 40], kind, 6), Chain([3000, 900], [60, 40], kind, 6)
    ws = w4.Workspace(DEV)
    chain.ws = {"gemm": ws, "attention": ws}
    for _ in range(3):
        want, got = twin.step(), chain.step()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        c = chain.cache
        q = want[3][:2].contiguous()
        one = [w4.attention(q, x.cache.data, x.cache.dev_table, x.lengths, c.pages, c.H, c.P, c.kind, workspace=w)
               for x, w in ((chain, ws), (twin, None))]
        assert torch.equal(*one)
        for x in (chain, twin):
            x.feed(want[0])
