"""GPU tests of sampling against the 64-bit definition (tests/step_reference.py).
Tokens have to be equal; the random numbers are seeded, and the reference says
how near they come to a border between two tokens."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import mixed_precision_w4a16_repack_amd as w4
from tests import step_reference as step
from tests.operator_reference import DTYPES
from tests.test_gpu_operators import BOTH, DEV, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    w4.load_library()
    yield
    torch.cuda.synchronize()


def check(x, u, dev=None, **settings):
    """x [M, V] act dtype, u [M]; settings: lists or tensors of M."""
    M = x.shape[0]
    kinds = dict(temperature=torch.float32, top_k=torch.int32, top_p=torch.float32, min_p=torch.float32)
    given = {k: torch.as_tensor(v, dtype=kinds[k]) for k, v in settings.items()}
    probs = torch.full((M,), 9.0, device=DEV)
    got = w4.sample(x.to(DEV) if dev is None else dev, u.to(DEV), probs=probs, **{k: v.to(DEV) for k, v in given.items()}).cpu()
    probs = probs.cpu()
    for r in range(M):
        one = {k: v[r].item() for k, v in given.items()}
        token, p, border = step.sample(x[r], u[r].item(), **one)
        # sums of fp64 roundings are 2^-40 off at most
        assert got[r].item() == token or border < 2.0**-38, f"row {r}: {got[r].item()} for {token} ({one}, u = {u[r].item()})"
        if got[r].item() == token:
            assert abs(probs[r].item() - p) <= 2.0**-23 * p, f"row {r}: probability {probs[r].item()} for {p}"
    return got


def rows(g, M, V, dtype, std=2.0):
    x = torch.randn(M, V, generator=g) * std + 6 * torch.relu(torch.randn(M, V, generator=g) - 2.5)
    return x.to(DTYPES[dtype])


SIZES = [(3, 1), (4, 2), (5, 7), (4, 8), (3, 63), (2, 511), (2, 513), (6, 1000), (4, 8192), (3, 8193), (3, 32003), (2, 128000),
         (1, 262147)]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("M,V", SIZES)
def test_sample_all(M, V, dtype):
    g = gen("sample", M, V, dtype)
    check(rows(g, M, V, dtype), torch.rand(M, generator=g))


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("M,V", [(64, 7), (64, 1000), (40, 32003)])
def test_sample_settings(M, V, dtype):
    g = gen("settings", M, V, dtype)

    def pick(*of):
        return [of[i] for i in torch.randint(len(of), (M,), generator=g).tolist()]

    check(rows(g, M, V, dtype), torch.rand(M, generator=g), temperature=pick(0.0, 0.3, 0.7, 1.0, 1.7, 50.0),
          top_k=pick(0, -3, 1, 2, 5, 40, 1000, 2**31 - 1), top_p=pick(1.0, 0.95, 0.5, 0.1, 1e-7, 0.0, -1.0, 2.0),
          min_p=pick(0.0, -1.0, 0.01, 0.1, 0.5, 1.0, 3.0))


@pytest.mark.parametrize("name,values", [("top_k", [1, 2, 3, 10, 100, 999]), ("top_p", [0.01, 0.3, 0.9, 0.999, 0.99999]),
                                         ("min_p", [1e-6, 0.001, 0.2, 0.999]), ("temperature", [0.01, 0.5, 2.0, 1000.0])])
def test_sample_each_setting_alone(name, values):
    g = gen("alone", name)
    M = 8 * len(values)
    check(rows(g, M, 1000, "bf16"), torch.rand(M, generator=g), **{name: values * 8})


def test_sample_bounds_of_the_uniform_numbers():
    g = gen("bounds")
    x = rows(g, 1, 5000, "f16").repeat(7, 1)
    u = torch.tensor([0.0, -1.0, float("nan"), 1 - 2.0**-24, 1.0, 5.0, float("inf")])
    got = check(x, torch.nan_to_num(u, nan=0.0).clamp(-1, 1), top_k=[50] * 7)
    dev = w4.sample(x.to(DEV), u.to(DEV), top_k=torch.full((7,), 50, dtype=torch.int32, device=DEV)).cpu()
    assert torch.equal(dev, got)
    order = torch.sort(x[0].float(), descending=True, stable=True)[1]
    assert got[0] == got[1] == got[2] == order[0] and got[3] == got[4] == got[5] == got[6] == order[49]


def test_sample_ties_go_to_the_lowest_index():
    V = 3000
    x = torch.zeros(6, V, dtype=torch.bfloat16)
    x[1, 100:] = -1
    x[2] = -0.0
    x[2, ::2] = 0.0  # zeros of both signs are equal
    x[3, 7::9] = 4
    u = torch.tensor([0.5, 0.99, 0.25, 0.001, 0.7, 0.2])
    check(x, u)
    check(x, u, top_k=[10] * 6)
    check(x, u, top_p=[0.5] * 6)
    got = check(x, u, temperature=[0.0] * 6)
    assert got.tolist() == [0, 0, 0, 7, 0, 0]


@pytest.mark.parametrize("V", [70000, 200000])
@pytest.mark.parametrize("value", [0.0, -3.0, -1e4])
def test_sample_values_more_frequent_than_a_count_holds(V, value):
    """One value 65536 times and more, alone, below a few others, and two such values."""
    g = gen("frequent", V, value)
    x = torch.full((4, V), value, dtype=torch.bfloat16)
    x[1, 5::1000] = 2.0
    x[2, : V // 2] = value - 1
    x[3, torch.randperm(V, generator=g)[: V // 3]] = value + 0.25
    for u in (0.0, 0.4, 0.75, 0.9999):
        check(x, torch.full((4,), u))
        check(x, torch.full((4,), u), top_k=[V - 3, 66000, 69999, 40000], top_p=[0.9, 1.0, 0.99, 0.5])


@pytest.mark.parametrize("dtype", BOTH)
def test_sample_forbidden_tokens(dtype):
    g = gen("forbidden", dtype)
    M, V = 8, 4099
    x = rows(g, M, V, dtype)
    x[0] = -float("inf")
    x[1, 1:] = -float("inf")
    x[2, torch.rand(V, generator=g) < 0.99] = -float("inf")
    x[3, ::3] = float("nan")
    x[4] = float("nan")
    x[5, [17, 40, 4000]] = float("inf")
    x[6] = torch.finfo(DTYPES[dtype]).min
    x[7, :4000] = torch.finfo(DTYPES[dtype]).min
    u = torch.rand(M, generator=g)
    got = check(x, u)
    assert got[0] == -1 and got[1] == 0 and got[4] == -1 and got[5].item() in (17, 40, 4000)
    for kw in (dict(temperature=[0.0] * M), dict(top_k=[5] * M), dict(top_p=[0.8] * M), dict(min_p=[0.3] * M),
               dict(temperature=[float("inf")] * M), dict(temperature=[1e-44] * M)):
        got = check(x, u, **kw)
        assert got[0] == -1 and got[4] == -1
    check(x, u, temperature=[float("nan")] * M)


def test_sample_strided_rows_and_outputs():
    g = gen("strided")
    wide = rows(g, 9, 3010, "f16").to(DEV)
    x = wide[:, 3:3002]  # odd addresses
    u = torch.rand(9, generator=g)
    check(x.cpu(), u, dev=x, top_p=[0.9] * 9)
    out = torch.full((9,), 5, device=DEV)
    assert w4.sample(x, u.to(DEV), out=out) is out
    assert torch.equal(out, w4.sample(x.contiguous(), u.to(DEV)))
    assert w4.sample(x[:0], u[:0].to(DEV)).shape == (0,)


def test_sample_follows_the_distribution():
    """Evenly spread numbers draw each token as often as its probability says, to one draw."""
    g = gen("spread")
    n = 4096
    x = rows(g, 1, 40, "bf16")
    u = (torch.arange(n) + 0.5) / n
    got = w4.sample(x.expand(n, 40).contiguous().to(DEV), u.to(DEV), temperature=torch.full((n,), 0.8, device=DEV)).cpu()
    p = torch.softmax(x[0].double() / 0.8, 0)
    assert bool(((torch.bincount(got, minlength=40).double() - n * p).abs() <= 1.0 + 1e-6).all())


def test_sample_repeats_in_a_graph_and_on_another_stream():
    g = gen("graph sample")
    M, V = 12, 32003
    x, u = rows(g, M, V, "bf16").to(DEV), torch.rand(M, generator=g).to(DEV)
    kw = dict(top_p=torch.full((M,), 0.9, device=DEV), top_k=torch.full((M,), 200, dtype=torch.int32, device=DEV))
    first = w4.sample(x, u, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = w4.sample(x, u, **kw)
    torch.cuda.current_stream().wait_stream(side)
    there.record_stream(torch.cuda.current_stream())
    assert torch.equal(first, there)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = w4.sample(x, u, **kw)
    for _ in range(4):
        u.copy_(torch.rand(M, generator=g).to(DEV))
        x.copy_(rows(g, M, V, "bf16").to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, w4.sample(x, u, **kw))
    assert np.unique(got.cpu().numpy()).size > 1


@pytest.mark.parametrize("dtype", BOTH)
def test_both_zeros_are_one_value_however_many_they_are(dtype):
    """More than 2^15 of each sign, and of one of them."""
    V = 150000
    g = gen("zeros")
    sign = torch.rand(3, V, generator=g)
    x = torch.zeros(3, V)
    x[0] = torch.where(sign[0] < 0.5, -0.0, 0.0)
    x[1] = torch.where(sign[1] < 0.4, -0.0, torch.where(sign[1] < 0.8, 0.0, 1.0))
    x[2, ::3] = -0.0
    x[2, 7] = 3.0
    check(x.to(DTYPES[dtype]), torch.tensor([0.61, 0.1, 0.83]))
    check(x.to(DTYPES[dtype]), torch.tensor([0.3, 0.97, 0.5]), top_k=[40000, 100000, 70000], top_p=[0.9, 0.5, 1.0])


@pytest.mark.parametrize("V", [70000, 200000])
@pytest.mark.parametrize("dtype", BOTH)
def test_sample_nans_of_any_pattern_that_are_most_of_a_row(V, dtype):
    """A NaN pattern of either sign, beside the infinities' in the order and far from them, more than 2^15 times: never
    drawn, counted nowhere, alone, under one finite logit, among others and beside an infinite one."""
    inf = 0x7C00 if dtype == "f16" else 0x7F80
    g = gen("nan", V, dtype)
    for payload in (1, 2, 62, 63, 64, 0x7FFF - inf):
        for sign in (0, 0x8000):
            bits = torch.full((5, V), (sign | inf | payload) - (0x10000 if sign else 0), dtype=torch.int16)
            x = bits.view(DTYPES[dtype])
            assert bool(x.isnan().all())
            x[1, 12345] = 1.0
            x[2, ::7] = rows(g, 1, len(range(0, V, 7)), dtype)[0]
            x[3, V - 1] = float("inf")
            x[3, 5] = 2.0
            x[4, ::2] = -3.0
            u = torch.rand(5, generator=g)
            for kw in ({}, dict(top_k=[40] * 5, top_p=[0.9] * 5, min_p=[0.05] * 5), dict(temperature=[0.0] * 5)):
                got = check(x, u, **kw)
                assert got[0] == -1 and got[1] == 12345 and got[3] == V - 1
