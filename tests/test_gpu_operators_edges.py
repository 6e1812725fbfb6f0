"""GPU tests of the operators between a layer's GEMMs at the ends of their
ranges: gates past exp's range, rows whose products leave fp32's, wide rows
in place, workspaces under capture. References in 64 bits
(tests/operator_reference.py); tolerances count the roundings made."""

from __future__ import annotations

import pytest
import torch

import mixed_precision_w4a16_repack_amd as w4
from tests import operator_reference as ref
from tests.operator_reference import DTYPES
from tests.test_gpu_operators import BOTH, DEV, check_codes, gen, randn

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
