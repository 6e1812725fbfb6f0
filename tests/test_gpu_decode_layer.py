"""GPU test of the decode-layer example: the operators chained as a user
chains them, against the same layer in plain fp32, and its captured graph
against eager steps."""

from __future__ import annotations

import pytest
import torch

import mixed_precision_w4a16_repack_amd as w4
from examples.decode_layer import Batch, DecodeLayer, capture

pytestmark = pytest.mark.gpu

SMALL = dict(hidden=512, heads=8, kv_heads=2, head_dim=64, inner=1024, page_size=32, pages=64)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    w4.load_library()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kind,window", [(w4.KV_ACT, 0), (w4.KV_INT8, 0), (w4.KV_INT8, 100)])
def test_step_against_plain_fp32(dtype, kind, window):
    layer = DecodeLayer(**SMALL, dtype=dtype, kv_kind=kind, window=window)
    batch = Batch(layer, [300, 1, 64, 31, 700], more=4)
    lengths, residual = batch.lengths + 1, batch.residual.clone()
    want, want_r = layer.plain_step(batch.x, batch.residual, batch.keys, batch.values, lengths)
    got = layer.step(batch.x, residual, batch.table, lengths)
    # Each rounding to 8 bits is off by a uniform share of max / 127: for about
    # normal rows (max of 4.5 deviations) 4.5 / 127 / sqrt(12) = 1.0 % of the
    # norm. Of them lie on the way: keys and values (a score's error of 1 % of
    # about 1 adds as much again), the norm's codes (both gate and up), the
    # product's codes (max nearer 10 deviations: 2.3 %). In squares: 0.010^2 * 2
    # + 2 * 0.010^2 + 0.023^2 = (3.0 %)^2; the 16-bit roundings add 2^-8 for each
    # of about six results. Twice that is allowed.
    assert ((got.float() - want).norm() / want.norm()).item() <= 2 * (0.030 + 6 * 2.0**-8)
    # The residual has the attention's output only, of much smaller norm.
    assert ((residual.float() - want_r).norm() / want_r.norm()).item() <= 2 * (0.014 + 3 * 2.0**-8)


@pytest.mark.parametrize("kind", [w4.KV_ACT, w4.KV_INT8])
def test_captured_steps_equal_eager_steps(kind):
    layer, twin = (DecodeLayer(**SMALL, kv_kind=kind) for _ in range(2))
    batch, eager = (Batch(x, [200, 5, 33], more=8) for x in (layer, twin))
    eager.table.copy_(batch.table)
    twin.cache.copy_(layer.cache)
    graph, y = capture(layer, batch)
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        eager.lengths.add_(1)
        want = twin.step(eager.x, eager.residual, eager.table, eager.lengths)
        assert torch.equal(got, want) and torch.equal(batch.residual, eager.residual)
        for b in (batch, eager):  # the next token's input
            b.x.copy_(want)
