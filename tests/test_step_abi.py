"""Argument checks of the operators for steps of several tokens a sequence and
of sampling (CPU only): every refusal comes before any HIP call, with the
documented status and message; the binding's own checks; the reference itself."""

from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import mixed_precision_w4a16_repack_amd as w4
from tests import step_reference as step

OK, INVALID, UNSUPPORTED, SIZE = 0, -1, -2, -3
P = ctypes.c_void_p(4096)


def at(n):
    return ctypes.c_void_p(4096 + n)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(w4.LIB_PATH):
        from mixed_precision_w4a16_repack_amd import build

        build.build()
    return w4.load_library()


def _append(lib, **kw):
    a = dict(q=P, qts=6144, qhs=128, Hq=32, qo=P, ots=4096, ohs=128, k=P, kts=6144, khs=128, v=P, vts=6144, vhs=128,
             T=4, pos=P, rates=P, pairs=64, near=0, slots=P, cache=P, nbytes=1 << 40, pages=4, H=8, D=128, P=64, kind=0,
             dtype=0)
    a.update(kw)
    return lib.w4a16_kv_append(*a.values(), None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), INVALID, "T=-1"),
    (dict(T=1 << 31), UNSUPPORTED, "too large for one launch"),
    (dict(T=1 << 27, Hq=1 << 10), UNSUPPORTED, "too large for one launch"),
    (dict(Hq=-1), INVALID, "q_heads=-1"),
    (dict(Hq=(1 << 20) + 1), UNSUPPORTED, "at most 2^20"),
    (dict(pairs=0), UNSUPPORTED, "pairs=0"),
    (dict(pairs=-8), UNSUPPORTED, "pairs=-8"),
    (dict(pairs=12), UNSUPPORTED, "multiple of 8"),
    (dict(pairs=72), UNSUPPORTED, "at most head_dim / 2 = 64"),
    (dict(near=2), INVALID, "neighbours=2"),
    (dict(dtype=7), INVALID, "dtype=7"),
    (dict(kind=-1), INVALID, "kind=-1"),
    (dict(D=80), UNSUPPORTED, "head_dim=80"),
    (dict(P=48), UNSUPPORTED, "page_size=48"),
    (dict(kts=-1), INVALID, "k strides must be >= 0"),
    (dict(vhs=(1 << 40) + 1), UNSUPPORTED, "v strides must be at most 2^40"),
    (dict(qhs=-1), INVALID, "q strides must be >= 0"),
    (dict(ots=-1), INVALID, "q_out strides must be >= 0"),
    (dict(k=None), INVALID, "must not be NULL"),
    (dict(v=None), INVALID, "must not be NULL"),
    (dict(pos=None), INVALID, "must not be NULL"),
    (dict(rates=None), INVALID, "must not be NULL"),
    (dict(slots=None), INVALID, "must not be NULL"),
    (dict(q=None), INVALID, "q and q_out must not be NULL"),
    (dict(qo=None), INVALID, "q and q_out must not be NULL"),
    (dict(cache=None), INVALID, "cache must not be NULL"),
    (dict(k=at(1)), INVALID, "2-byte aligned"),
    (dict(qo=at(1)), INVALID, "2-byte aligned"),
    (dict(slots=at(4)), INVALID, "8-byte aligned"),
    (dict(pos=at(2)), INVALID, "4-byte aligned"),
    (dict(rates=at(2)), INVALID, "4-byte aligned"),
    (dict(cache=at(8)), INVALID, "16-byte aligned"),
    (dict(nbytes=4 * 8 * 4 * 64 * 128 - 1), SIZE, "smaller than the 1048576 bytes"),
])
def test_append_rejects(lib, kw, status, needle):
    assert _append(lib, **kw) == status
    assert needle in w4.last_error()


def test_append_of_no_tokens_is_a_noop(lib):
    assert _append(lib, T=0, q=None, qo=None, k=None, v=None, pos=None, rates=None, slots=None, cache=None) == OK
    assert w4.last_error() == ""


def _sinks(lib, **kw):
    a = dict(q=P, qbs=4096, qhs=128, B=2, Hq=32, cache=P, nbytes=1 << 40, pages=4, H=8, D=128, P=64, kind=0, dtype=0,
             table=P, width=2, ld=2, lengths=P, window=8, sinks=4, scale=0.1, out=P, obs=4096, ohs=128, ws=None, wsb=0)
    a.update(kw)
    return lib.w4a16_attention_sinks(*a.values(), None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(sinks=-1), INVALID, "sinks=-1 must be >= 0"),
    (dict(window=-1), INVALID, "window=-1"),
    (dict(Hq=30), INVALID, "q_heads=30"),
    (dict(lengths=None), INVALID, "must not be NULL"),
    (dict(nbytes=100), SIZE, "cache_bytes=100"),
    (dict(), SIZE, "workspace of 0 bytes"),
    (dict(ws=at(16), wsb=1 << 30), INVALID, "256-byte aligned"),
])
def test_sinks_rejects(lib, kw, status, needle):
    assert _sinks(lib, **kw) == status
    assert needle in w4.last_error()


def test_sinks_workspace_size(lib):
    out = ctypes.c_size_t(0)
    assert lib.w4a16_attention_sinks_workspace_size(1, 32, 8, 128, 64, 4, 0, 0, 0, None) == INVALID
    assert lib.w4a16_attention_sinks_workspace_size(1, 32, 8, 128, 64, 4, 5, -1, 0, ctypes.byref(out)) == INVALID
    for window in (0, 100, 5000):
        assert w4.attention_workspace_size(1, 32, 8, 128, 64, 1 << 10, window, 0) == \
            w4.attention_workspace_size(1, 32, 8, 128, 64, 1 << 10, window, 0, 0)
    # first tokens count with a window only, and no more than the whole table
    assert w4.attention_workspace_size(1, 32, 8, 128, 64, 64, 0, 0, 1 << 40) == w4.attention_workspace_size(1, 32, 8, 128, 64, 64, 0, 0)
    assert w4.attention_workspace_size(1, 32, 8, 128, 64, 64, 10, 0, 1 << 40) <= w4.attention_workspace_size(1, 32, 8, 128, 64, 64, 0, 0)
    assert w4.attention_workspace_size(1, 32, 8, 128, 64, 1 << 20, 100, 0, 3000) > w4.attention_workspace_size(1, 32, 8, 128, 64, 1 << 20, 100, 0)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("B,width", [(1, 64), (1, 1 << 20), (9, 3)])
def test_sinks_workspace_of_windows_near_2_63(lib, B, width, kind):
    """Their sum with the first tokens leaves 64 bits: as without a window."""
    every = w4.attention_workspace_size(B, 32, 8, 128, 64, width, 0, kind)
    most = (1 << 63) - 1
    for window in (most, most - 1, most - 4, most - 32, most - 64, most - 100, 1 << 62, 1 << 40):
        for sinks in (0, 1, 4, 64, 1 << 30, 1 << 31, most):
            assert w4.attention_workspace_size(B, 32, 8, 128, 64, width, window, kind, sinks) == every, (window, sinks)


def _tokens(lib, **kw):
    a = dict(q=P, qts=4096, qhs=128, T=8, Hq=32, starts=P, B=2, tree=P, words=1, tld=1, cache=P, nbytes=1 << 40, pages=4,
             H=8, D=128, P=64, kind=0, dtype=0, table=P, width=2, ld=2, lengths=P, window=0, sinks=0, scale=0.1, out=P,
             ots=4096, ohs=128, ws=None, wsb=0)
    a.update(kw)
    return lib.w4a16_attention_tokens(*a.values(), None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), INVALID, "T=-1"),
    (dict(T=1 << 26), UNSUPPORTED, "T=67108864 tokens of q_heads=32"),
    (dict(B=-1), INVALID, "B=-1"),
    (dict(B=1 << 28), UNSUPPORTED, "too large for one launch"),
    (dict(Hq=0), INVALID, "q_heads=0"),
    (dict(Hq=30), INVALID, "q_heads=30 must be a positive multiple of kv_heads=8"),
    (dict(D=100), UNSUPPORTED, "head_dim=100"),
    (dict(P=40), UNSUPPORTED, "page_size=40"),
    (dict(kind=2), INVALID, "kind=2"),
    (dict(dtype=2), INVALID, "dtype=2"),
    (dict(width=-1), INVALID, "table_width=-1"),
    (dict(width=1 << 26, ld=1 << 26), UNSUPPORTED, "more than 2^31 tokens"),
    (dict(ld=1), INVALID, "table_ld=1 must be >= table_width=2"),
    (dict(words=0), INVALID, "tree_words=0"),
    (dict(words=1 << 17, tld=1 << 17), INVALID, "tree_words=131072"),
    (dict(words=2), INVALID, "tree_ld=1 must be >= tree_words=2"),
    (dict(tree=at(4)), INVALID, "tree must be 8-byte aligned"),
    (dict(window=-5), INVALID, "window=-5"),
    (dict(sinks=-5), INVALID, "sinks=-5"),
    (dict(scale=float("nan")), INVALID, "scale=nan"),
    (dict(qts=-1), INVALID, "q strides must be >= 0"),
    (dict(ohs=-1), INVALID, "out strides must be >= 0"),
    (dict(q=None), INVALID, "must not be NULL"),
    (dict(starts=None), INVALID, "must not be NULL"),
    (dict(table=None), INVALID, "must not be NULL"),
    (dict(lengths=None), INVALID, "must not be NULL"),
    (dict(out=None), INVALID, "must not be NULL"),
    (dict(q=at(1)), INVALID, "2-byte aligned"),
    (dict(starts=at(2)), INVALID, "4-byte aligned"),
    (dict(cache=at(4)), INVALID, "16-byte aligned"),
    (dict(nbytes=100), SIZE, "cache_bytes=100"),
    (dict(), SIZE, "workspace of 0 bytes"),
    (dict(tree=None, words=0, tld=0), SIZE, "workspace of 0 bytes"),
    (dict(ws=at(16), wsb=1 << 40), INVALID, "256-byte aligned"),
])
def test_tokens_rejects(lib, kw, status, needle):
    assert _tokens(lib, **kw) == status
    assert needle in w4.last_error()


def test_tokens_of_nothing_is_a_noop(lib):
    for kw in (dict(T=0), dict(B=0)):
        assert _tokens(lib, **kw, q=None, out=None, table=None, lengths=None, starts=None) == OK
        assert w4.last_error() == ""


def test_tokens_workspace_size(lib):
    out = ctypes.c_size_t(0)
    args = (64, 2, 32, 8, 128, 64, 4, 0)
    assert lib.w4a16_attention_tokens_workspace_size(*args, None) == INVALID
    assert lib.w4a16_attention_tokens_workspace_size(-1, *args[1:], ctypes.byref(out)) == INVALID
    assert lib.w4a16_attention_tokens_workspace_size(64, 2, 31, *args[3:], ctypes.byref(out)) == INVALID
    assert w4.attention_tokens_workspace_size(0, *args[1:]) == 0
    assert w4.attention_tokens_workspace_size(64, 0, *args[2:]) == 0
    need = w4.attention_tokens_workspace_size(8, 2, 32, 8, 128, 64, 2, 0)
    assert 0 < need and _tokens(lib, ws=P, wsb=need - 1) == SIZE and f"smaller than the {need} bytes" in w4.last_error()
    # bounded whatever the sizes
    assert w4.attention_tokens_workspace_size(1 << 20, 4096, 32, 8, 256, 64, 1 << 10, 0) < 512 << 20


def _sample(lib, **kw):
    a = dict(x=P, M=4, V=1000, ldl=1000, dtype=0, u=P, temperature=P, k=P, p=P, mp=P, tokens=P, probs=P)
    a.update(kw)
    return lib.w4a16_sample(*a.values(), None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dtype=2), INVALID, "dtype=2"),
    (dict(M=-1), INVALID, "M=-1"),
    (dict(M=1 << 23), UNSUPPORTED, "too large for one launch"),
    (dict(V=0), INVALID, "V=0 must be positive"),
    (dict(V=(1 << 22) + 1, ldl=1 << 23), UNSUPPORTED, "at most 2^22"),
    (dict(ldl=999), INVALID, "ldl=999 must be >= V=1000"),
    (dict(x=None), INVALID, "must not be NULL"),
    (dict(u=None), INVALID, "must not be NULL"),
    (dict(tokens=None), INVALID, "must not be NULL"),
    (dict(x=at(1)), INVALID, "2-byte aligned"),
    (dict(u=at(2)), INVALID, "4-byte aligned"),
    (dict(k=at(1)), INVALID, "4-byte aligned"),
    (dict(probs=at(2)), INVALID, "4-byte aligned"),
    (dict(tokens=at(4)), INVALID, "8-byte aligned"),
])
def test_sample_rejects(lib, kw, status, needle):
    assert _sample(lib, **kw) == status
    assert needle in w4.last_error()


def test_sample_of_no_rows_is_a_noop(lib):
    assert _sample(lib, M=0, x=None, u=None, tokens=None) == OK
    assert w4.last_error() == ""


def test_binding_refuses_cpu_tensors():
    kv, slots = torch.zeros(2, 1, 64, dtype=torch.float16), torch.zeros(2, dtype=torch.int64)
    cache, i32 = torch.zeros(1 << 14, dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.int32)
    for call in (lambda: w4.kv_append(kv, kv, kv, i32[:, 0], torch.zeros(8), slots, cache, 1, 32, w4.KV_ACT),
                 lambda: w4.attention_tokens(kv, i32[:, 0], cache, i32[:1], i32[:1, 0], 1, 1, 32, w4.KV_ACT),
                 lambda: w4.attention(kv, cache, i32, i32[:, 0], 1, 1, 32, w4.KV_ACT, window=3, sinks=1),
                 lambda: w4.sample(kv[:, 0], torch.zeros(2))):
        with pytest.raises(ValueError, match="must be a GPU tensor"):
            call()


# ---------------------------------------------------------------- the reference


def test_rows_see_a_prompt():
    seen = step.rows_see(5, 3)
    assert seen.int().tolist() == [[1, 1, 1, 0, 0], [1, 1, 1, 1, 0], [1, 1, 1, 1, 1]]
    assert step.rows_see(5, 3, window=2, sinks=1).int().tolist() == [[1, 1, 1, 0, 0], [1, 0, 1, 1, 0], [1, 0, 0, 1, 1]]
    assert step.rows_see(2, 4).int().tolist() == [[0, 0], [0, 0], [1, 0], [1, 1]]


def test_rows_see_a_tree():
    # 0 and 1 are roots, 2 hangs on 0, 3 has no bit
    words = torch.tensor([[0b0001], [0b0010], [0b0101], [0]])
    assert step.rows_see(6, 4, words=words).int().tolist() == [[1, 1, 1, 0, 0, 0], [1, 1, 0, 1, 0, 0], [1, 1, 1, 0, 1, 0], [0] * 6]
    # node 2 is a place further on: a window of 2 ends before the past's last token for it
    assert step.rows_see(6, 4, window=2, words=words).int().tolist() == [[0, 1, 1, 0, 0, 0], [0, 1, 0, 1, 0, 0], [0, 0, 1, 0, 1, 0], [0] * 6]


def test_random_trees_hold_their_nodes_and_parents():
    words = step.random_tree(np.random.default_rng(0), 130, 3)
    seen, depth = step.bits(words, 130)
    assert bool(seen.diagonal().all()) and not bool(seen.triu(1).any()) and int(depth.max()) < 130
    for i in range(130):
        for j in seen[i].nonzero()[:, 0].tolist():
            assert bool((seen[j] <= seen[i]).all())


def test_sample_reference_by_hand():
    x = torch.tensor([0.0, 2.0, 2.0, -float("inf"), 1.0], dtype=torch.float64)
    e1, e2 = np.exp(-1), np.exp(-2)
    total = 2 + e1 + e2
    for u, token in ((0.0, 1), (1 / total - 1e-6, 1), (1 / total + 1e-6, 2), (2 / total + 1e-6, 4), (0.99999, 0)):
        assert step.sample(x, u)[0] == token
    assert step.sample(x, 0.99, top_k=2)[0] == 2 and step.sample(x, 0.3, top_k=2)[1] == 0.5
    assert step.sample(x, 0.99, top_p=0.3)[0] == 1 and step.sample(x, 0.99, top_p=1.01 / total)[0] == 2
    assert step.sample(x, 0.99, min_p=0.3)[0] == 4 and step.sample(x, 0.99, min_p=0.5)[0] == 2
    assert step.sample(x, 0.9, temperature=0.0) == (1, 1.0, 1.0)
    assert step.sample(torch.full((3,), -float("inf")), 0.5)[0] == -1


def test_calls_run_with_their_tensors_device_current(monkeypatch):
    """Where another device is current, the entry runs inside a switch to the tensors' one, errors included."""
    current = [0]

    class Switch:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.former, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.former

    monkeypatch.setattr(w4, "_current_device", lambda: current[0])
    monkeypatch.setattr(w4.torch.cuda, "device", Switch)
    ran = []

    def entry(status):
        ran.append(current[0])
        return status

    w4._call(0, entry, 0)
    w4._call(1, entry, 0)
    with pytest.raises(RuntimeError, match="w4a16 status 1"):
        w4._call(2, entry, 1)
    assert ran == [0, 1, 2] and current == [0]


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_lds_limits_are_raised_on_each_device(tmp_path):
    """A kernel's limit is the device's: a call on another device raises its own, and calls at once never lower one."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = str(tmp_path / "lds_limit")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(root, "include"),
                    "-I", os.path.join(root, "mixed_precision_w4a16_repack_amd", "csrc"), "-isystem", "/opt/rocm/include",
                    os.path.join(root, "tests", "lds_limit.cpp"), "-o", exe], check=True, capture_output=True, text=True)
    res = subprocess.run([exe], capture_output=True, text=True)
    assert res.returncode == 0 and res.stdout.strip() == "ok", res.stdout
