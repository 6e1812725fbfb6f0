"""Argument checks of the operators between a layer's GEMMs (CPU only): every
refusal comes before any HIP call, with the documented status and message.
Also the cache's layout as the header states it: each byte of a record is one
element's, and the binding's own checks."""

from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest
import torch

import mixed_precision_w4a16_repack_amd as w4
from tests import operator_reference as ref

OK, INVALID, UNSUPPORTED, SIZE = 0, -1, -2, -3
P = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(w4.LIB_PATH):
        from mixed_precision_w4a16_repack_amd import build

        build.build()
    return w4.load_library()


def _norm(lib, out8=False, **kw):
    a = dict(x=P, M=4, K=4096, ldx=4096, dtype=0, weight=P, eps=1e-5, residual=P, ldr=4096, ro=P, ldro=4096, y=P,
             ldy=4096, xs=P)
    a.update(kw)
    head = (a["x"], a["M"], a["K"], a["ldx"], a["dtype"], a["weight"], a["eps"], a["residual"], a["ldr"], a["ro"],
            a["ldro"], a["y"], a["ldy"])
    return lib.w4a8_rmsnorm(*head, a["xs"], None) if out8 else lib.w4a16_rmsnorm(*head, None)


BOTH = [
    (dict(M=-1), INVALID, "M=-1"),
    (dict(K=0), INVALID, "K=0 must be positive"),
    (dict(K=(1 << 32) + 8, ldx=1 << 33, ldr=1 << 33, ldro=1 << 33, ldy=1 << 33), UNSUPPORTED, "at most 2^32"),
    (dict(M=1 << 31), UNSUPPORTED, "too large for one launch"),
    (dict(dtype=2), INVALID, "dtype=2"),
    (dict(ldx=4095), INVALID, "ldx=4095 must be >= K=4096"),
    (dict(ldx=(1 << 40) + 1), UNSUPPORTED, "ldx="),
    (dict(ldr=100), INVALID, "ldr=100 must be >= K=4096"),
    (dict(ldro=100), INVALID, "ldro=100 must be >= K=4096"),
    (dict(eps=-1.0), INVALID, "eps=-1"),
    (dict(eps=float("nan")), INVALID, "eps=nan"),
    (dict(eps=float("inf")), INVALID, "eps=inf"),
    (dict(x=None), INVALID, "must not be NULL"),
    (dict(weight=None), INVALID, "must not be NULL"),
    (dict(y=None), INVALID, "must not be NULL"),
    (dict(x=ctypes.c_void_p(4097)), INVALID, "2-byte aligned"),
    (dict(residual=ctypes.c_void_p(4097)), INVALID, "2-byte aligned"),
]


@pytest.mark.parametrize("kw,status,needle", BOTH + [
    (dict(ldy=4000), INVALID, "ldy=4000 must be >= K=4096"),
    (dict(y=ctypes.c_void_p(4097)), INVALID, "2-byte aligned"),
])
def test_rmsnorm_rejects(lib, kw, status, needle):
    assert _norm(lib, **kw) == status
    assert needle in w4.last_error()


@pytest.mark.parametrize("kw,status,needle", BOTH + [
    (dict(ldy=4000), INVALID, "ldq=4000 must be >= K=4096"),
    (dict(ldy=4100), UNSUPPORTED, "ldq % 8 == 0"),
    (dict(y=ctypes.c_void_p(4100)), UNSUPPORTED, "8-byte aligned"),
    (dict(xs=None), INVALID, "must not be NULL"),
    (dict(xs=ctypes.c_void_p(4098)), INVALID, "xs must be 4-byte aligned"),
    (dict(K=4092), UNSUPPORTED, "K=4092 must be divisible by 8"),
])
def test_rmsnorm_a8_rejects(lib, kw, status, needle):
    assert _norm(lib, True, **kw) == status
    assert needle in w4.last_error()


def _gate(lib, out8=False, **kw):
    a = dict(x=P, M=4, K=4096, ldx=8192, dtype=0, y=P, ldy=4096, xs=P)
    a.update(kw)
    head = (a["x"], a["M"], a["K"], a["ldx"], a["dtype"], a["y"], a["ldy"])
    return lib.w4a8_silu_mul(*head, a["xs"], None) if out8 else lib.w4a16_silu_mul(*head, None)


@pytest.mark.parametrize("out8", [False, True])
@pytest.mark.parametrize("kw,status,needle", [
    (dict(M=-3), INVALID, "M=-3"),
    (dict(K=-8), INVALID, "must be positive"),
    (dict(dtype=-1), INVALID, "dtype=-1"),
    (dict(ldx=8191), INVALID, "ldx=8191 must be >= 2*K=8192"),
    (dict(x=None), INVALID, "must not be NULL"),
    (dict(y=None), INVALID, "must not be NULL"),
    (dict(x=ctypes.c_void_p(4099)), INVALID, "2-byte aligned"),
])
def test_silu_mul_rejects(lib, out8, kw, status, needle):
    assert _gate(lib, out8, **kw) == status
    assert needle in w4.last_error()


def test_silu_mul_rejects_by_output(lib):
    assert _gate(lib, ldy=5) == INVALID and "ldy=5 must be >= K=4096" in w4.last_error()
    assert _gate(lib, True, ldy=5) == INVALID and "ldq=5 must be >= K=4096" in w4.last_error()
    assert _gate(lib, True, K=4092) == UNSUPPORTED and "divisible by 8" in w4.last_error()
    assert _gate(lib, True, y=ctypes.c_void_p(4100)) == UNSUPPORTED and "8-byte aligned" in w4.last_error()
    # rows of 14336 columns take 1024 threads each for codes, 7 workgroups of 256 else
    assert _gate(lib, True, M=1 << 22, K=14336, ldx=28672, ldy=14336) == UNSUPPORTED
    assert "too large for one launch" in w4.last_error()
    assert _gate(lib, M=3 << 20, K=14336, ldx=28672, ldy=14336) == UNSUPPORTED
    # rows of 2^20 columns take 512 workgroups each
    assert _gate(lib, M=1 << 23, K=1 << 20, ldx=1 << 21, ldy=1 << 20) == UNSUPPORTED
    assert "too large for one launch" in w4.last_error()


def test_rows_m_zero_is_a_noop(lib):
    for out8 in (False, True):
        assert _norm(lib, out8, M=0, x=None, y=None, weight=None) == OK
        assert _gate(lib, out8, M=0, x=None, y=None) == OK
        assert w4.last_error() == ""


@pytest.mark.parametrize("args,status,needle", [
    ((4, 8, 128, 64, 2), INVALID, "kind=2"),
    ((-1, 8, 128, 64, 0), INVALID, "pages=-1"),
    ((4, 0, 128, 64, 0), INVALID, "kv_heads=0"),
    ((4, 8, 96, 64, 0), UNSUPPORTED, "head_dim=96 not supported"),
    ((4, 8, 512, 64, 1), UNSUPPORTED, "head_dim=512 not supported"),
    ((4, 8, 128, 16, 0), UNSUPPORTED, "page_size=16"),
    ((4, 8, 128, 0, 0), UNSUPPORTED, "page_size=0"),
    ((4, 8, 128, 1 << 17, 0), UNSUPPORTED, "at most 2^16"),
    (((1 << 31) - 1, 1 << 16, 256, 1 << 16, 0), UNSUPPORTED, "2^50"),
])
def test_kv_cache_size_rejects(lib, args, status, needle):
    out = ctypes.c_size_t(0)
    assert lib.w4a16_kv_cache_size(*args, ctypes.byref(out)) == status
    assert needle in w4.last_error()


def test_kv_cache_size(lib):
    assert lib.w4a16_kv_cache_size(4, 8, 128, 64, 0, None) == INVALID
    assert w4.kv_cache_size(0, 8, 128, 64, w4.KV_ACT) == 0
    for kind in (w4.KV_ACT, w4.KV_INT8):
        for D in (64, 128, 192, 256):
            for page_size in (32, 96, 256):
                assert w4.kv_cache_size(7, 3, D, page_size, kind) == 7 * 3 * ref.record_bytes(D, page_size, kind)


@pytest.mark.parametrize("kind", [ref.KV_ACT, ref.KV_INT8])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("page_size", [32, 96])
def test_every_byte_of_a_record_belongs_to_one_element(D, page_size, kind):
    k, v, s = ref.places(D, page_size, kind)
    width = 2 if kind == ref.KV_ACT else 1
    bytes_ = [(p.reshape(-1, 1) + np.arange(width)).reshape(-1) for p in (k, v)]
    if s is not None:
        bytes_.append((s.reshape(-1, 1) + np.arange(4)).reshape(-1))
    assert np.array_equal(np.sort(np.concatenate(bytes_)), np.arange(ref.record_bytes(D, page_size, kind)))


def _kv(lib, write, **kw):
    a = dict(k=P, kts=1024, khs=128, v=P, vts=1024, vhs=128, T=4, slots=P, cache=P, nbytes=1 << 40, pages=4, H=8,
             D=128, P=64, kind=0, dtype=0)
    a.update(kw)
    if write:
        return lib.w4a16_kv_write(a["k"], a["kts"], a["khs"], a["v"], a["vts"], a["vhs"], a["T"], a["slots"],
                                  a["cache"], a["nbytes"], a["pages"], a["H"], a["D"], a["P"], a["kind"], a["dtype"],
                                  None)
    return lib.w4a16_kv_read(a["slots"], a["T"], a["cache"], a["nbytes"], a["pages"], a["H"], a["D"], a["P"],
                             a["kind"], a["dtype"], a["k"], a["kts"], a["khs"], a["v"], a["vts"], a["vhs"], None)


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), INVALID, "T=-1"),
    (dict(T=1 << 31), UNSUPPORTED, "too large for one launch"),
    (dict(dtype=7), INVALID, "dtype=7"),
    (dict(kind=-1), INVALID, "kind=-1"),
    (dict(D=80), UNSUPPORTED, "head_dim=80"),
    (dict(P=48), UNSUPPORTED, "page_size=48"),
    (dict(kts=-1), INVALID, "k strides must be >= 0"),
    (dict(vhs=(1 << 40) + 1), UNSUPPORTED, "v strides must be at most 2^40"),
    (dict(k=None), INVALID, "must not be NULL"),
    (dict(v=None), INVALID, "must not be NULL"),
    (dict(slots=None), INVALID, "must not be NULL"),
    (dict(cache=None), INVALID, "cache must not be NULL"),
    (dict(k=ctypes.c_void_p(4097)), INVALID, "2-byte aligned"),
    (dict(slots=ctypes.c_void_p(4100)), INVALID, "8-byte aligned"),
    (dict(cache=ctypes.c_void_p(4104)), INVALID, "16-byte aligned"),
    (dict(nbytes=4 * 8 * 4 * 64 * 128 - 1), SIZE, "smaller than the 1048576 bytes"),
    (dict(kind=1, nbytes=4 * 8 * (2 * 64 * 128 + 512) - 1), SIZE, "bytes of the cache"),
])
def test_kv_rejects(lib, write, kw, status, needle):
    assert _kv(lib, write, **kw) == status
    assert needle in w4.last_error()


def test_kv_t_zero_is_a_noop(lib):
    for write in (True, False):
        assert _kv(lib, write, T=0, k=None, v=None, slots=None, cache=None) == OK
        assert w4.last_error() == ""


def _attention(lib, **kw):
    a = dict(q=P, qbs=4096, qhs=128, B=2, Hq=32, cache=P, nbytes=1 << 40, pages=4, H=8, D=128, P=64, kind=0, dtype=0,
             table=P, width=2, ld=2, lengths=P, window=0, scale=0.1, out=P, obs=4096, ohs=128, ws=None, wsb=0)
    a.update(kw)
    return lib.w4a16_attention(a["q"], a["qbs"], a["qhs"], a["B"], a["Hq"], a["cache"], a["nbytes"], a["pages"],
                               a["H"], a["D"], a["P"], a["kind"], a["dtype"], a["table"], a["width"], a["ld"],
                               a["lengths"], a["window"], a["scale"], a["out"], a["obs"], a["ohs"], a["ws"], a["wsb"],
                               None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(B=-1), INVALID, "B=-1"),
    (dict(Hq=0), INVALID, "q_heads=0"),
    (dict(Hq=30), INVALID, "q_heads=30 must be a positive multiple of kv_heads=8"),
    (dict(H=0), INVALID, "kv_heads=0"),
    (dict(D=100), UNSUPPORTED, "head_dim=100"),
    (dict(P=40), UNSUPPORTED, "page_size=40"),
    (dict(kind=2), INVALID, "kind=2"),
    (dict(dtype=2), INVALID, "dtype=2"),
    (dict(width=-1), INVALID, "table_width=-1"),
    (dict(width=1 << 26, ld=1 << 26), UNSUPPORTED, "more than 2^31 tokens"),
    (dict(B=1 << 20, width=1 << 20, ld=1 << 20), UNSUPPORTED, "more than 2^43 tokens"),
    (dict(ld=1), INVALID, "table_ld=1 must be >= table_width=2"),
    (dict(window=-5), INVALID, "window=-5"),
    (dict(B=1 << 28), UNSUPPORTED, "too large for one launch"),
    (dict(scale=float("nan")), INVALID, "scale=nan"),
    (dict(scale=float("inf")), INVALID, "scale=inf"),
    (dict(qbs=-1), INVALID, "q strides must be >= 0"),
    (dict(ohs=-1), INVALID, "out strides must be >= 0"),
    (dict(q=None), INVALID, "must not be NULL"),
    (dict(table=None), INVALID, "must not be NULL"),
    (dict(lengths=None), INVALID, "must not be NULL"),
    (dict(out=None), INVALID, "must not be NULL"),
    (dict(q=ctypes.c_void_p(4097)), INVALID, "2-byte aligned"),
    (dict(lengths=ctypes.c_void_p(4098)), INVALID, "4-byte aligned"),
    (dict(cache=ctypes.c_void_p(4100)), INVALID, "16-byte aligned"),
    (dict(nbytes=100), SIZE, "cache_bytes=100"),
])
def test_attention_rejects(lib, kw, status, needle):
    assert _attention(lib, **kw) == status
    assert needle in w4.last_error()


def test_attention_b_zero_is_a_noop(lib):
    assert _attention(lib, B=0, q=None, out=None, table=None, lengths=None) == OK
    assert w4.last_error() == ""


def test_attention_workspace_size(lib):
    out = ctypes.c_size_t(0)
    assert lib.w4a16_attention_workspace_size(1, 32, 8, 128, 64, 4, 0, 0, None) == INVALID
    assert lib.w4a16_attention_workspace_size(1, 31, 8, 128, 64, 4, 0, 0, ctypes.byref(out)) == INVALID
    assert lib.w4a16_attention_workspace_size(1, 32, 8, 120, 64, 4, 0, 0, ctypes.byref(out)) == UNSUPPORTED
    assert lib.w4a16_attention_workspace_size(1, 32, 8, 128, 64, 4, -1, 0, ctypes.byref(out)) == INVALID
    assert w4.attention_workspace_size(0, 32, 8, 128, 64, 4, 0, w4.KV_ACT) == 0
    # bounded whatever the lengths, and never below the counter region
    small = w4.attention_workspace_size(1, 32, 8, 128, 64, 4, 0, w4.KV_ACT)
    assert w4.workspace_counter_bytes() < small < 1 << 20
    large = w4.attention_workspace_size(4096, 32, 8, 128, 64, 1 << 20, 0, w4.KV_ACT)
    assert large == w4.attention_workspace_size(256, 32, 8, 128, 64, 1 << 20, 0, w4.KV_ACT) < 64 << 20
    # a short window needs no more than a short table
    assert w4.attention_workspace_size(1, 32, 8, 128, 64, 1 << 20, 100, w4.KV_ACT) <= small


def test_attention_checks_its_workspace(lib):
    need = w4.attention_workspace_size(2, 32, 8, 128, 64, 2, 0, w4.KV_ACT)
    for ws, nbytes in ((None, 0), (None, need), (P, need - 1)):
        assert _attention(lib, ws=ws, wsb=nbytes) == SIZE
        assert f"smaller than the {need} bytes" in w4.last_error()
    assert _attention(lib, ws=ctypes.c_void_p(4096 + 16), wsb=need) == INVALID
    assert "256-byte aligned" in w4.last_error()


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(2, 8, dtype=torch.float16), torch.ones(8, dtype=torch.float16)
    kv, slots = torch.zeros(2, 1, 64, dtype=torch.float16), torch.zeros(2, dtype=torch.int64)
    cache, i32 = torch.zeros(1 << 14, dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.int32)
    for call in (lambda: w4.rmsnorm(x, w), lambda: w4.rmsnorm_a8(x, w), lambda: w4.silu_mul(x),
                 lambda: w4.silu_mul_a8(x), lambda: w4.kv_write(kv, kv, slots, cache, 1, 32, w4.KV_ACT),
                 lambda: w4.kv_read(slots, cache, 1, 1, 64, 32, w4.KV_ACT, torch.float16),
                 lambda: w4.attention(kv, cache, i32, i32[:, 0], 1, 1, 32, w4.KV_ACT)):
        with pytest.raises(ValueError, match="must be a GPU tensor"):
            call()
