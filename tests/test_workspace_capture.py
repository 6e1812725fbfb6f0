"""Workspaces under graph capture (CPU only: the capture is pretended)."""

from __future__ import annotations

import weakref

import pytest
import torch

import mixed_precision_w4a16_repack_amd as w4


@pytest.fixture
def capture(monkeypatch):
    """Sets whether the current stream counts as being captured."""
    state = {"on": False}
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["on"])
    monkeypatch.setattr(w4, "workspace_counter_bytes", lambda: 64)
    return lambda on: state.update(on=on)


def test_a_buffer_that_a_graph_holds_outlives_growth(capture):
    ws = w4.Workspace("cpu")
    small = ws.get(100)
    capture(True)
    held = ws.get(80)
    assert held is small
    capture(False)
    alive = weakref.ref(small)
    del held, small
    grown = ws.get(1000)
    assert grown.numel() == 1000 and not bool(grown.any())
    assert alive() is not None, "the graph's buffer was given back"


def test_former_buffers_stay_within_the_present_one(capture):
    ws = w4.Workspace("cpu")
    for n in range(100, 5000, 7):
        assert ws.get(n).numel() >= n
    assert sum(t.numel() for t in ws._former) <= ws.buf.numel()


def test_a_capture_leaves_no_uncleared_buffer_behind(capture):
    """What is allocated in a capture is cleared at replays only: eager calls must not find it."""
    ws = w4.Workspace("cpu")
    capture(True)
    first, second = ws.get(100), ws.get(100)
    assert first.numel() == second.numel() == 100 and first.data_ptr() != second.data_ptr()
    assert not bool(first[:64].any())
    capture(False)
    assert ws.buf is None
    eager = ws.get(100)
    assert eager.data_ptr() not in (first.data_ptr(), second.data_ptr()) and not bool(eager.any())
    # one that is too small for a captured call stays as it is
    capture(True)
    assert ws.get(200).numel() == 200 and ws.buf is eager
    capture(False)
    assert ws.get(100) is eager


def test_graphs_do_not_share_the_default_workspace(capture, monkeypatch):
    monkeypatch.setattr(w4, "_raw_stream", lambda index: 1234)
    monkeypatch.setattr(w4, "_workspaces", {})
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    eager = w4._default_workspace("cpu", "attention").get(100)
    capture(True)
    a = w4._default_workspace("cpu", "attention").get(100)
    b = w4._default_workspace("cpu", "attention").get(100)
    assert len({t.data_ptr() for t in (eager, a, b)}) == 3
    capture(False)
    assert w4._default_workspace("cpu", "attention").get(100) is eager
