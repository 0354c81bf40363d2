"""Who may use a cached workspace for how long, beside graph captures: the host's side, without a device."""
import contextlib
import weakref

import pytest
import torch

from block_scaled_fp8_02_gb300 import _binding as B

DEV = torch.device("cpu", 0)


@pytest.fixture
def capture(monkeypatch):
    """The cache on CPU tensors; state["id"] is the capture that every stream is in."""
    state = {"id": 0}
    monkeypatch.setattr(B, "_stream_ptr", lambda stream: 77 if stream is None else stream)
    monkeypatch.setattr(B, "_capture_id", lambda stream, sp: state["id"], raising=False)
    for name in ("_ws_cache", "_ws_graph", "_ws_held"):
        monkeypatch.setattr(B, name, {}, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda sp, device=None: None)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: None)
    return state


def test_a_buffer_that_a_graph_uses_outlives_its_replacement(capture):
    eager = weakref.ref(B.workspace_for(1000, DEV))
    capture["id"] = 1
    assert B.workspace_for(900, DEV) is eager()
    capture["id"] = 0
    larger = B.workspace_for(5000, DEV)
    assert larger.numel() >= 5000 and B.workspace_for(1000, DEV) is larger
    assert eager() is not None and eager() is not larger


def test_a_buffer_no_graph_has_seen_is_let_go(capture):
    first = weakref.ref(B.workspace_for(1000, DEV))
    B.workspace_for(5000, DEV)
    assert first() is None


def test_a_buffer_born_in_a_capture_is_for_that_capture_only(capture):
    """Its zeros are a node of that graph: whoever else got it could find anything."""
    capture["id"] = 1
    mine = B.workspace_for(1000, DEV)
    assert B.workspace_for(700, DEV) is mine
    assert B.workspace_for(700, DEV, 78) is not mine              # another stream of the capture
    capture["id"] = 2
    assert B.workspace_for(700, DEV) is not mine
    capture["id"] = 0
    assert B.workspace_for(700, DEV) is not mine


def test_a_failure_leaves_graphs_with_a_zeroed_buffer(capture):
    ws = B.workspace_for(1000, DEV)
    capture["id"] = 1
    assert B.workspace_for(1000, DEV) is ws
    capture["id"] = 0
    ws.fill_(1)                                                   # a kernel that gave up half-way
    B.drop_workspaces()
    assert (ws == 0).all() and B.workspace_for(1000, DEV) is not ws
