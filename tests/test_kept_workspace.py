"""The binding keeps a stream's last attention workspace and takes it again once nobody else holds it (no GPU: the
allocations are fakes).  Whether somebody does is told by reference counts, whose ground state is the interpreter's own affair:
some count what a caller's locals and arguments hold, some do not."""
import sys

import pytest
import torch

from gated_delta_rule_36_gb300 import binding as kb


@pytest.fixture
def allocations(monkeypatch):
    made = []

    def workspace(given, nbytes, device, stream):
        assert given is None
        made.append(nbytes)
        return torch.zeros(nbytes, dtype=torch.uint8)

    monkeypatch.setattr(kb, "_workspace", workspace)
    monkeypatch.setattr(kb, "_KEPT", {})
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False, raising=False)
    return made


def counting(shift):
    """sys.getrefcount as an interpreter reports it that counts `shift` more references for the same objects."""
    def through(o):
        return sys.getrefcount(o)
    x = object()
    extra = through(x) - sys.getrefcount(x)

    def count(o):
        return sys.getrefcount(o) - extra + shift
    return count


def take(nbytes=4096, raw=7):
    return kb._kept_workspace(nbytes, 0, None, raw)


@pytest.mark.parametrize("shift", [-2, -1, 0, 1])
def test_a_workspace_that_is_held_is_not_taken_again(allocations, monkeypatch, shift):
    monkeypatch.setattr(kb, "_refs", counting(shift))
    held = take()[0]
    second = take()[0]
    assert second.data_ptr() != held.data_ptr()
    view, at = second[:4], second.data_ptr()
    del second
    third = take()[0]
    assert third.data_ptr() != at                        # a view keeps it too
    storage, at = third.untyped_storage(), third.data_ptr()
    del third
    assert take()[1] != at and storage.data_ptr() == at  # ... and its storage
    assert held.numel() == 4096 and view.numel() == 4
    assert len(allocations) == 4


@pytest.mark.parametrize("shift", [-2, -1, 0, 1])
def test_a_workspace_that_is_dropped_is_taken_again(allocations, monkeypatch, shift):
    monkeypatch.setattr(kb, "_refs", counting(shift))
    at = take()[1]
    for _ in range(5):
        ws, where, room = take()
        assert where == ws.data_ptr() == at and room == 4096
        del ws
    assert take(2048)[1] == at and len(allocations) == 1
    assert take(8192)[2] == 8192 and take(8192, raw=8)[2] == 8192 and len(allocations) == 3     # a larger one; another stream's


def test_large_ones_are_not_kept(allocations):
    for _ in range(2):
        take(kb._KEPT_MOST + 1)
    assert not kb._KEPT and len(allocations) == 2


def test_no_more_than_some_streams_keep_one(allocations):
    """A program that makes a stream for each request does not keep a workspace for each."""
    held = take(raw=1000)[0]
    for raw in range(10 * kb._KEPT_STREAMS):
        take(raw=raw)
        assert len(kb._KEPT) <= kb._KEPT_STREAMS
    assert take(raw=1000)[1] != held.data_ptr()          # (one that is held is the caller's, whatever was kept)
    n = len(allocations)
    assert take(raw=5)[1] and take(raw=5)[1] and len(allocations) <= n + 1
