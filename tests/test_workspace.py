"""Who shares a scratch buffer: the cache is asked on CPU tensors, with the stream's handle made up."""
import threading

import pytest
import torch

from dora_adapter_linear_gb300 import _lib as L
from dora_adapter_linear_gb300 import ops


@pytest.fixture(autouse=True)
def made_up_stream(monkeypatch):
    monkeypatch.setattr(L, "current_stream", lambda device=None: 7)
    monkeypatch.setattr(L, "capture_id", lambda stream: 0, raising=False)
    monkeypatch.setattr(ops, "_WS", {})


def address(nbytes=1024):
    return ops.workspace(nbytes, torch.device("cpu")).data_ptr()


def test_calls_of_one_thread_share_a_buffer_that_grows():
    first = ops.workspace(1000, torch.device("cpu"))
    assert not first.any() and first.data_ptr() == address(300) == address(1000)
    assert ops.workspace(5000, torch.device("cpu")).numel() >= 5000


def test_two_threads_on_one_stream_have_a_buffer_each():
    """The launches of two calls may come in any order: on one buffer a call would read the other's partials."""
    mine, others = address(), []
    hold = threading.Barrier(3)

    def call():
        others.append(address())
        hold.wait(10)           # both threads live at once, as do their identifiers
    threads = [threading.Thread(target=call) for _ in range(2)]
    for t in threads:
        t.start()
    hold.wait(10)
    for t in threads:
        t.join()
    assert len({mine, *others}) == 3
    assert address() == mine


def test_a_capture_has_a_buffer_of_its_own(monkeypatch):
    """A graph writes where it was captured: neither a later call, however large, nor another graph may be there."""
    eager = ops.workspace(1024, torch.device("cpu"))
    captured = {}
    for number in (11, 12):
        monkeypatch.setattr(L, "capture_id", lambda stream: number)
        captured[number] = ops.workspace(1024, torch.device("cpu"))
        assert not captured[number][:256].any()
        assert address() == captured[number].data_ptr()         # calls of one capture follow one another
    assert len({eager.data_ptr(), *(t.data_ptr() for t in captured.values())}) == 3
    monkeypatch.setattr(L, "capture_id", lambda stream: 0)
    assert address() == eager.data_ptr()
    assert address(1 << 20) not in (eager.data_ptr(), *(t.data_ptr() for t in captured.values()))
    assert len(ops._WS) == 1            # what ended captures used is left to their graphs
