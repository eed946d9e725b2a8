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


def test_an_error_that_nobody_has_looked_at_outlives_its_buffer(monkeypatch):
    first = ops.workspace(1024, torch.device("cpu"))
    first[0], first[300] = 1, 9
    larger = ops.workspace(4096, torch.device("cpu"))
    assert larger.data_ptr() != first.data_ptr() and larger[0] == 1 and not larger[1:].any()
    cleared = []
    monkeypatch.setattr(torch.cuda, "synchronize", lambda: None)
    monkeypatch.setattr(L, "lora_check_device_error", lambda buf: 6 if buf[0] else 0)
    monkeypatch.setattr(L, "lora_clear_device_error", lambda buf: cleared.append(buf[:256].zero_()))
    with pytest.raises(L.LoraError) as e:
        ops.check_device_errors()
    assert e.value.status == 6 and len(cleared) == 1
    ops.check_device_errors()


@pytest.mark.gpu
def test_a_wait_that_ran_out_shows(monkeypatch):
    """The test hook's wait on a barrier that nothing arrives on, in the workspace of one of three streams."""
    monkeypatch.undo()
    from dora_adapter_linear_gb300.build import build
    build()
    device, streams = torch.device("cuda", 0), [torch.cuda.Stream() for _ in range(3)]
    ops.check_device_errors()
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            ws = ops.workspace(256, device)
            if i == 1:
                L.lora_debug_wait_timeout(ws, 2000)
                assert ops.workspace(1 << 22, device).data_ptr() != ws.data_ptr()
    with pytest.raises(L.LoraError) as e:
        ops.check_device_errors()
    assert e.value.status == 6
    ops.check_device_errors()
