"""CPU tests of the binding's workspaces: which calls share a buffer, and how long one is kept."""
import threading

import pytest
import torch

import speculative_decoding_verification_gb300 as sv


@pytest.fixture
def on(monkeypatch):
    """Sets the stream, and the capture, that the next calls find themselves on."""
    def set_(stream, capture=0):
        monkeypatch.setattr(sv, "_current_raw_stream", lambda index: stream)
        monkeypatch.setattr(sv, "_capture_id", lambda index, raw: capture)
    return set_


DEV = torch.device("cpu", 0)


@pytest.mark.parametrize("ws", ["own", "default"])
def test_streams_do_not_share(on, ws):
    ws = sv.Workspace() if ws == "own" else sv._default_ws
    on(101)
    a = ws.get(1000, DEV)
    on(102)
    b = ws.get(1000, DEV)
    assert a.data_ptr() != b.data_ptr()
    on(101)
    assert ws.get(900, DEV).data_ptr() == a.data_ptr()
    assert ws.get(5000, DEV).numel() >= 5000


def test_threads_do_not_share(on):
    """Launches of two calls on one stream may alternate, so host threads do not share either."""
    on(7)
    a, got = sv._default_ws.get(1000, DEV), []
    t = threading.Thread(target=lambda: got.append(sv._default_ws.get(1000, DEV)))
    t.start()
    t.join()
    assert got[0].data_ptr() != a.data_ptr()


def test_captured_buffers_are_kept_and_not_shared(on):
    ws = sv.Workspace()
    on(7)
    eager = ws.get(1000, DEV)
    on(7, capture=5)
    first = ws.get(1000, DEV)
    at = first.data_ptr()
    assert at != eager.data_ptr() and ws.get(600, DEV).data_ptr() == at   # calls of one capture follow one another
    larger = ws.get(1 << 20, DEV)
    assert larger.data_ptr() != at
    del first
    assert any(t.data_ptr() == at for bufs in ws._captured.values() for t in bufs)   # the graph still holds its address
    on(7, capture=6)
    assert ws.get(1000, DEV).data_ptr() not in (at, larger.data_ptr(), eager.data_ptr())
    on(7)
    assert ws.get(1000, DEV).data_ptr() == eager.data_ptr()


def test_calls_run_on_their_stream(monkeypatch):
    """A call with stream= allocates on that stream and marks the tensors that both streams use."""
    class Stream:
        device = torch.device("cuda", 0)
    mine, outer, seen = Stream(), Stream(), []

    class Context:
        def __init__(self, s):
            seen.append(("enter", s))

        def __enter__(self):
            pass

        def __exit__(self, *a):
            seen.append(("exit",))

    class Fake(torch.Tensor):
        is_cuda = True

        def record_stream(self, s):
            seen.append(("record", s))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: outer)
    monkeypatch.setattr(torch.cuda, "stream", Context)

    def f(x, y=None, stream=None):
        seen.append(("run", stream))
        return torch.zeros(1).as_subclass(Fake), None
    call = sv._on_stream(f)
    x = torch.zeros(1).as_subclass(Fake)
    call(x, y=3, stream=mine)
    assert seen == [("record", mine), ("enter", mine), ("run", mine), ("exit",), ("record", outer)]
    for args in ((x, None, None), (x, None, outer)):
        seen.clear()
        call(*args)
        assert seen == [("run", args[2])]
    seen.clear()
    call(x, None, mine)   # by position
    assert ("enter", mine) in seen
    for name in ("sv_verify", "sv_kv_attend", "sv_kv_append", "sv_kv_commit", "sv_rope", "sv_tree_verify", "sv_topk_rows"):
        assert hasattr(getattr(sv, name), "__wrapped__"), name
