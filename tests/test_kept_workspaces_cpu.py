"""Which workspaces the binding keeps between calls (allocation and streams replaced by
stand-ins; no GPU)."""

import threading
import weakref

import pytest
import torch

import implicit_gemm_conv_tcgen05_gb300 as igc

MB = 1 << 20


@pytest.fixture
def stream(monkeypatch):
    """The current stream's handle and whether it captures, to be set by the test."""
    state = {"handle": 0, "capturing": False}
    monkeypatch.setattr(igc, "_handle", lambda stream, dev: state["handle"])
    monkeypatch.setattr(igc, "_new", lambda shape, dtype, device, stream: torch.empty(
        shape, dtype=dtype))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    igc.release_workspaces()
    yield state
    igc.release_workspaces()


LIKE = torch.zeros(1)


def test_the_default_streams_is_kept_and_grows(stream):
    a = igc._workspace(None, 1000, LIKE, None)
    assert igc._workspace(None, 500, LIKE, None) is a
    b = igc._workspace(None, 2000, LIKE, None)
    assert b is not a and b.numel() >= 2000
    gone = weakref.ref(a)
    del a
    assert gone() is None
    assert igc._workspace(None, 1000, LIKE, None) is b


def test_other_streams_captures_and_large_ones_are_not_kept(stream):
    """A handle may come to name another stream once its own is destroyed, and a process may
    use many streams: nothing stays for them."""
    refs = []
    for handle in (7, 8, 7):
        stream["handle"] = handle
        refs.append(weakref.ref(igc._workspace(None, 1000, LIKE, None)))
    stream.update(handle=0, capturing=True)
    refs.append(weakref.ref(igc._workspace(None, 1000, LIKE, None)))
    stream["capturing"] = False
    refs.append(weakref.ref(igc._workspace(None, 33 * MB, LIKE, None)))
    refs.append(weakref.ref(igc._workspace(None, 1000, LIKE, 5)))   # a stream by argument
    assert all(r() is None for r in refs)


def test_release_drops_every_threads(stream):
    mine = weakref.ref(igc._workspace(None, 1000, LIKE, None))
    theirs, go, done = [], threading.Event(), threading.Event()

    def work():
        theirs.append(weakref.ref(igc._workspace(None, 1000, LIKE, None)))
        done.set()
        go.wait(30)

    t = threading.Thread(target=work)
    t.start()
    assert done.wait(30)
    assert mine() is not None and theirs[0]() is not None and theirs[0]() is not mine()
    igc.release_workspaces()
    assert mine() is None and theirs[0]() is None
    go.set()
    t.join()


def test_a_threads_goes_with_it(stream):
    refs = []
    t = threading.Thread(target=lambda: refs.append(
        weakref.ref(igc._workspace(None, 1000, LIKE, None))))
    t.start()
    t.join()
    assert refs[0]() is None
