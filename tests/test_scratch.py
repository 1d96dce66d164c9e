"""Whose device scratch a call takes.  The buffers are made on the CPU here: who gets which is the host's business."""
import threading
import types

import pytest
import torch

import lossless_draft_verification_online_amd as sdv

CPU = torch.device("cpu")


def drafting(monkeypatch):
    monkeypatch.setattr(sdv, "_CAPTURING", lambda: False)
    monkeypatch.setattr(sdv, "_SCRATCH", {})
    return lambda nbytes, stream=7: sdv._scratch(nbytes, CPU, 0, stream)


def verification(monkeypatch):
    monkeypatch.setattr(sdv, "_WORKSPACE", {})

    def take(nbytes, stream=7):
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device: types.SimpleNamespace(cuda_stream=stream))
        return sdv._workspace(nbytes, CPU)

    return take


@pytest.fixture(params=[drafting, verification])
def take(request, monkeypatch):
    return request.param(monkeypatch)


def in_thread(f):
    res = []
    t = threading.Thread(target=lambda: res.append(f()))
    t.start()
    t.join()
    return res[0]


def test_calls_of_one_thread_share_a_buffer_that_grows(take):
    first = take(1000)
    assert take(500) is first and take(1000) is first
    assert take(2000).numel() >= 2000 and take(2000) is not first
    assert take(1000, stream=8) is not take(1000)


def test_threads_on_one_stream_have_their_own(take):
    """Two threads' calls on one stream may alternate their launches."""
    barrier = threading.Barrier(3)
    got = []

    def call():
        ws = take(1000)
        barrier.wait()  # all alive at once
        got.append((ws.data_ptr(), take(1000).data_ptr()))
        barrier.wait()

    threads = [threading.Thread(target=call) for _ in range(2)]
    for t in threads:
        t.start()
    mine = take(1000)
    barrier.wait()
    barrier.wait()
    for t in threads:
        t.join()
    assert len({a for a, _ in got} | {mine.data_ptr()}) == 3 and all(a == b for a, b in got)


def test_a_thread_that_ended_leaves_the_others_theirs(take):
    mine = take(1000)
    in_thread(lambda: take(4000))
    assert take(1000) is mine
