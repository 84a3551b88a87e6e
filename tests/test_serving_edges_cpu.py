"""Host side of the serving calls: the workspaces that they keep, the scalars that they take and what they
refuse before any device work. No GPU: the device is the CPU and the stream a number of the test's."""

import gc
import threading
import weakref

import pytest
import torch

import differential_attention_02_gb300 as da


class Host:
    """Stands in for the device: `stream` is the current raw stream."""

    def __init__(self, monkeypatch):
        self.dev, self.stream = torch.device("cpu", 0), 1
        monkeypatch.setattr(da, "_raw_stream", lambda index: self.stream)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    def workspace(self, stream, nbytes=1000):
        self.stream = stream
        return da._serving_workspace(nbytes, self.dev)


@pytest.fixture
def host(monkeypatch):
    yield Host(monkeypatch)
    da.release_workspaces()


def test_kept_workspaces_are_of_a_thread_and_a_stream(host):
    a = host.workspace(1)
    assert host.workspace(1) is a and host.workspace(2) is not a
    assert host.workspace(1, 500) is a and host.workspace(1, 5000).numel() >= 5000
    assert host.workspace(1).data_ptr() % 256 == 0
    other = []
    t = threading.Thread(target=lambda: other.append(da._serving_workspace(1000, host.dev).data_ptr()))
    mine = host.workspace(1)
    t.start()
    t.join()
    assert other[0] != mine.data_ptr()


def test_kept_workspaces_end_with_their_thread(host):
    refs = []
    for _ in range(3):
        t = threading.Thread(target=lambda: refs.append(weakref.ref(da._serving_workspace(1000, host.dev))))
        t.start()
        t.join()
    del t
    gc.collect()
    assert all(r() is None for r in refs)


def test_kept_workspaces_are_bounded(host):
    refs = [weakref.ref(host.workspace(s)) for s in range(1, 41)]
    gc.collect()
    alive = [r() is not None for r in refs]
    assert alive == [False] * 36 + [True] * 4
    host.workspace(40, 9000)  # a stream's own growth drops no other's
    assert all(r() is not None for r in refs[36:39])


def test_kept_workspace_is_reachable(host):
    host.stream = 7
    assert da.kept_workspace() is None
    a = host.workspace(7)
    assert da.kept_workspace() is a and da.kept_workspace("cuda:0") is a and da.kept_workspace("cuda") is a
    host.stream = 8
    assert da.kept_workspace() is None
    assert da.kept_workspace(stream=type("Stream", (), {"cuda_stream": 7})()) is a
    da.release_workspaces()
    assert da.kept_workspace(stream=type("Stream", (), {"cuda_stream": 7})()) is None
