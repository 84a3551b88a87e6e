"""Host side of the serving calls: the workspaces that they keep, the scalars that they take and what they
refuse before any device work. No GPU: the device is the CPU and the stream a number of the test's."""

import gc
import threading
import weakref

import numpy as np
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


class Recorder:
    """Stands in for the library: every call returns OK and leaves its arguments, as ctypes converts them."""

    def __init__(self, real):
        self.calls = {}
        for name in ("diffattn_chunk_paged", "diffattn_chunk_paged_fp8", "diffattn_kv_append_chunk_paged",
                     "diffattn_kv_append_chunk_paged_fp8"):
            types = getattr(real, name).argtypes

            def call(*args, name=name, types=types):
                assert len(args) == len(types)
                for a, t in zip(args, types):
                    t.from_param(a)  # raises what the call would
                self.calls[name] = args
                return da.OK
            setattr(self, name, call)


@pytest.mark.parametrize("kind", [np.float32, np.float64, lambda x: torch.tensor(x, dtype=torch.float64), float])
def test_scalars_of_every_kind(host, monkeypatch, kind):
    """lam, lam_init, eps and the scales as Python, NumPy or 0-dim torch numbers, L and kv_group as NumPy or torch
    integers, as the one-token calls take them."""
    lib = Recorder(da.load_library())
    monkeypatch.setattr(da, "_lib", lib)
    monkeypatch.setattr(da, "_elsewhere", lambda dev, stream: None)
    f8, i32 = torch.float8_e4m3fn, torch.int32
    host.dev = torch.device("cpu")
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    k, v = torch.zeros(2, 2, 64, 64, dtype=torch.uint8).view(f8), torch.zeros(2, 2, 64, 128, dtype=torch.uint8).view(f8)
    rest = (torch.zeros(1, 2, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32))
    scales = tuple(kind(s) for s in (0.5, 0.25, 2.0))
    da.diffattn_kv_append_chunk_paged(q[:, :2], q[:, :2], torch.zeros(3, 2, 128, dtype=torch.bfloat16), k, k, v, *rest, scales=scales)
    assert lib.calls["diffattn_kv_append_chunk_paged_fp8"][-4:-1] == (0.5, 0.25, 2.0)
    ints = (int, np.int64, lambda x: torch.tensor(x))
    for to_int in ints:
        da.diffattn_chunk_paged(q, q, k, k, v, *rest, kind(0.75), kind(0.5), to_int(100), to_int(2), kind(0.125), scales=scales,
                                ws=torch.zeros(64, dtype=torch.uint8))
        args = lib.calls["diffattn_chunk_paged_fp8"]
        assert args[16:22] == (2, 64, 128, 0.75, 0.5, 0.125) and args[22:25] == (0.5, 0.25, 2.0) and args[10] == 100
    with pytest.raises(ValueError, match="scales"):
        da.diffattn_chunk_paged(q, q, k, k, v, *rest, 0.5, 0.5, 100, 2, scales=scales[:2])


def _chunk_args(dev="cpu"):
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    k, v = (torch.zeros(2, 2, 64, n, dtype=torch.bfloat16) for n in (64, 128))
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    return q, q, k, k, v, i32(1, 2), i32(2), i32(1), 0.5, 0.5, 100, 2


ELSEWHERE = torch.device("meta")  # another device than the operands', without memory


def test_workspaces_of_another_device_are_refused(host, monkeypatch):
    """A kernel would write to whatever address they have."""
    lib = Recorder(da.load_library())
    monkeypatch.setattr(da, "_lib", lib)
    monkeypatch.setattr(da, "_elsewhere", lambda dev, stream: None)
    da.diffattn_chunk_paged(*_chunk_args(), ws=torch.zeros(1 << 20, dtype=torch.uint8))
    lib.calls.clear()
    for ws in (torch.empty(1 << 20, dtype=torch.uint8, device=ELSEWHERE), torch.zeros(1, dtype=torch.uint8).expand(1 << 20),
               torch.zeros(1 << 20, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="ws"):
            da.diffattn_chunk_paged(*_chunk_args(), ws=ws)
    assert not lib.calls


def test_served_models_refuse_operands_of_another_device(monkeypatch):
    """Workspace, weights and gains, before any launch: the projections take no look at their devices."""
    monkeypatch.setattr(da, "_elsewhere", lambda dev, stream: None)
    launched = []
    for name in ("gemm", "gemm_residual", "gemm_swiglu", "add_rmsnorm", "diffattn_rope", "diffattn_kv_append_chunk_paged",
                 "diffattn_chunk_paged"):
        monkeypatch.setattr(da, name, lambda *a, name=name, **k: launched.append(name))
    bf = torch.bfloat16
    x, w_qkv, w_o = torch.zeros(3, 256, dtype=bf), torch.zeros(256, 512, dtype=bf), torch.zeros(128, 256, dtype=bf)
    w_gu, w_down, ws = torch.zeros(256, 256, dtype=bf), torch.zeros(128, 256, dtype=bf), torch.zeros(1 << 20, dtype=torch.uint8)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    rest = (1, [torch.zeros(2, 1, 64, n, dtype=bf) for n in (64, 64, 128)], i32(1, 2), i32(2), i32(1), 0.5, 0.5, 100)
    away = lambda t: torch.empty(t.shape, dtype=t.dtype, device=ELSEWHERE)  # noqa: E731
    gain, one = torch.ones(256), torch.ones(1)
    bad = [lambda: da.module_serve(x, away(w_qkv), w_o, *rest, ws=ws), lambda: da.module_serve(x, w_qkv, away(w_o), *rest, ws=ws),
           lambda: da.module_serve(x, w_qkv, w_o, *rest, ws=away(ws)),
           lambda: da.module_serve(x, w_qkv, w_o, *rest, ws=torch.zeros(1, dtype=torch.uint8).expand(1 << 20))]
    for i, w in enumerate((w_qkv, w_o, w_gu, w_down)):
        four = [w_qkv, w_o, w_gu, w_down]
        four[i] = away(w)
        bad.append(lambda four=four: da.layer_serve(x, *four, *rest, ws=ws))
    for g in (away(gain), one, gain.to(bf), torch.ones(512)[::2]):
        bad.append(lambda g=g: da.layer_serve(x, w_qkv, w_o, w_gu, w_down, *rest, ws=ws, norm1_weight=g))
        bad.append(lambda g=g: da.layer_serve(x, w_qkv, w_o, w_gu, w_down, *rest, ws=ws, norm2_weight=g))
    for call in bad:
        with pytest.raises(ValueError):
            call()
    assert not launched


def test_streams_of_another_device_are_refused(monkeypatch):
    """The call would run on the operands' device's current stream, in no order with the one asked for."""
    entered = []
    monkeypatch.setattr(torch.cuda, "stream", lambda s: entered.append(s))
    monkeypatch.setattr(da, "_current_device", lambda: 0)
    stream = lambda i: type("Stream", (), {"device": torch.device("cuda", i)})()  # noqa: E731
    for at in (1, 3):
        with pytest.raises(ValueError, match="stream"):
            da._elsewhere(torch.device("cuda", 0), stream(at))
    assert not entered
    same = stream(0)
    da._elsewhere(torch.device("cuda", 0), same)
    assert entered == [same] and da._elsewhere(torch.device("cuda", 0), None) is None


def test_rope_plans_have_their_whole_table():
    """A kernel reads rotary_dim / 2 values behind the table's address."""
    table, magnitude = da.rope_freqs(64)
    da.RopePlan(table, 64, False, magnitude)
    for bad in (table[:31], table[:16], table.to(torch.int32), table.double(), torch.zeros(64, dtype=torch.int64)[::2],
                table.view(2, 16), torch.zeros(1, dtype=torch.int64).expand(32)):
        with pytest.raises(ValueError, match="freqs"):
            da.RopePlan(bad, 64, False, magnitude)
    with pytest.raises(ValueError, match="operands"):
        da.diffattn_rope([], da.RopePlan(table, 64, False, magnitude))
