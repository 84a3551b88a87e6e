"""Host-side checks of the rotary positions, the ragged append and the chunk attention that
need no GPU: the frequency table, the workspace bounds and the refusals before any launch."""

import ctypes

import pytest
import torch

import differential_attention_02_gb300 as da
from differential_attention_02_gb300 import build as dab
from serving_reference import frequencies


@pytest.fixture(scope="module")
def lib():
    dab.build()
    return da.load_library()


vp = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731


@pytest.mark.parametrize("r", [8, 48, 64, 128])
@pytest.mark.parametrize("scaling", ["none", "linear", "ramp"])
@pytest.mark.parametrize("base", [1.0, 10000.0, 500000.0])
def test_frequency_table(lib, r, scaling, base):
    table, magnitude = da.rope_freqs(r, base, scaling, factor=8.0, original_length=4096)
    f, m = frequencies(r, base, scaling, 8.0, 4096)
    got = [(int(x) & (2 ** 64 - 1)) / 2.0 ** 64 * 2 * 3.141592653589793 for x in table]
    # both sides compute in double: a handful of roundings of 2^-53 relative, and 2^-64 turns of truncation
    torch.testing.assert_close(torch.tensor(got, dtype=torch.float64), f, rtol=1e-14, atol=1e-18)
    assert magnitude == pytest.approx(m, rel=1e-7)


def test_frequency_table_refusals(lib):
    buf, mag = (ctypes.c_uint64 * 64)(), ctypes.c_float()

    def call(r=64, base=1e4, kind=0, factor=8.0, orig=4096, fast=32.0, slow=1.0, out=buf, m=mag):
        return lib.diffattn_rope_freqs(r, base, kind, factor, orig, fast, slow,
                                       None if out is None else ctypes.cast(out, ctypes.c_void_p),
                                       None if m is None else ctypes.byref(m))
    assert call() == da.OK and call(kind=1) == da.OK and call(kind=2) == da.OK
    assert call(factor=0.0) == da.OK                           # not used by the plain kind
    for kw in (dict(r=0), dict(r=12), dict(r=-8), dict(base=0.5), dict(base=float("nan")), dict(base=float("inf")),
               dict(kind=3), dict(kind=-1), dict(kind=1, factor=0.5), dict(kind=1, factor=float("nan")),
               dict(kind=2, orig=0), dict(kind=2, fast=1.0, slow=1.0), dict(kind=2, slow=-1.0), dict(out=None), dict(m=None)):
        assert call(**kw) == da.ERR_INVALID_ARG, kw
    with pytest.raises(ValueError, match="scaling"):
        da.rope_freqs(64, scaling="other")


def _tensor(ptr=0x10000, sb=4096, sh=1024, sn=64):
    return da.Tensor4(ptr, sb, sh, sn)


def test_rope_refusals(lib):
    def call(x=None, y=None, heads=(2, 2), count=2, pos=None, B=1, N=4, d=64, rot=None, ind=da.BF16, outd=da.BF16, **null):
        t, o = [_tensor()] * 4, [_tensor(0x20000)] * 4
        if x is not None:
            t = [x] * 4
        if y is not None:
            o = [y] * 4
        rot = rot or da.Rotation(0x30000, 64, 0, 1.0)
        h = (ctypes.c_int * 4)(*(list(heads) + [0] * (4 - len(heads))))
        arr = da.Tensor4 * 4
        return lib.diffattn_rope(None if null.get("no_in") else bytes(arr(*t)), None if null.get("no_out") else bytes(arr(*o)),
                                 None if null.get("no_heads") else bytes(h), count, vp(pos), B, N, d,
                                 None if null.get("no_rot") else ctypes.byref(rot), 0, ind, outd, None)
    assert call(B=0) == da.OK and call(N=0) == da.OK and call(heads=(0, 0)) == da.OK
    for kw in (dict(B=-1), dict(N=-1), dict(d=60), dict(d=264), dict(d=0), dict(count=0), dict(count=5), dict(heads=(-1, 2)),
               dict(ind=7), dict(outd=-1), dict(no_in=1), dict(no_out=1), dict(no_heads=1), dict(no_rot=1),
               dict(rot=da.Rotation(0, 64, 0, 1.0)), dict(rot=da.Rotation(0x30004, 64, 0, 1.0)),
               dict(rot=da.Rotation(0x30000, 72, 0, 1.0)), dict(rot=da.Rotation(0x30000, 12, 0, 1.0)),
               dict(rot=da.Rotation(0x30000, 0, 0, 1.0)), dict(rot=da.Rotation(0x30000, 64, 0, float("inf"))),
               dict(x=_tensor(0)), dict(x=_tensor(0x10008)), dict(x=_tensor(sn=60)), dict(x=_tensor(sh=-1024)),
               dict(y=_tensor(0)), dict(y=_tensor(0x20004)),
               dict(y=_tensor(0x10000, sn=72)),                      # in place with other strides
               dict(y=_tensor(0x10000), outd=da.F32),                # in place with another type
               dict(B=1 << 20, N=1 << 20)):
        assert call(**kw) == da.ERR_INVALID_ARG, kw


def _append(lib, fp8=False, **kw):
    a = dict(T=4, B=2, Hk=2, d=64, Dv=128, maxp=4, pages=8, ind=da.BF16, new=_tensor(), vnew=_tensor(sn=128),
             k=_tensor(sn=64, sh=4096, sb=8192), v=_tensor(sn=128, sh=8192, sb=16384), table=0x3000, start=0x3100, lens=0x3200,
             rot=None, s=0.01)
    a.update(kw)
    args = [a["new"], a["new"], a["vnew"], a["ind"], a["k"], a["k"], a["v"], vp(a["table"]), a["maxp"], a["pages"],
            vp(a["start"]), vp(a["lens"]), None if a["rot"] is None else ctypes.byref(a["rot"]), a["T"], a["B"], a["Hk"],
            a["d"], a["Dv"]]
    if fp8:
        return lib.diffattn_kv_append_chunk_paged_fp8(*args, a["s"], 0.01, 0.01, None)
    return lib.diffattn_kv_append_chunk_paged(*args, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_refusals(lib, fp8):
    call = lambda **kw: _append(lib, fp8, **kw)  # noqa: E731
    assert call(T=0) == da.OK and call(B=0) == da.OK and call(Hk=0) == da.OK
    for kw in (dict(T=-1), dict(B=-1), dict(Hk=-1), dict(d=60), dict(Dv=4), dict(maxp=0), dict(pages=0), dict(ind=da.F32),
               dict(ind=9), dict(new=_tensor(0)), dict(new=_tensor(0x10002)), dict(new=_tensor(sn=68)), dict(vnew=_tensor(sn=64)),
               dict(k=_tensor(sn=48)), dict(v=_tensor(0)), dict(table=None), dict(start=None), dict(lens=None),
               dict(rot=da.Rotation(0x30000, 72, 0, 1.0)), dict(rot=da.Rotation(0, 64, 0, 1.0))):
        assert call(**kw) == da.ERR_INVALID_ARG, kw
    if fp8:
        for s in (0.0, -1.0, float("nan"), float("inf")):
            assert call(s=s) == da.ERR_INVALID_ARG


def _chunk(lib, fp8=False, **kw):
    a = dict(T=4, B=2, H=4, group=2, d=64, Dv=128, L=200, maxp=4, pages=8, q=_tensor(), k=_tensor(sn=64, sh=4096, sb=8192),
             v=_tensor(sn=128, sh=8192, sb=16384), table=0x3000, start=0x3100, lens=0x3200, out=0x40000, w=None, lam=0.5,
             li=0.2, eps=1e-5, outd=da.BF16, ws=0x100000, wsb=1 << 34, s=0.01)
    a.update(kw)
    args = [a["q"], a["q"], a["k"], a["k"], a["v"], vp(a["table"]), a["maxp"], a["pages"], vp(a["start"]), vp(a["lens"]),
            a["L"], vp(a["out"]), vp(a["w"]), a["T"], a["B"], a["H"], a["group"], a["d"], a["Dv"], a["lam"], a["li"], a["eps"]]
    tail = [a["outd"], vp(a["ws"]), a["wsb"], None]
    if fp8:
        return lib.diffattn_chunk_paged_fp8(*args, a["s"], 0.01, 0.01, *tail)
    return lib.diffattn_chunk_paged(*args, *tail)


@pytest.mark.parametrize("fp8", [False, True])
def test_chunk_refusals(lib, fp8):
    call = lambda **kw: _chunk(lib, fp8, **kw)  # noqa: E731
    assert call(T=0) == da.OK and call(B=0) == da.OK and call(H=0) == da.OK
    for kw in (dict(T=-1), dict(B=-1), dict(H=-1), dict(L=0), dict(group=0), dict(group=3), dict(maxp=0), dict(pages=0),
               dict(L=257), dict(outd=5), dict(lam=float("nan")), dict(li=float("inf")), dict(eps=-1.0), dict(q=_tensor(0)),
               dict(q=_tensor(0x10004)), dict(q=_tensor(sn=56)), dict(q=_tensor(sh=1004)), dict(k=_tensor(sn=60)),
               dict(v=_tensor(0)), dict(table=None), dict(start=None), dict(lens=None), dict(out=None), dict(out=0x40008),
               dict(w=0x50004)):
        assert call(**kw) == da.ERR_INVALID_ARG, kw
    assert call(d=32, Dv=64) == da.ERR_UNSUPPORTED
    assert call(d=64, Dv=64) == da.ERR_UNSUPPORTED
    assert call(H=256, group=256) == da.ERR_UNSUPPORTED
    need = da.chunk_workspace_bytes(4, 2, 4, 2, 200, 64, 128)
    for kw in (dict(ws=None), dict(ws=0x100010), dict(wsb=need - 1), dict(wsb=0)):
        assert call(**kw) == da.ERR_WORKSPACE, kw
    if fp8:
        assert call(s=0.0) == da.ERR_INVALID_ARG


def test_chunk_workspace_sizes(lib):
    n = ctypes.c_size_t()
    size = lambda *a: lib.diffattn_chunk_workspace_size(*a, ctypes.byref(n))  # noqa: E731
    assert size(0, 2, 4, 2, 100, 64, 128) == da.OK and n.value == 256
    assert size(4, 2, 4, 3, 100, 64, 128) == da.ERR_INVALID_ARG
    assert size(4, 2, 4, 2, 0, 64, 128) == da.ERR_INVALID_ARG
    assert size(-4, 2, 4, 2, 10, 64, 128) == da.ERR_INVALID_ARG
    assert size(4, 2, 256, 256, 10, 64, 128) == da.ERR_UNSUPPORTED
    assert lib.diffattn_chunk_workspace_size(4, 2, 4, 2, 10, 64, 128, None) == da.ERR_INVALID_ARG
    # one key tile at most: nothing to split, so only the plan's lists
    assert size(4, 2, 4, 2, 128, 64, 128) == da.OK and n.value < 4096
    # few rows make small slots: 2 maps x 2 heads x 1 token of up to 4 x 152 states of Dv floats and their statistics
    assert size(1, 1, 4, 2, 100000, 64, 128) == da.OK and n.value < 1 << 21


def test_python_wrappers_refuse_before_device_work(lib):
    bf, i32 = torch.bfloat16, torch.int32
    q = torch.zeros(3, 4, 64, dtype=bf)
    k, v = torch.zeros(5, 2, 64, 64, dtype=bf), torch.zeros(5, 2, 64, 128, dtype=bf)
    table, start, lens = torch.zeros(1, 4, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32)
    plan = da.RopePlan(torch.zeros(32, dtype=torch.int64), 64, False, 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        da.diffattn_chunk_paged(q, q, k, k, v, table, start, lens, 0.5, 0.2, L=64, kv_group=2)
    with pytest.raises(ValueError, match="CUDA"):
        da.diffattn_rope([torch.zeros(1, 2, 3, 64, dtype=bf)], plan)
    with pytest.raises(ValueError, match="CUDA"):
        da.diffattn_kv_append_chunk_paged(q[:, :2], q[:, :2], torch.zeros(3, 2, 128, dtype=bf), k, k, v, table, start, lens)


def test_serving_models_refuse_before_device_work(lib):
    """The served module and layer check shapes on the host; tensors on the CPU never reach a kernel."""
    x, w, wo = torch.zeros(3, 64), torch.zeros(64, 512), torch.zeros(128, 64)
    pages = [torch.zeros(2, 1, 64, n, dtype=torch.bfloat16) for n in (64, 64, 128)]
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    args = (pages, i32(0).view(1, 1), i32(0, 3), i32(3), 0.5, 0.5, 3)
    with pytest.raises(ValueError, match="CUDA"):
        da.module_serve(x, w, wo, 1, *args)
    with pytest.raises(ValueError, match="CUDA"):
        da.layer_serve(x, w, wo, w, wo, 1, *args)
