"""Edges of the chunk attention over an fp8 cache, on the GPU, against the float64 definition: score
scales at the ends of what the call takes, small weights behind a large one, and each of its three
kernels (few rows, 128-row tiles, the CTA pair's) with the options that the bf16 tests cover."""

import ctypes
import math

import pytest
import torch

import differential_attention_02_gb300 as da
import serving_reference as ref
from parity import errors
from test_gpu_chunk import LAM, LI, Case

pytestmark = pytest.mark.gpu
F8, BF = torch.float8_e4m3fn, torch.bfloat16

# New tokens and lengths of batches that go to the kernel for tiles of few rows, to it and the 128-row
# one in one call, to the 128-row one alone, and to the CTA pair's (d = 128).
KINDS = {"few": (64, [1, 5, 2], [65, 300, 700]), "both": (64, [1, 9, 2, 1], [65, 300, 700, 130]),
         "many": (64, [60, 1, 130], [60, 333, 500]), "wide": (128, [60, 1, 13], [60, 333, 500])}
kinds = pytest.mark.parametrize("kind", list(KINDS))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from differential_attention_02_gb300 import build
    build.build()
    da.load_library()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _case(kind, seed=0, group=2, **kw):
    d, n, lens = KINDS[kind]
    return Case(n, lens, 2 * group, group, d, True, seed=seed, **kw)


@pytest.mark.parametrize("k_scale", [1e-30, 1e-38, 1e-45])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -20, 1.0])
@kinds
def test_scores_that_vanish(kind, size, k_scale):
    """Rows of zeros, small rows and ordinary ones over K scales so small that every score is 0 to fp32:
    uniform weights over the visible keys (the masked ones stay out)."""
    c = _case(kind, seed=1)
    c.q = [(x.float() * size).to(BF) for x in c.q]
    c.scales = (k_scale, k_scale, ref.SCALES[2])
    c.check(c.run(), f"{kind} rows of {size}, K scale {k_scale}")


@kinds
def test_tiny_queries_and_a_large_scale(kind):
    """Query rows at the lower end of bf16's range against a K scale that brings their scores back to unit
    size: the rows' power of two has to cover the whole range."""
    c = _case(kind, seed=2)
    c.q = [(x.float() * 2.0 ** -122).to(BF) for x in c.q]
    g = torch.Generator().manual_seed(3)
    c.pools[:2] = [(torch.randn(p.shape, generator=g) * 16).to(F8) for p in c.pools[:2]]
    c.scales = (2.0 ** 118, 2.0 ** 118, ref.SCALES[2])
    c.check(c.run(), kind)


@pytest.mark.parametrize("at", [3, 5000])
@pytest.mark.parametrize("nats", [15.0, 17.0, 26 * math.log(2)])
@pytest.mark.parametrize("d,n", [(64, 2), (64, 20), (128, 2), (128, 20)])
def test_tail_behind_a_sink(d, n, nats, at):
    """One key far above a tail of 8191 whose scores are standard normal, its V row zero: the output is the
    tail's alone. A weight of the product is off by at most 2^-32 of the row's largest (half a step of
    fp16's smallest values, 2^-25, where the largest stands at 2^7 or more), so by 2^-32 / sqrt 3 RMS, and the
    tail's weights are e^(1 - nats) RMS (E[e^2z] = e^2), 0.2 nats less where the sink's e4m3 row is
    rounded up. The values are independent of both, so the output's relative RMS error is the weights'.
    Beside it, in quadrature, the path's own bound."""
    c = Case([n], [8192], 2, 1, d, True, seed=70)
    g = torch.Generator().manual_seed(4)
    u = torch.randn(d, generator=g)
    u = u / u.norm()
    for q in c.q:
        q.copy_((4 * d ** 0.5 * u + 0.02 * torch.randn(q.shape, generator=g)).to(BF))
    for p, s in zip(c.pools[:2], c.scales):
        p.copy_((torch.randn(p.shape, generator=g) * 0.25 / s).clamp(-448, 448).to(F8))
        p[int(c.table[0, at // 64]), :, at % 64] = (nats / 4 * u / s).clamp(-448, 448).to(F8)
    c.pools[2].view(torch.uint8)[int(c.table[0, at // 64]), :, at % 64] = 0
    _, rms = errors(c.run(), c.want().numpy())
    tol = math.hypot(3e-3, 2.0 ** -32 / math.sqrt(3) / math.exp(1 - nats - 0.2))
    print(f"d{d} n{n} {nats:.1f} nats: {rms:.2e} of {tol:.2e}")
    assert rms <= tol, f"rel-RMS {rms:.3e} against {tol:.3e}"


def test_error_word_of_a_kept_workspace():
    """A wait that runs out (the library's own test of it: a barrier that nothing completes, 1 s) in the
    workspace that a call without `ws` kept; the next call is right and leaves no error."""
    da.release_workspaces()
    c = _case("both", seed=6)
    dev = [x.cuda() for x in c.q] + [p.cuda() for p in c.pools]
    rest = (c.table.cuda(), _i32(c.starts), _i32(c.lens), LAM, LI)

    def call():
        return da.diffattn_chunk_paged(*dev, *rest, L=c.L, kv_group=2, scales=c.scales)
    assert da.kept_workspace() is None
    want = call()
    ws = da.kept_workspace()
    assert da.read_error(ws) == 0
    stream = torch.cuda.current_stream().cuda_stream
    assert da.load_library().diffattn_selftest_timeout(ctypes.c_void_p(ws.data_ptr()), ws.numel(), ctypes.c_void_p(stream)) == da.OK
    assert da.read_error(da.kept_workspace()) == (0x7F << 8) | 1
    assert torch.equal(call(), want) and da.kept_workspace() is ws and da.read_error(ws) == 0
