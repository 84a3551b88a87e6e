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


@kinds
@pytest.mark.parametrize("out_dtype", [torch.float32, BF, torch.float16])
def test_output_types_gain_and_layouts(kind, out_dtype):
    """16-bit outputs, the RMSNorm gain, queries as views of a projection and with heads outermost, pages whose
    rows do not follow one another."""
    c = _case(kind, seed=4)
    d = c.d
    gain = torch.linspace(0.5, 1.5, 2 * d)
    got = c.run(out_dtype=out_dtype, norm_weight=gain.cuda())
    want = c.want(norm_weight=gain)
    c.check((got.float() / gain.cuda()).to(out_dtype), f"{kind} gain", want / gain.double())
    proj = torch.cat(c.q, -1).cuda()
    heads = [x.transpose(0, 1).contiguous().transpose(0, 1).cuda() for x in c.q]
    padded = []
    for p in c.pools:
        big = torch.full((p.shape[0], p.shape[1], 66, p.shape[3] + 16), 0x7F, dtype=torch.uint8, device="cuda")  # NaN
        big[:, :, :64, :p.shape[3]] = p.cuda().view(torch.uint8)
        padded.append(big.view(F8)[:, :, :64, :p.shape[3]])
    plain = c.run(out_dtype=out_dtype)
    for q in ((proj[..., :d], proj[..., d:]), heads):
        alt = da.diffattn_chunk_paged(*q, *padded, c.table.cuda(), _i32(c.starts), _i32(c.lens), LAM, LI, L=c.L, kv_group=2,
                                      out_dtype=out_dtype, scales=c.scales)
        assert torch.equal(alt, plain)


@pytest.mark.parametrize("kind,n", [("few", [5, 4, 3, 4]), ("both", [5, 4, 3, 20]), ("many", [5, 40, 3, 140]),
                                    ("wide", [5, 4, 3, 140])])
def test_rows_without_keys_and_clamped_lengths(kind, n):
    """Lengths below the chunk (rows before position 0 see nothing), zero and negative ones, and lengths
    past L, which are clamped to it; the kernels' accumulators hold another call's values before."""
    d = KINDS[kind][0]
    full = [n[0], n[1], n[2], 300]
    c = Case(n, full, 2, 1, d, True, seed=5)
    c.run()  # leaves tensor memory and the workspace full
    lens = [3, 0, -7, 300]
    got = c.run(lens=lens)
    assert bool((got[:n[0] - 3] == 0).all()) and bool((got[n[0]:n[0] + n[1] + n[2]] == 0).all())
    c.check(got, f"{kind} short lengths", c.want(lens=[3, 0, 0, 300]))
    c.check(c.run(lens=[*full[:3], 10_000], L=300), f"{kind} clamped")


@pytest.mark.parametrize("d,group,n", [(64, g, [1, 50, 9]) for g in (3, 5, 7, 16, 100)] +
                         [(128, g, [1, 50, 9]) for g in (3, 6, 100)] + [(64, g, [1, 1, 1, 0]) for g in (3, 5, 7, 16)])
def test_group_sizes(d, group, n):
    """Groups that divide a tile's rows and groups that leave some unused; n of at most a token: few rows."""
    c = Case(n, [77, 50, 300, 64][:len(n)], group * (2 if group < 20 else 1), group, d, True, seed=group)
    c.check(c.run(), f"group {group}")


@kinds
def test_deterministic(kind):
    d, n, _ = KINDS[kind]
    c = Case(n, [6000, 5000, 2300, 900][:len(n)], 4, 2, d, True, seed=8)
    a = c.run()
    c.check(a, kind)
    for _ in range(3):
        assert torch.equal(c.run(), a)


def test_captured_call_whose_tiles_change_lists():
    """A call of two lists, captured, replayed with starts and lengths that move tiles from one to the other and
    leave either empty."""
    c = Case([1, 9, 2, 1], [900, 3000, 700, 130], 4, 2, 64, True, seed=9)
    dev = dict(q=[x.cuda() for x in c.q], pools=[p.cuda() for p in c.pools], table=c.table.cuda(), start=_i32(c.starts),
               lens=_i32(c.lens), out=torch.empty(c.T, 4, 128, device="cuda"))

    def call():
        da.diffattn_chunk_paged(*dev["q"], *dev["pools"], dev["table"], dev["start"], dev["lens"], LAM, LI, L=c.L, kv_group=2,
                                out=dev["out"], scales=c.scales)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for starts, lens in ((c.starts, c.lens), ([0, 9, 10, 12, 13], [900, 400, 700, 130]), ([0, 4, 7, 10, 13], [900, 3000, 700, 130]),
                         ([0, 13, 13, 13, 13], [850, 3000, 700, 130]), ([0, 0, 1, 3, 3], [900, 3000, 700, 130])):
        dev["start"].copy_(_i32(starts))
        dev["lens"].copy_(_i32(lens))
        dev["out"].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        want = ref.chunk_attention(*c.q, c.pools, c.table, starts, lens, LAM, LI, group=2, scales=c.scales)
        c.starts = starts
        c.check(dev["out"], f"{starts}", want)
        assert bool((dev["out"][starts[-1]:] == 7.0).all())


@pytest.mark.parametrize("scale", [0.0113, 1.0, 2.0 ** -61, 2.0 ** 61])
def test_append_fp8_stores_nan_as_the_single_token_append(scale):
    """NaN of both signs and any payload among ordinary values and infinities: e4m3's NaN, the code of the
    single-token append, with the quotient by the inverse (the first two scales) and by division."""
    bits = torch.cat([torch.arange(0x7F81, 0x8000), torch.arange(0xFF81, 0x10000), torch.tensor([0x7F80, 0xFF80])])
    nan = bits.to(torch.int32).to(torch.int16).view(BF)
    x = torch.randn(2, 1, 256, generator=torch.Generator().manual_seed(1)).to(BF)
    x.view(-1)[::2] = nan[:256]
    rows = [t.cuda() for t in (x[..., :64], x[..., 64:128], x[..., 128:])]
    make = lambda: [torch.zeros(1, 1, 64, w, dtype=torch.uint8, device="cuda") for w in (64, 64, 128)]  # noqa: E731
    a, b = make(), make()
    table = _i32([[0]])
    da.diffattn_kv_append_chunk_paged(*rows, *a, table, _i32([0, 2]), _i32([2]), scales=(scale,) * 3)
    for t in range(2):
        da.diffattn_kv_append_paged(*(r[t:t + 1].contiguous() for r in rows), *b, table, _i32([t + 1]), scales=(scale,) * 3)
    for p, q, r in zip(a, b, rows):
        assert torch.equal(p, q)
        assert torch.equal((p[0, 0, :2] & 0x7F) == 0x7F, r[:, 0].isnan())


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
