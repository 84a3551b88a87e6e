"""Differential attention of ragged new tokens over a paged cache, on the GPU, against the
float64 definition.

Tolerance: that of the framework's other 16-bit attention paths (parity.py): max-abs 1e-2
and relative RMS 3e-3 on fp32 outputs. Where it comes from: P is rounded to bf16 (half a
step 2^-8, uniform over a step: 2^-8 / sqrt 3 x 0.72 = 1.6e-3 RMS of a weight), the two maps'
errors add like their values, and the RMSNorm keeps relative errors; everything else is
fp32. Over an fp8 cache P is fp16 (2^-11). 16-bit outputs add half a step of their type."""

import pytest
import torch

import differential_attention_02_gb300 as da
import serving_reference as ref
from parity import assert_bf16_out_parity, assert_bf16_parity

pytestmark = pytest.mark.gpu
F8, BF = torch.float8_e4m3fn, torch.bfloat16
LAM, LI = 0.45, 0.47


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from differential_attention_02_gb300 import build
    build.build()
    da.load_library()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    """A ragged batch: queries and pools on the host, their copies on the GPU."""

    def __init__(self, n_new, lens, H, group, d, fp8=False, seed=0, pad=0, first=0):
        g = torch.Generator().manual_seed(1000 * d + seed)
        self.d, self.Dv, self.H, self.group, self.lens = d, 2 * d, H, group, lens
        self.starts = [first + sum(n_new[:b]) for b in range(len(n_new) + 1)]
        self.T = self.starts[-1] + pad
        self.scales = ref.SCALES if fp8 else None
        self.q = [torch.randn(self.T, H, d, generator=g).to(BF) for _ in range(2)]
        self.pools, self.table = ref.make_pool(lens, H // group, (d, d, 2 * d), F8 if fp8 else BF, seed=seed)
        self.L = max(max(lens), 1)

    def run(self, pools=None, table=None, lens=None, starts=None, ws=None, out_dtype=torch.float32, L=None, **kw):
        ws = ws if ws is not None else da.workspace(
            da.chunk_workspace_bytes(self.T, len(self.lens), self.H, self.group, L or self.L, self.d, self.Dv))
        dev = [p.cuda() for p in (pools or self.pools)]
        got = da.diffattn_chunk_paged(*(x.cuda() for x in self.q), *dev, (self.table if table is None else table).cuda(),
                                      _i32(starts or self.starts), _i32(lens or self.lens), LAM, LI, L=L or self.L,
                                      kv_group=self.group, ws=ws, out_dtype=out_dtype, scales=self.scales, **kw)
        assert da.read_error(ws) == 0
        return got

    def want(self, **kw):
        return ref.chunk_attention(*self.q, self.pools, self.table, self.starts, kw.pop("lens", self.lens), LAM, LI,
                                   group=self.group, scales=self.scales, **kw)

    def check(self, got, what, want=None):
        rows = slice(self.starts[0], self.starts[-1])
        if got.dtype == torch.float32:
            return assert_bf16_parity(got[rows], (self.want() if want is None else want)[rows].numpy(), what)
        return assert_bf16_out_parity(got[rows].float(), (self.want() if want is None else want)[rows].numpy(), what)


HEADS = [(64, 4, 1), (64, 4, 2), (128, 2, 1), (128, 4, 4)]  # d, H, group


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,H,group", HEADS)
@pytest.mark.parametrize("n,length", [(1, 1), (1, 64), (1, 65), (2, 2), (3, 127), (5, 128), (7, 129), (64, 64), (65, 200),
                                      (127, 127), (128, 128), (129, 129), (129, 1000), (300, 301), (16, 4097)])
def test_one_sequence(fp8, d, H, group, n, length):
    c = Case([n], [length], H, group, d, fp8, seed=n)
    c.check(c.run(), f"d{d} g{group} fp8={fp8} {n}/{length}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,H,group", HEADS)
def test_mixed_batch(fp8, d, H, group):
    """Decoding sequences, chunks, an empty one, a whole prompt; rows of no sequence before and behind."""
    c = Case([1, 200, 0, 1, 33, 130, 1], [700, 200, 50, 1, 1030, 1000, 64], H, group, d, fp8, seed=3, pad=5, first=2)
    out = torch.full((c.T, H, 2 * d), 7.0, device="cuda")
    got = c.run(out=out)
    c.check(got, "mixed")
    assert bool((got[:2] == 7.0).all()) and bool((got[c.starts[-1]:] == 7.0).all())  # left as they were


@pytest.mark.parametrize("d,group", [(64, 3), (64, 5), (64, 7), (64, 16), (64, 128), (128, 3), (128, 6), (128, 100)])
def test_group_sizes(d, group):
    """Groups that divide the 128 rows of a tile and groups that leave some unused."""
    c = Case([1, 50, 9], [77, 50, 300], group * (2 if group < 20 else 1), group, d, seed=group)
    c.check(c.run(), f"group {group}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_split_over_the_cache(fp8, d):
    """Few rows against long contexts: keys split over many entries and merged; ranges in which a row
    sees no key at all (the causal edge lies inside the last range)."""
    c = Case([3, 140, 1], [6000, 5000, 2300], 2, 1, d, fp8, seed=8)
    c.check(c.run(), "split")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_bytes_behind_the_lengths_do_not_matter(fp8, d):
    """NaN in every cache entry that no length covers (partial pages, unused pages): bit-identical."""
    c = Case([1, 30, 129, 2], [65, 190, 129, 640], 4, 2, d, fp8, seed=5)
    clean = c.run()
    dirty = c.run(pools=ref.poison(c.pools, c.table, c.lens))
    assert torch.equal(clean, dirty) and bool(torch.isfinite(clean).all())
    wide = torch.full((4, c.table.shape[1] + 7), 1 << 30, dtype=torch.int32)  # a wider table, rubbish behind
    wide[:, :c.table.shape[1]] = torch.where(c.table < 0, torch.tensor(-(1 << 30), dtype=torch.int32), c.table)
    assert torch.equal(c.run(table=wide), clean)


@pytest.mark.parametrize("d", [64, 128])
def test_rows_without_keys_and_clamped_lengths(d):
    """Lengths below the chunk (rows before position 0 see nothing), zero and negative lengths, and
    lengths past L, which are clamped to it."""
    c = Case([5, 4, 3, 140, 6], [5, 200, 3, 140, 300], 2, 1, d, seed=2)
    lens = [3, 0, -7, 100, 300]
    got = c.run(lens=lens)
    want = c.want(lens=[3, 0, 0, 100, 300])
    assert bool((got[:2] == 0).all()) and bool((got[5:12] == 0).all()) and bool((got[12:52] == 0).all())
    keep = want.clone()
    c.check(got, "short lengths", keep)
    again = c.run(lens=[5, 200, 3, 140, 10_000], L=300)  # 10,000 clamped to 300
    c.check(again, "clamped")


def test_pages_outside_the_pool_read_zeros():
    c = Case([4], [200], 2, 1, 64, seed=6)
    for bad in (-1, c.pools[0].shape[0], 1 << 30, -(1 << 30)):
        table = c.table.clone()
        table[0, 1] = bad
        pools = [p.clone() for p in c.pools]
        for p in pools:
            p[c.table[0, 1]] = 0
        assert torch.equal(c.run(table=table), c.run(pools=pools))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("out_dtype", [torch.float32, BF, torch.float16])
def test_output_types_gain_and_layouts(d, out_dtype):
    """16-bit outputs, the RMSNorm gain, queries as views of a projection (heads inside rows, halves side
    by side) and with heads outermost, pages with padded strides."""
    c = Case([60, 1, 130], [60, 333, 500], 4, 2, d, seed=4)
    gain = torch.linspace(0.5, 1.5, 2 * d)
    got = c.run(out_dtype=out_dtype, norm_weight=gain.cuda())
    want = c.want(norm_weight=gain)
    c.check((got.float() / gain.cuda()).to(torch.float32 if out_dtype == torch.float32 else out_dtype), "gain", want / gain.double())
    proj = torch.cat([x for x in c.q], -1).cuda()            # [T, H, 2 d]
    heads = [x.transpose(0, 1).contiguous().transpose(0, 1).cuda() for x in c.q]  # head stride outermost
    padded = []
    for p in c.pools:
        big = torch.full((p.shape[0], p.shape[1], 66, p.shape[3] + 8), float("nan"), dtype=BF, device="cuda")
        big[:, :, :64, :p.shape[3]] = p.cuda()
        padded.append(big[:, :, :64, :p.shape[3]])
    ws = da.workspace(da.chunk_workspace_bytes(c.T, 3, 4, 2, c.L, d, 2 * d))
    plain = c.run(out_dtype=out_dtype)
    for q in ((proj[..., :d], proj[..., d:]), heads):
        alt = da.diffattn_chunk_paged(*q, *padded, c.table.cuda(), _i32(c.starts), _i32(c.lens), LAM, LI, L=c.L, kv_group=2,
                                      ws=ws, out_dtype=out_dtype)
        assert torch.equal(alt, plain)


@pytest.mark.parametrize("fp8", [False, True])
def test_one_token_rows_agree_with_the_decode(fp8):
    c = Case([1] * 9, [1, 64, 65, 300, 2, 128, 1000, 777, 5], 4, 2, 64, fp8, seed=7)
    got = c.run()
    dec = da.diffattn_decode_paged(*(x.cuda() for x in c.q), *(p.cuda() for p in c.pools), c.table.clamp(min=0).cuda(),
                                   _i32(c.lens), LAM, LI, L=c.L, kv_group=2, scales=c.scales)
    assert_bf16_parity(got, dec.double().cpu().numpy(), "decode")


@pytest.mark.parametrize("group,n_new", [(2, [1, 8, 9, 1, 1, 1, 0, 2, 1, 1, 1, 40]), (1, [16, 17, 1, 0, 15, 1]), (16, [1, 1, 0, 1]),
                                         (5, [3, 4, 1, 2, 1, 1, 3, 1])])
def test_few_rows_beside_many(group, n_new):
    """fp8 batches whose sequences have at most 16 rows on average: tiles of up to 16 rows and longer ones
    run in kernels of their own; whole, split, and with NaN behind the lengths."""
    lens = [n + 37 * b * b + 5 for b, n in enumerate(n_new)]
    edge = 0 if group == 16 else 1  # rows of no sequence before and behind; they count into the average
    c = Case(n_new, lens, 2 * group, group, 64, True, seed=group, pad=2 * edge, first=edge)
    assert c.T * group <= 16 * len(n_new)
    out = torch.full((c.T, 2 * group, 128), 7.0, device="cuda")
    got = c.run(out=out)
    c.check(got, f"few beside many, group {group}")
    assert bool((got[:c.starts[0]] == 7.0).all()) and bool((got[c.starts[-1]:] == 7.0).all())
    dirty = c.run(pools=ref.poison(c.pools, c.table, c.lens))
    rows = slice(c.starts[0], c.starts[-1])
    assert torch.equal(got[rows], dirty[rows])


@pytest.mark.parametrize("order", ["rising", "falling", "sink"])
@pytest.mark.parametrize("n", [2, 20])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_moving_maxima(d, fp8, n, order):
    """Scores that rise key by key (the running maximum moves in every tile), that fall, and one early key
    far above a long tail whose small weights add up to as much (2^-10 of it each, 1030 keys). A shift of
    a row's scores multiplies its exponential's argument error only by fp32's 2^-24 x 60: 4e-6 of a weight."""
    c = Case([n], [1100], 2, 1, d, fp8, seed=40)
    u = torch.randn(d, generator=torch.Generator().manual_seed(1))
    u = u / u.norm()
    x = torch.arange(1100, dtype=torch.float32) / 1100
    want = {"rising": 30 * x, "falling": 30 * (1 - x), "sink": torch.where(torch.arange(1100) == 3, 6.93, 0.0)}[order]
    for q in c.q:  # scores: q k / sqrt d, with q = 4 sqrt d u plus a little noise
        q.copy_((4 * d ** 0.5 * u + 0.02 * torch.randn(q.shape, generator=torch.Generator().manual_seed(2))).to(BF))
    for p, s in zip(c.pools[:2], c.scales or (1.0, 1.0)):
        for i in range(18):
            k = min(64, 1100 - 64 * i)
            rows = (want[64 * i:64 * i + k, None] / 4 * u) / s
            p[int(c.table[0, i]), :, :k] = rows.clamp(-448, 448).to(p.dtype)
    c.check(c.run(), f"{order} d{d} fp8={fp8}")


def test_score_range():
    """Queries scaled so that the softmax is nearly flat and nearly one-hot."""
    for scale in (1e-4, 30.0):
        c = Case([40, 1], [300, 900], 2, 1, 64, seed=11)
        c.q = [(x.float() * scale).to(BF) for x in c.q]
        c.check(c.run(), f"scale {scale}")


def test_offsets_past_32_bits():
    """A pool whose last pages lie beyond 2^31 elements (and 2^32 bytes) from its start."""
    H, d, Dv, P = 16, 64, 128, 16500                     # 16,500 pages x 16 heads x 64 x 128 = 2.16e9 V elements
    c = Case([70], [130], H, 1, d, seed=9)
    dev = [torch.empty(P, H, 64, w, dtype=BF, device="cuda") for w in (d, d, Dv)]
    where = torch.tensor([[P - 1, 3, P - 2]], dtype=torch.int32)
    for p, src in zip(dev, c.pools):
        for i in range(3):
            p[int(where[0, i])] = src[int(c.table[0, i])].cuda()
    new = [torch.randn(70, H, w, generator=torch.Generator().manual_seed(1)).to(BF) for w in (d, d, Dv)]
    da.diffattn_kv_append_chunk_paged(*(x.cuda() for x in new), *dev, where.cuda(), _i32([0, 70]), _i32([130]))
    for p, src, x in zip(dev, c.pools, new):
        for i in range(70):
            src[int(c.table[0, (60 + i) // 64]), :, (60 + i) % 64] = x[i]
        assert torch.equal(p[P - 2].cpu().view(torch.int16)[:, :2], src[int(c.table[0, 2])].view(torch.int16)[:, :2])
    got = da.diffattn_chunk_paged(*(x.cuda() for x in c.q), *dev, where.cuda(), _i32([0, 70]), _i32([130]), LAM, LI, L=130)
    c.check(got, "far pages")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_serving_steps_together(fp8, d):
    """rope on Q, append with the rotation, attention: a prompt in two chunks, then two decoding steps,
    beside a second sequence; each output against the float64 definition of the whole sequence."""
    H, Hk, Dv, r = 4, 2, 2 * d, d // 2
    total = [150, 90]
    plan = da.rope_plan(r, scaling="ramp", factor=4.0, original_length=64, interleaved=True)
    f, m = ref.frequencies(r, scaling="ramp", factor=4.0, original=64)
    g = torch.Generator().manual_seed(d)
    seqs = [[torch.randn(n, h, w, generator=g).to(BF) for h, w in ((H, d), (H, d), (Hk, d), (Hk, d), (Hk, Dv))] for n in total]
    dt = F8 if fp8 else BF
    pools, table = ref.make_pool(total, Hk, (d, d, Dv), dt, seed=1)
    scales = ref.SCALES if fp8 else None
    dev = [p.cuda() for p in ref.poison(pools, table, [0, 0])]  # nothing but NaN before the first append
    done = [0, 0]
    worst = []
    for step in ([100, 0], [48, 88], [1, 1], [1, 1]):
        starts = [0, step[0], step[0] + step[1]]
        rows = [torch.cat([seqs[b][i][done[b]:done[b] + step[b]] for b in (0, 1)]).cuda() for i in range(5)]
        pos = torch.cat([torch.arange(done[b], done[b] + step[b]) for b in (0, 1)]).to(torch.int32).cuda()[None]
        done = [done[b] + step[b] for b in (0, 1)]
        q1, q2 = da.diffattn_rope([x.transpose(0, 1)[None] for x in rows[:2]], plan, positions=pos)
        da.diffattn_kv_append_chunk_paged(*rows[2:], *dev, table.cuda(), _i32(starts), _i32(done), rope=plan, scales=scales)
        got = da.diffattn_chunk_paged(q1[0].transpose(0, 1), q2[0].transpose(0, 1), *dev, table.cuda(), _i32(starts), _i32(done),
                                      LAM, LI, L=150, kv_group=2, scales=scales)
        # The reference rotates in float64 and rounds where the cache and Q are held in fewer bits; a code
        # next to a rounding border may differ, so the cache it attends to is the one on the GPU, checked
        # on its own by the append's tests.
        angle = (pos[0].cpu().double()[:, None] * f)[:, None]
        qr = [ref.rotate(x.cpu().double(), angle, m, True).to(BF) for x in rows[:2]]
        want = ref.chunk_attention(*qr, [p.cpu() for p in dev], table, starts, done, LAM, LI, group=2, scales=scales)
        worst.append(assert_bf16_parity(got, want.numpy(), f"step {step}"))
    assert len(worst) == 4


def test_deterministic():
    c = Case([3, 140, 1], [6000, 5000, 2300], 4, 2, 64, seed=8)
    a = c.run()
    for _ in range(3):
        assert torch.equal(c.run(), a)


def test_graph_replays_with_new_lengths_and_two_graphs_at_once():
    """One captured call serves other chunk starts and lengths; two captured calls replayed on two
    streams at the same time do not share partial states."""
    graphs = []
    for k in range(2):
        c = Case([2, 60], [5000 - k, 700], 4, 1, 64, seed=20 + k)
        dev = dict(q=[x.cuda() for x in c.q], pools=[p.cuda() for p in c.pools], table=c.table.cuda(), start=_i32(c.starts),
                   lens=_i32(c.lens), out=torch.empty(c.T, 4, 128, device="cuda"))
        call = lambda dev=dev, c=c: da.diffattn_chunk_paged(*dev["q"], *dev["pools"], dev["table"], dev["start"], dev["lens"],  # noqa: E731
                                                            LAM, LI, L=c.L, out=dev["out"])
        call()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call()
        graphs.append((c, dev, gr, c.run()))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for _, dev, _, _ in graphs:
            dev["out"].zero_()
        torch.cuda.synchronize()
        for s, (_, _, gr, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for _, dev, _, want in graphs:
            assert torch.equal(dev["out"], want)
    c, dev, gr, _ = graphs[0]
    dev["start"].copy_(_i32([0, 40, 62]))
    dev["lens"].copy_(_i32([300, 600]))
    gr.replay()
    torch.cuda.synchronize()
    want = ref.chunk_attention(*c.q, c.pools, c.table, [0, 40, 62], [300, 600], LAM, LI)
    assert_bf16_parity(dev["out"], want.numpy(), "replayed with other lengths")


def test_two_streams_at_once():
    cases = [Case([2, 90], [4000, 1500], 4, 1, 64, seed=30 + k) for k in range(2)]
    want = [c.run() for c in cases]
    dev = [dict(q=[x.cuda() for x in c.q], pools=[p.cuda() for p in c.pools], table=c.table.cuda(), start=_i32(c.starts),
                lens=_i32(c.lens)) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [da.diffattn_chunk_paged(*x["q"], *x["pools"], x["table"], x["start"], x["lens"], LAM, LI, L=c.L, stream=s)
               for c, x, s in zip(cases, dev, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_shape_refusals():
    c = Case([2], [10], 4, 2, 64, seed=1)
    q, pools = [x.cuda() for x in c.q], [p.cuda() for p in c.pools]
    rest = [c.table.cuda(), _i32(c.starts), _i32(c.lens), LAM, LI]

    def call(q=q, pools=pools, rest=rest, **kw):
        return da.diffattn_chunk_paged(*q, *pools, *rest, **{**dict(L=10, kv_group=2), **kw})
    call()
    bad = [lambda: call(q=[q[0].half(), q[1].half()]), lambda: call(q=[q[0], q[1][:1]]), lambda: call(kv_group=4),
           lambda: call(pools=[pools[0].half()] + pools[1:]), lambda: call(scales=(1.0, 1.0, 1.0)),
           lambda: call(rest=[rest[0].long()] + rest[1:]), lambda: call(rest=[rest[0], rest[1][:1]] + rest[2:]),
           lambda: call(rest=[rest[0].cpu()] + rest[1:]), lambda: call(out=torch.empty(2, 4, 64, device="cuda")),
           lambda: call(norm_weight=torch.ones(64, device="cuda")), lambda: call(pools=[p[:, :, :32] for p in pools]),
           lambda: call(q=[x.transpose(1, 2) for x in q]), lambda: call(out_dtype=torch.float64)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(da.DiffAttnError):
        call(L=65)  # past the table


def test_two_threads_on_one_stream():
    """Calls of two threads may interleave their launches on one stream: each has a workspace of its own."""
    import threading
    cases = [Case([2, 90], [4000, 1500], 4, 1, 64, seed=50), Case([3, 1, 7], [2000, 3000, 900], 4, 1, 64, True, seed=51)]
    want = [c.run() for c in cases]
    bad = []

    def work(c, want):
        dev = [x.cuda() for x in c.q], [p.cuda() for p in c.pools]
        rest = c.table.cuda(), _i32(c.starts), _i32(c.lens)
        for _ in range(40):
            got = da.diffattn_chunk_paged(*dev[0], *dev[1], *rest, LAM, LI, L=c.L, scales=c.scales)
            torch.cuda.current_stream().synchronize()
            if not torch.equal(got, want):
                bad.append(c)
    threads = [threading.Thread(target=work, args=a) for a in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_batches_of_next_to_nothing(d, fp8):
    """No sequence has a new token; one of a thousand has; a cache of a single token."""
    c = Case([3, 2], [100, 200], 4, 2, d, fp8, seed=60)
    out = torch.full((5, 4, 2 * d), 7.0, device="cuda")
    c.run(starts=[2, 2, 2], out=out)
    assert bool((out == 7.0).all())  # rows of no sequence
    n = [0] * 1000
    n[613] = 2
    lens = [1 + b % 60 for b in range(1000)]
    lens[613] = 333
    c = Case(n, lens, 2, 1, d, fp8, seed=61)
    c.check(c.run(), "one of a thousand")
    c = Case([1], [1], 2, 1, d, fp8, seed=62)
    c.check(c.run(L=1), "a cache of one token")
