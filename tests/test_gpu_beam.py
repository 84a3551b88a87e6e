"""Beam search's selection and the reordering of per-beam states on the GPU, against float64 references.

Tolerance of the scores. A term e^(x - m) of the sum is fp32: the difference is off by 2^-24 |x - m| and
its product with log2 e by as much again, so the term by 2^-22.5 |x - m| + 2^-22 (the instruction) of
itself. Weighted with the terms, |x - m| averages at most the logarithm of their number (22 bits: 16): 4e-6 of
the sum. Sums of up to 2^10 terms in fp32 before they are joined in 64 bits: 2^10 2^-24 = 6e-5 at the worst, all
roundings alike; of either sign, 6 sigma of 2^5 x 2^-24 / sqrt 3 = 7e-6. Together 1.1e-5 on the logarithm, and
half a step of fp32, 2^-24, of the score. A beam's candidates come in the order of its logits, whatever the sum;
those of different beams whose ranks are within twice 1.1e-5 may change places."""

import math

import pytest
import torch

import beam_reference as ref
import differential_attention_02_gb300 as da

pytestmark = pytest.mark.gpu
F32, BF, F16 = torch.float32, torch.bfloat16, torch.float16
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from differential_attention_02_gb300 import build
    build.build()
    da.load_library()


def _check(got, logits, scores, width, finished=None, lengths=None, eos=None, penalty=0.0):
    """A BeamChoice against the reference, on the same inputs."""
    want = ref.select(logits, scores, width, finished, lengths, eos, penalty)
    more = ref.select(logits, scores, min(width + 8, logits.shape[1] * logits.shape[2]), finished, lengths, eos, penalty)
    rank = lambda c: c[0] / max(c[4], 1) ** penalty if c[0] > -INF else -INF  # noqa: E731
    s = torch.tensor([[w[0] for w in row] for row in want], dtype=torch.float64)
    g = got.scores.double().cpu()
    assert torch.equal(torch.isfinite(g), torch.isfinite(s)), (g, s)
    some = torch.isfinite(s)
    off = ((g - s).abs() / (2.2e-5 + 2 ** -24 * s.abs()))[some]  # two that change places are another 1.1e-5 apart
    assert off.numel() == 0 or float(off.max()) <= 1, float(off.max())
    columns = [None if t is None else t.tolist() for t in got[1:]]
    for b, row in enumerate(want):
        found = list(zip(*(c[b] if c is not None else [None] * len(row) for c in columns)))
        known = {(c[1], c[2]): c for c in more[b]}
        for f, w in zip(found, row):
            c = known[f[:2]]  # the candidate that was chosen: nothing else is among the best
            assert f[2:] == tuple(v if t is not None else None for v, t in zip(c[3:], f[2:])), (f, c)
            assert f[:2] == w[1:3] or abs(rank(c) - rank(w)) <= 2.2e-5 * max(1.0, max(w[4], c[4], 1) ** -penalty), (f, w)
        for k in range(logits.shape[1]):  # in the order of the logits
            mine, theirs = [f[0] for f in found if f[1] == k], [c[1] for c in more[b] if c[2] == k]
            assert mine == theirs[:len(mine)], k


def _inputs(B, K, V, dtype, seed, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    logits = (torch.randn(B, K, V, generator=g) * spread).to(dtype)
    scores = -20 * torch.rand(B, K, generator=g)
    return g, logits, scores


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("B,K,V,W", [(1, 1, 1, 1), (1, 2, 3, 5), (2, 3, 17, 6), (3, 4, 255, 4), (2, 5, 1000, 10), (1, 4, 32000, 4),
                                     (2, 32, 4097, 64), (4, 8, 50001, 16), (1, 1, 262147, 64), (5, 1, 2049, 2), (1, 3, 300001, 33)])
def test_selection(B, K, V, W, dtype):
    _, logits, scores = _inputs(B, K, V, dtype, seed=V + W)
    got = da.diffattn_beam_select(logits.cuda(), scores.cuda(), width=W)
    assert got.finished is None and got.lengths is None
    _check(got, logits, scores, W)
    again = da.diffattn_beam_select(logits.cuda(), scores.cuda(), width=W)
    assert all(torch.equal(a, b) for a, b in zip(got[:3], again[:3]))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,K,V,W", [(1, 32, 16001, 64), (300, 2, 90, 5), (1, 2, 1 << 20, 64), (3, 1, 9000, 63), (2, 7, 40000, 33), (64, 16, 700, 32),
                                     (1, 1, 64, 64)])
def test_short_rows_and_many_kept(B, K, V, W, dtype):
    """Segments of a vector, of 256 logits and of a round, rows in one chunk and in many."""
    _, logits, scores = _inputs(B, K, V, dtype, seed=V)
    _check(da.diffattn_beam_select(logits.cuda(), scores.cuda(), W), logits, scores, W)


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("V,W", [(900, 9), (6000, 64), (50001, 16), (50001, 64), (262144, 8)])
def test_logits_in_order_and_nearly_all_masked(V, W, dtype):
    """The best side by side (ascending, descending, in blocks), a grammar's mask that leaves three tokens above the type's
    lowest value, and steps of equal values."""
    K = 2
    x = torch.stack([torch.linspace(-6, 6, V), torch.linspace(6, -6, V), (torch.arange(V) // 700 * 37 % 101).float() / 9,
                     torch.full((V,), torch.finfo(dtype).min), (torch.arange(V) % 97).float() / 10, torch.zeros(V)])
    x[3, [V // 3, V // 2, V - 1]] = torch.tensor([1.0, 3.0, 2.0])
    logits = x.clamp(torch.finfo(dtype).min, torch.finfo(dtype).max).to(dtype)[:, None].expand(6, K, V).contiguous()
    logits[:, 1] = logits[:, 1].roll(5, -1)
    scores = torch.tensor([[-1.0, -4.0]]).expand(6, K).contiguous()
    _check(da.diffattn_beam_select(logits.cuda(), scores.cuda(), W), logits, scores, W)


def test_scores_of_every_size():
    """Scores far from zero, where units of fp32 hide differences of logits, and dead beams at -1e9 as some programs have them."""
    g = torch.Generator().manual_seed(6)
    logits = torch.randn(4, 3, 3000, generator=g) * 2
    scores = torch.tensor([[-1e6, -1e6 - 1, -2e6], [0.0, -1e9, -1e9], [-3.0, -3e38, -INF], [1e4, 1e4, 5.0]])
    got = da.diffattn_beam_select(logits.cuda(), scores.cuda(), 6)
    _check(got, logits, scores, 6)
    assert got.parents[1].tolist() == [0] * 6


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("penalty", [0.0, 0.7, -0.5])
@pytest.mark.parametrize("B,K,V,W", [(4, 4, 1000, 8), (3, 6, 4099, 6), (2, 16, 30000, 32)])
def test_finished_beams_and_lengths(B, K, V, W, penalty, dtype):
    g, logits, scores = _inputs(B, K, V, dtype, seed=int(V + 10 * penalty))
    finished = torch.rand(B, K, generator=g) < 0.4
    finished[0] = True  # a sequence that is done: it offers its beams, and places are left
    lengths = torch.randint(0, 40, (B, K), generator=g, dtype=torch.int32)
    logits[1, 0, 7] = 40.0  # ends
    got = da.diffattn_beam_select(logits.cuda(), scores.cuda(), W, finished.cuda(), lengths.cuda(), 7, penalty)
    _check(got, logits, scores, W, finished, lengths, 7, penalty)
    assert W <= K or bool((got.parents[0] == -1).any())


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("V", [40, 5003, 140001])
def test_ties_go_to_the_lowest_beam_and_token(V, dtype):
    """Equal logits everywhere; few values; the best at the ends of the row and over its middle."""
    B, K, W = 4, 3, 9
    logits = torch.zeros(B, K, V)
    g = torch.Generator().manual_seed(V)
    logits[1] = torch.randint(0, 3, (K, V), generator=g).float()
    logits[2, :, 0] = logits[2, :, V - 1] = logits[2, :, V // 2:V // 2 + 3] = 2.0
    logits[3] = torch.linspace(-4, 4, V)  # the best lie side by side, at the end
    logits = logits.to(dtype)
    logits[3, 1] = logits[3, 1].flip(0)
    scores = torch.tensor([[-1.0, -1.0, -1.0], [-1.0, -1.5, -2.0], [-1.0, -1.0, -3.0], [-1.0, -2.0, -3.0]])
    got = da.diffattn_beam_select(logits.cuda(), scores.cuda(), W)
    want = ref.select(logits[:3], scores[:3], W)  # sums that are exact or alike in each beam: no two ranks change places
    assert got.tokens.tolist()[:3] == [[w[1] for w in row] for row in want]
    assert got.parents.tolist()[:3] == [[w[2] for w in row] for row in want]
    _check(got, logits, scores, W)
    assert got.tokens[0].tolist() == list(range(9)) and got.parents[0].tolist() == [0] * 9
    for k in range(K):  # beam by beam, where sums of another order would change nothing
        one = da.diffattn_beam_select(logits[:, k:k + 1].contiguous().cuda(), scores[:, k:k + 1].contiguous().cuda(), W)
        _check(one, logits[:, k:k + 1], scores[:, k:k + 1], W)
        assert one.tokens.tolist() == [[w[1] for w in row] for row in ref.select(logits[:, k:k + 1], scores[:, k:k + 1], W)]


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("V", [33, 2500, 70001])
def test_masks_infinities_and_nan(V, dtype):
    """Banned tokens (-inf and the type's lowest value), rows of which nothing is left, NaN, +inf, dead beams and NaN
    scores, alone and together."""
    B, K, W = 6, 4, 8
    g, logits, scores = _inputs(B, K, V, dtype, seed=V)
    low = torch.finfo(dtype).min
    logits[0] = -INF
    logits[0, 2, V - 1] = 1.0          # a single candidate in a whole sequence
    logits[1] = -INF                   # none
    logits[2, :, ::2] = -INF
    logits[2, 1, 1::2] = float("nan")  # a row of NaN and -inf
    logits[3, 0, 5] = INF
    logits[3, 1, [3, 11, V - 2]] = INF
    logits[3, 2] = INF
    logits[3, 3] = low
    logits[4, :, 1:] = low
    logits[4, 2] = float("nan")
    logits[4, 3, ::3] = float("nan")
    scores[4, 1] = float("nan")
    scores[5] = torch.tensor([-3.0, -INF, -INF, -INF])
    scores[2, 0] = -INF
    got = da.diffattn_beam_select(logits.cuda(), scores.cuda(), W)
    _check(got, logits, scores, W)
    assert got.parents[1].tolist() == [-1] * W and got.tokens[1].tolist() == [0] * W
    ended = da.diffattn_beam_select(logits.cuda(), scores.cuda(), W, eos=V - 1)
    _check(ended, logits, scores, W, eos=V - 1)
    assert bool(ended.finished[1].all()) and ended.tokens[1].tolist() == [V - 1] * W


@pytest.mark.parametrize("dtype", [F32, BF, F16])
def test_rows_of_any_stride_and_alignment(dtype):
    """Rows that begin at every place of a 16-byte vector, padded rows, shared rows, batches apart."""
    B, K, V, W = 3, 4, 5011, 7
    g = torch.Generator().manual_seed(3)
    scores = -5 * torch.rand(B, K, generator=g)
    whole = torch.full((B, K + 1, V + 64), 60.0).to(dtype)  # what lies around a row would win
    for shift in (0, 1, 2, 3, 5, 7, 8, 9):
        view = whole[:, :K, shift:shift + V]
        view.copy_((torch.randn(B, K, V, generator=g) * 2).to(dtype))
        on = whole.cuda()[:, :K, shift:shift + V]
        _check(da.diffattn_beam_select(on, scores.cuda(), W), view, scores, W)
        whole.fill_(60.0)
    row = (torch.randn(1, 1, V, generator=g) * 2).to(dtype)
    shared = row.cuda().expand(B, K, V)
    _check(da.diffattn_beam_select(shared, scores.cuda(), W), row.expand(B, K, V), scores, W)


def test_the_outputs_may_be_the_inputs():
    B, K, V = 5, 4, 3000
    g, logits, scores = _inputs(B, K, V, BF, seed=9)
    finished, lengths = torch.rand(B, K, generator=g) < 0.3, torch.randint(0, 9, (B, K), generator=g, dtype=torch.int32)
    want = da.diffattn_beam_select(logits.cuda(), scores.cuda(), None, finished.cuda(), lengths.cuda(), 2, 0.5)
    out = da.BeamChoice(scores.cuda(), *(torch.empty(B, K, dtype=torch.int32, device="cuda") for _ in range(2)), finished.cuda(), lengths.cuda())
    got = da.diffattn_beam_select(logits.cuda(), out.scores, None, out.finished, out.lengths, 2, 0.5, out=out)
    assert got is out and all(torch.equal(a, b) for a, b in zip(want, got))


def test_selection_on_other_streams_and_from_graphs():
    """Two streams at once, and two graphs of one pool of memory replayed on new inputs."""
    B, K, V, W = 2, 4, 70001, 8
    cases = [_inputs(B, K, V, BF, seed=s)[1:] for s in range(4)]
    want = [da.diffattn_beam_select(l.cuda(), s.cuda(), W) for l, s in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ins = [(l.cuda(), s.cuda()) for l, s in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            got[i].append(da.diffattn_beam_select(*ins[i], W, stream=st))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for g in got[i] for a, b in zip(g[:3], want[i][:3]))
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = da.diffattn_beam_select(*ins[i], W)
        graphs.append((g, out))
    for step in (2, 3):
        for i in range(2):
            for a, b in zip(ins[i], cases[(step + i) % 4]):
                a.copy_(b)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(graphs[i][1][:3], want[(step + i) % 4][:3]))


# ---------------------------------------------------------------- reordering
def _reordered(t, parents, lens=None):
    B, K = parents.shape
    out, old = t.clone(), t.clone()
    for i in range(B * K):
        p = int(parents[i // K, i % K])
        if 0 <= p < K:
            src = i // K * K + p
            if lens is None:
                out[i] = old[src]
            else:
                n = min(max(int(lens[src]), 0), t.shape[2])
                out[i, :, :n] = old[src, :, :n]
    return out


@pytest.mark.parametrize("B,K", [(1, 1), (3, 2), (2, 4), (4, 5), (2, 8), (1, 13), (2, 16), (1, 17), (2, 32)])
def test_reorder_rows(B, K):
    """Rows of every type, width and alignment: cycles, children of one parent, itself, none, and values outside."""
    g = torch.Generator().manual_seed(K)
    parents = torch.randint(-1, K + 1, (B, K), generator=g, dtype=torch.int32)
    parents[0] = (torch.arange(K) + 1) % K  # a cycle of all
    S = B * K
    base = torch.randint(0, 1000, (S, 40), generator=g)
    states = [torch.randint(0, 255, (S, 7), generator=g, dtype=torch.uint8), torch.randn(S, 3, 5, generator=g).to(BF),
              torch.randint(0, 9, (S, 777), generator=g, dtype=torch.int32), torch.randn(S, 4096, generator=g), torch.randn(S, generator=g),
              torch.randn(S, 2, 8, 16, generator=g).to(F16), torch.rand(S, generator=g) < 0.5, base[:, 3:20], torch.zeros(S, 0),
              torch.randn(S, 64, generator=g).to(torch.float8_e4m3fn)]
    on = [t.cuda() for t in states]
    on[7] = base.cuda()[:, 3:20]  # rows inside wider ones
    got = da.diffattn_beam_reorder(on, parents.cuda())
    assert got is on
    for t, x in zip(states, on):
        bits = (lambda v: v.view(torch.uint8)) if t.dtype == torch.float8_e4m3fn else (lambda v: v)
        assert torch.equal(bits(x.cpu()), _reordered(bits(t), parents))


@pytest.mark.parametrize("dtype", [BF, torch.float8_e4m3fn])
@pytest.mark.parametrize("B,K,H,L,d", [(1, 2, 1, 1, 64), (2, 4, 3, 100, 64), (3, 5, 2, 65, 128), (1, 32, 1, 40, 64)])
def test_reorder_caches(B, K, H, L, d, dtype):
    """Contiguous caches: the parent's tokens are moved, and what lies behind them stays."""
    g = torch.Generator().manual_seed(L)
    S = B * K
    parents = torch.randint(-1, K, (B, K), generator=g, dtype=torch.int32)
    lens = torch.randint(0, L + 1, (S,), generator=g, dtype=torch.int32)
    lens[0], lens[-1] = L, L + 7 if S > 1 else L  # clamped
    states = [torch.randn(S, H, L, w, generator=g).to(dtype) for w in (d, d, 2 * d)]
    on = [t.cuda() for t in states]
    token_major = torch.randn(S, L, H, d, generator=g).to(dtype)  # tokens outside, heads inside
    on.append(token_major.cuda().transpose(1, 2))
    states.append(token_major.transpose(1, 2))
    da.diffattn_beam_reorder(on, parents.cuda(), lens.cuda())
    for t, x in zip(states, on):
        assert torch.equal(x.cpu().contiguous().view(torch.uint8), _reordered(t.contiguous(), parents, lens).view(torch.uint8))


def test_reorder_many_states_and_long_rows():
    """More states than a launch takes, of mixed units, and rows beyond a MiB."""
    g = torch.Generator().manual_seed(0)
    parents = torch.tensor([[1, 0, 0], [2, 2, 1]], dtype=torch.int32)
    states = [torch.randn(6, 8 + i % 5, generator=g) for i in range(120)] + [torch.randn(6, (1 << 18) * 2 + 13, generator=g)]
    on = [t.cuda() for t in states]
    da.diffattn_beam_reorder(on, parents.cuda())
    assert all(torch.equal(x.cpu(), _reordered(t, parents)) for t, x in zip(states, on))
