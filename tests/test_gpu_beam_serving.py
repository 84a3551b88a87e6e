"""A beam search through the paged serving calls, as a program runs it: a layer over the cache, the vocabulary,
the selection, and the beams' pages."""

import math

import pytest
import torch

import beam_reference as ref
import differential_attention_02_gb300 as da

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16
LAM, LI, EOS = 0.45, 0.47, 3


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from differential_attention_02_gb300 import build
    build.build()
    da.load_library()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Model:
    """Two served layers between an embedding and a vocabulary."""

    def __init__(self, dm=256, h=2, d=64, V=520, d_ff=256, seed=0):
        g = torch.Generator().manual_seed(seed)
        w = lambda k, n, s=1.0: (torch.randn(k, n, generator=g) * s * k ** -0.5).to(BF).cuda()  # noqa: E731
        self.h, self.d, self.V = h, d, V
        self.embedding = torch.randn(V, dm, generator=g).to(BF).cuda()
        self.layers = [(w(dm, 3 * h * 2 * d), w(h * 2 * d, dm), da.interleave_gate_up(w(dm, d_ff), w(dm, d_ff)), w(d_ff, dm)) for _ in range(2)]
        self.head = w(dm, V, 3.0)
        self.rope = da.rope_plan(d)

    def run(self, tokens, pools, table, q_start, lens, positions, L):
        x = self.embedding[tokens.long()].float()
        for weights, pages in zip(self.layers, pools):
            x = da.layer_serve(x, *weights, self.h, pages, table, q_start, lens, LAM, LI, L, rope=self.rope, positions=positions)
        return da.add_rmsnorm(x)[1]

    def pools(self, P):
        return [tuple(torch.full((P, self.h, 64, w), float("nan"), dtype=BF, device="cuda") for w in (self.d, self.d, 2 * self.d))
                for _ in self.layers]


def _search(m, prompts, K, steps, graph=False, vocabulary=None):
    """(final choice, histories [B][K] of tokens) of a beam search after the prompts."""
    B, L = len(prompts), max(map(len, prompts)) + steps + 1
    S, M = B * K, -(-L // 64) + 1
    P = S * M + 2
    pools = m.pools(P)
    handle = da.page_pools(*pools)
    empty = (torch.full((S, M), -1, dtype=torch.int32, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda"),
             torch.zeros(P, dtype=torch.int32, device="cuda"))
    # the prompts, each in its group's first row
    first = [len(prompts[i // K]) if i % K == 0 else 0 for i in range(S)]
    plan = da.diffattn_pages_fork(*empty, _i32([[-1] * K] * B), new_lens=_i32(first))
    starts = [sum(first[:i]) for i in range(S + 1)]
    rows = m.run(_i32([t for p in prompts for t in p]), pools, plan.table, _i32(starts), plan.lens,
                 _i32([i for p in prompts for i in range(len(p))]), L)
    last = torch.tensor([starts[(i // K) * K + 1] - 1 for i in range(S)], device="cuda")
    scores = torch.tensor([[0.0] + [-math.inf] * (K - 1)] * B, device="cuda")
    zeros = torch.zeros(B, K, dtype=torch.int32, device="cuda")
    kw = dict(eos=EOS, length_penalty=0.6, vocabulary=vocabulary)
    choice, plan = da.beam_step(rows[last], m.head, scores, handle, *plan[:3], torch.zeros(B, K, dtype=torch.bool, device="cuda"), zeros, **kw)
    histories = [[[choice.tokens[b, k].item()] for k in range(K)] for b in range(B)]
    q_start = torch.arange(S + 1, dtype=torch.int32, device="cuda")

    def step():
        x = m.run(choice.tokens.view(-1), pools, plan.table, q_start, plan.lens, plan.lens - 1, L)
        da.beam_step(x, m.head, choice.scores, handle, plan.table, plan.lens, plan.refs, choice.finished, choice.lengths, choice=choice,
                     plan=plan, **kw)
    captured = None
    for i in range(steps):
        if graph and i == 1:
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                step()
        step() if captured is None else captured.replay()
        histories = [[(histories[b][p] + ([t] if not f or t != EOS or histories[b][p][-1] != EOS else [])) if p >= 0 else []
                      for t, p, f in zip(*(x[b].tolist() for x in (choice.tokens, choice.parents, choice.finished)))] for b in range(B)]
    assert plan.info[1].item() == 0
    held = [p for row, n in zip(plan.table.tolist(), plan.lens.tolist()) for p in row[:ref.pages(n)]]
    assert plan.refs.tolist() == [held.count(p) for p in range(P)]
    return choice, histories


def _log_probabilities(m, prompt, tokens):
    """Sum of the log-probabilities of `tokens` after the prompt, the whole text served in one pass. Logits are those of
    the kernels' own 16-bit rows, taken to fp32 sums."""
    text = prompt + tokens[:-1]
    n = len(text)
    M = -(-n // 64)
    pools = m.pools(M)
    x = m.run(_i32(text), pools, _i32([list(range(M))]), _i32([0, n]), _i32([n]), _i32(list(range(n))), n)
    logp = torch.log_softmax((x.double() @ m.head.double()), -1)
    return sum(float(logp[len(prompt) - 1 + i, t]) for i, t in enumerate(tokens))


@pytest.mark.parametrize("K,steps", [(1, 6), (4, 12), (3, 70)])
def test_beams_have_the_scores_of_their_texts(K, steps):
    """Every hypothesis at the end, served again from the start in one pass, has the sum of log-probabilities that the
    search kept through its forks and copies: its cache was its own text's all along.

    Bound per token: the two passes' normalised rows differ by twice the layer's error (3.4e-3 each, in two layers:
    1e-2 of their RMS of one), a logit of deviation 3 is a sum over them: 3e-2 RMS; the log-softmax is that and the
    mean's. 6 sigma of independent tokens' sums: 6 x 4e-2 x sqrt(tokens)."""
    m = Model(seed=K)
    g = torch.Generator().manual_seed(K)
    prompts = [torch.randint(4, m.V, (n,), generator=g).tolist() for n in (5, 64, 150)]
    choice, histories = _search(m, prompts, K, steps)
    for b, prompt in enumerate(prompts):
        for k in range(K):
            tokens = histories[b][k]
            want = _log_probabilities(m, prompt, tokens)
            got = choice.scores[b, k].item()
            assert abs(got - want) <= 0.24 * len(tokens) ** 0.5, (b, k, got, want)
            assert choice.lengths[b, k].item() == len(tokens)
        if K > 1:
            assert len({tuple(h) for h in histories[b]}) == K
    if K == 1:  # greedy
        for b, prompt in enumerate(prompts):
            text = prompt + histories[b][0]
            better = text[:-1] + [(text[-1] + 1) % m.V]
            assert _log_probabilities(m, prompt, better[len(prompt):]) < choice.scores[b, 0].item() + 0.5


def test_a_captured_step_is_the_eager_one():
    m = Model(seed=9)
    prompts = [[7, 8, 9, 10], [11] * 63]
    a, b = _search(m, prompts, 4, 8), _search(m, prompts, 4, 8, graph=True)
    assert a[1] == b[1] and all(torch.equal(x, y) for x, y in zip(a[0], b[0]))


def test_columns_beyond_the_vocabulary_are_never_chosen():
    m = Model(seed=4)
    m.head[:, 400:] *= 50
    choice, histories = _search(m, [[5, 6, 7]], 4, 4, vocabulary=400)
    assert max(t for h in histories[0] for t in h) < 400


def test_a_step_of_no_sequences():
    """An empty batch: empty choices, and the plan of the others' counts alone."""
    m = Model(seed=2)
    refs = _i32([0, 2, 0, 1])
    choice, plan = da.beam_step(m.head.new_empty(0, m.head.shape[0]), m.head, torch.empty(0, 4, device="cuda"), da.page_pools(*m.pools(4)),
                                torch.empty(0, 3, dtype=torch.int32, device="cuda"), _i32([]), refs, eos=EOS,
                                finished=torch.empty(0, 4, dtype=torch.bool, device="cuda"))
    assert choice.tokens.shape == (0, 4) and plan.table.shape == (0, 3) and plan.copies.shape == (0, 3)
    assert torch.equal(plan.refs, refs) and plan.info.tolist() == [0, 0, 2, 2]
