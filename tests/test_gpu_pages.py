"""Forks, compactions and copies of a paged cache's pages on the GPU: whole numbers and bytes, equal to the
references' that take one row and page after the other."""

import random

import pytest
import torch

import beam_reference as ref
import differential_attention_02_gb300 as da

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn
PAGE = 64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from differential_attention_02_gb300 import build
    build.build()
    da.load_library()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _table(x, M):
    return _i32(x).view(len(x), M)


def _fork(table, lens, refs, parents=None, grow=0, new_lens=None, done=None, out=None):
    """The kernel's plan, checked against the reference's."""
    M = len(table[0])
    args = [_table(table, M), _i32(lens), _i32(refs)]
    if out == "in place":
        out = da.PagePlan(*args, _i32([[7] * 3] * len(table)), _i32([0] * 4))
    p = da.diffattn_pages_fork(*args, None if parents is None else _i32(parents), grow, None if new_lens is None else _i32(new_lens),
                               None if done is None else torch.tensor(done, device="cuda"), out=out)
    want = ref.fork(table, lens, refs, parents, grow, new_lens, done)
    for name, got, w in zip(p._fields, p, want):
        assert got.tolist() == w, name
    return want


def _state(rng, S, M, P, shared=True):
    """A random consistent state: rows that share prefixes, in shuffled pages."""
    order = list(range(P))
    rng.shuffle(order)
    table, lens, refs = [], [], [0] * P
    for i in range(S):
        n = rng.choice([0, 1, 63, 64, 65, rng.randint(0, M * PAGE), rng.randint(0, M * PAGE)])
        n = min(n, M * PAGE)
        row = []
        if shared and i and rng.random() < 0.5:
            j = rng.randrange(i)
            row = table[j][:rng.randint(0, min(lens[j], n) // PAGE)]
        while len(row) < ref.pages(n) and order:
            row.append(order.pop())
        n = min(n, len(row) * PAGE)
        row = row[:ref.pages(n)]
        for p in row:
            refs[p] += 1
        table.append(row + [rng.choice([-1, 0, 5]) for _ in range(M - len(row))])  # what lies behind is none of theirs
        lens.append(n)
    return table, lens, refs


@pytest.mark.parametrize("seed", range(12))
def test_random_forks(seed):
    """Every kind of step on random states, in place and apart."""
    rng = random.Random(seed)
    S, M = rng.choice([1, 2, 7, 24, 60, 130]), rng.choice([1, 2, 5, 16, 33, 140])
    P = rng.choice([max(4, S * M // 2), S * M + 3, S * M + 1500])
    table, lens, refs = _state(rng, S, M, P)
    for step in range(4):
        K = rng.choice([k for k in (1, 2, 3, 4, 5, S) if S % k == 0])
        parents = rng.choice([None, [[rng.choice([-1, 0, k, rng.randrange(K), K]) for k in range(K)] for _ in range(S // K)]])
        new_lens = rng.choice([None, [rng.randint(-1, M * PAGE + 70) if rng.random() < 0.5 else n + 1 for n in lens]])
        done = rng.choice([None, [rng.random() < 0.3 for _ in range(S)]])
        table, lens, refs, _, _ = _fork(table, lens, refs, parents, rng.choice([0, 1, 5, 64, 200, -3]), new_lens, done,
                                        rng.choice([None, "in place"]))


def test_a_life_of_sequences_keeps_its_counts():
    """Prompts, growth, sharing, roll-back and ends: the counts are always those of the table's rows, no page is held by
    two begun rows, and in the end all pages are free."""
    rng = random.Random(5)
    S, M, P = 12, 9, 60
    table, lens, refs = [[-1] * M] * S, [0] * S, [0] * P
    for step in range(30):
        if step == 29:
            parents, new = None, [0] * S
        else:
            parents = [[rng.choice([i, i, i, rng.randrange(S), -1]) for i in range(S)]]
            new = [rng.choice([lens[p] + 1, lens[p] + 70, max(0, lens[p] - 30)]) if p >= 0 else rng.randint(0, 200) for p in parents[0]]
        table, lens, refs, copies, info = _fork(table, lens, refs, parents, 0, new)
        held = [p for row, n in zip(table, lens) for p in row[:ref.pages(n)] if p >= 0]
        assert refs == [held.count(p) for p in range(P)]
        begun = [row[n // PAGE] for row, n in zip(table, lens) if n % PAGE and row[n // PAGE] >= 0]
        assert len(set(begun)) == len(begun) and all(refs[p] == 1 for p in begun)
    assert info == [0, 0, P, 0]


def test_beams_from_one_prompt():
    """Four beams continue one prompt: whole pages shared, three copies of the begun one; then two of them go on."""
    table, lens, refs = [[5, 2, 9, -1]] + [[-1] * 4] * 3, [150, 0, 0, 0], [0, 0, 1, 0, 0, 1, 0, 0, 0, 1]
    table, lens, refs, copies, info = _fork(table, lens, refs, [[0, 0, 0, 0]], 1)
    assert table == [[5, 2, 9, -1], [5, 2, 0, -1], [5, 2, 1, -1], [5, 2, 3, -1]] and lens == [151] * 4
    assert copies[:3] == [[9, 0, 22], [9, 1, 22], [9, 3, 22]] and info == [3, 0, 4, 6]
    table, lens, refs, copies, info = _fork(table, lens, refs, [[2, 2, 0, -1]], 1)
    assert table == [[5, 2, 1, -1], [5, 2, 0, -1], [5, 2, 9, -1], [-1] * 4] and copies[0] == [1, 0, 23] and info[0] == 1


def test_a_begun_page_that_others_hold_is_copied():
    """A kept prefix whose count is one higher: no row may write its begun page."""
    _fork([[3, 1], [3, 1]], [100, 100], [0, 3, 0, 3, 0], [[0, 1]], 1)
    _fork([[3, 1], [3, 1]], [100, 100], [0, 2, 0, 2, 0, 0], [[0, 1]], 1)
    _fork([[3, 1], [3, 1]], [100, 100], [0, 1, 0, 1, 0, 0], [[1, 1]], 1)   # counts too low
    _fork([[3, 1], [1, 3]], [64, 100], [0, 2, 0, 2, 0, 0], None, 1)        # a whole page of one is the other's begun one


def test_pages_that_cannot_be_had():
    """A full pool, a full table, and entries outside the pool."""
    want = _fork([[0, 1], [2, -1], [-1, -1]], [100, 64, 0], [1, 1, 1, 0], [[0, 0, 1]], 0, [128, 101, 65])
    assert want[4][1] == 1
    _fork([[0, 1], [2, 3]], [128, 128], [1, 1, 1, 1, 0], None, 70)         # beyond the table
    _fork([[7, -3, 2], [0, 99, 1]], [180, 150], [1, 1, 1, 0, 0], [[1, 1]], 3)
    _fork([[-1, -1], [99, 0]], [30, 10], [0, 0, 0], None, 1)               # begun pages that are none
    _fork([[0]], [1000], [1], None, 1)                                     # a length beyond the table
    _fork([[0], [1]], [-5, 3], [-4, 1], None, 1)                           # a count below zero is free


def test_sizes_at_the_limits():
    for S, M, P in ((4096, 1, 5000), (4096, 9, 70000), (1, 5000, 6000), (3000, 8, 20000), (1025, 3, 3500)):
        rng = random.Random(S)
        table, lens, refs = _state(rng, S, M, P, shared=False)
        K = S if S % 4 else 4
        parents = [[rng.randrange(K) if rng.random() < 0.3 else k for k in range(K)] for _ in range(S // K)]
        _fork(table, lens, refs, parents, 1)
    p = da.diffattn_pages_fork(_i32([]).view(0, 4), _i32([]), _i32([1, 0, -2]))
    assert p.refs.tolist() == [1, 0, 0] and p.info.tolist() == [0, 0, 2, 1]


def test_pages_at_even_distances():
    """A fixed reservation a sequence, 128 or 8192 pages apart."""
    for S, step in ((64, 128), (512, 128), (100, 8192)):
        table = [[i * step, i * step + 1] for i in range(S)]
        refs = [0] * (S * step)
        for row in table:
            refs[row[0]] = refs[row[1]] = 1
        _fork(table, [100] * S, refs, [[max(0, i - i % 3) for i in range(S)]], 1)


def test_a_pool_of_many_pages():
    """More pages than 32 a thread."""
    rng = random.Random(3)
    P, S, M = 400000, 6, 40
    refs = [rng.choice([1, 1, 1, 1, 0, -1]) for _ in range(P)]
    table = [[rng.randrange(P) for _ in range(M)] for _ in range(S)]
    for row in table:
        for p in row:
            refs[p] = max(refs[p], 0) + 1
    lens = [M * PAGE - 5 * i for i in range(S)]
    _fork(table, lens, refs, [[0, 0, 1, 5, 5, -1]], 3)
    _fork(table, lens, refs, None, 0, [0, 2500, 0, 0, 2000, 10])
    args = [_table(table, M), _i32(lens), _i32(refs)]
    p = da.diffattn_pages_compact(*args)
    want = ref.compact(table, lens, refs)
    assert (p.table.tolist(), p.refs.tolist(), p.copies.tolist(), p.info.tolist(), p.moved.tolist()) == want


@pytest.mark.parametrize("seed", range(10))
def test_random_compactions(seed):
    rng = random.Random(seed)
    S, M, P = rng.choice([0, 1, 5, 40]), rng.choice([1, 3, 20]), rng.choice([1, 2, 7, 64, 1500, 5000])
    table, lens, refs = _state(rng, S, M, P)
    for p in range(P):
        if rng.random() < 0.2:
            refs[p] += rng.choice([1, -2 if refs[p] == 0 else 1])  # holders of other tables, counts below zero
    most = rng.choice([None, None, 0, P // 4])
    args = [_table(table, M) if S else _i32([]).view(0, M), _i32(lens), _i32(refs)]
    out = None
    if most is not None or seed % 2:
        most = P // 2 if most is None else most
        mine = args if seed % 4 < 2 else [a.clone() for a in args]  # in place, or apart
        out = da.PagePlan(mine[0], args[1], mine[2], _i32([[5] * 3] * most).view(most, 3), _i32([0] * 4), _i32([9] * P))
    p = da.diffattn_pages_compact(*args, out=out)
    table, refs, copies, info, moved = ref.compact(table, lens, refs, most)
    assert (p.table.tolist(), p.refs.tolist(), p.copies.tolist(), p.info.tolist(), p.moved.tolist()) == (table, refs, copies, info, moved)


def _pools(P, H, d, dtype, layers, seed, strided=False):
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(layers):
        if strided:  # K1, K2 and V side by side, tokens outside the heads
            x = torch.randn(P, 64, H + 1, 4 * d, generator=g).to(dtype).cuda().transpose(1, 2)[:, :H]
            out.append((x[..., :d], x[..., d:2 * d], x[..., 2 * d:]))
        else:
            out.append(tuple(torch.randn(P, H, 64, w, generator=g).to(dtype).cuda() for w in (d, d, 2 * d)))
    return out


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("P,H,d,layers,n", [(2, 1, 64, 1, 1), (40, 3, 64, 2, 13), (30, 2, 128, 1, 15), (9, 5, 72, 1, 4), (16, 1, 64, 17, 3)])
def test_copies(P, H, d, layers, n, dtype, strided):
    """Whole and begun pages, entries that are skipped, and every other byte as it was."""
    if dtype == F8 and d % 16:
        d = 80
    rng = random.Random(P)
    pools = _pools(P, H, d, dtype, layers, seed=n, strided=strided)
    order = list(range(P))
    rng.shuffle(order)
    copies = [[order[i], order[n + i] if n + i < P else -1, rng.choice([64, 1, 63, 31, rng.randint(0, 70), -2])] for i in range(n)]
    copies += [[-1, 0, 64], [P, 0, 64], [0, P + 3, 64], [0, -1, 64]]
    flat = [t for p in pools for t in p]
    before = [t.cpu().contiguous() for t in flat]
    handle = da.page_pools(*pools)
    da.diffattn_pages_copy(handle, _i32(copies))
    for t, b in zip(flat, before):
        assert torch.equal(t.cpu().contiguous().view(torch.uint8), ref.copied(b, copies).view(torch.uint8))
    # only the entries that a plan's info counts
    before = [t.cpu().contiguous() for t in flat]
    back = [[b, a, r] for a, b, r in copies]
    da.diffattn_pages_copy(handle, _i32(back), _i32([n // 2, 0, 0, 0]))
    for t, b in zip(flat, before):
        assert torch.equal(t.cpu().contiguous().view(torch.uint8), ref.copied(b, back[:n // 2]).view(torch.uint8))


def test_copies_far_into_a_large_pool():
    """Byte offsets beyond 32 bits."""
    P = 70000
    pool = torch.zeros(P, 4, 64, 128, dtype=torch.uint8, device="cuda")
    pool[P - 1] = 3
    pool[1] = 5
    da.diffattn_pages_copy(da.page_pools(pool), _i32([[P - 1, 0, 64], [1, P - 2, 10]]))
    assert bool((pool[0] == 3).all()) and bool((pool[P - 2, :, :10] == 5).all()) and not bool(pool[P - 2, :, 10:].any())
    assert not bool(pool[2:P - 2].any())


def test_plans_and_copies_from_a_graph():
    """A step in place, captured once and replayed: fork and copies follow the parents that lie in the buffer."""
    rng = random.Random(1)
    S, K, M, P = 8, 4, 6, 64
    table, lens, refs = [[-1] * M] * S, [0] * S, [0] * P
    table, lens, refs, _, _ = ref.fork(table, lens, refs, None, 0, [70, 0, 0, 0, 130, 0, 0, 0])
    pools = _pools(P, 2, 64, BF, 1, seed=0)
    handle = da.page_pools(*pools)
    plan = da.PagePlan(_table(table, M), _i32(lens), _i32(refs), _i32([[0] * 3] * S), _i32([0] * 4))
    parents = _i32([[0, 0, 0, 0]] * 2)
    host = [t.cpu() for t in pools[0]]

    def step():
        da.diffattn_pages_fork(plan.table, plan.lens, plan.refs, parents, grow=1, out=plan)
        da.diffattn_pages_copy(handle, plan.copies, plan.info)
    graph = None
    for i in range(5):
        if i == 1:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        now = [[0] * K] * 2 if i == 0 else [[rng.randrange(K) for _ in range(K)] for _ in range(2)]
        parents.copy_(_i32(now))
        table, lens, refs, copies, info = ref.fork(table, lens, refs, now, 1)
        host = [ref.copied(t, copies) for t in host]
        step() if graph is None else graph.replay()
        assert (plan.table.tolist(), plan.lens.tolist(), plan.refs.tolist(), plan.info.tolist()) == (table, lens, refs, info)
        assert all(torch.equal(t.cpu(), h) for t, h in zip(pools[0], host))


def test_copies_alone_in_a_graph():
    """Captured with no plan before them: after nothing, and after a copy of the list."""
    pools = _pools(20, 2, 64, BF, 2, seed=3)
    handle = da.page_pools(*pools)
    host = [t.cpu() for p in pools for t in p]
    lists = [[[1, 2, 64], [3, 4, 10]], [[2, 5, 7], [-1, 0, 64]], [[4, 6, 64], [5, 7, 33]]]
    copies, staged = _i32(lists[0]), _i32(lists[0])
    da.diffattn_pages_copy(handle, copies)
    host = [ref.copied(t, lists[0]) for t in host]
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        da.diffattn_pages_copy(handle, copies)
    with torch.cuda.graph(graphs[1]):
        copies.copy_(staged)
        da.diffattn_pages_copy(handle, copies)
    for graph, now in zip(graphs, lists[1:]):
        staged.copy_(_i32(now))
        if graph is graphs[0]:
            copies.copy_(staged)
        graph.replay()
        host = [ref.copied(t, now) for t in host]
        assert all(torch.equal(t.cpu(), h) for t, h in zip((t for p in pools for t in p), host))
