"""Host side of the beam search and page calls: refusals before any launch, workspace bounds, and the
references' own agreement with torch. No GPU."""

import ctypes
import math

import pytest
import torch

import beam_reference as ref
import differential_attention_02_gb300 as da
from differential_attention_02_gb300 import build as dab

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    dab.build()
    return da.load_library()


def _select(lib, **kw):
    a = dict(logits=0x10000, sb=4000, sk=1000, dt=da.BF16, scores=0x20000, fin=None, lens=None, eos=-1, pen=0.0, B=2, K=4, V=1000, W=8,
             so=0x30000, tok=0x31000, par=0x32000, fo=None, lo=None, ws=0x100000, wsb=1 << 30)
    a.update(kw)
    return lib.diffattn_beam_select(*a.values(), None)


def test_select_refusals(lib):
    assert _select(lib, B=0) == da.OK and _select(lib, B=0, fin=0x40000, eos=5, fo=0x41000, lens=0x42000, lo=0x43000, pen=1.0) == da.OK
    for kw in (dict(B=-1), dict(K=0), dict(K=33), dict(V=0), dict(V=(1 << 20) + 1), dict(W=0), dict(W=65), dict(W=3, K=1, V=2), dict(B=65536),
               dict(dt=7), dict(eos=-2), dict(eos=1000), dict(fin=0x40000), dict(fo=0x40000), dict(pen=NAN), dict(pen=INF), dict(pen=0.5),
               dict(lo=0x40000), dict(logits=None), dict(logits=0x10001), dict(logits=0x10002, dt=da.F32), dict(scores=None),
               dict(scores=0x20002), dict(so=None), dict(tok=None), dict(par=None), dict(par=0x32001), dict(sb=-4), dict(sk=-4),
               dict(lens=0x40002)):
        assert _select(lib, **kw) == da.ERR_INVALID_ARG, kw
    for kw in (dict(ws=None), dict(ws=0x100080), dict(wsb=256)):
        assert _select(lib, **kw) == da.ERR_WORKSPACE, kw


def test_workspace_sizes(lib):
    n = ctypes.c_size_t()
    assert lib.diffattn_beam_workspace_size(2, 4, 1000, 8, None) == da.ERR_INVALID_ARG
    assert lib.diffattn_beam_workspace_size(2, 33, 1000, 8, ctypes.byref(n)) == da.ERR_INVALID_ARG
    assert da.beam_workspace_bytes(0, 1, 1, 1) >= 256 and da.beam_workspace_bytes(64, 8, 1000, 16) >= 512 * 16 * 8


def _state(**kw):
    a = dict(ptr=0x10000, ss=4096, sp=1024, sr=64, parts=4, rows=16, width=64, by_len=0)
    a.update(kw)
    return da._PACK_STATE(*a.values())


def test_reorder_refusals(lib):
    def call(state=None, count=1, parents=0x20000, lens=None, B=2, K=4, null=False):
        return lib.diffattn_beam_reorder(None if null else (state or _state()) * max(count, 1), count, parents, lens, B, K, None)
    assert call(B=0) == da.OK and call(count=0) == da.OK and call(count=0, null=True) == da.OK
    for kw in (dict(B=-1), dict(B=65536), dict(K=0), dict(K=33), dict(count=-1), dict(null=True), dict(parents=None), dict(parents=0x20002),
               dict(lens=0x20001), dict(state=_state(by_len=1)), dict(state=_state(ptr=0)), dict(state=_state(parts=-1)),
               dict(state=_state(rows=-1)), dict(state=_state(width=-16)), dict(state=_state(ss=-4)), dict(state=_state(sr=-4)),
               dict(state=_state(rows=1 << 20, width=1 << 12)), dict(state=_state(rows=1 << 10, width=1 << 18), B=60000)):
        assert call(**kw) == da.ERR_INVALID_ARG, kw


def _fork(lib, **kw):
    a = dict(table=0x10000, lens=0x20000, refs=0x30000, parents=0x40000, new=None, done=None, grow=1, to=0x50000, lo=0x60000, ro=0x70000,
             copies=0x80000, info=0x90000, B=2, K=4, M=16, P=100)
    a.update(kw)
    return lib.diffattn_pages_fork(*a.values(), None)


def test_fork_refusals(lib):
    for kw in (dict(B=-1), dict(K=0), dict(B=1025), dict(M=0), dict(P=0), dict(M=1 << 29), dict(table=None), dict(lens=None), dict(refs=None),
               dict(to=None), dict(lo=None), dict(ro=None), dict(copies=None), dict(info=None), dict(table=0x10002), dict(parents=0x40001),
               dict(new=0x40002), dict(to=0x10004), dict(lo=0x20004), dict(ro=0x30004), dict(ro=0x30000 - 396)):
        assert _fork(lib, **kw) == da.ERR_INVALID_ARG, kw


def test_compact_refusals(lib):
    def call(**kw):
        a = dict(table=0x10000, lens=0x20000, refs=0x30000, to=0x50000, ro=0x70000, moved=0x80000, copies=0x90000, most=50, info=0xa0000,
                 S=8, M=16, P=100)
        a.update(kw)
        return lib.diffattn_pages_compact(*a.values(), None)
    for kw in (dict(S=-1), dict(S=4097), dict(M=0), dict(P=0), dict(most=-1), dict(most=51), dict(table=None), dict(lens=None), dict(refs=None),
               dict(to=None), dict(ro=None), dict(moved=None), dict(copies=None), dict(info=None), dict(to=0x10004), dict(ro=0x30008),
               dict(moved=0x80001)):
        assert call(**kw) == da.ERR_INVALID_ARG, kw


def test_copy_refusals(lib):
    pool = lambda **kw: da._PACK_POOL(*{**dict(ptr=0x10000, sp=65536, sh=8192, sr=128, heads=4, width=128), **kw}.values())  # noqa: E731

    def call(p=None, count=1, copies=0x20000, n=None, most=4, P=100, null=False):
        return lib.diffattn_pages_copy(None if null else (p or pool()) * max(count, 1), count, copies, n, most, P, None)
    assert call(count=0) == da.OK and call(most=0, copies=None) == da.OK
    for kw in (dict(count=-1), dict(most=-1), dict(P=0), dict(null=True), dict(copies=None), dict(copies=0x20002), dict(n=0x20001),
               dict(p=pool(ptr=0)), dict(p=pool(ptr=0x10008)), dict(p=pool(sp=100)), dict(p=pool(sh=-16)), dict(p=pool(sr=120)),
               dict(p=pool(heads=0)), dict(p=pool(width=0)), dict(p=pool(width=24)), dict(p=pool(width=1 << 21))):
        assert call(**kw) == da.ERR_INVALID_ARG, kw


ELSEWHERE = torch.device("meta")  # another device than the operands', without memory


@pytest.fixture
def no_launch(monkeypatch):
    monkeypatch.setattr(da, "_elsewhere", lambda dev, stream: None)
    monkeypatch.setattr(da, "_check", lambda *a: pytest.fail("launched"))
    monkeypatch.setattr(da, "_raw_stream", lambda index: pytest.fail("launched"))


def test_select_checks_its_tensors(no_launch):
    z, i32 = torch.zeros, torch.int32
    logits, scores, ended, n = z(2, 3, 50), z(2, 3), z(2, 3, dtype=torch.bool), z(2, 3, dtype=i32)
    away = lambda t: torch.empty(t.shape, dtype=t.dtype, device=ELSEWHERE)  # noqa: E731
    out = lambda **kw: da.BeamChoice(**{**dict(scores=z(2, 3), tokens=z(2, 3, dtype=i32), parents=z(2, 3, dtype=i32),  # noqa: E731
                                               finished=None, lengths=None), **kw})
    for args, kw in (((logits[0], scores), {}), ((logits.transpose(1, 2), scores), {}), ((logits[..., ::2], scores), {}),
                     ((logits.double(), scores), {}), ((logits, scores.double()), {}), ((logits, scores[:1]), {}), ((logits, scores.T), {}),
                     ((logits, away(scores)), {}), ((logits, scores), dict(finished=ended)), ((logits, scores), dict(finished=n, eos=1)),
                     ((logits, scores), dict(finished=away(ended), eos=1)), ((logits, scores), dict(lengths=n.long())),
                     ((logits, scores), dict(lengths=n[:, :2])), ((logits, scores), dict(out=out(tokens=z(2, 3)))),
                     ((logits, scores), dict(out=out(scores=z(2, 4)))), ((logits, scores), dict(out=out(parents=away(n)))),
                     ((logits, scores), dict(width=2, out=out()))):
        with pytest.raises(ValueError):
            da.diffattn_beam_select(*args, **kw)


def test_page_calls_check_their_tensors(no_launch):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    table, lens, refs = i32(6, 4), i32(6), i32(20)
    plan = lambda **kw: da.PagePlan(**{**dict(table=i32(6, 4), lens=i32(6), refs=i32(20), copies=i32(6, 3), info=i32(4)), **kw})  # noqa: E731
    bad = [((table.long(), lens, refs), {}), ((table[0], lens, refs), {}), ((table, lens[:5], refs), {}), ((table, lens, refs.float()), {}),
           ((table, lens, i32(2, 10)), {}), ((i32(6, 8)[:, ::2], lens, refs), {}),
           ((table, lens, torch.empty(20, dtype=torch.int32, device=ELSEWHERE)), {})]
    for args, kw in bad:
        with pytest.raises(ValueError):
            da.diffattn_pages_fork(*args, **kw)
        with pytest.raises(ValueError):
            da.diffattn_pages_compact(*args, **kw)
    for kw in (dict(parents=i32(6)), dict(parents=i32(2, 2)), dict(parents=i32(2, 3).long()), dict(new_lens=i32(5)), dict(done=i32(6)),
               dict(done=torch.zeros(5, dtype=torch.bool)), dict(out=plan(table=i32(6, 5))), dict(out=plan(copies=i32(5, 3))),
               dict(out=plan(info=i32(3))), dict(out=plan(refs=i32(20).long()))):
        with pytest.raises(ValueError):
            da.diffattn_pages_fork(table, lens, refs, **kw)
    for kw in (dict(out=plan()), dict(out=plan(copies=i32(11, 3), moved=i32(20))), dict(out=plan(copies=i32(10, 2), moved=i32(20))),
               dict(out=plan(copies=i32(10, 3), moved=i32(19)))):
        with pytest.raises(ValueError):
            da.diffattn_pages_compact(table, lens, refs, **kw)


def test_pools_and_states_are_checked(no_launch):
    bf = torch.bfloat16
    page = torch.zeros(5, 2, 64, 64, dtype=bf)
    assert len(da.page_pools((page, page), page).tensors) == 3 and len(da.page_pools([(page, page), (page,)]).tensors) == 3
    for bad in ((), (page[0],), (page, page[:4]), (page[:, :, :32],), (page[..., ::2],), (page[:, :, :1].expand(5, 2, 64, 64),),
                (page, torch.empty(5, 2, 64, 64, dtype=bf, device=ELSEWHERE))):
        with pytest.raises(ValueError):
            da.page_pools(*bad)
    pools, i32 = da.page_pools(page), lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    for args in ((i32(4, 2),), (i32(12),), (i32(4, 3).long(),), (i32(4, 3), i32(1)), (i32(3, 4).T,)):
        with pytest.raises(ValueError):
            da.diffattn_pages_copy(pools, *args)
    state, parents = torch.zeros(6, 10), i32(2, 3)
    for args in (([state], i32(6)), ([state], parents.long()), ([state[:5]], parents), ([state[:, ::2]], parents), ([state[:1].expand(6, 10)], parents),
                 ([torch.zeros(6, 2, 9, 64)], parents, i32(5)), ([state], parents, i32(6)), ([torch.zeros(6, 2, 9, 64)[..., ::2]], parents, i32(6)),
                 ([torch.zeros(6, 2, 1, 64).expand(6, 2, 9, 64)], parents, i32(6)),
                 ([torch.empty(6, 10, device=ELSEWHERE)], parents)):
        with pytest.raises(ValueError):
            da.diffattn_beam_reorder(*args)


def test_beam_step_checks_its_tensors(no_launch, monkeypatch):
    monkeypatch.setattr(da, "gemm", lambda *a, **k: pytest.fail("launched"))
    bf, i32 = torch.bfloat16, lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    pools = da.page_pools(torch.zeros(5, 2, 64, 64, dtype=bf))
    x, w, scores = torch.zeros(6, 32, dtype=bf), torch.zeros(32, 80, dtype=bf), torch.zeros(2, 3)
    for args, kw in (((x[:5], w, scores, pools, i32(6, 4), i32(6), i32(5)), {}), ((x, w, scores[0], pools, i32(6, 4), i32(6), i32(5)), {}),
                     ((x, w, scores, pools, i32(5, 4), i32(5), i32(5)), {}), ((x, w, scores, pools, i32(6, 4), i32(6), i32(6)), {}),
                     ((x, w, scores, pools, i32(6, 4), i32(6), i32(5)), dict(vocabulary=81)),
                     ((x, w.to(ELSEWHERE), scores, pools, i32(6, 4), i32(6), i32(5)), {})):
        with pytest.raises(ValueError):
            da.beam_step(*args, **kw)


def test_numbers_beyond_31_bits_are_refused(no_launch):
    """They would reach the library cut off: a width of 2^32 + 3 as 3."""
    far, on = 1 << 32, dict(device=ELSEWHERE)  # (without memory)
    logits, scores = torch.zeros(2, 3, 50), torch.zeros(2, 3)
    for kw in (dict(width=0), dict(width=-far + 3), dict(width=far + 3), dict(eos=far + 5), dict(eos=-far + 5), dict(eos=50), dict(eos=-1)):
        with pytest.raises(ValueError):
            da.diffattn_beam_select(logits, scores, **kw)
    with pytest.raises(ValueError):
        da.diffattn_beam_select(torch.empty(1, 1, far + 50, **on), torch.empty(1, 1, **on))
    with pytest.raises(ValueError):
        da.diffattn_beam_select(torch.empty(far + 1, 1, 2, **on), torch.empty(far + 1, 1, **on))
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, **on)  # noqa: E731
    for grow in (far + 1, -far - 1, 1 << 31):
        with pytest.raises(ValueError):
            da.diffattn_pages_fork(i32(6, 4), i32(6), i32(20), grow=grow)
    for state in ((i32(far + 1, 1), i32(far + 1), i32(20)), (i32(1, far + 1), i32(1), i32(20)), (i32(6, 4), i32(6), i32(far + 20))):
        with pytest.raises(ValueError):
            da.diffattn_pages_fork(*state)
        with pytest.raises(ValueError):
            da.diffattn_pages_compact(*state)
    with pytest.raises(ValueError):
        da.diffattn_beam_reorder([torch.empty(far + 2, 4, **on)], i32(far // 2 + 1, 2))
    with pytest.raises(ValueError):
        da.diffattn_pages_copy(da.page_pools(torch.empty(5, 2, 64, 64, **on)), i32(far + 3, 3))


def test_the_reference_selects_like_a_sort():
    """beam_reference.select against torch's log_softmax and a stable sort over beams and tokens."""
    g = torch.Generator().manual_seed(1)
    logits, scores = torch.randn(3, 4, 90, generator=g).double(), -torch.rand(3, 4, generator=g)
    all_ = (scores.double()[..., None] + torch.log_softmax(logits, -1)).flatten(1)
    v, i = all_.sort(stable=True, dim=-1, descending=True)
    want = ref.select(logits, scores, 12)
    for b in range(3):
        assert [w[2] * 90 + w[1] for w in want[b]] == i[b, :12].tolist()
        assert max(abs(w[0] - x) for w, x in zip(want[b], v[b].tolist())) < 1e-12
    assert ref.select(torch.full((1, 1, 4), -math.inf), torch.zeros(1, 1), 2) == [[(-math.inf, 0, -1, True, 0)] * 2]


def test_the_reference_forks_keep_texts():
    """Texts held in the reference's pages survive its forks and compactions."""
    import random
    rng = random.Random(2)
    S, M, P = 6, 5, 40
    table, lens, refs, texts = [[-1] * M] * S, [0] * S, [0] * P, [[] for _ in range(S)]
    pool = [[None] * 64 for _ in range(P)]
    for step in range(60):
        parents = [[rng.choice([i, i, rng.randrange(S), -1]) for i in range(S)]]
        new = [max(0, (lens[p] if p >= 0 else 0) + rng.choice([1, 1, 40, -20])) for p in parents[0]]
        new = [min(n, M * 64) for n in new]
        old = lens
        table, lens, refs, copies, info = ref.fork(table, lens, refs, parents, 0, new)
        pages = [list(p) for p in pool]
        for src, dst, rows in copies:
            if src >= 0:
                pool[dst][:rows] = pages[src][:rows]
        assert info[1] == 0
        before, texts = texts, []
        for i, p in enumerate(parents[0]):
            text = (before[p] if p >= 0 else [])[:min(new[i], old[p] if p >= 0 else 0)]
            for at in range(len(text), new[i]):
                text = text + [rng.random()]
                pool[table[i][at // 64]][at % 64] = text[-1]
            texts.append(text)
        if step % 9 == 0:
            table, refs, copies, _, _ = ref.compact(table, lens, refs)
            pages = [list(p) for p in pool]
            for src, dst, rows in copies:
                if src >= 0:
                    pool[dst] = pages[src]
        for i in range(S):
            assert [pool[table[i][at // 64]][at % 64] for at in range(lens[i])] == texts[i]
