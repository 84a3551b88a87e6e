"""Beam search and the pages of a cache, as cases that can be timed and compared.

Five operators around the paged serving of many sequences:

- select: the best continuations over a sequence's beams and the vocabulary, from logits;
- reorder: per-beam states (contiguous caches, token histories) take the rows of their parents, in place;
- fork: which pages each sequence holds after some continue others, grow, roll back, start or end; full
  pages shared, the begun page copied where two would write it;
- compact: the held pages moved to the front of the pool;
- copy: whole or begun pages copied inside every pool of a cache.

`own` selects the framework's kernels; without it `run` computes the same in elementary torch operations.
"""

import math
import random

import torch

own = False

PAGE = 64
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one sequence with four beams: latency
        dict(name="select_step", op="select", B=1, K=4, W=4, V=32000, dtype="f32", finished=False, alpha=0.0, masked=False),
        # twice as many candidates as beams, some hypotheses ended, tokens banned, odd rows, lengths weighed
        dict(name="select_masked", op="select", B=5, K=5, W=10, V=50001, dtype="f16", finished=True, alpha=0.7, masked=True),
        # a serving batch
        dict(name="select_batch", op="select", B=32, K=4, W=8, V=131072, dtype="bf16", finished=True, alpha=0.0, masked=False),
        # many beams over a large vocabulary of odd size: no row but the first is aligned
        dict(name="select_wide", op="select", B=32, K=8, W=16, V=200003, dtype="bf16", finished=False, alpha=0.0, masked=False),
        # contiguous caches of 64 sequences with the decode workload's heads, ragged lengths
        dict(name="reorder_cache", op="reorder", B=16, K=4, H=16, d=64, L=2048, T=0),
        # token histories and a row of features of each beam, odd sizes: latency
        dict(name="reorder_rows", op="reorder", B=3, K=7, H=0, d=0, L=0, T=777),
        # a step of beam search over a paged cache: beams share their prompt, each gets a page for its next token
        dict(name="fork_beams", op="fork", B=16, K=4, H=4, d=64, cache="bf16", layers=2, L=4096, kind="beams"),
        # a step of a serving batch: sequences end, others take their places with prompts of their own, drafted
        # tokens are taken back, one prompt is continued by several
        dict(name="fork_turnover", op="fork", B=1, K=192, H=2, d=128, cache="fp8", layers=1, L=8192, kind="turnover"),
        # half of a large pool is held, in scattered pages
        dict(name="compact_half", op="compact", S=96, P=4096, H=4, d=64, cache="bf16", layers=1, fill=0.5),
        # a few pages of a nearly full pool
        dict(name="compact_few", op="compact", S=9, P=300, H=2, d=128, cache="fp8", layers=2, fill=0.93),
        # whole pages
        dict(name="copy_pages", op="copy", P=2048, n=700, H=8, d=64, cache="bf16", layers=1, begun=False),
        # three begun pages: latency
        dict(name="copy_begun", op="copy", P=64, n=3, H=4, d=64, cache="bf16", layers=2, begun=True),
    ]


def _log(rng, lo, hi):
    """A whole number whose logarithm is spread evenly over [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select", "select", "reorder", "fork", "fork", "compact", "copy"])
    if op == "select":
        V, K = _log(rng, 100, 262144), rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        B = _log(rng, 1, max(1, min(128, (32 * 8 * 200003) // (K * V))))
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        if dtype == "f32":
            B = max(1, B // 2)
        return dict(op=op, B=B, K=K, W=rng.choice([K, 2 * K]), V=V, dtype=dtype, finished=rng.random() < 0.5,
                    alpha=rng.choice([0.0, 0.0, 0.6, 1.0]), masked=rng.random() < 0.4)
    K = rng.choice([1, 2, 3, 4, 5, 8, 13, 16])
    if op == "reorder":
        B, T = _log(rng, 1, 64 // K), rng.choice([0, 0, _log(rng, 1, 4096)])
        H, d = (0, 0) if T else (rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([64, 128]))
        return dict(op=op, B=B, K=max(K, 2), H=H, d=d, L=0 if T else _log(rng, 1, (2048 * 16 * 64) // (H * d)), T=T)
    cache = dict(H=rng.choice([1, 2, 4, 5]), d=rng.choice([64, 128]), cache=rng.choice(["bf16", "fp8"]))
    size = cache["H"] * cache["d"] // 64
    if op == "fork":
        kind = rng.choice(["beams", "turnover"])
        S = _log(rng, 1, 192)
        B, K = (max(1, S // K), K) if kind == "beams" else (1, S)
        return dict(op=op, B=B, K=K, layers=rng.choice([1, 1, 2]), L=_log(rng, 1, max(64, min(8192, 64 * 8192 // (B * K * size)))),
                    kind=kind, **cache)
    P = _log(rng, 16, max(16, 8192 // size))
    if op == "compact":
        return dict(op=op, S=_log(rng, 1, min(128, P // 4)), P=P, layers=1, fill=round(rng.uniform(0.1, 0.95), 3), **cache)
    return dict(op=op, P=P, n=_log(rng, 1, P // 2 - 1), layers=rng.choice([1, 2]), begun=rng.random() < 0.5, **cache)


def _rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _parents(rng, B, K):
    """Parents as a selection gives them: the best beam has several children, some beams have none."""
    return [[rng.choice([0, rng.randrange(K), rng.randrange(K), k]) for k in range(K)] for _ in range(B)]


def _fork(case):
    """Of each row: its length, the rows that it shares its first pages with and how many, its parent (or -1), and its new
    length. The same for every seed of a case."""
    rng, B, K, L = _rng(case), case["B"], case["K"], case["L"]
    if case["kind"] == "beams":
        lens, owner, shared, parents = [], [], [], _parents(rng, B, K)
        for b in range(B):
            n = rng.randint(max(1, L // 2), L)
            lens += [n] * K
            owner += [b * K] * K
            shared += [rng.randint(0, n // PAGE)] * K
        return lens, owner, shared, parents, None
    lens = [rng.choice([0, rng.randint(1, L), rng.randint(1, L), rng.randint(1, L)]) for _ in range(K)]
    rows = []
    for i, n in enumerate(lens):
        what = rng.random()
        if what < 0.1:      # ends
            rows.append((-1, 0))
        elif what < 0.2 or n == 0:  # another one's prompt takes the place
            rows.append((-1, rng.randint(1, max(1, L // 4))))
        elif what < 0.25:   # continues another sequence's text
            p = rng.randrange(K)
            rows.append((p, lens[p] + 1))
        elif what < 0.45:   # drafted tokens taken back
            rows.append((i, max(0, n - rng.randint(1, 70))))
        else:
            rows.append((i, n + rng.choice([1, 1, 1, 4])))
    return lens, list(range(K)), [0] * K, [[p for p, _ in rows]], [[n for _, n in rows]]


def _pages(n):
    return -(-n // PAGE)


def _sizes(case):
    """Rows, columns and pages of a fork's table and pool."""
    lens, owner, shared, _, new = _fork(case)
    S, M = len(lens), _pages(max(lens + (new[0] if new else []) + [1]) + 4)
    held = sum(_pages(n) - (h if o != i else 0) for i, (n, o, h) in enumerate(zip(lens, owner, shared)))
    return S, M, held + S + 5 + (sum(_pages(n) for n in new[0]) if new else 0)


# ---------------------------------------------------------------- inputs
def _pools(case, P, g):
    """K1, K2 and V pages of each layer."""
    out = []
    for w in (case["d"], case["d"], 2 * case["d"]) * case["layers"]:
        x = torch.randn(P, case["H"], PAGE, w, generator=g, device="cuda")
        out.append((x * 90).clamp(-448, 448).to(torch.float8_e4m3fn) if case["cache"] == "fp8" else x.to(torch.bfloat16))
    return out


def _cuda(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.rand(*shape, generator=g, device="cuda")  # noqa: E731
    s = dict(case=case)
    if case["op"] == "select":
        B, K, V = case["B"], case["K"], case["V"]
        x = torch.randn(B, K, V, generator=g, device="cuda").mul_(2.5)
        if case["masked"]:
            x.masked_fill_(rand(B, K, V) < 0.3, -math.inf)
            x[:, :, 1::7] = torch.finfo(DTYPES[case["dtype"]]).min
            x[0, K - 1] = -math.inf  # nothing may follow this one
        s["logits"] = x.to(DTYPES[case["dtype"]])
        s["scores"] = -(1 + 20 * rand(B, K)).sort(-1).values
        if case["masked"]:
            s["scores"][B - 1, 1:] = -math.inf  # a sequence that has just begun
        s["lengths"] = (5 + 60 * rand(B, K)).to(torch.int32)
        s["finished"] = rand(B, K) < 0.2 if case["finished"] else None
        return s
    if case["op"] == "reorder":
        B, K, rng = case["B"], case["K"], _rng(case)
        s["parents"] = _cuda(_parents(rng, B, K))
        S = B * K
        if case["T"]:
            s["states"] = [torch.randint(0, 50000, (S, case["T"]), generator=g, device="cuda", dtype=torch.int32), rand(S, 1025)]
            s["lens"] = None
        else:
            s["states"] = [torch.randn(S, case["H"], case["L"], w, generator=g, device="cuda").to(torch.bfloat16)
                           for w in (case["d"], case["d"], 2 * case["d"])]
            s["lens"] = _cuda(_reorder_lens(case))
        return s
    if case["op"] == "fork":
        lens, owner, shared, parents, new = _fork(case)
        S, M, P = _sizes(case)
        first = [_pages(n) - (h if o != i else 0) for i, (n, o, h) in enumerate(zip(lens, owner, shared))]
        order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
        n, own_pages = _cuda([_pages(x) for x in lens])[:, None].long(), _cuda(first)[:, None].long()
        start = own_pages.cumsum(0) - own_pages
        col = torch.arange(M, device="cuda")
        at = (start + col - (n - own_pages)).clamp(0, P - 1)
        table = torch.where(col < n, order[at], -1)
        o = _cuda(owner).long()
        s["table"] = torch.where(col < (n - own_pages), table[o], table).to(torch.int32).contiguous()
        s["refs"] = torch.zeros(P + 1, dtype=torch.int32, device="cuda").index_add_(
            0, s["table"].flatten() % (P + 1), torch.ones(S * M, dtype=torch.int32, device="cuda"))[:P].contiguous()
        s["lens"], s["parents"], s["pools"] = _cuda(lens), _cuda(parents), _pools(case, P, g)
        s["new_lens"] = None if new is None else _cuda(new).view(-1)
    elif case["op"] == "compact":
        P, counts = case["P"], _held(case)
        order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
        n = _cuda(counts)[:, None].long()
        M = max(max(counts), 1)
        col = torch.arange(M, device="cuda")
        s["table"] = torch.where(col < n, order[(n.cumsum(0) - n + col).clamp(max=P - 1)], -1).to(torch.int32).contiguous()
        # a page that two sequences share, where there are two
        if len(counts) > 1 and counts[0] and counts[1]:
            s["table"][1, 0] = s["table"][0, 0]
        s["refs"] = torch.zeros(P + 1, dtype=torch.int32, device="cuda").index_add_(
            0, s["table"].flatten() % (P + 1), torch.ones(s["table"].numel(), dtype=torch.int32, device="cuda"))[:P].contiguous()
        s["lens"], s["pools"] = _cuda([max(0, PAGE * c - 5) for c in counts]), _pools(case, P, g)
    else:
        P, N = case["P"], case["n"]
        order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
        rows = torch.randint(1, PAGE, (N,), generator=g, device="cuda").to(torch.int32) if case["begun"] else torch.full_like(order[:N], PAGE)
        s["copies"] = torch.stack((order[:N], order[N:2 * N], rows), 1).contiguous()
        s["pools"] = _pools(case, P, g)
    if own:
        import differential_attention_02_gb300 as da
        s["handle"] = da.page_pools(s["pools"])
    return s


def _reorder_lens(case):
    rng = _rng(case)
    n = [rng.randint(max(1, case["L"] // 2), case["L"]) for _ in range(case["B"])]
    n[-1] = case["L"]
    return [x for x in n for _ in range(case["K"])]


def _held(case):
    """Pages of each sequence."""
    rng, total = _rng(case), int(case["P"] * case["fill"])
    cuts = sorted(rng.randint(0, total) for _ in range(case["S"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


# ---------------------------------------------------------------- the plain forms
EOS = 2


def _plain_select(s):
    case = s["case"]
    B, K, W, V = case["B"], case["K"], case["W"], case["V"]
    x = s["logits"].float()
    m = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    # scores that lie next to each other are told apart in 64 bits
    total = torch.exp(x - m).sum(-1, keepdim=True, dtype=torch.float64)
    logp = x.double().sub_(m.double()).sub_(torch.log(total))
    score = logp.add_(s["scores"].double()[..., None]).masked_fill_(total == 0, -math.inf)
    length = s["lengths"] + 1
    if s["finished"] is not None:
        ended = s["finished"][..., None]
        score.masked_fill_(ended, -math.inf)
        score[..., EOS] = torch.where(s["finished"], s["scores"].double(), score[..., EOS])
        length = length - s["finished"].int()
    rank = score / length.clamp(min=1).double().pow(case["alpha"])[..., None]
    rank, score = rank.flatten(1), score.flatten(1)
    last = rank.topk(W, -1).values[:, -1:]
    more, same = rank > last, rank == last
    chosen = more | (same & (same.cumsum(-1, dtype=torch.int32) <= W - more.sum(-1, keepdim=True)))
    at = torch.where(chosen, torch.arange(K * V, device="cuda"), K * V).topk(W, -1, largest=False, sorted=True).values
    at = at.gather(1, rank.gather(1, at).sort(stable=True, dim=-1, descending=True).indices)
    got = score.gather(1, at)
    none = got == -math.inf
    parents, tokens = at // V, at % V
    out = dict(scores=got.float(), tokens=tokens.masked_fill(none, EOS).int(), parents=parents.masked_fill(none, -1).int(),
               lengths=length.gather(1, parents).masked_fill(none, 0))
    if s["finished"] is not None:
        out["finished"] = none | (tokens == EOS) | s["finished"].gather(1, parents)
    return out


def _from(parents, rows):
    """The row that each takes, of all: its group's parent, or itself."""
    return torch.where(parents >= 0, parents + torch.arange(parents.shape[0], device="cuda")[:, None] * parents.shape[1],
                       rows.view(parents.shape)).view(-1).long()


def _plain_reorder(s):
    rows = torch.arange(s["parents"].numel(), device="cuda")
    source = _from(s["parents"], rows)
    if s["lens"] is None:
        new = [x[source] for x in s["states"]]
    else:
        seen = torch.arange(s["case"]["L"], device="cuda") < s["lens"][source, None]
        new = [torch.where(seen[:, None, :, None], x[source], x) for x in s["states"]]
    torch._foreach_copy_(s["states"], new)
    return s["states"]


def _copied(pools, copies):
    """Copies the begun rows of pages; entries with a source of -1 are none."""
    src, dst, rows = (c.long() for c in copies.unbind(1))
    at = torch.where(src >= 0, dst, pools[0].shape[0] + torch.arange(len(src), device="cuda"))  # none: behind the pool
    keep = torch.arange(PAGE, device="cuda")[None, :] < rows[:, None]
    for p in pools:
        bits = p.view(torch.uint8) if p.element_size() == 1 else p.view(torch.int16)
        new = torch.where(keep[:, None, :, None], bits[src.clamp(min=0)], bits[dst.clamp(min=0)])
        some = at < p.shape[0]
        bits.index_copy_(0, at[some], new[some])
    return pools


def _counted(refs, pages, by):
    """Counts of the pages, `by` added at each; pages outside the pool are none."""
    P = refs.shape[0]
    inside = (pages >= 0) & (pages < P)
    return torch.cat((refs, refs[:1])).index_add_(0, torch.where(inside, pages, P).flatten().long(), (by * inside).flatten().int())[:P]


def _plain_fork(s):
    table, lens, refs = s["table"], s["lens"], s["refs"]
    (S, M), P = table.shape, refs.shape[0]
    parent = s["parents"].view(-1)
    rows, col = torch.arange(S, device="cuda"), torch.arange(M, device="cuda")
    source, alive = _from(s["parents"], rows), parent >= 0
    before = torch.where(alive, lens[source], 0)
    new = before + alive.int() if s["new_lens"] is None else s["new_lens"]
    kept = torch.minimum(before, new)
    full, begun = (kept // PAGE)[:, None], kept % PAGE > 0
    taken = table[source]
    count = _counted(refs, table, -(col < (lens[:, None] + PAGE - 1) // PAGE).int())
    count = _counted(count, taken, (col < full).int())
    # the begun page stays with the first row that has it, if no other holds it; the others get copies
    tail = torch.where(begun, taken.gather(1, full.long().clamp(max=M - 1))[:, 0], -1)
    tail = torch.where(tail < P, tail, -1)
    first = torch.full((P + 1,), S, device="cuda").scatter_reduce_(0, torch.where(tail >= 0, tail, P).long(), rows, "amin")
    stays = (tail >= 0) & (first[tail.long()] == rows) & (count[tail.long()] <= 0)
    count = _counted(count, tail, stays.int()).clamp(min=0)
    needs = (col >= full + stays[:, None]) & (col < (new[:, None] + PAGE - 1) // PAGE)
    number = needs.flatten().cumsum(0).view(S, M) - 1
    free = torch.argsort((count > 0).int(), stable=True).int()
    left = (count <= 0).sum()
    page = torch.where(needs & (number < left), free[number.clamp(0, P - 1)], -1)
    count = _counted(count, page, torch.ones_like(page))
    out = torch.where(col < full, taken, torch.where((col == full) & stays[:, None], tail[:, None], page))
    copy_to = torch.where((tail >= 0) & ~stays, page.gather(1, full.long().clamp(max=M - 1))[:, 0], -1)
    order = torch.argsort((copy_to < 0).int(), stable=True)
    copies = torch.stack((tail, copy_to, kept % PAGE), 1).int().masked_fill((copy_to < 0)[:, None], -1)[order]
    missing = (needs.sum() - left).clamp(min=0)
    info = torch.stack(((copy_to >= 0).sum(), missing, (count <= 0).sum(), (count > 0).sum())).int()
    return dict(table=out.int(), lens=new.int(), refs=count, copies=copies, info=info, pools=_copied(s["pools"], copies))


def _plain_compact(s):
    table, refs = s["table"], s["refs"]
    (S, M), P = table.shape, refs.shape[0]
    page = torch.arange(P, device="cuda")
    held = refs > 0
    up = torch.argsort(held.int(), stable=True)                                  # free pages upwards first
    down = P - 1 - torch.argsort((~held).flip(0).int(), stable=True)             # held pages downwards first
    n = P // 2
    moves = (down[:n] > up[:n]) & (page[:n] < held.sum()) & (page[:n] < (~held).sum())
    src, dst = torch.where(moves, down[:n], P), torch.where(moves, up[:n], P)
    moved = torch.cat((torch.where(held, page, -1), page[:1])).index_copy_(0, torch.where(moves, down[:n], P), torch.where(moves, up[:n], 0))[:P]
    counts = torch.cat((refs.clamp(min=0), refs[:1])).index_copy_(0, dst, torch.cat((refs, refs[:1]))[src]).index_fill_(0, src, 0)[:P]
    col = torch.arange(M, device="cuda")
    inside = (col < (s["lens"][:, None] + PAGE - 1) // PAGE) & (table >= 0) & (table < P)
    out = torch.where(inside, moved[table.long().clamp(0, P - 1)], -1).int()
    copies = torch.stack((src, dst, torch.full_like(src, PAGE)), 1).masked_fill(~moves[:, None], -1).int()
    info = torch.stack((moves.sum(), moves.sum() * 0, (~held).sum(), held.sum())).int()
    return dict(table=out, refs=counts, moved=moved.int(), copies=copies, info=info, pools=_copied(s["pools"], copies))


# ---------------------------------------------------------------- one pass
def run(state):
    s, case = state, state["case"]
    if own:
        import differential_attention_02_gb300 as da
        if case["op"] == "select":
            c = da.diffattn_beam_select(s["logits"], s["scores"], width=case["W"], lengths=s["lengths"], finished=s["finished"],
                                        eos=EOS, length_penalty=case["alpha"])
            out = dict(scores=c.scores, tokens=c.tokens, parents=c.parents, lengths=c.lengths)
            if s["finished"] is not None:
                out["finished"] = c.finished
            return out
        if case["op"] == "reorder":
            return da.diffattn_beam_reorder(s["states"], s["parents"], lens=s["lens"])
        if case["op"] == "fork":
            p = da.diffattn_pages_fork(s["table"], s["lens"], s["refs"], s["parents"], new_lens=s["new_lens"], grow=1)
            da.diffattn_pages_copy(s["handle"], p.copies, p.info)
            return dict(table=p.table, lens=p.lens, refs=p.refs, copies=p.copies, info=p.info, pools=s["pools"])
        if case["op"] == "compact":
            p = da.diffattn_pages_compact(s["table"], s["lens"], s["refs"])
            da.diffattn_pages_copy(s["handle"], p.copies, p.info)
            return dict(table=p.table, refs=p.refs, moved=p.moved, copies=p.copies, info=p.info, pools=s["pools"])
        da.diffattn_pages_copy(s["handle"], s["copies"])
        return s["pools"]
    if case["op"] == "copy":
        return _copied(s["pools"], s["copies"])
    return {"select": _plain_select, "reorder": _plain_reorder, "fork": _plain_fork, "compact": _plain_compact}[case["op"]](s)


def _page_bytes(case):
    """Bytes of a token in all pools."""
    return case["layers"] * case["H"] * 4 * case["d"] * (1 if case["cache"] == "fp8" else 2)


def work(case):
    if case["op"] == "select":
        rows = case["B"] * case["K"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": rows * case["V"] * size + rows * 9 + case["B"] * case["W"] * 17, "flops": 4 * rows * case["V"]}
    if case["op"] == "reorder":
        parents = _parents(_rng(case), case["B"], case["K"])
        if case["T"]:
            row = [4 * case["T"] + 4 * 1025] * (case["B"] * case["K"])
        else:
            row = [n * case["H"] * 4 * case["d"] * 2 for n in _reorder_lens(case)]
        total = 0
        for b, group in enumerate(parents):
            moved = [p for k, p in enumerate(group) if p != k]
            total += row[b * case["K"]] * (len(moved) + len(set(moved)))
        return {"bytes": max(total, 4 * case["B"] * case["K"]), "flops": 0}
    if case["op"] == "fork":
        lens, _, _, parents, new = _fork(case)
        S, M, P = _sizes(case)
        group = len(parents[0])
        tails, seen = 0, set()
        for i, p in enumerate(q for g in parents for q in g):
            p = p if p < 0 else i // group * group + p
            kept = 0 if p < 0 else min(lens[p], new[0][i] if new else lens[p] + 1)
            if kept % PAGE:
                tails += (kept % PAGE) if (p, kept // PAGE) in seen else 0
                seen.add((p, kept // PAGE))
        return {"bytes": sum(4 * _pages(n) for n in lens) + 4 * S * M + 8 * P + 24 * S + 2 * tails * _page_bytes(case), "flops": 0}
    if case["op"] == "compact":
        P, held = case["P"], int(case["P"] * case["fill"])
        moves = int(held * (P - held) / P)  # of held pages behind place `held`, for scattered ones
        return {"bytes": 12 * P + 8 * held + 2 * moves * PAGE * _page_bytes(case), "flops": 0}
    return {"bytes": 12 * case["n"] + 2 * case["n"] * (PAGE // 2 if case["begun"] else PAGE) * _page_bytes(case), "flops": 0}


# ---------------------------------------------------------------- the definition, one row and page after the other
def _exact_select(s):
    case = s["case"]
    B, K, W, V = case["B"], case["K"], case["W"], case["V"]
    out = dict(scores=[], tokens=[], parents=[], lengths=[], finished=[])
    for b in range(B):
        found = []
        for k in range(K):
            score, n = float(s["scores"][b, k]), int(s["lengths"][b, k])
            if s["finished"] is not None and bool(s["finished"][b, k]):
                if score > -math.inf:
                    found.append((-score / max(n, 1) ** case["alpha"], k, EOS, score, n, True))
                continue
            x = s["logits"][b, k].double()
            lse = torch.logsumexp(x, 0)
            if not math.isfinite(score) or not bool(torch.isfinite(lse)):
                continue
            y = x - lse
            low = torch.topk(y, min(W, V)).values[-1]
            for v in torch.nonzero(y >= low)[:, 0].tolist() if bool(low > -math.inf) else torch.nonzero(y > -math.inf)[:, 0].tolist():
                t = score + float(y[v])
                found.append((-t / max(n + 1, 1) ** case["alpha"], k, v, t, n + 1, v == EOS))
        found = sorted(found)[:W] + [(0, -1, EOS, -math.inf, 0, True)] * max(0, W - len(found))
        for name, i in (("scores", 3), ("tokens", 2), ("parents", 1), ("lengths", 4), ("finished", 5)):
            out[name].append([f[i] for f in found])
    out["scores"] = torch.tensor(out["scores"], dtype=torch.float64)
    out.update({n: torch.tensor(out[n], dtype=torch.int32) for n in ("tokens", "parents", "lengths")})
    out["finished"] = torch.tensor(out["finished"])
    if s["finished"] is None:
        del out["finished"]
    return out


def _exact_copies(pools, copies):
    out = [p.double() for p in pools]
    for new, p in zip(out, pools):
        for src, dst, rows in copies:
            new[dst, :, :rows] = p[src, :, :rows].double()
    return out


def _listed_copies(copies, n):
    return torch.tensor(copies + [[-1] * 3] * (n - len(copies)), dtype=torch.int32).view(n, 3)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "select":
        return _exact_select(s)
    if case["op"] == "reorder":
        old = [x.double().cpu() if case["T"] else x for x in s["states"]]
        out = [x.double().clone() for x in old]
        for b, group in enumerate(s["parents"].tolist()):
            for k, p in enumerate(group):
                i, j = b * case["K"] + k, b * case["K"] + p
                for x, y in zip(out, old):
                    if s["lens"] is None:
                        x[i] = y[j]
                    else:
                        x[i, :, :int(s["lens"][j])] = y[j, :, :int(s["lens"][j])].double()
        return [o.to(torch.int32) if i == 0 and case["T"] else o for i, o in enumerate(out)]
    if case["op"] == "copy":
        return _exact_copies(s["pools"], s["copies"].tolist())
    table, lens, refs = s["table"].tolist(), s["lens"].tolist(), s["refs"].tolist()
    P, M = len(refs), len(table[0])
    if case["op"] == "compact":
        used, free = [p for p in range(P) if refs[p] > 0], [p for p in range(P) if refs[p] <= 0]
        moved = [p if refs[p] > 0 else -1 for p in range(P)]
        copies = []
        for src, dst in zip(reversed(used), free):
            if dst > src:
                break
            moved[src], refs[dst], refs[src] = dst, refs[src], 0
            copies.append([src, dst, PAGE])
        table = [[moved[p] if c < _pages(n) and p >= 0 else -1 for c, p in enumerate(row)] for row, n in zip(table, lens)]
        return dict(table=torch.tensor(table, dtype=torch.int32), refs=torch.tensor(refs, dtype=torch.int32),
                    moved=torch.tensor(moved, dtype=torch.int32), copies=_listed_copies(copies, P // 2),
                    info=torch.tensor([len(copies), 0, len(free), len(used)], dtype=torch.int32), pools=_exact_copies(s["pools"], copies))
    parents, group = s["parents"].flatten().tolist(), case["K"]
    for row, n in zip(table, lens):
        for p in row[:_pages(n)]:
            refs[p] -= 1
    rows = []
    for i, p in enumerate(parents):
        p = p if p < 0 else i // group * group + p
        before = 0 if p < 0 else lens[p]
        new = (before + (p >= 0)) if s["new_lens"] is None else int(s["new_lens"][i])
        kept = min(before, new)
        row = table[p][:kept // PAGE]
        for q in row:
            refs[q] += 1
        rows.append((new, kept, row, table[p][kept // PAGE] if kept % PAGE else -1))
    held, copies, missing, out = set(), [], 0, []
    for new, kept, row, tail in rows:  # the begun pages that stay
        if tail >= 0 and tail not in held and refs[tail] <= 0:
            held.add(tail)
            refs[tail] = 1
            row.append(tail)
    free = [p for p in range(P) if refs[p] <= 0]
    for new, kept, row, tail in rows:
        first = len(row)
        while len(row) < _pages(new):
            row.append(free.pop(0) if free else -1)
            missing += row[-1] < 0
            if row[-1] >= 0:
                refs[row[-1]] = 1
        if tail >= 0 and first == kept // PAGE and row[first] >= 0:
            copies.append([tail, row[first], kept % PAGE])
        out.append(row + [-1] * (M - len(row)))
    info = [len(copies), missing, len(free), P - len(free)]
    return dict(table=torch.tensor(out, dtype=torch.int32), lens=torch.tensor([r[0] for r in rows], dtype=torch.int32),
                refs=torch.tensor(refs, dtype=torch.int32), copies=_listed_copies(copies, len(rows)),
                info=torch.tensor(info, dtype=torch.int32), pools=_exact_copies(s["pools"], copies))
