"""The serving and training operators around differential attention, as cases that can be timed and compared.

Three operators over Q1, Q2, K1, K2 and V:

- rope: the position rotation of the query and key halves, and its transpose for gradients;
- append: writing the keys and values of many new tokens of many sequences into a paged cache,
  K1 and K2 rotated on the way, into bf16 or fp8 (e4m3) pages;
- chunk: differential attention of the new tokens of many sequences (a prompt's chunk, a few drafted
  tokens, a single one) over that paged cache, query heads sharing KV heads.

`own` selects the framework's kernels; without it `run` computes the same in elementary torch operations.
"""

import math
import random

import torch

own = False

PAGE = 64
LAM, LAM_INIT, EPS = 0.55, 0.47, 1e-5
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the rotation of a training step's or a prompt's Q and K: the repository's prefill workload
        dict(name="rope_prefill", op="rope", B=4, H=16, H_kv=16, N=2048, d=64, rotary=64, interleaved=False, scaling="none",
             dtype="bf16", backward=False, far=0),
        # the gradients of the module workload on their way back through the rotation (the backward's are fp32)
        dict(name="rope_gradients", op="rope", B=2, H=8, H_kv=8, N=4096, d=128, rotary=128, interleaved=True, scaling="linear",
             dtype="f32", backward=True, far=0),
        # one decoding step of 33 sequences at far positions, half of each head rotated, scaled for long contexts
        dict(name="rope_step", op="rope", B=1, H=16, H_kv=4, N=33, d=64, rotary=32, interleaved=False, scaling="ramp", dtype="f16",
             backward=False, far=1_000_000),
        # four prompts' chunks into the cache of the decode workload's heads
        dict(name="append_chunk", op="append", B=4, H_kv=16, d=64, Dv=128, chunk=2048, L=8192, ragged=True, cache="bf16", rotary=64,
             interleaved=False, scaling="none"),
        # the module's wide heads into an fp8 cache, odd lengths, part of the head rotated
        dict(name="append_fp8_wide", op="append", B=5, H_kv=8, d=128, Dv=256, chunk=777, L=4000, ragged=True, cache="fp8", rotary=96,
             interleaved=True, scaling="ramp"),
        # one decoding step of 64 sequences: latency
        dict(name="append_step", op="append", B=64, H_kv=16, d=64, Dv=128, chunk=1, L=8192, ragged=True, cache="bf16", rotary=64,
             interleaved=False, scaling="none"),
        # the last chunks of four 8192-token prompts
        dict(name="chunk_prefill", op="chunk", B=4, H=16, group=1, d=64, Dv=128, chunk=2048, L=8192, ragged=False, cache="bf16"),
        # a short chunk far into one long context, four query heads to a KV head
        dict(name="chunk_long", op="chunk", B=1, H=16, group=4, d=64, Dv=128, chunk=500, L=65000, ragged=False, cache="bf16"),
        # a serving batch: most sequences decode, some bring a piece of their prompt
        dict(name="chunk_mixed", op="chunk", B=32, H=16, group=4, d=64, Dv=128, chunk=333, L=4096, ragged=True, cache="bf16"),
        # the module's wide heads
        dict(name="chunk_wide", op="chunk", B=2, H=8, group=1, d=128, Dv=256, chunk=1024, L=4096, ragged=False, cache="bf16"),
        # five drafted tokens a sequence are checked against an fp8 cache
        dict(name="chunk_fp8_verify", op="chunk", B=16, H=16, group=2, d=64, Dv=128, chunk=5, L=8192, ragged=False, cache="fp8"),
        # a single token of a single sequence: latency
        dict(name="chunk_step", op="chunk", B=1, H=16, group=1, d=64, Dv=128, chunk=1, L=8192, ragged=False, cache="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number whose logarithm is spread evenly over [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "chunk", "chunk"])
    d = rng.choice([64, 64, 128])
    group = rng.choice([1, 1, 2, 4, 8])
    H_kv = rng.choice([1, 2, 4, 5, 8, 16])
    rot = dict(rotary=rng.choice([8, 16, 32, 48, 64] + ([96, 120, 128] if d == 128 else [])), interleaved=rng.random() < 0.5,
               scaling=rng.choice(["none", "linear", "ramp"]))
    if op == "rope":
        H_kv = rng.choice([2, 4, 8, 16])
        B, N = _log(rng, 1, 8), _log(rng, 1, 4096)
        return dict(op="rope", B=B, H=min(16, H_kv * group), H_kv=H_kv, N=N, d=d, dtype=rng.choice(["bf16", "f16", "f32"]),
                    backward=rng.random() < 0.5, far=rng.choice([0, 0, 100_000, 4_000_000]), **rot)
    cache = rng.choice(["bf16", "bf16", "fp8"])
    if op == "append":
        B = _log(rng, 1, 64)
        chunk = _log(rng, 1, max(1, 8192 // B))
        L = max(chunk, _log(rng, 1, max(1, 65536 // B)))
        return dict(op="append", B=B, H_kv=H_kv, d=d, Dv=2 * d, chunk=chunk, L=L, ragged=rng.random() < 0.7, cache=cache, **rot)
    H = min(16, H_kv * group)
    H -= H % H_kv
    B = _log(rng, 1, 32)
    # the largest listed one has 4 x 16 heads x 2048 x 8192 pairs of a query and a key
    chunk = _log(rng, 1, max(1, 2048 // B))
    L = max(chunk, _log(rng, 1, max(1, min(65536 // B, (1 << 27) // (B * chunk)))))
    return dict(op="chunk", B=B, H=H, group=H // H_kv, d=d, Dv=2 * d, chunk=chunk, L=L, ragged=rng.random() < 0.7, cache=cache)


def _lengths(case):
    """New tokens and length (with them) of each sequence: the same for every seed of a case."""
    B, chunk, L = case["B"], case["chunk"], case["L"]
    if not case["ragged"]:
        return [chunk] * B, [L] * B
    rng = random.Random("%d %d %d" % (B, chunk, L))
    # two in three bring a single token, as in a serving batch; the first has the longest chunk and the last the longest context
    new = [chunk if b == 0 else 1 if case["op"] == "chunk" and rng.random() < 0.67 else rng.randint(1, chunk) for b in range(B)]
    lens = [rng.randint(n, L) for n in new]
    lens[-1] = L
    return new, lens


# ---------------------------------------------------------------- inputs
def _frequencies(case):
    """Angle per position of each rotated pair, and the factor of the rotated values."""
    r, base, factor, original = case["rotary"], 10000.0, 8.0, 4096
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if case["scaling"] == "linear":
        return [x / factor for x in f], 1.0
    if case["scaling"] == "ramp":
        g = [min(1.0, max(0.0, (original * x / (2 * math.pi) - 1.0) / (32.0 - 1.0))) for x in f]
        return [x / factor * (1 - w) + x * w for x, w in zip(f, g)], 0.1 * math.log(factor) + 1
    return f, 1.0


def _rope_plan(case):
    import differential_attention_02_gb300 as da
    return da.rope_plan(case["rotary"], base=10000.0, interleaved=case["interleaved"], scaling=case["scaling"], factor=8.0,
                        original_length=4096)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s = dict(case=case)
    if case["op"] != "chunk":
        f, s["magnitude"] = _frequencies(case)
        s["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        if own:
            s["plan"] = _rope_plan(case)
    if case["op"] == "rope":
        B, N, d, dt = case["B"], case["N"], case["d"], DTYPES[case["dtype"]]
        # tokens outermost, as a projection writes them: [B, N, H, 2 d] with the two halves of a head side by side
        q, k = rand(B, N, case["H"], 2 * d).to(dt), rand(B, N, case["H_kv"], 2 * d).to(dt)
        halves = [t[..., i * d:(i + 1) * d].transpose(1, 2) for t in (q, k) for i in (0, 1)]
        s["x"] = halves if case["dtype"] != "f32" else [h.contiguous() for h in halves]  # gradients have rows of their own
        s["positions"] = None
        if case["far"]:
            s["positions"] = torch.randint(0, case["far"], (B, N), generator=g, device="cuda", dtype=torch.int32)
        return s
    B, H_kv, d, Dv = case["B"], case.get("H_kv") or case["H"] // case["group"], case["d"], case["Dv"]
    new, lens = _lengths(case)
    starts = [sum(new[:b]) for b in range(B + 1)]
    s["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    T, L = starts[-1], max(lens)
    max_pages = -(-L // PAGE)
    counts = torch.tensor([-(-n // PAGE) for n in lens], device="cuda")
    P = int(counts.sum()) + 3
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    at = torch.arange(max_pages, device="cuda")
    first = counts.cumsum(0) - counts
    s["table"] = torch.where(at < counts[:, None], order[(first[:, None] + at).clamp(max=P - 1)], 0).contiguous()
    widths = (d, d, Dv)
    if case["cache"] == "fp8":
        s["scales"] = (0.0113, 0.0127, 0.0109)  # 448 of them is about five standard deviations
        s["pages"] = [(rand(P, H_kv, PAGE, w) / c).clamp(-448, 448).to(torch.float8_e4m3fn) for w, c in zip(widths, s["scales"])]
    else:
        s["scales"] = None
        s["pages"] = [rand(P, H_kv, PAGE, w).to(torch.bfloat16) for w in widths]
    if case["op"] == "append":
        rows = rand(T, H_kv * (2 * d + Dv)).to(torch.bfloat16)  # one projection's [K | V]: each head's K1 and K2 side by side
        k = rows[:, :2 * d * H_kv].unflatten(1, (H_kv, 2 * d))
        s["new"] = [k[..., :d], k[..., d:], rows[:, 2 * d * H_kv:].unflatten(1, (H_kv, Dv))]
    else:
        q = rand(T, case["H"], 2 * d).to(torch.bfloat16)
        s["q"] = [q[..., :d], q[..., d:]]
        s["L"] = L
    return s


# ---------------------------------------------------------------- the plain forms
def _turned(x, cos, sin, interleaved):
    """Each pair of the first channels of x turned by its angle; the channels behind them as they are."""
    r = 2 * cos.shape[-1]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    y = (a * cos - b * sin, a * sin + b * cos)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat((y, x[..., r:]), -1)


def _angles(s, positions):
    a = positions.double()[..., None] * s["freq"]
    return torch.cos(a).float() * s["magnitude"], torch.sin(a).float() * s["magnitude"]


def _plain_rope(s):
    case = s["case"]
    positions = s["positions"]
    if positions is None:
        positions = torch.arange(case["N"], device="cuda").expand(case["B"], -1)
    cos, sin = _angles(s, positions)
    cos, sin = cos[:, None], (-sin if case["backward"] else sin)[:, None]  # over the heads
    return [_turned(x.float(), cos, sin, case["interleaved"]).to(x.dtype) for x in s["x"]]


def _tokens(s):
    """Of each new token: its sequence, its number in the chunk, and its position."""
    start, lens = s["q_start"].long(), s["seq_lens"].long()
    t = torch.arange((s.get("new") or s["q"])[0].shape[0], device="cuda")
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    i = t - start[b]
    return b, i, lens[b] - (start[b + 1] - start[b]) + i


def _plain_append(s):
    case = s["case"]
    b, _, pos = _tokens(s)
    page, row = s["table"][b, pos // PAGE].long(), pos % PAGE
    cos, sin = _angles(s, pos)
    cos, sin = cos[:, None], sin[:, None]
    turn = lambda x: _turned(x.float(), cos, sin, case["interleaved"])  # noqa: E731
    rows = [turn(s["new"][0]), turn(s["new"][1]), s["new"][2].float()]
    if s["scales"] is None:
        s["pages"][0][page, :, row] = rows[0].to(torch.bfloat16)
        s["pages"][1][page, :, row] = rows[1].to(torch.bfloat16)
        s["pages"][2][page, :, row] = rows[2].to(torch.bfloat16)
    else:
        held = [(x / c).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x, c in zip(rows, s["scales"])]
        s["pages"][0].view(torch.uint8)[page, :, row] = held[0]
        s["pages"][1].view(torch.uint8)[page, :, row] = held[1]
        s["pages"][2].view(torch.uint8)[page, :, row] = held[2]
    return s["pages"]


def _plain_chunk(s):
    case = s["case"]
    B, H, G, d = case["B"], case["H"], case["group"], case["d"]
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    lens, N = s["seq_lens"].long(), case["chunk"]
    at = torch.arange(N, device="cuda")
    rows = (s["q_start"][:-1].long()[:, None] + at).clamp(max=s["q"][0].shape[0] - 1)
    # [B, H_kv, G N, d] and [B, H_kv, L, width]: the sequences padded to the longest chunk and length
    q1, q2 = (x[rows].float().unflatten(2, (H // G, G)).permute(0, 2, 3, 1, 4).flatten(2, 3) for x in s["q"])
    held = [p.view(torch.uint8)[s["table"].long()].view(p.dtype) if s["scales"] else p[s["table"].long()] for p in s["pages"]]
    k1, k2, v = (x.transpose(1, 2).flatten(2, 3)[:, :, :s["L"]].float() for x in held)
    if s["scales"]:
        k1, k2, v = k1 * s["scales"][0], k2 * s["scales"][1], v * s["scales"][2]
    pos = (lens - n)[:, None] + at
    seen = torch.arange(s["L"], device="cuda") <= pos.clamp(max=s["L"] - 1)[..., None]  # [B, N, L]
    hidden = ~seen.repeat(1, G, 1)[:, None]

    def weights(q, k):
        x = (q @ k.transpose(-1, -2)).mul_(1 / math.sqrt(d)).masked_fill_(hidden, -math.inf)
        x = x.sub_(x.amax(-1, keepdim=True)).exp_()
        return x.div_(x.sum(-1, keepdim=True))

    a = weights(q1, k1).sub_(weights(q2, k2).mul_(LAM))
    o = a @ v
    y = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS) * (1 - LAM_INIT)
    y = y.unflatten(2, (G, N)).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [B, N, H, Dv]
    b, i, _ = _tokens(s)
    return y[b, i].to(torch.bfloat16)


# ---------------------------------------------------------------- one pass
def run(state):
    s, case = state, state["case"]
    if own:
        import differential_attention_02_gb300 as da
        if case["op"] == "rope":
            return list(da.diffattn_rope(s["x"], s["plan"], positions=s["positions"], backward=case["backward"]))
        if case["op"] == "append":
            da.diffattn_kv_append_chunk_paged(*s["new"], *s["pages"], s["table"], s["q_start"], s["seq_lens"], rope=s["plan"],
                                              scales=s["scales"])
            return s["pages"]
        return da.diffattn_chunk_paged(*s["q"], *s["pages"], s["table"], s["q_start"], s["seq_lens"], LAM, LAM_INIT, L=s["L"],
                                       kv_group=case["group"], eps=EPS, out_dtype=torch.bfloat16, scales=s["scales"])
    return {"rope": _plain_rope, "append": _plain_append, "chunk": _plain_chunk}[case["op"]](s)


def work(case):
    if case["op"] == "rope":
        rows = case["B"] * case["N"] * 2 * (case["H"] + case["H_kv"])
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * rows * case["d"] * size + (4 * case["B"] * case["N"] if case["far"] else 0),
                "flops": 3 * rows * case["rotary"]}
    new, lens = _lengths(case)
    d, Dv, held = case["d"], case["Dv"], 1 if case["cache"] == "fp8" else 2
    if case["op"] == "append":
        rows = sum(new) * case["H_kv"]
        return {"bytes": rows * (2 * d + Dv) * (2 + held), "flops": 3 * rows * 2 * case["rotary"]}
    H, H_kv = case["H"], case["H"] // case["group"]
    pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(new, lens))  # of a query and a key that it sees
    return {"bytes": sum(lens) * H_kv * (2 * d + Dv) * held + sum(new) * H * (2 * d + Dv) * 2,
            "flops": pairs * H * (4 * d + 2 * Dv)}


# ---------------------------------------------------------------- the definition in 64 bits
def _pairs_turned(x, angle, magnitude, interleaved, sign):
    """The rotation as a product with e^(i angle) of each pair taken as a complex number."""
    n = angle.shape[-1]
    re = torch.arange(n, device=x.device) * (2 if interleaved else 1)
    im = re + (1 if interleaved else n)
    z = torch.complex(x[..., re], x[..., im]) * torch.polar(torch.full_like(angle, magnitude), sign * angle)
    y = x.clone()
    y[..., re], y[..., im] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        pos = s["positions"] if s["positions"] is not None else torch.arange(case["N"], device="cuda")[None].repeat(case["B"], 1)
        angle = (pos.double()[:, :, None] * s["freq"])[:, None]
        return [_pairs_turned(x.double(), angle, s["magnitude"], case["interleaved"], -1.0 if case["backward"] else 1.0)
                for x in s["x"]]
    new, lens = _lengths(case)
    starts = [sum(new[:b]) for b in range(case["B"] + 1)]
    if case["op"] == "append":
        out = [p.double() for p in s["pages"]]
        for b, (n, m) in enumerate(zip(new, lens)):
            pos = torch.arange(m - n, m, device="cuda")
            page, row = s["table"][b].long()[pos // PAGE], pos % PAGE
            angle = (pos.double()[:, None] * s["freq"])[:, None]
            for k in range(3):
                x = s["new"][k][starts[b]:starts[b + 1]].double()
                if k < 2:
                    x = _pairs_turned(x, angle.expand(-1, x.shape[1], -1), s["magnitude"], case["interleaved"], 1.0)
                if s["scales"]:
                    x = (x / s["scales"][k]).clamp(-448, 448)
                out[k][page, :, row] = x
        return out
    H, G, d, Dv = case["H"], case["group"], case["d"], case["Dv"]
    if sum(n * m for n, m in zip(new, lens)) * H * (4 * d + 2 * Dv) > 4e12:
        return None
    y = torch.empty(starts[-1], H, Dv, dtype=torch.float64, device="cuda")
    for b, (n, m) in enumerate(zip(new, lens)):
        used = s["table"][b, :-(-m // PAGE)].long()
        held = [p.view(torch.uint8)[used].view(p.dtype) if s["scales"] else p[used] for p in s["pages"]]
        kv = [x.double().permute(1, 0, 2, 3).reshape(H // G, -1, x.shape[-1])[:, :m] * (s["scales"][i] if s["scales"] else 1.0)
              for i, x in enumerate(held)]
        future = torch.triu(torch.ones(n, m, dtype=torch.bool, device="cuda"), diagonal=m - n + 1)
        for h in range(H):
            qh = [x[starts[b]:starts[b + 1], h].double() for x in s["q"]]
            maps = [torch.softmax((qh[i] @ kv[i][h // G].T / math.sqrt(d)).masked_fill(future, -math.inf), -1) for i in (0, 1)]
            o = (maps[0] - LAM * maps[1]) @ kv[2][h // G]
            y[starts[b]:starts[b + 1], h] = o / torch.sqrt(o.square().mean(-1, keepdim=True) + EPS) * (1 - LAM_INIT)
    return y
