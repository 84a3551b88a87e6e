"""Float64 references of the rotary positions, the ragged paged append and the chunk
attention, written from their definitions (NumPy-like torch on the CPU, no package code),
and the builders of paged caches that the tests share."""

import math

import torch

PAGE = 64


def frequencies(r, base=10000.0, scaling="none", factor=1.0, original=0, fast=32.0, slow=1.0):
    """Radians per position of each pair, and the magnitude (float64)."""
    f = torch.tensor([base ** (-2.0 * j / r) for j in range(r // 2)], dtype=torch.float64)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ramp":
        g = ((original * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        return f / factor * (1 - g) + f * g, 0.1 * math.log(factor) + 1
    return f, 1.0


def rotate(x, angle, magnitude=1.0, interleaved=False, backward=False):
    """x [..., d] float64, angle [..., r / 2] broadcastable over the leading dimensions."""
    h = angle.shape[-1]
    c, s = magnitude * torch.cos(angle), magnitude * torch.sin(angle) * (-1 if backward else 1)
    ia = torch.arange(h) * 2 if interleaved else torch.arange(h)
    ib = ia + 1 if interleaved else ia + h
    y = x.clone()
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    return y


def make_pool(lens, H_kv, widths, dtype, seed, spare=3, fill=None):
    """Pools [P, H_kv, 64, w] per width, and the shuffled block table [B, max_pages] whose unused
    entries are -1. `fill`: value of every byte pattern that no sequence owns (default: random)."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-n // PAGE) for n in lens]
    maxp = max(max(counts), 1)
    P = sum(counts) + spare
    perm = torch.randperm(P, generator=g)
    table = torch.full((len(lens), maxp), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = perm[at:at + c].to(torch.int32)
        at += c
    pools = [torch.randn(P, H_kv, PAGE, w, generator=g) for w in widths]
    if dtype == torch.float8_e4m3fn:
        pools = [(p / s).clamp(-448, 448).to(dtype) for p, s in zip(pools, SCALES)]
    else:
        pools = [p.to(dtype) for p in pools]
    return pools, table


SCALES = (0.0113, 0.0127, 0.0109)


def poison(pools, table, lens):
    """Copies of the pools with NaN in every entry that no sequence's length covers."""
    out = []
    for p in pools:
        bits = torch.uint8 if p.dtype == torch.float8_e4m3fn else torch.int16
        q = torch.full_like(p.view(bits), 0x7F if bits == torch.uint8 else 0x7FC1)
        for b, n in enumerate(lens):
            for i in range(-(-n // PAGE)):
                k = min(PAGE, n - i * PAGE)
                q[table[b, i], :, :k] = p.view(bits)[table[b, i], :, :k]
        out.append(q.view(p.dtype))
    return out


def gather(pool, table, b, n, scale=1.0):
    """The first n entries of sequence b: [H_kv, n, w] float64."""
    used = table[b, :-(-n // PAGE)].long()
    bits = pool.view(torch.uint8)[used].view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else pool[used]
    x = bits.float().double() * scale
    return x.permute(1, 0, 2, 3).reshape(pool.shape[1], -1, pool.shape[3])[:, :n]


def chunk_attention(q1, q2, pools, table, starts, lens, lam, lam_init, group=1, eps=1e-5, norm_weight=None, scales=None):
    """[T, H, Dv] float64; rows of no sequence are NaN (not computed)."""
    T, H, d = q1.shape
    Dv = pools[2].shape[3]
    sc = scales or (1.0, 1.0, 1.0)
    y = torch.full((T, H, Dv), float("nan"), dtype=torch.float64)
    for b, n_keys in enumerate(lens):
        s, e = starts[b], starts[b + 1]
        n = e - s
        if n == 0:
            continue
        pos = torch.arange(n_keys - n, n_keys)
        if n_keys == 0:
            y[s:e] = 0
            continue
        k1, k2, v = (gather(p, table, b, n_keys, c) for p, c in zip(pools, sc))
        hidden = torch.arange(n_keys)[None] > pos[:, None]
        for h in range(H):
            o = 0
            for q, k, w in ((q1, k1, 1.0), (q2, k2, -lam)):
                x = (q[s:e, h].double() @ k[h // group].T / math.sqrt(d)).masked_fill(hidden, -math.inf)
                x = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e300))
                o = o + w * (x / x.sum(-1, keepdim=True).clamp(min=1e-300)) @ v[h // group]
            o = o / torch.sqrt(o.square().mean(-1, keepdim=True) + eps) * (1 - lam_init)
            o[pos < 0] = 0
            y[s:e, h] = o if norm_weight is None else o * norm_weight.double()
    return y
