"""The position rotation and the ragged paged append on the GPU, against float64 references.

Tolerance of the rotation, per element of a pair (a, b) at magnitude m, before the rounding
to the output type: the fixed-point angle is exact to 2^-32 turns and rounded to fp32 within
2^-25 turns (1.9e-7 rad); sincospi adds at most 2 ulp of values up to 1 (2.4e-7); scaling,
two products and a sum round four times by 2^-24 (2.4e-7). Together 6.7e-7 m (|a| + |b|); the
tests take 8e-7. The stored value adds half a step of its type relative to it."""

import math

import pytest
import torch

import differential_attention_02_gb300 as da
import serving_reference as ref

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from differential_attention_02_gb300 import build
    build.build()
    da.load_library()


def _angles(positions, r, **scaling):
    f, m = ref.frequencies(r, **scaling)
    return positions.double()[..., None] * f, m


def _bound(x, y, h, m, interleaved, dtype):
    """Allowed error of the rotated x (float64 result y): see the top."""
    ia = torch.arange(h) * 2 if interleaved else torch.arange(h)
    ib = ia + 1 if interleaved else ia + h
    s = torch.zeros_like(x)
    pair = x[..., ia].abs() + x[..., ib].abs()
    s[..., ia], s[..., ib] = pair, pair
    half = torch.finfo(dtype).eps / 2
    smallest = torch.finfo(dtype).smallest_normal * half  # half the smallest step, below the normal range
    return 8e-7 * m * s * (1 + half) + half * y.abs() + smallest


def _check(got, x, y, h, m, interleaved, dtype):
    err = (got.double().cpu() - y).abs()
    assert bool((err <= _bound(x, y, h, m, interleaved, dtype)).all()), float((err - _bound(x, y, h, m, interleaved, dtype)).max())


CASES = [  # B, H, H_kv, N, d, rotary
    (1, 1, 1, 1, 8, 8), (2, 3, 1, 5, 64, 64), (1, 16, 4, 33, 64, 32), (3, 2, 2, 130, 128, 96), (2, 5, 5, 7, 40, 24),
    (1, 7, 2, 1000, 128, 128), (1, 2, 1, 3, 256, 200), (5, 1, 3, 1, 64, 8)]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
                                             (torch.float32, torch.float32), (torch.float32, torch.bfloat16),
                                             (torch.bfloat16, torch.float32), (torch.float16, torch.bfloat16),
                                             (torch.float32, torch.float16)])
def test_rotation_matches_the_definition(case, interleaved, dtype, out_dtype):
    B, H, Hk, N, d, r = case
    g = torch.Generator().manual_seed(d + N)
    x = [torch.randn(B, h, N, d, generator=g).to(dtype) for h in (H, H, Hk, Hk)]
    plan = da.rope_plan(r, interleaved=interleaved)
    got = da.diffattn_rope([t.cuda() for t in x], plan, out_dtype=out_dtype)
    angle, m = _angles(torch.arange(N), r)
    for a, b in zip(got, x):
        assert a.dtype == out_dtype and a.shape == b.shape
        y = ref.rotate(b.double(), angle, m, interleaved)
        _check(a, b.double(), y, r // 2, m, interleaved, out_dtype)
        assert torch.equal(a[..., r:].cpu(), b[..., r:].to(out_dtype))  # the channels behind are copied


@pytest.mark.parametrize("scaling", [dict(scaling="linear", factor=4.0), dict(scaling="ramp", factor=8.0, original=4096)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_scaled_frequencies_at_far_positions(scaling, interleaved):
    g = torch.Generator().manual_seed(3)
    B, H, N, d, r = 2, 3, 50, 64, 48
    pos = torch.randint(0, 1 << 22, (B, N), generator=g, dtype=torch.int32)
    pos[0, :3] = torch.tensor([0, 1, (1 << 22) - 1], dtype=torch.int32)
    x = torch.randn(B, H, N, d, generator=g)
    kw = {("original_length" if k == "original" else k): v for k, v in scaling.items()}
    got, = da.diffattn_rope([x.cuda()], da.rope_plan(r, interleaved=interleaved, **kw), positions=pos.cuda())
    angle, m = _angles(pos[:, None], r, **scaling)
    # the reference's own angle: position x frequency in double, 2^22 rad x 2^-52, far below the bound
    _check(got, x.double(), ref.rotate(x.double(), angle, m, interleaved), r // 2, m, interleaved, torch.float32)


def test_extreme_positions_are_exact_in_the_angle():
    """Positions at both ends of int32 against exact integer arithmetic on the same table."""
    r = 64
    pos = torch.tensor([[2 ** 31 - 1, -(2 ** 31), -1, -12345, 0, 2 ** 30 + 1]], dtype=torch.int32)
    x = torch.randn(1, 2, 6, r, generator=torch.Generator().manual_seed(9))
    plan = da.rope_plan(r)
    got, = da.diffattn_rope([x.cuda()], plan, positions=pos.cuda())
    table, _ = da.rope_freqs(r)
    turns = [[((int(p) * (int(f) & (2 ** 64 - 1))) % 2 ** 64) / 2.0 ** 64 for f in table] for p in pos[0]]
    angle = 2 * math.pi * torch.tensor(turns, dtype=torch.float64)[None, None]
    _check(got, x.double(), ref.rotate(x.double(), angle), r // 2, 1.0, False, torch.float32)


def test_strided_views_in_place_and_magnitude():
    """Q1, Q2 as the column blocks of a projection's output, rotated where they lie."""
    B, N, H, d = 2, 37, 3, 64
    base = torch.randn(B * N, H * 2 * d, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    view = lambda t: t.unflatten(0, (B, N)).unflatten(2, (H, 2 * d)).permute(0, 2, 1, 3)  # noqa: E731
    dev = base.cuda()
    q1, q2 = view(dev)[..., :d], view(dev)[..., d:]
    plan = da.rope_plan(32, magnitude=0.75)
    back = da.diffattn_rope([q1], plan, out=[q1])
    assert back[0].data_ptr() == q1.data_ptr()
    angle, _ = _angles(torch.arange(N), 32)
    want = ref.rotate(view(base)[..., :d].double(), angle, 0.75)
    _check(q1, view(base)[..., :d].double(), want, 16, 0.75, False, torch.bfloat16)
    assert torch.equal(q2.cpu(), view(base)[..., d:])  # the neighbours are untouched
    # an operand with no heads beside one that has some
    empty = torch.empty(B, 0, N, d, dtype=torch.bfloat16, device="cuda")
    a, b = da.diffattn_rope([empty, q2], plan)
    assert a.shape == empty.shape and b.shape == q2.shape


@pytest.mark.parametrize("interleaved", [False, True])
def test_backward_is_the_gradient(interleaved):
    """The gradient of sum(w * rope(x)) against the formula (the transpose) and against central
    differences of the forward: the map is linear, so a difference with step 1 is exact up to the
    forward's own rounding, 2 x 8e-7 (|a| + |b|) m |w| per element with |a|, |b| <= 1."""
    B, H, N, d, r = 1, 2, 9, 32, 24
    g = torch.Generator().manual_seed(6)
    w = torch.randn(B, H, N, d, generator=g)
    pos = torch.randint(0, 5000, (B, N), generator=g, dtype=torch.int32)
    plan = da.rope_plan(r, interleaved=interleaved, scaling="ramp", factor=4.0, original_length=512)
    got, = da.diffattn_rope([w.cuda()], plan, positions=pos.cuda(), backward=True)
    angle, m = _angles(pos[:, None], r, scaling="ramp", factor=4.0, original=512)
    _check(got, w.double(), ref.rotate(w.double(), angle, m, interleaved, backward=True), r // 2, m, interleaved, torch.float32)
    for c in range(d):  # all rows at once: a row's output depends on the row alone
        e = torch.zeros(B, H, N, d)
        e[..., c] = 0.5
        hi, = da.diffattn_rope([e.cuda()], plan, positions=pos.cuda())
        lo, = da.diffattn_rope([-e.cuda()], plan, positions=pos.cuda())
        diff = ((hi - lo).double().cpu() * w.double()).sum(-1)
        tol = 2 * (2 * 8e-7 * m) * w.double().abs().amax(-1) + 1e-7
        assert bool(((got[..., c].double().cpu() - diff).abs() <= tol).all())


def test_other_stream_and_graph():
    x = torch.randn(2, 4, 100, 64, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    plan = da.rope_plan(64)
    want, = da.diffattn_rope([x], plan)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, = da.diffattn_rope([x], plan, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out, = da.diffattn_rope([x], plan)
    out.zero_()
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_rope_shape_refusals():
    plan = da.rope_plan(64)
    x = torch.zeros(1, 2, 3, 64, device="cuda")
    bad = [lambda: da.diffattn_rope([x, x.to(torch.bfloat16)], plan), lambda: da.diffattn_rope([x[0]], plan),
           lambda: da.diffattn_rope([x] * 5, plan), lambda: da.diffattn_rope([x, x[:, :, :2]], plan),
           lambda: da.diffattn_rope([x], plan, positions=torch.zeros(1, 3, device="cuda")),
           lambda: da.diffattn_rope([x], plan, positions=torch.zeros(1, 4, dtype=torch.int32, device="cuda")),
           lambda: da.diffattn_rope([x], plan, out=[x[:, :1]]), lambda: da.diffattn_rope([x.double()], plan),
           lambda: da.diffattn_rope([x.transpose(2, 3)], plan)]
    for call in bad:
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------- append
APPEND = [  # new tokens, lengths, H_kv, d, Dv, rotary (0: none)
    ([1], [1], 1, 64, 128, 64), ([1, 1, 1], [5, 64, 65], 2, 64, 128, 64), ([130, 0, 1, 63], [130, 40, 129, 200], 3, 64, 128, 32),
    ([200, 77], [1000, 77], 5, 128, 256, 96), ([3, 64, 5], [3, 64, 5], 1, 24, 40, 16), ([1] * 40, list(range(1, 41)), 16, 64, 128, 0),
    ([300], [4000], 4, 128, 256, 128)]


def _append_reference(pools, table, new, starts, lens, r, interleaved, scales, **scaling):
    """Float64 values of every written entry: list of (operand, page, row, token)."""
    out = []
    f, m = ref.frequencies(r, **scaling) if r else (torch.zeros(0, dtype=torch.float64), 1.0)
    for b, n_keys in enumerate(lens):
        n = starts[b + 1] - starts[b]
        for i in range(n):
            pos = n_keys - n + i
            if pos < 0 or pos // 64 >= table.shape[1]:
                continue
            page = int(table[b, pos // 64])
            if not 0 <= page < pools[0].shape[0]:
                continue
            for k in range(3):
                x = new[k][starts[b] + i].double()
                y = ref.rotate(x, (pos * f)[None].expand(x.shape[0], -1), m, interleaved) if r and k < 2 else x
                out.append((k, page, pos % 64, x, y))
    return out, m


@pytest.mark.parametrize("case", APPEND)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("in_dtype", [torch.bfloat16, torch.float16])
def test_append_bf16(case, interleaved, in_dtype):
    n_new, lens, Hk, d, Dv, r = case
    pools, table = ref.make_pool(lens, Hk, (d, d, Dv), torch.bfloat16, seed=d)
    starts = [sum(n_new[:b]) for b in range(len(n_new) + 1)]
    T = starts[-1] + 2  # two rows behind the last sequence
    g = torch.Generator().manual_seed(T)
    new = [torch.randn(T, Hk, w, generator=g).to(in_dtype) for w in (d, d, Dv)]
    dev = [p.cuda() for p in pools]
    plan = da.rope_plan(r, interleaved=interleaved) if r else None
    da.diffattn_kv_append_chunk_paged(*(x.cuda() for x in new), *dev, table.cuda(), _i32(starts), _i32(lens), rope=plan)
    entries, m = _append_reference(pools, table, new, starts, lens, r, interleaved, None)
    got = [p.cpu() for p in dev]
    touched = [torch.zeros(p.shape[0], 64, dtype=torch.bool) for p in pools]
    for k, page, row, x, y in entries:
        touched[k][page, row] = True
        have = got[k][page, :, row]
        if k == 2 or not r:
            assert torch.equal(have, x.to(in_dtype).to(torch.bfloat16))
        else:
            _check(have, x, y, r // 2, m, interleaved, torch.bfloat16)
            assert torch.equal(have[:, r:], x[:, r:].to(in_dtype).to(torch.bfloat16))
    for k in range(3):  # everything else is left as it was, bit for bit
        keep = ~touched[k]
        a, b = got[k].view(torch.int16).transpose(1, 2), pools[k].view(torch.int16).transpose(1, 2)
        assert torch.equal(a[keep], b[keep])


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("case", APPEND[1:5])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_fp8(case, interleaved):
    """Each stored code is e4m3 of a value within the rotation's bound of the exact one (divided in
    fp32, half a step of 2^-24): the exact quotient's code, or its neighbour when the quotient lies
    that close to the middle between the two."""
    n_new, lens, Hk, d, Dv, r = case
    pools, table = ref.make_pool(lens, Hk, (d, d, Dv), F8, seed=d)
    starts = [sum(n_new[:b]) for b in range(len(n_new) + 1)]
    new = [(torch.randn(starts[-1], Hk, w, generator=torch.Generator().manual_seed(w)) * 2).to(torch.bfloat16) for w in (d, d, Dv)]
    new[2][0, 0, :2] = torch.tensor([1e4, -1e4])  # saturates
    dev = [p.cuda() for p in pools]
    plan = da.rope_plan(r, interleaved=interleaved)
    call = lambda: da.diffattn_kv_append_chunk_paged(*(x.cuda() for x in new), *dev, table.cuda(), _i32(starts), _i32(lens),  # noqa: E731
                                                     rope=plan, scales=ref.SCALES)
    if d % 16 or Dv % 16:  # rows of one-byte values that are no multiple of 16 bytes long
        with pytest.raises(da.DiffAttnError):
            call()
        return
    call()
    entries, m = _append_reference(pools, table, new, starts, lens, r, interleaved, ref.SCALES)
    got = [p.cpu() for p in dev]
    codes = lambda v: v.clamp(-448, 448).to(torch.float32).to(F8).to(torch.float32)  # noqa: E731
    for k, page, row, x, y in entries:
        s = ref.SCALES[k]
        tol = (_bound(x, y, r // 2, m, interleaved, torch.float32) if k < 2 else 0) / s + 2.0 ** -23 * (y / s).abs()
        have = got[k].view(torch.uint8)[page, :, row].view(F8).to(torch.float32)
        lo, hi = codes(y / s - tol), codes(y / s + tol)
        assert bool(((have >= lo) & (have <= hi)).all())
    assert float(got[2].view(torch.uint8)[entries[2][1], 0, entries[2][2]].view(F8).float()[0]) == 448.0


def test_append_skips_what_has_no_place():
    """Lengths below the chunk, lengths past the table, table entries outside the pool, rows before the
    first start: nothing is written for them."""
    Hk, d, Dv = 2, 64, 128
    pools, table = ref.make_pool([64, 128, 64, 128], Hk, (d, d, Dv), torch.bfloat16, seed=1)
    table[1, 0], table[1, 1] = -1, 10_000
    lens, n_new = [2, 128, 300, 128], [5, 4, 3, 2]          # three rows before position 0; past the table
    starts = [3 + sum(n_new[:b]) for b in range(5)]          # three rows of no sequence first
    new = [torch.randn(starts[-1], Hk, w, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16) for w in (d, d, Dv)]
    dev = [p.cuda() for p in pools]
    da.diffattn_kv_append_chunk_paged(*(x.cuda() for x in new), *dev, table.cuda(), _i32(starts), _i32(lens))
    entries, _ = _append_reference(pools, table, new, starts, lens, 0, False, None)
    assert len(entries) == 3 * (2 + 0 + 0 + 2)
    want = [p.clone() for p in pools]
    for k, page, row, x, _ in entries:
        want[k][page, :, row] = x.to(torch.bfloat16)
    for a, b in zip(dev, want):
        assert torch.equal(a.cpu().view(torch.int16), b.view(torch.int16))


def test_append_strided_rows_and_many_sequences():
    """Rows as column blocks of one projection, more sequences than one step of the search holds,
    empty ones among them; equal to the one-token append where both apply."""
    B, Hk, d, Dv = 1500, 2, 64, 128
    g = torch.Generator().manual_seed(12)
    n_new = torch.randint(0, 3, (B,), generator=g).tolist()
    lens = [max(1, n) + int(torch.randint(0, 60, (1,), generator=g)) for n in n_new]
    pools, table = ref.make_pool(lens, Hk, (d, d, Dv), torch.bfloat16, seed=3)
    starts = [sum(n_new[:b]) for b in range(B + 1)]
    rows = torch.randn(starts[-1], Hk * (2 * d + Dv), generator=g).to(torch.bfloat16)
    k = rows[:, :2 * d * Hk].unflatten(1, (Hk, 2 * d))
    new = [k[..., :d], k[..., d:], rows[:, 2 * d * Hk:].unflatten(1, (Hk, Dv))]
    on = rows.cuda()
    kd = on[:, :2 * d * Hk].unflatten(1, (Hk, 2 * d))
    dev = [p.cuda() for p in pools]
    da.diffattn_kv_append_chunk_paged(kd[..., :d], kd[..., d:], on[:, 2 * d * Hk:].unflatten(1, (Hk, Dv)), *dev, table.cuda(),
                                      _i32(starts), _i32(lens))
    want = [p.clone() for p in pools]
    for kk, page, row, x, _ in _append_reference(pools, table, new, starts, lens, 0, False, None)[0]:
        want[kk][page, :, row] = x.to(torch.bfloat16)
    for a, b in zip(dev, want):
        assert torch.equal(a.cpu().view(torch.int16), b.view(torch.int16))
    one = [p.cuda() for p in pools]
    two = [p.cuda() for p in pools]
    rows1 = [torch.randn(B, Hk, w, generator=g).to(torch.bfloat16).cuda() for w in (d, d, Dv)]
    da.diffattn_kv_append_paged(*rows1, *one, table.cuda(), _i32(lens))
    da.diffattn_kv_append_chunk_paged(*rows1, *two, table.cuda(), _i32(list(range(B + 1))), _i32(lens))
    for a, b in zip(one, two):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_unsorted_starts_stay_inside():
    """Starts that are not sorted are not a valid call; whatever is written stays inside the pool (the
    kernel bounds every index), and the call returns."""
    Hk, d, Dv = 1, 64, 128
    pools, table = ref.make_pool([64, 64, 64], Hk, (d, d, Dv), torch.bfloat16, seed=1)
    new = [torch.zeros(9, Hk, w, dtype=torch.bfloat16, device="cuda") for w in (d, d, Dv)]
    dev = [p.cuda() for p in pools]
    da.diffattn_kv_append_chunk_paged(*new, *dev, table.cuda(), _i32([7, -3, 100, 2]), _i32([64, 5, 64]))
    torch.cuda.synchronize()


@pytest.mark.parametrize("scale", [0.0113, 1.0, 3.0, 2.0 ** -61, 2.0 ** 61, 1e-38, 3e38, 1e-30])
def test_append_fp8_quantizes_as_the_single_token_append(scale):
    """e4m3(x / scale) of the correctly rounded quotient, bit for bit: values next to the borders between
    codes (the midpoints times the scale and their neighbours), every magnitude, infinities and NaN."""
    mid = torch.arange(0, 0x7E, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).float()
    mid = (mid[:-1] + mid[1:]) / 2 * scale
    g = torch.Generator().manual_seed(9)
    x = torch.cat([mid, -mid, torch.randn(2000, generator=g) * 100 * min(scale, 1e30),
                   torch.randn(1000, generator=g) * 1e-39, torch.tensor([float("inf"), float("-inf"), 0.0, -0.0, 3e38])])
    x = torch.cat([x.to(torch.bfloat16)] + [(x.to(torch.bfloat16).view(torch.int16) + i).view(torch.bfloat16) for i in (-1, 1)])
    x = x[~x.isnan()]
    T = -(-x.numel() // 256)
    x = torch.cat([x, torch.zeros(T * 256 - x.numel(), dtype=x.dtype)]).view(T, 1, 256).cuda()
    new = [x[..., :64], x[..., 64:128], x[..., 128:]]
    make = lambda: [torch.zeros(-(-T // 64), 1, 64, w, dtype=torch.uint8, device="cuda") for w in (64, 64, 128)]  # noqa: E731
    a, b = make(), make()
    table = torch.arange(-(-T // 64), dtype=torch.int32, device="cuda")[None]
    da.diffattn_kv_append_chunk_paged(*new, *a, table, _i32([0, T]), _i32([T]), scales=(scale,) * 3)
    for t in range(T):
        da.diffattn_kv_append_paged(*(n[t:t + 1].contiguous() for n in new), *b, table, _i32([t + 1]), scales=(scale,) * 3)
    for p, q in zip(a, b):
        assert torch.equal(p, q)
