"""The module and the layer with rotary positions, in training form and over a paged cache, on the
GPU, against float64 references that round where the path holds 16 bits.

Tolerance of the paged paths, relative RMS: the attention's own 3e-3 (parity.py). Beside it, in
quadrature: a projection that rounds to the other neighbour than the reference's (fp32 sums are off
by 1e-6 of a value, half a bf16 step is 2^-9 of one: one value in a thousand is a whole step 2^-8
off, 2^-8 / sqrt 1000 = 1.2e-4 RMS); the attention's output rounded to the operands' type (half a
step over sqrt 3 and x 0.72: bf16 1.6e-3, fp16 2e-4); W_O's fp32 sums (1e-6). Together 3.0e-3 for
fp16 and sqrt(3^2 + 1.6^2) = 3.4e-3 for bf16 operands. A single element of [T, d_model] is a sum
over h * Dv >= 512 such errors, near normal: at most 6 sigma among 1e5 of them, and a row's sigma
up to twice the mean's (its P has few large weights): 12 x the relative RMS of the outputs' RMS."""

import numpy as np
import pytest
import torch

import differential_attention_02_gb300 as da
import serving_reference as ref
from oracle import diffattn_oracle as orc

pytestmark = pytest.mark.gpu
F8, BF, F16 = torch.float8_e4m3fn, torch.bfloat16, torch.float16
LAM, LI = 0.45, 0.47
RMS = {F16: 3.0e-3, BF: 3.4e-3}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from differential_attention_02_gb300 import build
    build.build()
    da.load_library()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _close(got, want, tol, what):
    err = got.double().cpu() - want
    size = want.square().mean().sqrt()
    rms, top = float(err.square().mean().sqrt() / size), float(err.abs().max() / size)
    print(f"{what}: rel-RMS {rms:.2e}, max/RMS {top:.2e}")
    assert rms <= tol and top <= 12 * tol, f"{what}: rel-RMS {rms:.3e}, max/RMS {top:.3e} against {tol:.1e}"


class Model:
    """One module's (and layer's) weights, standard normal over the root of their height: projections of
    normalised rows come out with unit variance."""

    def __init__(self, dm, h, group, d, dtype, d_ff=256, seed=0):
        g = torch.Generator().manual_seed(seed)
        w = lambda k, n: (torch.randn(k, n, generator=g) * k ** -0.5).to(dtype)  # noqa: E731
        self.dm, self.h, self.hk, self.group, self.d, self.Dv, self.dtype = dm, h, h // group, group, d, 2 * d, dtype
        self.w_q, self.w_k, self.w_v = w(dm, h * 2 * d), w(dm, self.hk * 2 * d), w(dm, self.hk * 2 * d)
        self.w_qkv = torch.cat([self.w_q, self.w_k, self.w_v], 1)
        self.w_o, self.w_gate, self.w_up, self.w_down = w(h * 2 * d, dm), w(dm, d_ff), w(dm, d_ff), w(d_ff, dm)
        self.g = g

    def project(self, x, dtype):
        """The five operands of x [.., dm], rounded to dtype: [.., heads, width]."""
        q, k, v = ((x.double() @ w.double()).to(dtype) for w in (self.w_q, self.w_k, self.w_v))
        q, k, v = q.unflatten(-1, (self.h, -1)), k.unflatten(-1, (self.hk, -1)), v.unflatten(-1, (self.hk, -1))
        d = self.d
        return q[..., :d], q[..., d:], k[..., :d], k[..., d:], v


@pytest.mark.parametrize("positions", [False, True])
@pytest.mark.parametrize("d,h,dtype", [(64, 4, BF), (128, 2, F16), (32, 8, BF)])
def test_module_with_rope(d, h, dtype, positions):
    """module_fwd(rope=...): Q and K rotated in place between the projections and the attention. Q and K are
    fp16, rounded once more by the rotation: 2^-11 roundings, in the quadrature above without weight."""
    B, N, dm = 2, 150, 256
    m = Model(dm, h, 1, d, dtype, seed=d)
    x = torch.randn(B, N, dm, generator=m.g).to(dtype)
    pos = torch.randint(0, 9000, (B, N), generator=m.g, dtype=torch.int32) if positions else None
    kw = dict(scaling="ramp", factor=4.0, original_length=64)
    plan = da.rope_plan(d // 2, interleaved=positions, **kw)
    f, mag = ref.frequencies(d // 2, scaling="ramp", factor=4.0, original=64)
    dev = {k: getattr(m, k).cuda() for k in ("w_q", "w_k", "w_v", "w_o", "w_qkv")}
    ws = da.workspace(256)
    run = lambda **k: da.module_fwd(x.cuda(), dev["w_q"], dev["w_k"], dev["w_v"], dev["w_o"], h, LAM, LI, ws=ws,  # noqa: E731
                                    out_dtype=torch.float32, rope=plan, positions=None if pos is None else pos.cuda(), **k)
    if d == 32:  # the 16-bit prefill has no such heads, and refuses them with or without a rotation
        with pytest.raises(da.DiffAttnError):
            run(w_qkv=dev["w_qkv"])
        return
    got = run(w_qkv=dev["w_qkv"])
    assert da.read_error(ws) == 0
    assert torch.equal(got, run())  # three projections give the same columns
    p = (torch.arange(N).expand(B, N) if pos is None else pos).double()
    angle = (p[..., None] * f)[:, :, None]
    ops = m.project(x, F16)
    rot = [ref.rotate(t.double(), angle, mag, positions).to(F16) for t in ops[:4]] + [ops[4]]
    att = orc.diffattn_fwd(*(t.transpose(1, 2) for t in rot), LAM, LI)
    want = torch.from_numpy(att.reshape(B, N, -1)) @ m.w_o.double()
    _close(got, want, RMS[dtype], f"module with rope d{d} {dtype}")
    with pytest.raises(ValueError):  # positions without a rotation
        da.module_fwd(x.cuda(), dev["w_q"], dev["w_k"], dev["w_v"], dev["w_o"], h, LAM, LI, positions=_i32([[0]]))


def test_layer_with_rope_is_the_module_with_rope():
    """layer_fwd(rope=...) against its own parts: the same kernels in the same order, bit for bit."""
    m = Model(256, 2, 1, 64, BF, seed=1)
    x = torch.randn(1, 130, 256, generator=m.g).to(BF).cuda()
    plan = da.rope_plan(64)
    c = lambda n: getattr(m, n).cuda()  # noqa: E731
    w_gu = da.interleave_gate_up(c("w_gate"), c("w_up"))
    got = da.layer_fwd(x, c("w_q"), c("w_k"), c("w_v"), c("w_o"), w_gu, c("w_down"), 2, LAM, LI, w_qkv=c("w_qkv"), rope=plan)
    _, n1 = da.add_rmsnorm(x)
    att = da._module_attention(n1, c("w_q"), c("w_k"), c("w_v"), 2, LAM, LI, 1e-5, None, None, None, BF, rope=plan)
    y, y16, sq = da.gemm_residual(att, c("w_o"), x.view(130, 256), c16_dtype=BF, want_row_sq=True)
    want, _, _ = da.gemm_residual(da.gemm_swiglu(y16, w_gu, row_sq=sq, sq_count=256, out_dtype=BF), c("w_down"), y)
    assert torch.equal(got[0], want)
    plain = da.layer_fwd(x, c("w_q"), c("w_k"), c("w_v"), c("w_o"), w_gu, c("w_down"), 2, LAM, LI, w_qkv=c("w_qkv"))
    assert float((plain - got).abs().max()) > 0.1  # the rotation is not without effect


class Serving:
    """Two sequences served through a shared cache: prompts in chunks, then single tokens."""

    def __init__(self, m, total, fp8, r, seed=0):
        self.m, self.total, self.fp8 = m, total, fp8
        self.x = [torch.randn(n, m.dm, generator=m.g).to(m.dtype) for n in total]
        self.plan = da.rope_plan(r, base=5e5)
        self.f, _ = ref.frequencies(r, base=5e5)
        pools, self.table = ref.make_pool(total, m.hk, (m.d, m.d, m.Dv), F8 if fp8 else BF, seed=seed)
        self.pools = tuple(p.cuda() for p in ref.poison(pools, self.table, [0] * len(total)))
        self.scales = ref.SCALES if fp8 else None
        self.done = [0] * len(total)
        self.dev = {k: getattr(m, k).cuda() for k in ("w_qkv", "w_o", "w_gate", "w_up", "w_down")}

    def step(self, n, pad=0):
        """Row arguments of the step that adds n[b] tokens to sequence b, and the rows (pad rows behind)."""
        rows = torch.cat([x[a:a + k] for x, a, k in zip(self.x, self.done, n)] + [torch.full((pad, self.m.dm), 3.0).to(self.m.dtype)])
        pos = torch.cat([torch.arange(a, a + k) for a, k in zip(self.done, n)] + [torch.zeros(pad, dtype=torch.int64)])
        self.starts = [sum(n[:b]) for b in range(len(n) + 1)]
        self.done = [a + k for a, k in zip(self.done, n)]
        self.pos = pos.to(torch.int32)
        return rows, (self.m.h, self.pools, self.table.cuda(), _i32(self.starts), _i32(self.done), LAM, LI, max(self.total),
                      self.m.group, self.plan, self.pos.cuda(), self.scales)

    def attention(self, rows):
        """float64 attention [T, h * Dv] of the normalised rows over the cache as it stands (checked on its own)."""
        m = self.m
        angle = (self.pos.double()[:, None] * self.f)[:, None]
        q1, q2, k1, k2, v = m.project(rows, BF)
        q = [ref.rotate(t.double(), angle).to(BF) for t in (q1, q2)]
        pools = [p.cpu() for p in self.pools]
        att = ref.chunk_attention(*q, pools, self.table, self.starts, self.done, LAM, LI, group=m.group, scales=self.scales)
        att[self.starts[-1]:] = 0
        # The new entries. Each rounding is off by at most half a step: bf16 2^-8 of the value, K one more time
        # than here, and its RMS 2^-8 / sqrt 3. e4m3 (3 bits) 2^-4 of the value, so the RMS of the errors is at
        # most 2^-4 of the values' RMS (2^-4 / sqrt 3 = 0.036 for errors spread evenly over a step and values
        # just above a power of two, 0.024 for values spread evenly between two); the grid below the smallest
        # normal, 2^-9 x 2^-1 x 0.0127 = 1.2e-5, is nothing beside an RMS of one.
        new = [ref.rotate(t.double(), angle) for t in (k1, k2)] + [v.double()]
        for p, x, s in zip(pools, new, self.scales or (1, 1, 1)):
            for b, (a, e) in enumerate(zip(self.starts, self.starts[1:])):
                if e > a:
                    got = ref.gather(p, self.table, b, self.done[b], s)[:, self.done[b] - (e - a):].transpose(0, 1)
                    rel = float((got - x[a:e]).square().mean().sqrt() / x[a:e].square().mean().sqrt())
                    assert rel <= (2 ** -4 if self.fp8 else 2 ** -8), rel
        return att.flatten(1)


STEPS = ([100, 0, 7], [48, 88, 1], [1, 1, 1], [1, 1, 120])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,h,group,dtype", [(64, 4, 1, BF), (64, 8, 4, F16), (128, 4, 2, F16), (128, 2, 2, BF)])
def test_module_serve_steps(d, h, group, dtype, fp8):
    m = Model(256, h, group, d, dtype, seed=d + h)
    s = Serving(m, [150, 90, 129], fp8, d // 2)
    for n in STEPS:
        rows, args = s.step(n, pad=3)
        got = da.module_serve(rows.cuda(), s.dev["w_qkv"], s.dev["w_o"], *args, out_dtype=torch.float32)
        assert bool((got[s.starts[-1]:] == 0).all())
        _close(got, s.attention(rows) @ m.w_o.double(), RMS[dtype], f"module d{d} g{group} fp8={fp8} step {n}")


@pytest.mark.parametrize("dtype", [BF, F16])
def test_layer_serve_steps(dtype):
    """The layer: the residual stream and the feed-forward around the served module. The branches add to
    rows of unit size, so that the module's bound covers attention's part; SwiGLU's 16-bit operand, its
    16-bit output and the normalised copy of Y round three times more (1.6e-3 each for bf16)."""
    m = Model(256, 4, 2, 64, dtype, d_ff=512, seed=3)
    s = Serving(m, [150, 90, 129], False, 32)
    w_gu = da.interleave_gate_up(s.dev["w_gate"], s.dev["w_up"])
    gains = [1 + 0.1 * torch.randn(n, generator=m.g) for n in (256, 256)]
    for n in STEPS:
        rows, args = s.step(n)
        got = da.layer_serve(rows.float().cuda(), s.dev["w_qkv"], s.dev["w_o"], w_gu, s.dev["w_down"], *args,
                             norm1_weight=gains[0].cuda(), norm2_weight=gains[1].cuda())
        x = rows.double().numpy()
        n1 = torch.from_numpy(orc.rmsnorm_rows(x, 1e-5, gains[0].numpy())).to(dtype)
        y = x + s.attention(n1).numpy() @ m.w_o.double().numpy()
        want = y + orc.swiglu_ffn(orc.rmsnorm_rows(y, 1e-5, gains[1].numpy()), m.w_gate, m.w_up, m.w_down)
        tol = {BF: (3.4e-3 ** 2 + 3 * 1.6e-3 ** 2) ** 0.5, F16: 3.1e-3}[dtype]
        _close(got, torch.from_numpy(want), tol, f"layer {dtype} step {n}")


def test_serving_agrees_with_the_whole_prompt():
    """A prompt served in one call, in ragged chunks and by module_fwd: the same rows up to the paths'
    roundings (each within its bound of the exact value: twice the bound apart at most). Beside the
    attention, module_fwd keeps its V and P as the others do (bf16 Q, K, V)."""
    m = Model(256, 4, 1, 64, F16, seed=9)
    dev = {k: getattr(m, k).cuda() for k in ("w_q", "w_k", "w_v", "w_o")}
    outs = []
    for steps in ([[200]], [[64], [1], [100], [35]]):
        s = Serving(m, [200], False, 64)
        s.x = [torch.randn(200, 256, generator=torch.Generator().manual_seed(2)).to(F16)]
        part = []
        for n in steps:
            rows, args = s.step(n)
            part.append(da.module_serve(rows.cuda(), s.dev["w_qkv"], s.dev["w_o"], *args, out_dtype=torch.float32))
        outs.append(torch.cat(part))
    whole = da.module_fwd(s.x[0][None].cuda(), dev["w_q"], dev["w_k"], dev["w_v"], dev["w_o"], 4, LAM, LI,
                          out_dtype=torch.float32, qkv_dtype=BF, rope=s.plan)[0]
    _close(outs[0], outs[1].double().cpu(), 2 * RMS[F16], "one call against chunks")
    _close(whole, outs[0].double().cpu(), 2 * RMS[F16], "whole prompt")


def test_serving_graph_streams_and_empty_batches():
    """One captured decoding step replayed for the following tokens; the same step on another stream; a
    batch without rows; refusals."""
    m = Model(256, 4, 2, 64, BF, seed=5)
    make = lambda: Serving(m, [80, 140], False, 32)  # noqa: E731
    m.g.manual_seed(11)
    a = make()
    m.g.manual_seed(11)
    b = make()
    w = (a.dev["w_qkv"], a.dev["w_o"])
    for s in (a, b):
        rows, args = s.step([70, 130])
        da.module_serve(rows.cuda(), *w, *args)
    side, graph, buf = torch.cuda.Stream(), None, None
    for i in range(4):
        rows, args = a.step([1, 1])
        rows_b, args_b = b.step([1, 1])
        torch.cuda.synchronize()
        want = da.module_serve(rows_b.cuda(), *w, *args_b, stream=side)
        if graph is None:
            buf = [rows.cuda(), *args]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = da.module_serve(buf[0], *w, *buf[1:])
        buf[0].copy_(rows)
        for at in (4, 5, 11):  # q_start, seq_lens, positions
            buf[at].copy_(args[at - 1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want), i
    for p, q in zip(a.pools, b.pools):
        assert torch.equal(p.view(torch.int16), q.view(torch.int16))
    _, args = a.step([0, 0])
    empty = torch.empty(0, 256, dtype=BF, device="cuda")
    assert da.module_serve(empty, *w, *args).shape == (0, 256)
    rows, args = b.step([1, 0])
    for bad in (dict(kv_group=3), dict(rope=None), dict(positions=None), dict(positions=_i32([0, 0]))):
        names = ("n_heads", "pages", "block_table", "q_start", "seq_lens", "lam", "lam_init", "L", "kv_group", "rope",
                 "positions", "scales")
        with pytest.raises(ValueError):
            da.module_serve(rows.cuda(), *w, **{**dict(zip(names, args)), **bad})
    with pytest.raises(ValueError):
        da.module_serve(rows.cuda(), w[0][:, :-128], w[1], *args)


@pytest.mark.parametrize("dtype,interleaved", [(BF, False), (F16, True)])
def test_training_run(dtype, interleaved):
    """rotation, fwd_train, bwd_saved, transposed rotation: gradients with respect to the operands before the
    rotation, against the chain rule in float64 on the operands as rounded, and against central differences
    of the float64 forward along random directions. Bounds: those of the backward pass (its products round to
    the operands' type: 5e-3 RMS bf16, 1e-3 fp16, maximum twice that); the rotation in fp32 adds 1e-6.
    A difference along a random direction u is a sum over all elements of err * u: normal with
    sigma = |err| |u_i| <= bound * |grad| for unit-variance u; 4 sigma."""
    B, H, N, d, Dv = 1, 2, 140, 64, 128
    tol, top = {BF: (5e-3, 1e-2), F16: (1e-3, 2e-3)}[dtype]
    g = torch.Generator().manual_seed(77)
    raw = [torch.randn(B, H, N, w, generator=g).to(dtype) for w in (d, d, d, d, Dv)]
    dy = torch.randn(B, N, H, Dv, generator=g).to(dtype)
    pos = (torch.arange(N) * 3 + 5).to(torch.int32)[None]
    plan = da.rope_plan(48, interleaved=interleaved, magnitude=0.9)
    f, _ = ref.frequencies(48)
    angle = (pos.double()[..., None] * f)[:, None]
    qk = da.diffattn_rope([t.cuda() for t in raw[:4]], plan, positions=pos.cuda())
    out, saved = da.diffattn_fwd_train(*qk, raw[4].cuda(), LAM, LI)
    grads = da.diffattn_bwd(*qk, raw[4].cuda(), dy.cuda(), LAM, LI, saved=saved)
    names = ("dq1", "dq2", "dk1", "dk2")
    back = da.diffattn_rope([grads[k] for k in names], plan, positions=pos.cuda(), backward=True,
                            out=[grads[k] for k in names])
    rounded = [ref.rotate(t.double(), angle, 0.9, interleaved).to(dtype) for t in raw[:4]]
    same = [float((a.cpu() != b).float().mean()) for a, b in zip(qk, rounded)]
    assert max(same) < 2e-3  # a value next to a rounding border may fall on its other side
    want = orc.diffattn_bwd(*rounded, raw[4], dy, LAM, LI)
    for k, got in zip(names, back):
        exp = ref.rotate(torch.from_numpy(want[k]), angle, 0.9, interleaved, backward=True)
        err = got.double().cpu() - exp
        rr, ma = float(err.norm() / exp.norm()), float(err.abs().max() / exp.abs().max())
        print(f"{k}: rel-RMS {rr:.2e}, max {ma:.2e}")
        assert rr <= tol and ma <= top, (k, rr, ma)
    loss = lambda ops: float((torch.from_numpy(orc.diffattn_fwd(  # noqa: E731
        *(ref.rotate(t, angle, 0.9, interleaved) for t in ops), raw[4].double(), LAM, LI)) * dy.double()).sum())
    base = [t.double() for t in raw[:4]]
    for i, got in enumerate(back):
        u = torch.randn(B, H, N, d, generator=g).double()
        hi, lo = ([t + sgn * 1e-4 * u if j == i else t for j, t in enumerate(base)] for sgn in (1, -1))
        diff = (loss(hi) - loss(lo)) / 2e-4
        grad = got.double().cpu()
        # the operands' own rounding (half a step 2^-8 or 2^-11) moves the gradient in the same relative measure
        assert abs(float((grad * u).sum()) - diff) <= 4 * 2 * tol * float(grad.norm()), names[i]
    assert np.isfinite(float(out.float().abs().max()))
