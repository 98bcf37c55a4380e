"""Rotary positions and per-head query/key norms on the GPU against the fp64
definitions (oracle/rope.py), element by element.

Tolerances (u = half a step of the output type relative to the value: bf16
2^-8, fp16 2^-11, fp32 2^-24):
  rotation  u |ref| + 2^-20 m |pair|:  the angle is held to 2^-25 of a turn's
            half (pi 2^-24), cosine and sine each round (2^-23 together) and
            so do the products and the sum (3 * 2^-24); their sum is below
            2^-21 of the pair's length.
  norm      2^-18 m |pair| instead: the mean square sums at most 16 terms in a
            row and 5 levels of a tree (21 * 2^-24 of a positive sum, half of
            it after the root), plus rsqrt, division and two products.
  gradient  2^-17 of r (max|g w| + |x| r^2 mean|g w x|): the same sums, now
            with cancellation, so relative to the absolute values.
  weights   2^-17 sum|g x r|: at most 64 terms in a row per thread at these
            sizes, then 48 levels and rows of partial sums (112 * 2^-24).
fp16 results below 2^-14 round in steps of 2^-24 (half a step 2^-25).
"""
import pytest
import torch

import context_attention_fwd_gb300 as ctx
from oracle import rope as ref

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ctx.load_library(build_if_missing=True)


def _rand(g, B, S, H, D, dt, layout="bshd"):
    t = torch.randn((B, S, H, D) if layout == "bshd" else (S, B, H, D), generator=g).to(dt).cuda()
    return t if layout == "bshd" else t.permute(1, 0, 2, 3)


def _pair_len(x, rot, inter):
    """Length of each element's pair (its own magnitude past rot), fp64."""
    n = x.abs().clone()
    if inter:
        h = torch.hypot(x[..., 0:rot:2], x[..., 1:rot:2])
        n[..., 0:rot:2], n[..., 1:rot:2] = h, h
    else:
        h = torch.hypot(x[..., :rot // 2], x[..., rot // 2:rot])
        n[..., :rot // 2], n[..., rot // 2:rot] = h, h
    return n


def close(name, got, want, bound, dt):
    err = (got.double().cpu() - want).abs()
    tol = HALF[dt] * want.abs() * (1 + 2.0 ** -10) + bound + (2.0 ** -25 if dt == FP else 1e-38)
    bad = err > tol
    assert not bad.any(), f"{name}: {int(bad.sum())} off, worst {(err / tol).max().item():.2f} of the tolerance"


def _positions(g, B, S, kind):
    """(argument for the call, int64 [B,S] on the CPU, offset)."""
    if kind == "offset":
        return None, (77 + torch.arange(S)).expand(B, S), 77
    if kind == "shared":
        p = torch.randint(-(1 << 31), 1 << 31, (S,), generator=g)
        return p.cuda(), p.expand(B, S), 0
    p = torch.randint(0, 1 << 40, (B, S), generator=g)
    return p.cuda(), p, 0


CASES = [  # B, S, Hq, Hk, D, rot, interleaved, dtype, layout, positions
    (1, 1, 1, 0, 64, 64, False, BF, "bshd", "offset"),
    (2, 37, 24, 4, 256, 64, False, BF, "bshd", "each"),
    (1, 130, 24, 24, 128, 128, True, BF, "bshd", "shared"),
    (3, 33, 16, 16, 64, 64, False, FP, "sbhd", "each"),
    (1, 50, 3, 1, 80, 80, True, F32, "sbhd", "shared"),
    (2, 19, 5, 2, 96, 48, False, BF, "bshd", "each"),       # rot / 2 not a multiple of 16
    (1, 23, 4, 2, 96, 34, True, FP, "bshd", "each"),        # single-pair kernel
    (1, 21, 2, 2, 6, 2, False, F32, "bshd", "offset"),      # tiny heads
    (1, 9, 7, 3, 512, 512, False, F32, "bshd", "each"),
    (1, 9, 2, 1, 512, 510, True, BF, "bshd", "shared"),
    (1, 9, 2, 1, 510, 254, False, BF, "bshd", "shared"),
    (2, 19, 5, 2, 128, 50, False, BF, "bshd", "each"),      # half pairs whose halves are not whole groups:
    (1, 37, 24, 4, 80, 40, False, FP, "sbhd", "shared"),    # partners through shared memory, in twos
    (1, 11, 3, 2, 64, 22, False, F32, "bshd", "each"),      # or one by one
    (1, 7, 9, 1, 512, 6, False, BF, "bshd", "offset"),
    (1, 7, 2, 2, 16, 10, False, F32, "bshd", "offset"),
    (1, 40, 3, 2, 48, 48, False, BF, "bshd", "each"),       # three groups of a row's four lanes
    (2, 3000, 4, 2, 64, 16, True, BF, "bshd", "shared"),    # many tokens: one unit per token
    (1, 5000, 16, 2, 64, 28, False, BF, "bshd", "shared"),
    (16, 1, 24, 4, 256, 256, True, FP, "bshd", "each"),     # newest tokens
]


@pytest.mark.parametrize("B,S,Hq,Hk,D,rot,inter,dt,layout,pos", CASES)
def test_rotation_and_its_gradient(B, S, Hq, Hk, D, rot, inter, dt, layout, pos):
    g = torch.Generator().manual_seed(B * 1000 + S)
    table = ctx.rope_table(rot, interleaved=inter, magnitude=1.25)
    arg, p, off = _positions(g, B, S, pos)
    ang = ref.angles(table.turns, p)
    q = _rand(g, B, S, Hq, D, dt, layout)
    k = _rand(g, B, S, Hk, D, dt, layout) if Hk else None
    for call, back in ((ctx.rope_fwd, False), (ctx.rope_bwd, True)):
        for name, x, y in zip("qk", (q, k), call(q, k, table, positions=arg, offset=off)):
            if x is None:
                assert y is None
                continue
            assert y.dtype == dt and (y.stride(0) >= y.stride(1)) == (x.stride(0) >= x.stride(1))
            x64 = x.double().cpu()
            close(name, y, ref.rotate(x64, ang, rot, inter, 1.25, transpose=back),
                  2.0 ** -20 * 1.25 * _pair_len(x64, rot, inter), dt)


@pytest.mark.parametrize("D,rot", [(64, 64), (80, 32), (128, 36), (256, 128)])
@pytest.mark.parametrize("Hq,Hk,S,inter,dt", [
    (3, 1, 300, False, BF), (8, 2, 3000, True, BF), (6, 2, 7, False, F32), (1, 1, 3000, True, FP), (5, 3, 200, True, F32),
    (2, 9, 3000, False, FP), (8, 8, 300, False, BF)])
def test_few_heads_of_both_sides(Hq, Hk, S, inter, dt, D, rot):
    """Queries' and keys' heads that share a pass, stored differently."""
    test_rotation_and_its_gradient(2, S, Hq, Hk, D, rot, inter, dt, "bshd", "each")
    g = torch.Generator().manual_seed(S)
    table = ctx.rope_table(rot, interleaved=inter)
    q, k = _rand(g, 2, S, Hq, D, dt), _rand(g, 2, S, Hk + 2, D, dt, "sbhd")[:, :, 1:-1]
    a, b = ctx.rope_fwd(q, k, table, offset=5)
    assert torch.equal(a, ctx.rope_fwd(q, None, table, offset=5)[0])
    assert torch.equal(b, ctx.rope_fwd(k, None, table, offset=5)[0])
    ctx.rope_fwd(q, k, table, offset=5, q_out=q, k_out=k)
    assert torch.equal(q, a) and torch.equal(k, b)


@pytest.mark.parametrize("wdt", [None, torch.float32, "same"])
@pytest.mark.parametrize("B,S,Hq,Hk,D,rot,inter,dt,layout,pos", CASES)
def test_norm_and_its_gradient(B, S, Hq, Hk, D, rot, inter, dt, layout, pos, wdt):
    g = torch.Generator().manual_seed(B * 1000 + S + 1)
    table = ctx.rope_table(rot, interleaved=inter, magnitude=1.25)
    arg, p, off = _positions(g, B, S, pos)
    ang, eps, m = ref.angles(table.turns, p), 1e-3, 1.25
    xs = [_rand(g, B, S, H, D, dt, layout) if H else None for H in (Hq, Hk)]
    gs = [_rand(g, B, S, H, D, dt, layout) if H else None for H in (Hq, Hk)]
    ws = [None if wdt is None or x is None else
          (1 + 0.3 * torch.randn(D, generator=g)).to(dt if wdt == "same" else wdt).cuda() for x in xs]
    ys = ctx.qk_norm_rope_fwd(*xs, *ws, table, positions=arg, offset=off, eps=eps)
    dq, dk, dwq, dwk = ctx.qk_norm_rope_bwd(*gs, *xs, *ws, table, positions=arg, offset=off, eps=eps)
    for name, x, gy, w, y, dx, dw in zip("qk", xs, gs, ws, ys, (dq, dk), (dwq, dwk)):
        if x is None:
            assert y is None and dx is None and dw is None
            continue
        x64, g64 = x.double().cpu(), gy.double().cpu()
        w64 = None if w is None else w.double().cpu()
        n = ref.norm(x64, w64, eps)
        close(f"{name} out", y, ref.rotate(n, ang, rot, inter, m), 2.0 ** -18 * m * _pair_len(n, rot, inter), dt)
        gr = ref.rotate(g64, ang, rot, inter, m, transpose=True)
        dx_ref, dw_ref = ref.norm_grad(gr, x64, w64, eps)
        r = 1.0 / torch.sqrt((x64 * x64).mean(-1, keepdim=True) + eps)
        gw = m * _pair_len(g64, rot, inter) * (1.0 if w64 is None else w64.abs())
        size = r * (gw + x64.abs() * r * r * (gw * x64.abs()).mean(-1, keepdim=True))
        close(f"d{name}", dx, dx_ref, 2.0 ** -17 * size, dt)
        if w is None:
            assert dw is None
        else:
            assert dw.dtype == F32
            bound = 2.0 ** -17 * (m * _pair_len(g64, rot, inter) * (x64 * r).abs()).flatten(0, 2).sum(0)
            close(f"dw{name}", dw, dw_ref, bound, F32)


def test_norm_alone_without_a_table():
    g = torch.Generator().manual_seed(3)
    q = _rand(g, 2, 40, 6, 128, BF)
    w = (1 + 0.3 * torch.randn(128, generator=g)).cuda()
    y, _ = ctx.qk_norm_rope_fwd(q, None, w, None, None)
    n = ref.norm(q.double().cpu(), w.double().cpu(), 1e-6)
    close("q", y, n, 2.0 ** -18 * n.abs(), BF)


@pytest.mark.parametrize("batched", [False, True])
@pytest.mark.parametrize("D", [128, 132])  # 16-byte groups, single pairs
def test_several_position_axes(batched, D):
    """Frames, rows and columns on 22/21/21 pairs; the pairs of one 8-wide
    group straddle a section boundary."""
    g = torch.Generator().manual_seed(9)
    B, S, secs = 2, 75, (22, 21, 21)
    table = ctx.rope_table(128, sections=secs, interleaved=True)
    p = torch.randint(-5, 4000, (B, S, 3) if batched else (S, 3), generator=g)
    wide = torch.repeat_interleave(torch.arange(3), torch.tensor(secs))
    ang = ref.angles(table.turns, (p if batched else p.expand(B, S, 3))[..., wide])
    q, k = _rand(g, B, S, 4, D, BF), _rand(g, B, S, 2, D, BF)
    for x, y in zip((q, k), ctx.rope_fwd(q, k, table, positions=p.cuda())):
        x64 = x.double().cpu()
        close("axes", y, ref.rotate(x64, ang, 128, True), 2.0 ** -20 * _pair_len(x64, 128, True), BF)
    with pytest.raises(ValueError, match="positions"):
        ctx.rope_fwd(q, k, table)
    with pytest.raises(ValueError, match="positions"):
        ctx.rope_fwd(q, k, table, positions=p[..., :2].cuda())


@pytest.mark.parametrize("shift,rot", [(0, 32), (0, 20), (1, 32)])  # 16-byte rows (twice); off the boundary (single pairs)
def test_views_of_one_projection_in_place(shift, rot):
    """q and k as views of a packed [B,S,(Hq+2Hk) D] projection, rotated in
    place: v, the padding and everything around the views stay as they were."""
    g = torch.Generator().manual_seed(4)
    B, S, Hq, Hk, D = 2, 45, 6, 2, 64
    width = (Hq + 2 * Hk) * D + 24
    buf = torch.randn(B * S * width + 64, generator=g).to(BF).cuda()
    before = buf.clone()
    rows = buf[shift:shift + B * S * width].view(B, S, width)
    q = rows[:, :, :Hq * D].unflatten(2, (Hq, D))
    k = rows[:, :, Hq * D:(Hq + Hk) * D].unflatten(2, (Hk, D))
    q0, k0 = q.double().cpu(), k.double().cpu()
    w = (1 + 0.3 * torch.randn(D, generator=g)).cuda()
    table = ctx.rope_table(rot)
    ctx.qk_norm_rope_fwd(q, k, w, w, table, offset=5, q_out=q, k_out=k)
    ang = ref.angles(table.turns, (5 + torch.arange(S)).expand(B, S))
    for x, x0 in ((q, q0), (k, k0)):
        n = ref.norm(x0, w.double().cpu(), 1e-6)
        close("view", x, ref.rotate(n, ang, rot, False), 2.0 ** -18 * _pair_len(n, rot, False), BF)
    mask = torch.zeros_like(buf, dtype=torch.bool)
    mask[shift:shift + B * S * width].view(B, S, width)[:, :, :(Hq + Hk) * D] = True
    assert torch.equal(buf[~mask].view(torch.int16), before[~mask].view(torch.int16))


def test_gradient_against_differences():
    """fp32 gradients against central differences of the fp64 definition
    (difference error below 1e-8; the gradient's own tolerance as above)."""
    g = torch.Generator().manual_seed(6)
    B, S, H, D, rot = 1, 3, 2, 32, 16
    table = ctx.rope_table(rot)
    x, gy = _rand(g, B, S, H, D, F32), _rand(g, B, S, H, D, F32)
    w = (1 + 0.3 * torch.randn(D, generator=g)).cuda()
    dx, _, dw, _ = ctx.qk_norm_rope_bwd(gy, None, x, None, w, None, table, offset=9, eps=1e-3)
    ang = ref.angles(table.turns, (9 + torch.arange(S)).expand(B, S))
    x64, w64, g64 = x.double().cpu(), w.double().cpu(), gy.double().cpu()
    f = lambda x, w: (ref.rotate(ref.norm(x, w, 1e-3), ang, rot, False) * g64).sum()
    h = 1e-5
    for i in range(x64.numel()):
        e = torch.zeros(x64.numel(), dtype=torch.float64)
        e[i] = h
        e = e.view_as(x64)
        d = (f(x64 + e, w64) - f(x64 - e, w64)) / (2 * h)
        assert abs(d - dx.flatten()[i].item()) < 1e-8 + 2.0 ** -17 * 20
    for i in range(D):
        e = torch.zeros(D, dtype=torch.float64)
        e[i] = h
        d = (f(x64, w64 + e) - f(x64, w64 - e)) / (2 * h)
        assert abs(d - dw[i].item()) < 1e-8 + 2.0 ** -17 * 20


def test_rows_of_nan_and_zero_stay_apart():
    """A row of NaN, of infinities or of zeros changes no other row, and a zero
    row normalises to zero (eps > 0)."""
    g = torch.Generator().manual_seed(8)
    q = _rand(g, 1, 64, 4, 128, BF)
    table = ctx.rope_table(128)
    clean, _ = ctx.qk_norm_rope_fwd(q, None, None, None, table)
    bad = q.clone()
    bad[0, 5, 1] = float("nan")
    bad[0, 9, 2, 3] = float("inf")
    bad[0, 11, 0] = 0
    y, _ = ctx.qk_norm_rope_fwd(bad, None, None, None, table)
    assert torch.isnan(y[0, 5, 1]).all() and (y[0, 11, 0] == 0).all()
    keep = torch.ones(64, 4, dtype=torch.bool)
    keep[5, 1] = keep[9, 2] = keep[11, 0] = False
    assert torch.equal(y[0][keep.cuda()], clean[0][keep.cuda()])


def test_repeats_and_graph_replay_are_bit_equal():
    """The weight gradients sum in a fixed order; a captured backward replays
    on new values of its inputs."""
    g = torch.Generator().manual_seed(12)
    B, S, Hq, Hk, D = 1, 900, 8, 4, 128
    table = ctx.rope_table(D, interleaved=True)
    q, k, gq, gk = (_rand(g, B, S, h, D, BF) for h in (Hq, Hk, Hq, Hk))
    w = (1 + 0.3 * torch.randn(D, generator=g)).cuda()
    call = lambda out=None: ctx.qk_norm_rope_bwd(gq, gk, q, k, w, w, table, **(out or {}))
    first = call()
    for _ in range(3):
        for a, b in zip(first, call()):
            assert torch.equal(a, b)
    out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dwq=torch.empty(D, device="cuda"),
               dwk=torch.empty(D, device="cuda"),
               workspace=torch.empty(ctx.load_library().ctx_qk_norm_rope_workspace_size(D), dtype=torch.uint8, device="cuda"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    graph.replay()
    for n, a in zip(("dq", "dk", "dwq", "dwk"), first):
        assert torch.equal(a, out[n])
    q.copy_(_rand(g, B, S, Hq, D, BF))
    graph.replay()
    for n, a in zip(("dq", "dk", "dwq", "dwk"), call()):
        assert torch.equal(a, out[n])


def test_side_stream_and_outputs_not_written_elsewhere():
    g = torch.Generator().manual_seed(13)
    q = _rand(g, 1, 300, 4, 128, BF)
    table = ctx.rope_table(128)
    want, _ = ctx.rope_fwd(q, None, table)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y, _ = ctx.rope_fwd(q, None, table)
    s.synchronize()
    assert torch.equal(y, want)


def test_long_strides_pass_32_bits():
    """Rows more than 2^31 elements apart (a view of one large buffer)."""
    far = (1 << 31) + 8
    buf = torch.zeros(far + 4 * 64 * 2, dtype=BF, device="cuda")
    q = buf.as_strided((2, 4, 1, 64), (far, 64, 64, 1))
    g = torch.Generator().manual_seed(14)
    q.copy_(torch.randn(2, 4, 1, 64, generator=g))
    q0 = q.double().cpu()
    table = ctx.rope_table(64)
    ctx.rope_fwd(q, None, table, q_out=q)
    ang = ref.angles(table.turns, torch.arange(4).expand(2, 4))
    close("far", q, ref.rotate(q0, ang, 64, False), 2.0 ** -20 * _pair_len(q0, 64, False), BF)


def test_refusals_on_the_gpu():
    q = torch.zeros(1, 4, 2, 64, dtype=BF, device="cuda")
    table = ctx.rope_table(64)
    with pytest.raises(ValueError):
        ctx.rope_fwd(q, q.float(), table)
    with pytest.raises(ctx.CtxError):
        ctx.rope_fwd(q, q[:, :2], table)
    with pytest.raises(ValueError):
        ctx.rope_fwd(q, None, table, positions=torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        ctx.rope_fwd(q, None, table, positions=torch.zeros(5, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        ctx.rope_fwd(q, None, ctx.rope_table(64, device="cpu"))
    with pytest.raises(ValueError):
        ctx.qk_norm_rope_fwd(q, None, torch.ones(32, device="cuda"), None, table)
    w = torch.ones(64, device="cuda")
    for ws in (torch.empty(1 << 22, dtype=torch.uint8), torch.empty(1 << 23, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            ctx.qk_norm_rope_bwd(q, None, q, None, w, None, table, workspace=ws)
    with pytest.raises(ctx.CtxError):
        ctx.qk_norm_rope_bwd(q, None, q, None, w, None, table, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ctx.CtxError):
        ctx.rope_fwd(q, None, ctx.rope_table(128))
    with pytest.raises(ctx.CtxError):
        ctx.rope_fwd(q, None, table, q_out=torch.zeros(1, 4, 3, 64, dtype=BF, device="cuda"))
