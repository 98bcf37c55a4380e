"""Windowed attention with sinks on the GPU against the fp64 definition
(oracle/window.py), through the public calls.

Tolerance: the norm of the error within 8e-3 of the tensor's norm and no
element off by more than 2e-2 of the largest.  A rounding to bf16 is off by at
most 2^-8 of the value, 2^-8 / sqrt(3) = 2.3e-3 in the mean; the forward
rounds the probabilities and the output, the backward P, dS, the output that
delta is taken from and the gradient (four roundings: 4.6e-3 in the mean,
1.6e-2 at worst).  lse is fp32: 1e-3 as in the other parity tests."""
import random

import pytest
import torch

import context_attention_fwd_gb300 as ctx
from oracle import window as ref
from seeded_inputs import AttnShape, attn_inputs
from test_guard_bands_gpu import Guarded, GuardedLse

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ctx.load_library(build_if_missing=True)
    yield
    assert ctx.device_status() == 0


def close(name, got, want):
    g, r = got.double().cpu(), want
    assert torch.isfinite(g).all(), f"{name}: non-finite values"
    if r.abs().max() < 1e-9:  # identically zero but for fp64 noise
        assert g.abs().max() < 1e-3, name
        return
    nrm, mx = ((g - r).norm() / r.norm()).item(), ((g - r).abs().max() / r.abs().max()).item()
    assert nrm <= 8e-3 and mx <= 2e-2, f"{name}: norm-rel {nrm:.3e}, max-rel {mx:.3e}"


def run(sh, left, right, sinks, causal, offsets=None, P=None, scale=None):
    q, k, v, do = attn_inputs(sh)
    d = [t.cuda() for t in (q, k, v, do)]
    kw = dict(sinks=sinks, causal=causal, chunk_offsets=offsets, scale=scale)
    P = sh.P if P is None else P
    out, lse = ctx.attn_window_fwd(*d[:3], P, (left, right), **kw)
    grads = ctx.attn_window_bwd(*d[:3], out, lse, d[3], P, (left, right), **kw)
    torch.cuda.synchronize()
    assert ctx.device_status() == 0
    return (q, k, v, do), (out, lse, *grads)


def check(sh, left, right, sinks, causal, **kw):
    (q, k, v, do), (out, lse, dq, dk, dv) = run(sh, left, right, sinks, causal, **kw)
    args = (left, right, sinks, causal, kw.get("scale"))
    o_ref, l_ref = ref.attn_fwd(q, k, v, *args)
    close("out", out, o_ref)
    assert (lse.double().cpu() - l_ref).abs().max() < 1e-3
    for name, g, r in zip(("dq", "dk", "dv"), (dq, dk, dv), ref.attn_bwd(q, k, v, do, *args)):
        close(name, g, r)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("S,left,right,sinks,causal", [
    (1, 0, 0, 0, True), (2, 1, 0, 1, True), (127, 5, 0, 0, True), (128, 127, 0, 4, True), (129, 128, 0, 0, True),
    (300, 0, 0, 0, True),            # every row sees itself alone
    (300, 0, 0, 3, True),            # itself and the sinks
    (700, 100, 0, 4, True), (700, 127, 0, 128, True), (700, 128, 0, 129, True), (700, 1, 0, 700, True),
    (700, -1, 0, 4, True),           # unlimited to the left: plain causal
    (700, 64, 64, 0, False), (700, 200, 3, 5, False), (700, 0, 130, 300, False), (513, 10, -1, 0, False),
    (513, -1, -1, 0, False),         # nothing masked
])
def test_window_shapes(D, S, left, right, sinks, causal):
    check(AttnShape(B=1, S=S, Hq=2, Hkv=1, D=D, P=1), left, right, sinks, causal)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("left,right,sinks,causal", [
    (100, 0, 4, True), (40, 30, 4, False), (300, 0, 130, True), (0, 0, 1, True), (50, 0, 300, True), (63, 64, 1, False)])
def test_sink_walks_cut_into_parts(D, left, right, sinks, causal):
    """Enough query tiles that the sink tiles' walks are cut (20 tiles, windows
    of under eight)."""
    check(AttnShape(B=2, S=2500, Hq=2, Hkv=1, D=D, P=3), left, right, sinks, causal)


def _cases(n=40, seed=515):
    rng = random.Random(seed)
    out = []
    for i in range(n):
        D = rng.choice([64, 128, 256])
        Hkv = rng.choice([1, 2, 3])
        S = rng.randint(1, 1500 if D < 256 else 1200)
        P = rng.randint(1, min(S, 9))
        offsets = None
        if P > 1 and rng.random() < 0.4:
            offsets = [0] + sorted(rng.sample(range(1, S), P - 1)) + [S]
        causal = rng.random() < 0.5
        left, right = rng.choice([0, rng.randint(0, 300), rng.randint(0, S), -1]), rng.choice([0, rng.randint(0, 300), -1])
        sinks = rng.choice([0, 0, rng.randint(1, 8), rng.randint(1, 200), rng.randint(1, S), S + 5])
        sh = AttnShape(B=rng.choice([1, 1, 2]), S=S, Hq=Hkv * rng.choice([1, 2, 6]), Hkv=Hkv, D=D, P=P,
                       layout=rng.choice(["bshd", "sbhd"]))
        out.append((i, sh, left, right, sinks, causal, offsets))
    return out


@pytest.mark.parametrize("i,sh,left,right,sinks,causal,offsets", _cases(),
                         ids=lambda v: str(v) if isinstance(v, int) else None)
def test_random_windows(i, sh, left, right, sinks, causal, offsets):
    check(sh, left, right, sinks, causal, offsets=offsets)


def test_more_tiles_than_a_grid_axis_holds():
    """65538 KV tiles (a grid's y and z axes hold 65535) and offsets past
    2^31 elements: the last rows against the definition on their own slab,
    which under a causal window of 100 holds all they depend on."""
    S, Hq, D, left, n, edge = 128 * 65537 + 5, 4, 64, 99, 512, 128
    g = torch.Generator(device="cuda").manual_seed(11)
    q, k, v, do = (torch.empty(1, S, h, D, device="cuda", dtype=torch.bfloat16).normal_(generator=g) for h in (Hq, 1, 1, Hq))
    out, lse = ctx.attn_window_fwd(q, k, v, 1, (left, 0), causal=True)
    grads = ctx.attn_window_bwd(q, k, v, out, lse, do, 1, (left, 0), causal=True)
    a = S - n
    slab = [t[:, a:].cpu() for t in (q, k, v, do)]
    o_ref, l_ref = ref.attn_fwd(*slab[:3], left, 0, 0, True)
    close("out", out[:, a + edge:], o_ref[:, edge:])
    assert (lse[:, :, a + edge:].double().cpu() - l_ref[:, :, edge:]).abs().max() < 1e-3
    for name, t, r in zip(("dq", "dk", "dv"), grads, ref.attn_bwd(*slab, left, 0, 0, True)):
        close(name, t[:, a + edge:], r[:, edge:])


def test_custom_scale():
    check(AttnShape(B=1, S=400, Hq=2, Hkv=2, D=128, P=2), 90, 0, 2, True, scale=0.2)


@pytest.mark.parametrize("D", [128, 256])
def test_result_does_not_depend_on_chunks_and_matches_the_plain_call(D):
    sh = AttnShape(B=1, S=900, Hq=4, Hkv=2, D=D, P=1)
    base = run(sh, 200, 0, 4, True)[1]
    for P, offsets in ((2, None), (5, [0, 1, 300, 301, 899, 900])):
        for i, (a, b) in enumerate(zip(base, run(sh, 200, 0, 4, True, P=P, offsets=offsets)[1])):
            if i == 2:  # dq is reduced in no fixed order
                assert (a.float() - b.float()).abs().max() <= 2e-2 * a.float().abs().max()
            else:
                assert torch.equal(a, b)
    (q, k, v, do), got = run(sh, -1, -1, 0, True)
    d = [t.cuda() for t in (q, k, v, do)]
    out, lse = ctx.attn_fwd(*d[:3], 1, causal=True)
    for a, b in zip(got, (out, lse, *ctx.attn_bwd(*d[:3], out, lse, d[3], 1, causal=True))):
        assert (a.float() - b.float()).abs().max() <= 2e-2 * b.float().abs().max()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("left,right,sinks,causal,P", [(100, 0, 4, True, 3), (40, 30, 130, False, 64)])
def test_outputs_and_workspace_stay_inside(D, left, right, sinks, causal, P):
    """Strided views in sentinel-filled buffers, and a workspace of exactly the
    size asked for between two bands."""
    sh = AttnShape(B=2, S=1300, Hq=4, Hkv=2, D=D, P=P, layout="sbhd")
    q, k, v, do = attn_inputs(sh)
    d = [t.cuda() for t in (q, k, v, do)]
    out, dq = (Guarded(sh.B, sh.S, sh.Hq, D, sh.layout) for _ in range(2))
    dk, dv = (Guarded(sh.B, sh.S, sh.Hkv, D, sh.layout, pad_d=32, pad_row=16) for _ in range(2))
    lse = GuardedLse(sh.B, sh.Hq, sh.S)
    kw = dict(sinks=sinks, causal=causal)
    n = ctx.window_workspace_size(sh.B, sh.S, sh.Hq, sh.Hkv, D, P, (left, right), sinks, causal)
    ws = torch.full((n + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
    ctx.attn_window_fwd(*d[:3], P, (left, right), out=out.view, lse=lse.view, **kw)
    ctx.attn_window_bwd(*d[:3], out.view, lse.view, d[3], P, (left, right), dq=dq.view, dk=dk.view, dv=dv.view,
                        workspace=ws[4096:4096 + n], **kw)
    torch.cuda.synchronize()
    for name, g in (("out", out), ("dq", dq), ("dk", dk), ("dv", dv), ("lse", lse)):
        assert g.untouched(), name
    assert (ws[:4096] == 0x5A).all() and (ws[4096 + n:] == 0x5A).all()
    close("out", out.view, ref.attn_fwd(q, k, v, left, right, sinks, causal)[0])
    for name, g, r in zip(("dq", "dk", "dv"), (dq, dk, dv), ref.attn_bwd(q, k, v, do, left, right, sinks, causal)):
        close(name, g.view, r)
    with pytest.raises(ctx.CtxError) as e:
        ctx.attn_window_bwd(*d[:3], out.view, lse.view, d[3], P, (left, right), workspace=ws[4096:4096 + n - 256], **kw)
    assert e.value.code == 3


@pytest.mark.parametrize("D", [128, 256])
def test_dk_dv_repeat_bit_for_bit(D):
    a = run(AttnShape(B=1, S=2500, Hq=4, Hkv=2, D=D, P=2), 100, 0, 4, True)[1]
    b = run(AttnShape(B=1, S=2500, Hq=4, Hkv=2, D=D, P=2), 100, 0, 4, True)[1]
    for i in (0, 1, 3, 4):
        assert torch.equal(a[i], b[i])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_tiles_out_of_reach_are_not_read(D):
    """NaN in keys and values that no tile of a query meets changes nothing."""
    sh = AttnShape(B=1, S=1280, Hq=2, Hkv=2, D=D, P=1)
    q, k, v, do = (t.cuda() for t in attn_inputs(sh))
    out, lse = ctx.attn_window_fwd(q, k, v, 1, (128, 0), causal=True)
    k2, v2 = k.clone(), v.clone()
    k2[:, :256] = float("nan")
    v2[:, :256] = float("inf")
    out2, lse2 = ctx.attn_window_fwd(q, k2, v2, 1, (128, 0), causal=True)
    assert torch.equal(out[:, 640:], out2[:, 640:]) and torch.equal(lse[..., 640:], lse2[..., 640:])


def test_graph_replay_and_side_stream():
    sh = AttnShape(B=1, S=1500, Hq=4, Hkv=2, D=128, P=2)
    q, k, v, do = (t.cuda() for t in attn_inputs(sh))
    kw = dict(sinks=4, causal=True)
    ws = torch.empty(ctx.window_workspace_size(1, 1500, 4, 2, 128, 2, (100, 0), 4, True), dtype=torch.uint8, device="cuda")
    bufs = [torch.empty_like(q), torch.empty(1, 4, 1500, device="cuda"), torch.empty_like(q), torch.empty_like(k),
            torch.empty_like(k)]

    def step(o):
        ctx.attn_window_fwd(q, k, v, 2, (100, 0), out=o[0], lse=o[1], **kw)
        ctx.attn_window_bwd(q, k, v, o[0], o[1], do, 2, (100, 0), dq=o[2], dk=o[3], dv=o[4], workspace=ws, **kw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(bufs)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(bufs)
    q.copy_(attn_inputs(sh, seed=5)[0])
    graph.replay()
    torch.cuda.synchronize()
    fresh = [torch.empty_like(b) for b in bufs]
    step(fresh)
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(bufs, fresh)):
        if i == 2:
            assert (a.float() - b.float()).abs().max() <= 2e-2 * b.float().abs().max()
        else:
            assert torch.equal(a, b)


def test_gradient_against_differences():
    """dq, dk, dv against central differences of the fp64 definition, along
    random directions (difference error below 1e-6 of the norm)."""
    sh = AttnShape(B=1, S=150, Hq=2, Hkv=1, D=64, P=1)
    (q, k, v, do), (_, _, *grads) = run(sh, 20, 0, 3, True)
    g = torch.Generator().manual_seed(1)
    x = [t.double() for t in (q, k, v)]
    f = lambda x: (ref.attn_fwd(*x, 20, 0, 3, True)[0] * do.double()).sum()
    for n in range(3):
        for _ in range(4):
            d = torch.randn(x[n].shape, generator=g, dtype=torch.float64)
            hi, lo = list(x), list(x)
            hi[n], lo[n] = x[n] + 1e-4 * d, x[n] - 1e-4 * d
            want = (f(hi) - f(lo)) / 2e-4
            got = (grads[n].double().cpu() * d).sum()
            # 8e-3 of the gradient's norm against a unit-variance direction: 6 sigma
            assert (got - want).abs() <= 6 * 8e-3 * grads[n].double().norm().cpu()


@pytest.mark.parametrize("D", [128, 256])
def test_missing_arrival_is_reported_and_the_next_call_is_right(D):
    """The windowed kernels' bounded waits: with the loads stopped after the
    first step the call reports a timeout, and the next one computes."""
    sh = AttnShape(B=1, S=900, Hq=2, Hkv=1, D=D, P=1)
    q, k, v, do = (t.cuda() for t in attn_inputs(sh))
    kw = dict(sinks=4, causal=True)
    out, lse = ctx.attn_window_fwd(q, k, v, 1, (200, 0), **kw)
    torch.cuda.synchronize()
    try:
        ctx.debug_set(ctx.DEBUG_SKIP_ARRIVAL, 100)
        ctx.attn_window_fwd(q, k, v, 1, (200, 0), **kw)
        assert ctx.device_status() == 5
        ctx.attn_window_bwd(q, k, v, out, lse, do, 1, (200, 0), **kw)
        assert ctx.device_status() == 5
    finally:
        ctx.debug_set()
    check(sh, 200, 0, 4, True)


def test_refusals():
    sh = AttnShape(B=1, S=64, Hq=2, Hkv=1, D=64, P=1)
    q, k, v, _ = (t.cuda() for t in attn_inputs(sh))
    with pytest.raises(ValueError):
        ctx.attn_window_fwd(q, k, v, 1, (-2, 0))
    with pytest.raises(ValueError):
        ctx.attn_window_fwd(q, k, v, 1, 5, sinks=-1)
    with pytest.raises(ValueError):
        ctx.attn_window_fwd(q.float(), k, v, 1, 5)
    with pytest.raises(ctx.CtxError):
        ctx.attn_window_fwd(q, k, v, 65, 5)
    out, lse = ctx.attn_window_fwd(q, k, v, 1, 5)
    with pytest.raises(ValueError):
        ctx.attn_window_bwd(q, k, v, out, lse, q, 1, 5, workspace=torch.empty(1 << 24, dtype=torch.uint8))
    with pytest.raises(ValueError):
        ctx.attn_window_bwd(q, k, v, out, lse[:, :, :-1], q, 1, 5)


def test_integers_past_32_bits_are_refused():
    q = torch.randn(1, 8, 2, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="32 bits"):
        ctx.attn_window_fwd(q, q, q, (1 << 32) + 1, 4)
    with pytest.raises(ValueError, match="expected a tensor"):
        ctx.attn_window_fwd(q, q.tolist(), q, 1, 4)
    out, _ = ctx.attn_window_fwd(q, q, q, 1, 1 << 40)  # a window may be any length
    assert torch.equal(out, ctx.attn_window_fwd(q, q, q, 1, -1)[0])
