"""The operators together, as a training step uses them: query/key norm and
rotation of one packed projection, windowed attention with sinks, and the
gradients back to the projection and the norm weights, against fp64 autograd
of the whole chain.

Tolerance: 2e-2 of each tensor's norm.  On top of the roundings of
test_window_gpu.py (8e-3), the rotated q and k are rounded to bf16 before the
scores: 2^-8 / sqrt(3) per element of two factors gives scores (of unit-norm
rows times sqrt(D)) an error of 3.3e-3, and so the probabilities and all that
follows from them; their gradients dq, dk are rounded once more before the
norm's backward (2.3e-3)."""
import math

import pytest
import torch

import context_attention_fwd_gb300 as ctx
from oracle import rope as rref
from oracle import window as wref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,Hq,Hkv,win,sinks,causal,graph", [
    (128, 4, 2, 100, 4, True, False), (64, 6, 2, 60, 0, False, False), (256, 4, 1, 150, 3, True, True)])
def test_training_step(D, Hq, Hkv, win, sinks, causal, graph):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ctx.load_library(build_if_missing=True)
    g = torch.Generator().manual_seed(D)
    B, S, rot, eps = 2, 333, D // 2, 1e-6
    qkv = torch.randn(B, S, Hq + 2 * Hkv, D, generator=g).bfloat16()
    wq, wk = (1 + 0.2 * torch.randn(D, generator=g) for _ in range(2))
    do = torch.randn(B, S, Hq, D, generator=g).bfloat16()
    table = ctx.rope_table(rot, interleaved=D == 64)
    pos = torch.arange(S).expand(B, S) + torch.tensor([[0], [1000]])
    left, right = win, 0 if causal else win

    x, w1, w2, dod, posd = qkv.cuda(), wq.cuda(), wk.cuda(), do.cuda(), pos.cuda()
    dx = torch.empty_like(x)
    parts = lambda t: (t[:, :, :Hq], t[:, :, Hq:Hq + Hkv], t[:, :, Hq + Hkv:])

    def step():
        q, k, v = parts(x)
        qr, kr = ctx.qk_norm_rope_fwd(q, k, w1, w2, table, positions=posd, eps=eps)
        out, lse = ctx.attn_window_fwd(qr, kr, v, 2, (left, right), sinks=sinks, causal=causal)
        dq, dk, dv = parts(dx)  # written in place of the packed gradient
        dqr, dkr, dvr = ctx.attn_window_bwd(qr, kr, v, out, lse, dod, 2, (left, right), sinks=sinks, causal=causal)
        dv.copy_(dvr)
        _, _, dw1, dw2 = ctx.qk_norm_rope_bwd(dqr, dkr, q, k, w1, w2, table, positions=posd, eps=eps, dq=dq, dk=dk)
        return out, dw1, dw2

    got = step()
    if graph:  # the whole step captured and replayed on another projection
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        s.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            got = step()
        qkv = torch.randn(qkv.shape, generator=g).bfloat16()
        x.copy_(qkv)
        dx.zero_()
        cg.replay()
    torch.cuda.synchronize()
    assert ctx.device_status() == 0

    leaves = [t.double().requires_grad_() for t in (qkv, wq, wk)]
    ang = rref.angles(table.turns, pos)

    def rotate(t):  # rotate() of oracle/rope.py without its in-place writes
        c, s = torch.cos(ang)[:, :, None], torch.sin(ang)[:, :, None]
        if table.interleaved:
            a, b = t[..., 0:rot:2], t[..., 1:rot:2]
            y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
        else:
            a, b = t[..., :rot // 2], t[..., rot // 2:rot]
            y = torch.cat([a * c - b * s, b * c + a * s], -1)
        return torch.cat([y, t[..., rot:]], -1)

    q, k, v = parts(leaves[0])
    q, k = rotate(rref.norm(q, leaves[1], eps)), rotate(rref.norm(k, leaves[2], eps))
    G = Hq // Hkv
    sc = torch.einsum("bihd,bjhd->bhij", q, k.repeat_interleave(G, 2)) / math.sqrt(D)
    sc = sc.masked_fill(~wref.visible(S, left, right, sinks, causal), -math.inf)
    out = torch.einsum("bhij,bjhd->bihd", torch.softmax(sc, -1), v.repeat_interleave(G, 2))
    want = torch.autograd.grad(out, leaves, do.double())
    for name, a, b in (("out", got[0], out.detach()), ("dqkv", dx, want[0]), ("dwq", got[1], want[1]), ("dwk", got[2], want[2])):
        err = ((a.double().cpu() - b).norm() / b.norm()).item()
        assert err <= 2e-2, f"{name}: {err:.3e}"
