"""The newest tokens over a cache, on the GPU, against the fp64 definition.

Tolerance as in test_window_gpu.py for the forward (P and the output round to
bf16: 2^-8 / sqrt(3) each in the mean): norm within 6e-3, no element off by
more than 2e-2 of the largest; lse 1e-3."""
import random

import pytest
import torch

import context_attention_fwd_gb300 as ctx
from oracle import window as ref
from test_guard_bands_gpu import Guarded, GuardedLse

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ctx.load_library(build_if_missing=True)
    yield
    assert ctx.device_status() == 0


def inputs(B, T, cap, Hq, Hkv, D, seed=0, layout="bshd"):
    """q, k, v on the GPU; the cache stored [B,cap,H,D] or [B,H,cap,D]."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(BF).cuda()
    q = r(B, T, Hq, D)
    if layout == "bhsd":
        return q, r(B, Hkv, cap, D).transpose(1, 2), r(B, Hkv, cap, D).transpose(1, 2)
    return q, r(B, cap, Hkv, D), r(B, cap, Hkv, D)


def close(out, lse, want, lse_want):
    g = out.double().cpu()
    assert torch.isfinite(g).all()
    assert ((g - want).norm() <= 6e-3 * want.norm()) and ((g - want).abs().max() <= 2e-2 * want.abs().max())
    l = lse.double().cpu()
    assert torch.equal(torch.isinf(l), torch.isinf(lse_want))
    ok = torch.isfinite(lse_want)
    assert not ok.any() or (l[ok] - lse_want[ok]).abs().max() < 1e-3


def check(B, T, cap, Hq, Hkv, D, lengths, left, sinks, layout="bshd", scale=None):
    q, k, v = inputs(B, T, cap, Hq, Hkv, D, seed=B + T + cap, layout=layout)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = ctx.attn_decode(q, k, v, n, window=left, sinks=sinks, scale=scale)
    clamped = [cap] * B if lengths is None else [min(max(x, 0), cap) for x in lengths]
    want, lw = ref.decode(q.cpu(), k.cpu(), v.cpu(), clamped, left, sinks, scale)
    close(out, lse, want, lw)
    return out, lse


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,cap,Hq,Hkv,lengths,left,sinks", [
    (1, 1, 1, 1, None, -1, 0), (1, 1, 4, 2, [1, 1], 0, 0), (1, 15, 4, 2, [15, 1], -1, 0), (1, 16, 4, 2, [16, 0], -1, 0),
    (1, 17, 6, 1, [17, 9], 3, 2), (1, 500, 24, 4, [500, 333], -1, 0), (1, 500, 24, 4, [500, 7], 100, 4),
    (1, 1000, 8, 8, [999, 1000], 63, 200), (2, 300, 16, 2, [300, 1], -1, 0), (3, 200, 8, 2, [200, 2], 50, 4),
    (5, 130, 12, 1, [130, 64], 0, 3), (4, 4, 4, 4, [4, 3], -1, 0), (17, 64, 3, 1, [64, 20], 10, 1),
    (1, 3000, 32, 8, [2999, 1500], -1, 0),        # split over CTAs
    (1, 3000, 20, 1, [3000, 12], -1, 5),          # two blocks of 16 query rows, split
    (2, 2500, 12, 2, [2500, 2], 2000, 4),
    (1, 300, 4, 2, [1000, -5], -1, 0),            # lengths beyond the cache and below zero are clamped
])
def test_decode_shapes(D, T, cap, Hq, Hkv, lengths, left, sinks):
    B = 1 if lengths is None else len(lengths)
    check(B, T, cap, Hq, Hkv, D, lengths, left, sinks, layout="bhsd" if cap % 2 else "bshd")


def _cases(n=30, seed=99):
    rng = random.Random(seed)
    out = []
    for i in range(n):
        cap = rng.choice([rng.randint(1, 80), rng.randint(1, 1500)])
        B, Hkv = rng.randint(1, 4), rng.choice([1, 2, 4])
        T = rng.choice([1, 1, 2, rng.randint(1, 9)])
        out.append((i, B, T, cap, Hkv * rng.choice([1, 3, 8]), Hkv, rng.choice([64, 128, 256]),
                    [rng.randint(0, cap) for _ in range(B)], rng.choice([-1, 0, rng.randint(0, 200)]),
                    rng.choice([0, 4, rng.randint(0, 300)]), rng.choice(["bshd", "bhsd"])))
    return out


@pytest.mark.parametrize("i,B,T,cap,Hq,Hkv,D,lengths,left,sinks,layout", _cases(),
                         ids=lambda v: str(v) if isinstance(v, int) else None)
def test_random_caches(i, B, T, cap, Hq, Hkv, D, lengths, left, sinks, layout):
    check(B, T, cap, Hq, Hkv, D, lengths, left, sinks, layout=layout)


def test_custom_scale():
    check(1, 1, 300, 4, 2, 128, [277], -1, 0, scale=0.3)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("left,sinks,T", [(-1, 0, 1), (100, 3, 1), (100, 3, 2)])
def test_unseen_rows_of_the_cache_are_not_read(D, left, sinks, T):
    """NaN and infinities in every row that no query sees: before the window
    (past the sinks) and beyond each sequence's length, tile interiors included."""
    B, cap = 3, 700
    lengths = [700, 523, 150]
    q, k, v = inputs(B, T, cap, 8, 2, D, seed=4)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    want = ctx.attn_decode(q, k, v, n, window=left, sinks=sinks)
    for b, ln in enumerate(lengths):
        first = 0 if left < 0 else max(0, ln - T - left)
        for t, bad in ((k, float("nan")), (v, float("inf"))):
            t[b, ln:] = bad
            t[b, min(sinks, first):first] = bad
    for a, b in zip(want, ctx.attn_decode(q, k, v, n, window=left, sinks=sinks)):
        assert torch.equal(a, b)


def test_empty_sequences_give_zero_and_no_nan():
    q, k, v = inputs(4, 2, 600, 8, 2, 128, seed=6)
    k.fill_(float("nan"))
    v.fill_(float("nan"))
    out, lse = ctx.attn_decode(q, k, v, torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert (out == 0).all() and (lse == float("-inf")).all()


def test_decoding_token_by_token_matches_the_windowed_forward():
    """As it is used: norm + rotation, the windowed forward over a prompt, then
    the same step for one token at a time against the cache."""
    g = torch.Generator().manual_seed(21)
    S, N, Hq, Hkv, D, win, sinks = 300, 12, 8, 2, 128, 99, 4
    qkv = torch.randn(1, S + N, Hq + 2 * Hkv, D, generator=g).to(BF).cuda()
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).cuda() for _ in range(2))
    table = ctx.rope_table(64, scaling="yarn", factor=4.0, original_len=256)
    split = lambda x: (x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:])
    q, k, v = split(qkv)
    q, k = ctx.qk_norm_rope_fwd(q, k, wq, wk, table)
    full, lse = ctx.attn_window_fwd(q, k, v, 1, (win, 0), sinks=sinks, causal=True)
    cache_k = torch.full((1, S + N, Hkv, D), float("nan"), dtype=BF, device="cuda")
    cache_v = torch.full_like(cache_k, float("nan"))
    cache_k[:, :S], cache_v[:, :S] = k[:, :S], v[:, :S]
    length = torch.full((1,), S, dtype=torch.int32, device="cuda")
    for i in range(S, S + N):
        tq, tk, tv = split(qkv[:, i:i + 1])
        tq, _ = ctx.qk_norm_rope_fwd(tq, tk, wq, wk, table, offset=i, k_out=cache_k[:, i:i + 1])
        cache_v[:, i:i + 1] = tv
        length += 1
        out, l = ctx.attn_decode(tq, cache_k, cache_v, length, window=win, sinks=sinks)
        assert torch.equal(cache_k[:, i], k[:, i])
        # two roundings of P and one of the output on each side
        assert (out.float() - full[:, i:i + 1].float()).norm() <= 1.2e-2 * full[:, i:i + 1].float().norm()
        assert (l[..., 0] - lse[..., i]).abs().max() < 2e-3


@pytest.mark.parametrize("D,cap,left", [(64, 3000, -1), (128, 3000, -1), (256, 3000, -1), (128, 200, 50)])
def test_outputs_and_workspace_stay_inside(D, cap, left):
    B, T, Hq, Hkv = 2, 3, 6, 2
    q, k, v = inputs(B, T, cap, Hq, Hkv, D, seed=8)
    n = torch.tensor([cap, 2], dtype=torch.int32, device="cuda")
    out, lse = Guarded(B, T, Hq, D), GuardedLse(B, Hq, T)
    need = ctx.decode_workspace_size(B, T, Hq, Hkv, D, cap, left, 4)
    ws = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
    ctx.attn_decode(q, k, v, n, window=left, sinks=4, out=out.view, lse=lse.view, workspace=ws[4096:4096 + need])
    torch.cuda.synchronize()
    assert out.untouched() and lse.untouched()
    assert (ws[:4096] == 0x5A).all() and (ws[4096 + need:] == 0x5A).all()
    close(out.view, lse.view, *ref.decode(q.cpu(), k.cpu(), v.cpu(), [cap, 2], left, 4))


def test_graph_replay_with_new_lengths_and_repeatability():
    B, cap = 2, 2800
    q, k, v = inputs(B, 1, cap, 16, 2, 128, seed=9)
    n = torch.tensor([5, 2000], dtype=torch.int32, device="cuda")
    ws = torch.empty(max(256, ctx.decode_workspace_size(B, 1, 16, 2, 128, cap)), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(B, 16, 1, device="cuda")
    call = lambda o, l: ctx.attn_decode(q, k, v, n, out=o, lse=l, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(out, lse)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, lse)
    for lengths in ([5, 2000], [2800, 0], [1, 777]):
        n.copy_(torch.tensor(lengths, dtype=torch.int32))
        graph.replay()
        a, b = call(torch.empty_like(q), torch.empty_like(lse))
        torch.cuda.synchronize()
        assert torch.equal(a, out) and torch.equal(b, lse)
        close(out, lse, *ref.decode(q.cpu(), k.cpu(), v.cpu(), lengths, -1, 0))


def test_offsets_past_32_bits():
    """Sequences more than 2^31 elements apart in one large cache."""
    far = (1 << 31) + 64
    buf = torch.zeros(far + 300 * 64, dtype=BF, device="cuda")
    k = buf.as_strided((2, 300, 1, 64), (far, 64, 64, 1))
    q, k0, v = inputs(2, 1, 300, 2, 1, 64, seed=10)
    k.copy_(k0)
    out, lse = ctx.attn_decode(q, k, v, torch.tensor([300, 211], dtype=torch.int32, device="cuda"))
    close(out, lse, *ref.decode(q.cpu(), k0.cpu(), v.cpu(), [300, 211], -1, 0))


def test_refusals():
    q, k, v = inputs(2, 1, 64, 4, 2, 64)
    n = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    for bad in (n.long(), n[:1], n.cpu()):
        with pytest.raises(ValueError):
            ctx.attn_decode(q, k, v, bad)
    with pytest.raises(ValueError):
        ctx.attn_decode(q, k, v, n, window=-2)
    with pytest.raises(ctx.CtxError):
        ctx.attn_decode(q, k, v[:, :32], n)
    with pytest.raises(ctx.CtxError) as e:
        ctx.attn_decode(*inputs(1, 1, 3000, 8, 2, 128), workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 3
    with pytest.raises(ValueError):
        ctx.attn_decode(*inputs(1, 1, 3000, 8, 2, 128), workspace=torch.empty(1 << 24, dtype=torch.uint8))


def test_two_streams_at_once():
    """Calls in flight on two streams, each with its own outputs and workspace."""
    a = inputs(1, 1, 20000, 8, 2, 128, seed=1)
    b = inputs(2, 1, 9000, 12, 4, 64, seed=2)
    want = [ctx.attn_decode(*x, window=w, sinks=4) for x, w in ((a, -1), (b, 5000))]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        with torch.cuda.stream(s1):
            got.append((0, ctx.attn_decode(*a, window=-1, sinks=4)))
        with torch.cuda.stream(s2):
            got.append((1, ctx.attn_decode(*b, window=5000, sinks=4)))
    torch.cuda.synchronize()
    for i, (out, lse) in got:
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
