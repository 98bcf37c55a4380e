"""Host-side checks of the windowed attention calls (no GPU)."""
import ctypes
import math

import pytest
import torch

import context_attention_fwd_gb300 as ctx
from oracle import window as ref

FAKE = 1 << 20  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    return ctx.load_library(build_if_missing=True)


def _t(B=1, S=64, H=4, D=64, data=FAKE):
    return ctx._Tensor(data, B, S, H, D, 0, 0, 0)


def _fwd(lib, q=None, k=None, out=None, P=2, left=5, right=0, sinks=1, lse=FAKE, layout=0):
    q, k, out = q or _t(), k or _t(H=2), out or _t()
    b = ctypes.byref
    return lib.ctx_attn_window_fwd(b(q), b(k), b(k), P, None, layout, 1, left, right, sinks, 0.0, b(out),
                                   ctypes.c_void_p(lse), None)


@pytest.mark.parametrize("kw,code", [
    (dict(left=-2), 1), (dict(right=-2), 1), (dict(sinks=-1), 1), (dict(P=0), 1), (dict(P=65), 1), (dict(lse=None), 1),
    (dict(layout=3), 1), (dict(k=_t(H=3)), 1), (dict(q=_t(D=96), k=_t(H=2, D=96), out=_t(D=96)), 2),
    (dict(q=_t(data=None)), 1), (dict(out=_t(S=32)), 1), (dict(q=_t(data=FAKE + 2)), 2)])
def test_forward_refuses_before_launch(lib, kw, code):
    assert _fwd(lib, **kw) == code


def test_backward_refuses_before_launch(lib):
    b, P = ctypes.byref, ctypes.c_void_p
    q, k = _t(), _t(H=2)

    def call(left=5, sinks=1, ws=256, wsb=1 << 30, dk=None):
        return lib.ctx_attn_window_bwd(b(q), b(k), b(k), b(q), P(FAKE), b(q), 2, None, 0, 1, left, 0, sinks, 0.0, b(q),
                                       b(dk or k), b(k), P(ws), wsb, None)

    assert call(left=-3) == 1 and call(sinks=-1) == 1
    assert call(ws=None) == 3 and call(wsb=100) == 3 and call(ws=128) == 3
    strided = ctx._Tensor(FAKE, 1, 64, 2, 64, 64 * 256, 256, 128)
    assert call(dk=strided) == 2  # dk and dv stored differently


def test_workspace_size(lib):
    n = lambda S, P, left, sinks, D=128: ctx.window_workspace_size(1, S, 4, 2, D, P, (left, 0), sinks, True)
    # few KV tiles: room for a head split's partial rows (two query heads a group)
    def base(S):  # row statistics and the fp32 dq accumulator of whole tiles
        slots = 4 * -(-S // 128) * 128
        return 2 * slots * 4 + slots * 128 * 4

    assert n(1000, 4, 100, 0) == n(1000, 9, 100, 0) == base(1000) + 2 * 2 * 1000 * 2 * 128 * 4
    # many: none
    assert n(60000, 4, 100, 0) == base(60000)
    # sinks add the partial rows of at most 64 parts (and head splits) over all sink tiles
    for S, P, left, sinks in ((32760, 8, 1023, 4), (65536, 64, 0, 1), (32760, 1, 100, 2000), (9000, 3, 10, 9000)):
        extra = n(S, P, left, sinks) - n(S, P, left, 0)
        rows = min(S, sinks + 128)
        assert 0 <= extra <= 2 * 64 * 2 * rows * 2 * 128 * 4 + 256
        assert extra <= 2 * (64 + 64) * 2 * 2 * 128 * 128 * 4 * 2
    assert lib.ctx_attn_window_workspace_size(1, 1000, 4, 2, 128, 4, 1, -2, 0, 0) == 0
    assert lib.ctx_attn_window_workspace_size(1, 1000, 4, 3, 128, 4, 1, 5, 0, 0) == 0
    assert lib.ctx_attn_window_workspace_size(1, 3, 4, 2, 128, 4, 1, 5, 0, 0) == 0


def test_binding_refuses():
    x = torch.zeros(1, 8, 2, 64)
    for window, sinks in (((-2, 0), 0), ((0, -2), 0), (5, -1)):
        with pytest.raises(ValueError):
            ctx.window_workspace_size(1, 8, 2, 2, 64, 1, window, sinks)
    with pytest.raises(ValueError):
        ctx.attn_window_fwd(x, x, x, 1, 3)
    with pytest.raises(ValueError):
        ctx.attn_window_fwd(x.bfloat16(), x.bfloat16(), x.bfloat16(), 1, 3)


@pytest.mark.parametrize("left,right,sinks,causal", [(3, 0, 2, True), (2, 4, 0, False), (0, 1, 9, False), (-1, -1, 0, True)])
def test_reference_against_differences_and_a_row_by_row_softmax(left, right, sinks, causal):
    g = torch.Generator().manual_seed(2)
    q, k, v, do = (torch.randn(1, 17, h, 4, generator=g, dtype=torch.float64) for h in (2, 1, 1, 2))
    out, lse = ref.attn_fwd(q, k, v, left, right, sinks, causal)
    for i in range(17):
        keys = [j for j in range(17) if (j <= i or not causal) and
                (j < sinks or ((left < 0 or j >= i - left) and (causal or right < 0 or j <= i + right)))]
        for h in range(2):
            s = [float(q[0, i, h] @ k[0, j, 0]) / 2.0 for j in keys]
            z = sum(math.exp(x) for x in s)
            assert abs(math.log(z) - lse[0, h, i]) < 1e-12
            want = sum(math.exp(x) / z * v[0, j, 0] for x, j in zip(s, keys))
            assert (want - out[0, i, h]).abs().max() < 1e-12
    grads = ref.attn_bwd(q, k, v, do, left, right, sinks, causal)
    f = lambda q, k, v: (ref.attn_fwd(q, k, v, left, right, sinks, causal)[0] * do).sum()
    for n, x in enumerate((q, k, v)):
        for i in range(0, x.numel(), 7):
            e = torch.zeros(x.numel(), dtype=torch.float64)
            e[i] = 1e-5
            args = [q, k, v]
            hi, lo = list(args), list(args)
            hi[n], lo[n] = x + e.view_as(x), x - e.view_as(x)
            assert abs((f(*hi) - f(*lo)) / 2e-5 - grads[n].flatten()[i]) < 1e-8
