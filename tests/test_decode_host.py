"""Host-side checks of the decode call (no GPU)."""
import ctypes

import pytest
import torch

import context_attention_fwd_gb300 as ctx
from oracle import window as ref

FAKE = 1 << 20  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    return ctx.load_library(build_if_missing=True)


def _t(B=2, S=64, H=4, D=64, data=FAKE, strides=(0, 0, 0)):
    return ctx._Tensor(data, B, S, H, D, *strides)


def _call(lib, q=None, k=None, v=None, out=None, lengths=FAKE, layout=0, left=5, sinks=1, lse=FAKE, ws=256, wsb=1 << 30):
    q, out = q or _t(S=1), out or _t(S=1)
    k = k or _t(H=2)
    v = v or k
    b, P = ctypes.byref, ctypes.c_void_p
    return lib.ctx_attn_decode(b(q), b(k), b(v), P(lengths), layout, left, sinks, 0.0, b(out), P(lse), P(ws), wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(left=-2), 1), (dict(sinks=-1), 1), (dict(layout=2), 1), (dict(lse=None), 1), (dict(lse=FAKE + 2), 1),
    (dict(lengths=FAKE + 1), 1), (dict(k=_t(H=3)), 1), (dict(k=_t(B=3, H=2)), 1), (dict(k=_t(S=0, H=2)), 1),
    (dict(q=_t(S=0), out=_t(S=0)), 1), (dict(out=_t(S=2)), 1), (dict(v=_t(H=2, S=32)), 1), (dict(q=_t(S=1, data=None)), 1),
    (dict(q=_t(S=1, D=96), out=_t(S=1, D=96), k=_t(H=2, D=96)), 2), (dict(k=_t(H=2, data=FAKE + 4)), 2),
    (dict(k=_t(H=2, strides=(8192, 132, 64))), 2)])
def test_refuses_before_launch(lib, kw, code):
    assert _call(lib, **kw) == code


def test_workspace(lib):
    # one sequence over a long cache is split, and needs room for the parts
    n = ctx.decode_workspace_size(1, 1, 32, 8, 128, 65536)
    assert n > 0 and n % 256 == 0
    k = _t(1, 65536, 8, 128)
    q = _t(1, 1, 32, 128)
    for ws, wsb in ((None, n), (256, n - 1), (128, n)):
        assert _call(lib, q=q, k=k, out=q, left=-1, ws=ws, wsb=wsb) == 3
    # many sequences fill the GPU by themselves
    assert ctx.decode_workspace_size(512, 1, 32, 8, 128, 4096) == 0
    # a short window leaves too few tiles to split
    assert ctx.decode_workspace_size(1, 1, 32, 8, 128, 65536, window=10) == 0
    assert lib.ctx_attn_decode_workspace_size(1, 1, 32, 7, 128, 100, -1, 0) == 0
    assert lib.ctx_attn_decode_workspace_size(1, 1, 32, 8, 96, 100, -1, 0) == 0
    with pytest.raises(ValueError):
        ctx.decode_workspace_size(1, 1, 32, 8, 128, 65536, window=-2)


def test_reference_is_the_last_rows_of_the_windowed_forward():
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(1, 40, h, 8, generator=g, dtype=torch.float64) for h in (4, 2, 2))
    for left, sinks in ((-1, 0), (7, 0), (7, 3), (0, 0)):
        full, lse = ref.attn_fwd(q, k, v, left, 0, sinks, True)
        out, l = ref.decode(q[:, -3:], k, v, [40], left, sinks)
        assert (out - full[:, -3:]).abs().max() < 1e-12 and (l - lse[:, :, -3:]).abs().max() < 1e-12
    out, l = ref.decode(q[:, :3], k, v, [1], -1, 0)  # two queries before the start
    assert (out[:, :2] == 0).all() and torch.isinf(l[:, :, :2]).all() and (out[0, 2, 0] - v[0, 0, 0]).abs().max() < 1e-12


def test_binding_refuses():
    x = torch.zeros(1, 8, 2, 64).bfloat16()
    with pytest.raises(ValueError):
        ctx.attn_decode(x, x.float(), x)
    with pytest.raises(ValueError):
        ctx.attn_decode(x, x, x)  # not on a GPU
