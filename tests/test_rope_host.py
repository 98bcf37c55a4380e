"""Host-side checks of the rotary and query/key norm calls (no GPU): the
frequency table against high-precision arithmetic, the fp64 definitions
against differences, and the refusal of every malformed argument before
anything is launched."""
import ctypes
import decimal
import math

import pytest
import torch

import context_attention_fwd_gb300 as ctx
from oracle import rope as ref

PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module")
def lib():
    return ctx.load_library(build_if_missing=True)


def _u64(table):
    return [t + (1 << 64) if t < 0 else t for t in table.turns.tolist()]


@pytest.mark.parametrize("rot,theta", [(64, 10000.0), (128, 500000.0), (2, 10000.0), (256, 10000.0)])
def test_table_holds_turns_per_position(rot, theta):
    """Each entry is theta^(-2i/rot) / (2 pi) of 2^64, within fp64's rounding
    of the power and the quotient (8 ulp of 2^-53)."""
    decimal.getcontext().prec = 60
    for i, t in enumerate(_u64(ctx.rope_table(rot, theta=theta, device="cpu"))):
        want = decimal.Decimal(theta) ** (decimal.Decimal(-2 * i) / rot) / (2 * PI) * (1 << 64)
        assert abs(decimal.Decimal(t) - want) <= want * 8 / (1 << 53) + 1


def test_table_scalings():
    base = [t / 2.0 ** 64 for t in _u64(ctx.rope_table(64, device="cpu"))]
    lin = [t / 2.0 ** 64 for t in _u64(ctx.rope_table(64, scaling="linear", factor=4.0, device="cpu"))]
    assert all(abs(a / 4 - b) <= 1e-14 for a, b in zip(base, lin))
    ntk = [t / 2.0 ** 64 for t in _u64(ctx.rope_table(64, scaling="ntk", factor=4.0, device="cpu"))]
    assert abs(ntk[0] - base[0]) < 1e-14                # the fastest pair is kept
    assert abs(ntk[-1] - base[-1] / 4) < 1e-12 * base[-1] * 1e3  # the slowest is divided by the factor
    y = ctx.rope_table(64, scaling="yarn", factor=8.0, original_len=4096, device="cpu")
    yarn = [t / 2.0 ** 64 for t in _u64(y)]
    for a, b in zip(base, yarn):
        turns = a * 4096  # over the original length
        if turns > 40:
            assert abs(a - b) < 1e-14
        elif turns < 0.7:
            assert abs(a / 8 - b) < 1e-14
        assert a / 8 - 1e-14 <= b <= a + 1e-14
    assert y.magnitude == pytest.approx(0.1 * math.log(8.0) + 1.0)
    assert ctx.rope_table(64, scaling="yarn", factor=8.0, original_len=4096, magnitude=1.0, device="cpu").magnitude == 1.0


def test_table_sections_have_their_own_frequencies():
    t = ctx.rope_table(128, sections=(22, 21, 21), device="cpu")
    assert t.turns[:22].tolist() == ctx.rope_table(44, device="cpu").turns.tolist()
    assert t.turns[22:43].tolist() == ctx.rope_table(42, device="cpu").turns.tolist()
    own = ctx.rope_table(4, inv_freq=[0.5, 0.0], device="cpu")
    assert own.turns[1] == 0 and abs(_u64(own)[0] / 2.0 ** 64 - 0.5 / (2 * math.pi)) < 1e-16


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=64, theta=1.0), dict(rot_dim=64, theta=math.inf),
    dict(rot_dim=64, factor=0.5), dict(rot_dim=64, scaling="other"), dict(rot_dim=64, scaling="yarn", factor=2.0),
    dict(rot_dim=64, sections=(16, 15)), dict(rot_dim=64, sections=(32, 0)), dict(rot_dim=64, sections=(8, 8, 8, 4, 4)),
    dict(rot_dim=2, scaling="ntk", factor=2.0), dict(rot_dim=4, inv_freq=[1.0]), dict(rot_dim=2, inv_freq=[7.0]),
    dict(rot_dim=2, inv_freq=[-1.0]), dict(rot_dim=2, inv_freq=[math.nan])])
def test_table_refuses(kw):
    with pytest.raises(ValueError):
        ctx.rope_table(device="cpu", **kw)


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_gradient_against_differences(interleaved):
    """The fp64 formulas the GPU tests use, against central differences of the
    forward (error of a central difference at h = 1e-5: below 1e-8 here)."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(2, 3, 2, 8, generator=g, dtype=torch.float64)
    w = torch.randn(8, generator=g, dtype=torch.float64)
    dy = torch.randn(2, 3, 2, 8, generator=g, dtype=torch.float64)
    ang = torch.randn(2, 3, 3, generator=g, dtype=torch.float64)
    f = lambda x, w: (ref.rotate(ref.norm(x, w, 1e-3), ang, 6, interleaved, 1.2) * dy).sum()
    dx, dw = ref.norm_grad(ref.rotate(dy, ang, 6, interleaved, 1.2, transpose=True), x, w, 1e-3)
    h = 1e-5
    for t, d, args in ((x, dx, 0), (w, dw, 1)):
        for i in range(t.numel()):
            e = torch.zeros(t.numel(), dtype=torch.float64)
            e[i] = h
            e = e.view_as(t)
            hi, lo = (f(x + e, w), f(x - e, w)) if args == 0 else (f(x, w + e), f(x, w - e))
            assert abs((hi - lo) / (2 * h) - d.flatten()[i]) < 1e-8


FAKE = 1 << 20  # never dereferenced: validation fails first


def _t(B=1, S=8, H=4, D=64, data=FAKE, strides=(0, 0, 0)):
    return ctx._Tensor(data, B, S, H, D, *strides)


def _rope(**kw):
    r = ctx._Rope(FAKE, 64, 0, 1, (ctypes.c_int * 4)(0, 0, 0, 0), 1.0, None, 0, 0, 0, 0)
    for n, v in kw.items():
        setattr(r, n, (ctypes.c_int * 4)(*v) if n == "sections" else v)
    return r


def _fwd(lib, q=None, k=None, rope=None, dtype=0, layout=0, qo=None, ko=None):
    ref_ = lambda t: None if t is None else ctypes.byref(t)
    return lib.ctx_rope_fwd(ref_(q), ref_(k), ref_(rope), dtype, layout, ref_(qo), ref_(ko), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(qo=None), 1), (dict(rope=None), 1), (dict(k=_t()), 1), (dict(ko=_t()), 1),
    (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(layout=2), 1),
    (dict(q=_t(S=0), qo=_t(S=0)), 1), (dict(q=_t(B=0), qo=_t(B=0)), 1), (dict(q=_t(H=0), qo=_t(H=0)), 1),
    (dict(q=_t(D=514), qo=_t(D=514)), 2), (dict(q=_t(D=63), qo=_t(D=63)), 2),
    (dict(qo=_t(S=9)), 1), (dict(qo=_t(H=5)), 1), (dict(q=_t(data=None)), 1),
    (dict(q=_t(strides=(-8, 256, 64))), 1), (dict(q=_t(strides=(2048, 0, 64))), 1), (dict(q=_t(strides=(2048, 256, 32))), 1),
    (dict(q=_t(data=FAKE + 1)), 2), (dict(q=_t(data=FAKE + 2), dtype=2), 2),
    (dict(rope=_rope(turns=None)), 1), (dict(rope=_rope(rot_dim=66)), 1), (dict(rope=_rope(rot_dim=0)), 1),
    (dict(rope=_rope(rot_dim=7)), 1), (dict(rope=_rope(n_axes=0)), 1), (dict(rope=_rope(n_axes=5)), 1),
    (dict(rope=_rope(n_axes=2, sections=(16, 16, 0, 0))), 1),  # several axes need positions
    (dict(rope=_rope(n_axes=2, sections=(16, 15, 0, 0), positions=FAKE)), 1),
    (dict(rope=_rope(n_axes=2, sections=(33, -1, 0, 0), positions=FAKE)), 1),
    (dict(rope=_rope(magnitude=math.nan)), 1), (dict(rope=_rope(magnitude=math.inf)), 1),
    (dict(rope=_rope(positions=FAKE + 4)), 2), (dict(rope=_rope(turns=FAKE + 4)), 2),
    (dict(rope=_rope(positions=FAKE, pos_stride_s=-1)), 1)])
def test_rope_refuses_before_launch(lib, kw, code):
    args = dict(q=_t(), rope=_rope(), qo=_t())
    args.update(kw)
    assert _fwd(lib, **args) == code


def test_norm_refuses_before_launch(lib):
    b = ctypes.byref
    P = ctypes.c_void_p
    q, r = _t(), _rope()

    def bwd(gq=q, gk=None, q=q, k=None, wq=FAKE, wk=None, wt=2, eps=1e-6, dq=q, dk=None, dwq=FAKE, dwk=None,
            ws=256, wsb=1 << 30, rope=r):
        o = lambda t: None if t is None else b(t)
        return lib.ctx_qk_norm_rope_bwd(o(gq), o(gk), o(q), o(k), P(wq), P(wk), wt, eps, o(rope), 0, 0, o(dq), o(dk),
                                        P(dwq), P(dwk), P(ws), wsb, None)

    assert bwd(ws=None) == 3 and bwd(wsb=16) == 3 and bwd(ws=128) == 3
    assert bwd(eps=-1.0) == 1 and bwd(eps=math.nan) == 1 and bwd(wt=7) == 1
    assert bwd(wq=None) == 1            # a weight gradient without its weight
    assert bwd(dwk=FAKE) == 1           # k's without k
    assert bwd(gq=None) == 1 and bwd(q=None) == 1 and bwd(dq=None) == 1 and bwd(gk=_t()) == 1
    assert bwd(wq=FAKE + 2) == 2        # misaligned fp32 weights
    assert bwd(gq=_t(S=4)) == 1
    assert lib.ctx_qk_norm_rope_workspace_size(63) == 0 and lib.ctx_qk_norm_rope_workspace_size(514) == 0
    assert lib.ctx_qk_norm_rope_workspace_size(128) > 0


def test_binding_refuses_host_tensors_and_types():
    x = torch.zeros(1, 4, 2, 64)
    t = ctx.rope_table(64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        ctx.rope_fwd(x, None, t)
    with pytest.raises(ValueError, match="dtype"):
        ctx.rope_fwd(x.double(), None, t)
    with pytest.raises(ValueError, match="dims"):
        ctx.rope_fwd(x[0], None, t)
    with pytest.raises(ValueError, match="table"):
        ctx.rope_fwd(x, None, None)
    with pytest.raises(ValueError, match="go together"):
        ctx.qk_norm_rope_bwd(x, x, x, None, None, None, t)


def test_table_is_checked_when_made_by_hand():
    good = ctx.rope_table(8, device="cpu")
    for kw in (dict(rot_dim=10), dict(turns=good.turns[:3]), dict(turns=good.turns.int()), dict(sections=(2, 1)),
               dict(turns=torch.zeros(8, dtype=torch.int64)[::2])):
        with pytest.raises(ValueError):
            ctx.RopeTable(**{**dict(turns=good.turns, rot_dim=8, interleaved=False, sections=(4,), magnitude=1.0), **kw})


def test_packed_table_has_the_c_layout():
    """The packed bytes are the ctypes structure of the same fields."""
    t = ctx.rope_table(8, sections=(1, 2, 1), interleaved=True, magnitude=1.5, device="cpu")
    r = ctx._Rope(t.turns.data_ptr(), 8, 1, 3, (ctypes.c_int * 4)(1, 2, 1, 0), 1.5, None, 0, 0, 0, 0)
    assert t._head == bytes(r)
