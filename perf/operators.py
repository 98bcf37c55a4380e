"""Timed cases of the operators around the attention calls: rotary positions,
per-head norms of queries and keys fused with the rotation, attention with a
sliding window and sink tokens (forward and backward), and its form for the
newest tokens of a key/value cache.

A case is one call at one size.  ``run`` makes it through the library when
``own`` is set, and otherwise in a plain form of elementary torch operations
in fp32 (fp64 for angles and long sums).  ``exact`` states the operators'
definitions once more in fp64.

Definitions.
  rotary   pair i of a head turns by  a = position * f_i ; (x1, x2) ->
           m (x1 cos a - x2 sin a, x2 cos a + x1 sin a).  The pair is elements
           (i, i + R/2) of the first R ("half") or (2i, 2i + 1)
           ("interleaved"); elements from R on stay as they are.
  norm     x / sqrt(mean(x^2) + eps) * w over the head, then the rotation.
  window   key j is visible to query i iff
           (j < sinks and (not causal or j <= i)) or
           (i - left <= j <= i + right and (not causal or j <= i));
           a side of -1 is unlimited.
  decode   query t of T sits at position length - T + t of its sequence's
           cache and sees it causally, under the same window and sinks.
"""
import math
import random

import torch

own = False
DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def _rope(name, kind, B, S, Hq, Hkv, D, rot, style, dtype, layout="bshd", sections="", scaling="none", factor=1.0,
          orig=0, theta=10000.0, pos="offset", offset=0):
    return {"name": name, "kind": kind, "B": B, "S": S, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "style": style,
            "dtype": dtype, "layout": layout, "sections": sections, "scaling": scaling, "factor": factor, "orig": orig,
            "theta": theta, "pos": pos, "offset": offset}


def _win(name, kind, B, S, Hq, Hkv, D, P, left, right, sinks, causal, layout="bshd"):
    return {"name": name, "kind": kind, "B": B, "S": S, "Hq": Hq, "Hkv": Hkv, "D": D, "P": P, "left": left,
            "right": right, "sinks": sinks, "causal": causal, "layout": layout}


def _dec(name, B, T, cap, Hq, Hkv, D, left, sinks, fill):
    return {"name": name, "kind": "decode", "B": B, "T": T, "cap": cap, "Hq": Hq, "Hkv": Hkv, "D": D, "left": left,
            "sinks": sinks, "fill": fill}


def listed():
    return [
        # the newest token of each of 16 running sequences of the 24/4-head
        # D=256 language model, a quarter of the head rotated
        _rope("rope_newest_d256", "rope_fwd", 16, 1, 24, 4, 256, 64, "half", "bf16", pos="ragged"),
        # the 65536-token hybrid workload (32/8 heads), context stretched 8x
        _rope("rope_long_d128", "rope_fwd", 1, 65536, 32, 8, 128, 128, "interleaved", "bf16", scaling="yarn",
              factor=8.0, orig=8192),
        # gradients through the rotation, sequence-first storage, odd length
        _rope("rope_grad_seqfirst", "rope_bwd", 1, 1001, 16, 16, 64, 64, "half", "fp16", layout="sbhd"),
        # the newest tokens of 64 sequences before a decode step
        _rope("norm_rope_newest_d256", "norm_rope_fwd", 64, 1, 24, 4, 256, 64, "half", "bf16", pos="ragged"),
        # queries and keys of the long video workload: three position axes
        # (frames, rows, columns) on 22/21/21 pairs of the head
        _rope("norm_rope_video", "norm_rope_fwd", 1, 32760, 24, 24, 128, 128, "interleaved", "bf16",
              sections="22,21,21", pos="grid"),
        # its training step: gradients of q, k and both weights
        _rope("norm_rope_video_grad", "norm_rope_bwd", 1, 32760, 24, 24, 128, 128, "interleaved", "bf16",
              sections="22,21,21", pos="grid"),
        # a short bidirectional window, sequence-first, uneven chunks
        _win("window_fwd_seqfirst", "window_fwd", 1, 1001, 16, 16, 64, 4, 100, 100, 0, False, layout="sbhd"),
        # the long workload under a 1024-token causal window with 4 sinks
        _win("window_fwd_long", "window_fwd", 1, 32760, 24, 24, 128, 8, 1023, 0, 4, True),
        # training step of grouped heads at the joint-sequence size
        _win("window_grad_gqa", "window_bwd", 1, 4608, 24, 8, 128, 4, 511, 511, 16, False),
        # training step of the D=256 language model on a long sequence
        _win("window_grad_d256", "window_bwd", 1, 16384, 24, 4, 256, 8, 2047, 0, 4, True),
        # one sequence, the whole history of a 65536-token cache
        _dec("decode_history", 1, 1, 65536, 32, 8, 128, -1, 0, "full"),
        # 64 sequences of ragged lengths under a window with sinks
        _dec("decode_window_batch", 64, 1, 4096, 24, 4, 256, 1023, 4, "ragged"),
    ]


def _logint(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b + 1)))))))


def draw(rng):
    kind = rng.choice(["rope_fwd", "rope_bwd", "norm_rope_fwd", "norm_rope_bwd", "window_fwd", "window_fwd",
                       "window_bwd", "window_bwd", "decode", "decode"])
    heads = [(24, 24), (24, 8), (24, 4), (32, 8), (16, 16), (8, 8), (8, 2), (6, 2), (3, 1)]
    if kind in ("rope_fwd", "rope_bwd", "norm_rope_fwd", "norm_rope_bwd"):
        Hq, Hkv = rng.choice(heads)
        D = rng.choice([64, 80, 96, 128, 256])
        rot = rng.choice([D, D, D // 2, D // 4, 2 * rng.randint(1, D // 2)])
        rot -= rot % 2
        B = rng.choice([1, 1, 2, 7, 16])
        limit = 65536 * 40 * 128 // (B * (Hq + Hkv) * D * (2 if kind.startswith("norm") else 1))
        S = _logint(rng, 1, max(1, min(65536, limit)))
        sections, pos = "", rng.choice(["offset", "ragged", "ragged"])
        if rng.random() < 0.3 and rot >= 12:
            a, b = rng.randint(1, rot // 6), rng.randint(1, rot // 6)
            sections, pos = f"{rot // 2 - a - b},{a},{b}", "grid"
        scaling = "none" if sections else rng.choice(["none", "linear", "ntk", "yarn"])
        if rot <= 2 and scaling in ("ntk", "yarn"):
            scaling = "linear"
        return _rope("", kind, B, S, Hq, Hkv, D, rot, rng.choice(["half", "interleaved"]),
                     rng.choice(["bf16", "bf16", "fp16", "fp32"]), layout=rng.choice(["bshd", "bshd", "sbhd"]),
                     sections=sections, scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 16.0]),
                     orig=8192 if scaling == "yarn" else 0, theta=rng.choice([10000.0, 500000.0]), pos=pos,
                     offset=rng.randint(0, 1 << 20) if pos == "offset" else 0)
    if kind in ("window_fwd", "window_bwd"):
        Hq, Hkv = rng.choice(heads)
        D = rng.choice([64, 128, 256])
        B = rng.choice([1, 1, 2, 3])
        budget = 16384 * 24 * 256 // (B * Hq * D)
        # a row that sees itself alone has no gradient but that of v
        S = _logint(rng, 1 if kind == "window_fwd" else 16, max(16, min(32768, budget)))
        left = rng.choice([_logint(rng, 1, 2048), _logint(rng, 64, 2048)])
        causal = rng.random() < 0.6
        right = 0 if causal else rng.choice([left, _logint(rng, 1, 512)])
        if not causal:
            left = min(left, 1024)
            right = min(right, 1024)
        sinks = rng.choice([0, 1, 4, 16, rng.randint(1, 200)])
        return _win("", kind, B, S, Hq, Hkv, D, rng.randint(1, min(S, 8)), left, right, sinks, causal,
                    layout=rng.choice(["bshd", "bshd", "sbhd"]))
    Hq, Hkv = rng.choice(heads)
    D = rng.choice([64, 128, 256])
    B = rng.choice([1, 2, 5, 16, 64])
    cap = _logint(rng, 1, max(1, min(65536, 65536 * 8 * 128 * 2 // (B * Hkv * D))))
    T = min(cap, rng.choice([1, 1, 1, 2, 4]))
    left = rng.choice([-1, _logint(rng, 1, 4096)])
    return _dec("", B, T, cap, Hq, Hkv, D, left, rng.choice([0, 4, 16]), rng.choice(["full", "ragged"]))


# ------------------------------------------------------------------ inputs
def _gen(case, seed):
    return torch.Generator(device=DEV).manual_seed(seed * 7919 + 17)


def _randn(g, B, S, H, D, dtype, layout, scale=None):
    shape = (B, S, H, D) if layout == "bshd" else (S, B, H, D)
    t = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    if scale is not None:
        t = t * scale
    t = t.to(dtype)
    return t if layout == "bshd" else t.permute(1, 0, 2, 3)


def _sections(case):
    return [int(n) for n in case["sections"].split(",")] if case["sections"] else [case["rot"] // 2]


def _positions(case, g):
    """None (positions run on from ``offset``), or int64 [B,S] / [S,axes]."""
    B, S = case["B"], case["S"]
    if case["pos"] == "offset":
        return None
    if case["pos"] == "ragged":  # each sequence runs on from its own length
        first = torch.randint(0, 1 << 17, (B, 1), generator=g, device=DEV, dtype=torch.int64)
        return first + torch.arange(S, device=DEV, dtype=torch.int64)
    s = torch.arange(S, device=DEV, dtype=torch.int64)  # frames, rows and columns of a latent grid
    return torch.stack([s // 1560, s // 52 % 30, s % 52], dim=-1).contiguous()


def prepare(case, seed):
    g = _gen(case, seed)
    kind, B, Hq, Hkv, D = case["kind"], case["B"], case["Hq"], case["Hkv"], case["D"]
    st = {"case": case}
    if "rope" in kind:
        S, dt, lay = case["S"], _DT[case["dtype"]], case["layout"]
        st["positions"] = _positions(case, g)
        st["freq"] = _freq(case).to(DEV)
        if own:
            import context_attention_fwd_gb300 as ctx
            st["table"] = ctx.rope_table(
                case["rot"], theta=case["theta"], interleaved=case["style"] == "interleaved",
                sections=_sections(case) if case["sections"] else None, scaling=case["scaling"],
                factor=case["factor"], original_len=case["orig"] or None, device=DEV)
        if kind.startswith("norm"):
            # projections of a model: channels of unequal size, weights near one
            chan = torch.exp(0.5 * torch.randn(D, generator=g, device=DEV))
            st["wq"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)
            st["wk"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)
            st["q"] = _randn(g, B, S, Hq, D, dt, lay, chan)
            st["k"] = _randn(g, B, S, Hkv, D, dt, lay, chan)
        else:
            st["q"] = _randn(g, B, S, Hq, D, dt, lay)
            st["k"] = _randn(g, B, S, Hkv, D, dt, lay)
        if kind.endswith("bwd"):
            st["gq"] = _randn(g, B, S, Hq, D, dt, lay)
            st["gk"] = _randn(g, B, S, Hkv, D, dt, lay)
        return st
    if kind.startswith("window"):
        S, lay = case["S"], case["layout"]
        st["q"], st["k"], st["v"] = (_randn(g, B, S, h, D, torch.bfloat16, lay) for h in (Hq, Hkv, Hkv))
        if kind == "window_bwd":  # the forward's results and the incoming gradient
            st["do"] = _randn(g, B, S, Hq, D, torch.bfloat16, lay)
            out, st["lse"] = _window_fwd(case, st["q"], st["k"], st["v"])
            st["out"] = out if lay == "bshd" else out.permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3)
        return st
    T, cap = case["T"], case["cap"]
    st["q"] = _randn(g, B, T, Hq, D, torch.bfloat16, "bshd")
    st["k"] = _randn(g, B, cap, Hkv, D, torch.bfloat16, "bshd")
    st["v"] = _randn(g, B, cap, Hkv, D, torch.bfloat16, "bshd")
    if case["fill"] == "full":
        st["lengths"] = torch.full((B,), cap, dtype=torch.int32, device=DEV)
    else:
        st["lengths"] = torch.randint(T, cap + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    return st


# ------------------------------------------------------------------ plain forms
def _freq(case):
    """Radians per position of every rotated pair, fp64."""
    out = []
    for n in _sections(case):
        i, d, theta = torch.arange(n, dtype=torch.float64), 2 * n, case["theta"]
        f = case["factor"]
        if case["scaling"] == "ntk":
            theta = theta * f ** (d / (d - 2.0))
        w = theta ** (-2.0 * i / d)
        if case["scaling"] == "linear":
            w = w / f
        elif case["scaling"] == "yarn":
            turn = lambda r: d * math.log(case["orig"] / (r * 2 * math.pi)) / (2 * math.log(theta))
            lo, hi = max(math.floor(turn(32.0)), 0), min(math.ceil(turn(1.0)), d - 1)
            ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
            w = w / f * ramp + w * (1.0 - ramp)
        out.append(w)
    return torch.cat(out)


def _magnitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "yarn" and case["factor"] > 1 else 1.0


def _cos_sin(case, st):
    B, S = case["B"], case["S"]
    pos = st["positions"]
    if pos is None:
        pos = (case["offset"] + torch.arange(S, device=DEV, dtype=torch.int64))[None]
    elif case["pos"] == "grid":
        ax = torch.repeat_interleave(torch.arange(len(_sections(case)), device=DEV),
                                     torch.tensor(_sections(case), device=DEV))
        pos = pos[:, ax][None]  # [1,S,pairs]
    if pos.dim() == 2:
        pos = pos[:, :, None]
    a = pos.double() * st["freq"]
    m = _magnitude(case)
    return (torch.cos(a) * m).float()[:, :, None], (torch.sin(a) * m).float()[:, :, None]  # [B,S,1,pairs]


def _turn(case, x, c, s, inverse=False):
    """The rotation of fp32 [B,S,H,D] (its transpose when ``inverse``)."""
    R = case["rot"]
    if inverse:
        s = -s
    if case["style"] == "half":
        x1, x2 = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], dim=-1)
    else:
        x1, x2 = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([x1 * c - x2 * s, x2 * c + x1 * s], dim=-1).flatten(-2)
    return torch.cat([y, x[..., R:]], dim=-1) if R < case["D"] else y


_EPS = 1e-6


def _norm_grad(case, g, x, w, c, s):
    dt, x = x.dtype, x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
    g = _turn(case, g.float(), c, s, inverse=True)
    n = x * r
    dw = (g * n).sum(dim=(0, 1, 2), dtype=torch.float64).float()
    gw = g * w
    return (r * (gw - n * (gw * n).mean(-1, keepdim=True))).to(dt), dw


def _blocks(case, n_keys_of):
    """Query row ranges whose scores fit in about 1 GB."""
    S, i = case["S"], 0
    per = case["B"] * case["Hq"] * max(1, n_keys_of)
    blk = max(64, min(1024, (1 << 28) // per))
    while i < S:
        yield i, min(S, i + blk)
        i += blk


def _keys(case, i0, i1):
    """(sink count, first, last + 1) of the keys any of the rows may see."""
    S, left, right, sinks = case["S"], case["left"], case["right"], case["sinks"]
    lo = 0 if left < 0 else max(0, i0 - left)
    hi = S if right < 0 else min(S, i1 + right)
    if case["causal"]:
        hi = i1
    else:
        hi = max(hi, min(sinks, S))
    return min(sinks, lo), lo, hi


def _mask(case, i, j):
    left, right, sinks = case["left"], case["right"], case["sinks"]
    i, j = i[:, None], j[None, :]
    ok = torch.ones_like(i - j, dtype=torch.bool)
    if left >= 0:
        ok = ok & (j >= i - left)
    if right >= 0:
        ok = ok & (j <= i + right)
    ok = ok | (j < sinks)
    return ok & (j <= i) if case["causal"] else ok


def _span(case):
    left = case["S"] if case["left"] < 0 else case["left"]
    right = 0 if case["causal"] else (case["S"] if case["right"] < 0 else case["right"])
    return min(case["S"], 1024 + left + right + case["sinks"])


def _score_blocks(case, q, k):
    """Per block of rows: the rows, key ranges, grouped q, keys and masked scores."""
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    G, scale = Hq // Hkv, D ** -0.5
    ar = torch.arange(case["S"], device=DEV)
    for i0, i1 in _blocks(case, _span(case)):
        ns, lo, hi = _keys(case, i0, i1)
        take = lambda t: torch.cat([t[:, :ns], t[:, lo:hi]], dim=1).float().permute(0, 2, 1, 3)  # [B,Hkv,n,D]
        qb = q[:, i0:i1].float().unflatten(2, (Hkv, G)).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * (i1 - i0), D)
        kb = take(k)
        s = (qb @ kb.transpose(-1, -2)).view(B, Hkv, G, i1 - i0, -1) * scale
        ok = _mask(case, ar[i0:i1], torch.cat([ar[:ns], ar[lo:hi]]))
        s = torch.where(ok, s, torch.full((), -math.inf, device=DEV))
        yield (i0, i1, ns, lo, hi), take, qb, kb, s


def _window_fwd(case, q, k, v):
    B, S, Hq, Hkv, D = case["B"], case["S"], case["Hq"], case["Hkv"], case["D"]
    out = torch.empty(B, S, Hq, D, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(B, Hq, S, dtype=torch.float32, device=DEV)
    for (i0, i1, _, _, _), take, _, _, s in _score_blocks(case, q, k):
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        l = p.sum(-1, keepdim=True)
        o = (p / l).flatten(2, 3) @ take(v)
        out[:, i0:i1] = o.view(B, Hkv, Hq // Hkv, i1 - i0, D).permute(0, 3, 1, 2, 4).flatten(2, 3).to(torch.bfloat16)
        lse[:, :, i0:i1] = (m + torch.log(l)).view(B, Hq, i1 - i0)
    return out, lse


def _window_bwd(case, q, k, v, out, lse, do):
    B, S, Hq, Hkv, D = case["B"], case["S"], case["Hq"], case["Hkv"], case["D"]
    G, scale = Hq // Hkv, D ** -0.5
    dq = torch.empty(B, S, Hq, D, dtype=torch.bfloat16, device=DEV)
    dk = torch.zeros(B, S, Hkv, D, dtype=torch.float32, device=DEV)
    dv = torch.zeros(B, S, Hkv, D, dtype=torch.float32, device=DEV)
    group = lambda t, n: t.float().unflatten(2, (Hkv, G)).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    for (i0, i1, ns, lo, hi), take, qb, kb, s in _score_blocks(case, q, k):
        n = i1 - i0
        ob, gb = group(out[:, i0:i1], n), group(do[:, i0:i1], n)
        p = torch.exp(s - lse[:, :, i0:i1].reshape(B, Hkv, G, n, 1)).flatten(2, 3)
        ds = p * (gb @ take(v).transpose(-1, -2) - (ob * gb).sum(-1, keepdim=True)) * scale
        dq[:, i0:i1] = (ds @ kb).view(B, Hkv, G, n, D).permute(0, 3, 1, 2, 4).flatten(2, 3).to(torch.bfloat16)
        for acc, part in ((dk, ds.transpose(-1, -2) @ qb), (dv, p.transpose(-1, -2) @ gb)):
            part = part.permute(0, 2, 1, 3)
            acc[:, :ns] += part[:, :ns]
            acc[:, lo:hi] += part[:, ns:]
    return dq, dk.to(torch.bfloat16), dv.to(torch.bfloat16)


def _decode(case, q, k, v, lengths):
    B, T, cap, Hq, Hkv, D = (case[n] for n in ("B", "T", "cap", "Hq", "Hkv", "D"))
    G, left, sinks = Hq // Hkv, case["left"], case["sinks"]
    n = lengths.long()[:, None]
    if left < 0 or sinks + left + T >= cap:
        j = torch.arange(cap, device=DEV)[None].expand(B, cap)
        kb, vb = k, v
    else:  # the sinks, then the last left + T keys (repeated sinks are masked)
        j = torch.cat([torch.arange(sinks, device=DEV)[None].expand(B, sinks),
                       n - (left + T) + torch.arange(left + T, device=DEV)[None]], dim=1)
        take = j.clamp(0, cap - 1)[:, :, None, None].expand(-1, -1, Hkv, D)
        kb, vb = torch.gather(k, 1, take), torch.gather(v, 1, take)
        j = torch.where((torch.arange(j.shape[1], device=DEV)[None] >= sinks) & (j < sinks), torch.full_like(j, -1), j)
    pos = (n - T + torch.arange(T, device=DEV)[None])[:, :, None]
    jj = j[:, None]
    ok = (jj >= 0) & (jj <= pos)
    if left >= 0:
        ok = ok & ((jj >= pos - left) | (jj < sinks))
    qb = q.float().unflatten(2, (Hkv, G)).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, D)
    s = (qb @ kb.float().permute(0, 2, 3, 1)).view(B, Hkv, G, T, -1) * D ** -0.5
    s = torch.where(ok[:, None, None], s, torch.full((), -math.inf, device=DEV))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    o = ((p / l).flatten(2, 3) @ vb.float().permute(0, 2, 1, 3)).view(B, Hkv, G, T, D)
    return (o.permute(0, 3, 1, 2, 4).flatten(2, 3).to(torch.bfloat16), (m + torch.log(l)).view(B, Hq, T))


def run(state):
    case = state["case"]
    kind = case["kind"]
    if own:
        import context_attention_fwd_gb300 as ctx
        if kind == "rope_fwd":
            return ctx.rope_fwd(state["q"], state["k"], state["table"], positions=state["positions"],
                                offset=case["offset"])
        if kind == "rope_bwd":
            return ctx.rope_bwd(state["gq"], state["gk"], state["table"], positions=state["positions"],
                                offset=case["offset"])
        if kind == "norm_rope_fwd":
            return ctx.qk_norm_rope_fwd(state["q"], state["k"], state["wq"], state["wk"], state["table"],
                                        positions=state["positions"], offset=case["offset"], eps=_EPS)
        if kind == "norm_rope_bwd":
            return ctx.qk_norm_rope_bwd(state["gq"], state["gk"], state["q"], state["k"], state["wq"], state["wk"],
                                        state["table"], positions=state["positions"], offset=case["offset"], eps=_EPS)
        if kind == "decode":
            return ctx.attn_decode(state["q"], state["k"], state["v"], state["lengths"], window=case["left"],
                                   sinks=case["sinks"])
        window = (case["left"], case["right"])
        if kind == "window_fwd":
            return ctx.attn_window_fwd(state["q"], state["k"], state["v"], case["P"], window, sinks=case["sinks"],
                                       causal=case["causal"])
        return ctx.attn_window_bwd(state["q"], state["k"], state["v"], state["out"], state["lse"], state["do"],
                                   case["P"], window, sinks=case["sinks"], causal=case["causal"])
    if "rope" in kind:
        c, s = _cos_sin(case, state)
        if kind == "rope_fwd":
            return tuple(_turn(case, state[n].float(), c, s).to(state[n].dtype) for n in ("q", "k"))
        if kind == "rope_bwd":
            return tuple(_turn(case, state[n].float(), c, s, inverse=True).to(state[n].dtype) for n in ("gq", "gk"))
        if kind == "norm_rope_fwd":
            out = []
            for n, w in (("q", "wq"), ("k", "wk")):
                x = state[n].float()
                x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * state[w]
                out.append(_turn(case, x, c, s).to(state[n].dtype))
            return tuple(out)
        dq, dwq = _norm_grad(case, state["gq"], state["q"], state["wq"], c, s)
        dk, dwk = _norm_grad(case, state["gk"], state["k"], state["wk"], c, s)
        return dq, dk, dwq, dwk
    if kind == "window_fwd":
        return _window_fwd(case, state["q"], state["k"], state["v"])
    if kind == "window_bwd":
        return _window_bwd(case, state["q"], state["k"], state["v"], state["out"], state["lse"], state["do"])
    return _decode(case, state["q"], state["k"], state["v"], state["lengths"])


# ------------------------------------------------------------------ work
def _pairs(case):
    """Visible (query, key) pairs of one head."""
    S, total = case["S"], 0
    for i in range(S):
        lo = 0 if case["left"] < 0 else max(0, i - case["left"])
        hi = i if case["causal"] or case["right"] == 0 else (S - 1 if case["right"] < 0 else min(S - 1, i + case["right"]))
        sink = min(case["sinks"], S) if not case["causal"] else min(case["sinks"], i + 1)
        extra = min(sink, lo) + (max(0, sink - hi - 1))
        total += hi - lo + 1 + extra
    return total


def work(case):
    kind, B, Hq, Hkv, D = case["kind"], case["B"], case["Hq"], case["Hkv"], case["D"]
    if "rope" in kind:
        e = B * case["S"] * (Hq + Hkv) * D
        size = 4 if case["dtype"] == "fp32" else 2
        if kind == "norm_rope_bwd":
            return {"bytes": 3 * e * size, "flops": 14 * e}
        return {"bytes": 2 * e * size, "flops": (7 if kind == "norm_rope_fwd" else 3) * e}
    if kind.startswith("window"):
        S = case["S"]
        qe, ke, flops = B * S * Hq * D * 2, B * S * Hkv * D * 2, B * Hq * D * _pairs(case)
        if kind == "window_fwd":
            return {"bytes": 2 * qe + 2 * ke + 4 * B * Hq * S, "flops": 4 * flops}
        return {"bytes": 4 * qe + 4 * ke + 4 * B * Hq * S, "flops": 10 * flops}
    T, cap = case["T"], case["cap"]
    n = cap if case["fill"] == "full" else (cap + T) / 2  # mean length of a ragged batch
    if case["left"] >= 0:
        n = min(n, case["left"] + T + case["sinks"])
    e = B * n * D
    return {"bytes": int(4 * e * Hkv + 4 * B * T * Hq * D), "flops": int(4 * e * Hq * T)}


# ------------------------------------------------------------------ definitions in fp64
def _exact_freq(case):
    out = []
    for n in _sections(case):
        for p in range(n):
            d, base, f = 2 * n, case["theta"], case["factor"]
            if case["scaling"] == "ntk":
                base *= math.pow(f, d / (d - 2))
            w = 1.0 / math.pow(base, 2 * p / d)
            if case["scaling"] == "linear":
                w /= f
            if case["scaling"] == "yarn":
                # pairs that turn more than 32 times over the original length keep
                # their frequency, those under one turn are slowed by the factor
                edge = [d * math.log(case["orig"] / (2 * math.pi * r)) / (2 * math.log(base)) for r in (32.0, 1.0)]
                a, b = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), d - 1)
                t = min(max((p - a) / max(b - a, 1e-3), 0.0), 1.0)
                w = (1 - t) * w + t * w / f
            out.append(w)
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def _exact_rotate(case, st, x, sign):
    """The rotation as a complex product; x fp64 [B,S,H,D]."""
    B, S, R = case["B"], case["S"], case["rot"]
    pos = st["positions"]
    if pos is None:
        pos = torch.arange(case["offset"], case["offset"] + S, device=DEV).expand(B, S)
    if case["pos"] == "grid":
        cols = [ax for ax, n in enumerate(_sections(case)) for _ in range(n)]
        ang = torch.stack([pos[:, ax].double() for ax in cols], -1).expand(B, S, R // 2) * _exact_freq(case)
    else:
        ang = torch.einsum("bs,p->bsp", pos.double(), _exact_freq(case))
    m = 1.0 + 0.1 * math.log(case["factor"]) if case["scaling"] == "yarn" and case["factor"] > 1 else 1.0
    z = torch.polar(torch.full_like(ang, m), sign * ang)[:, :, None]
    if case["style"] == "half":
        y = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * z
        y = torch.cat([y.real, y.imag], -1)
    else:
        y = torch.view_as_real(torch.complex(x[..., 0:R:2].contiguous(), x[..., 1:R:2].contiguous()) * z).flatten(-2)
    return torch.cat([y, x[..., R:]], -1)


def _exact_norm(case, st, x, w):
    return _exact_rotate(case, st, x / (x.pow(2).sum(-1, keepdim=True) / case["D"] + _EPS).sqrt() * w, 1.0)


def _exact_rows(case, q, k, v, r0, r1):
    """Attention of query rows [r0, r1) in fp64 over every key any of them sees."""
    B, S, Hq, Hkv = case["B"], case["S"], case["Hq"], case["Hkv"]
    row = torch.arange(r0, r1, device=DEV).view(-1, 1)
    col = torch.arange(S, device=DEV).view(1, -1)
    dist = row - col
    vis = torch.ones_like(dist, dtype=torch.bool)
    if case["left"] >= 0:
        vis &= dist <= case["left"]
    if case["right"] >= 0:
        vis &= -dist <= case["right"]
    vis |= col < case["sinks"]
    if case["causal"]:
        vis &= dist >= 0
    used = vis.any(0).nonzero().flatten()
    vis = vis[:, used]
    rep = Hq // Hkv
    ks = k[:, used].repeat_interleave(rep, 2)
    vs = v[:, used].repeat_interleave(rep, 2)
    s = torch.einsum("bihd,bjhd->bhij", q[:, r0:r1], ks) / math.sqrt(case["D"])
    s = s.masked_fill(~vis, -math.inf)
    lse = torch.logsumexp(s, -1)
    return torch.einsum("bhij,bjhd->bihd", (s - lse[..., None]).exp(), vs), lse


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if "rope" in kind:
        names = ("gq", "gk") if kind == "rope_bwd" else ("q", "k")
        xs = [st[n].double() for n in names]
        if kind == "rope_fwd":
            return tuple(_exact_rotate(case, st, x, 1.0) for x in xs)
        if kind == "rope_bwd":
            return tuple(_exact_rotate(case, st, x, -1.0) for x in xs)
        ws = [st["wq"].double(), st["wk"].double()]
        if kind == "norm_rope_fwd":
            return tuple(_exact_norm(case, st, x, w) for x, w in zip(xs, ws))
        grads = []
        for x, w, g in zip(xs, ws, ("gq", "gk")):
            x, w = x.detach().requires_grad_(), w.requires_grad_()
            grads.append(torch.autograd.grad(_exact_norm(case, st, x, w), (x, w), st[g].double()))
        return grads[0][0], grads[1][0], grads[0][1], grads[1][1]
    if kind.startswith("window"):
        S = case["S"]
        # fp64 runs at about a TFLOP/s here
        if work(case)["flops"] * 1.6 * (1 + 512 / max(1, _span(case) - 1024 + 64)) > 1.5e13:
            return None
        q, k, v = (st[n].double() for n in ("q", "k", "v"))
        step = max(32, min(512, (1 << 26) // (case["B"] * case["Hq"] * _span(case))))
        if kind == "window_fwd":
            parts = [_exact_rows(case, q, k, v, i, min(S, i + step)) for i in range(0, S, step)]
            return torch.cat([p[0] for p in parts], 1), torch.cat([p[1] for p in parts], 2)
        leaves = [t.detach().requires_grad_() for t in (q, k, v)]
        sums = [torch.zeros_like(t) for t in leaves]
        for i in range(0, S, step):
            j = min(S, i + step)
            o, _ = _exact_rows(case, *leaves, i, j)
            for acc, gr in zip(sums, torch.autograd.grad(o, leaves, st["do"][:, i:j].double())):
                acc += gr
        return tuple(sums)
    B, T, Hq, Hkv, D = (case[n] for n in ("B", "T", "Hq", "Hkv", "D"))
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(st["lengths"].tolist()):
        for t in range(T):
            p = n - T + t
            if p < 0:
                continue
            first = 0 if case["left"] < 0 else max(0, p - case["left"])
            idx = torch.cat([torch.arange(min(case["sinks"], first)), torch.arange(first, p + 1)]).to(DEV)
            kk = st["k"][b, idx].double().repeat_interleave(Hq // Hkv, 1)
            vv = st["v"][b, idx].double().repeat_interleave(Hq // Hkv, 1)
            s = torch.einsum("hd,jhd->hj", st["q"][b, t].double(), kk) / math.sqrt(D)
            lse[b, :, t] = torch.logsumexp(s, -1)
            out[b, t] = torch.einsum("hj,jhd->hd", torch.softmax(s, -1), vv)
    return out, lse
