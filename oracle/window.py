"""Attention under a sliding window with sink tokens, in fp64, from its
definition: the full score matrix with masked entries at -infinity, and the
analytic gradient.  CPU code for the tests; shares nothing with the CUDA path."""
from __future__ import annotations

import math

import torch


def visible(S, left, right, sinks, causal):
    """Boolean [S,S]: key j (column) visible to query i (row)."""
    i, j = torch.arange(S)[:, None], torch.arange(S)[None]
    ok = torch.ones(S, S, dtype=torch.bool)
    if left >= 0:
        ok &= j >= i - left
    if right >= 0 and not causal:
        ok &= j <= i + right
    ok |= j < sinks
    return ok & (j <= i) if causal else ok


def _probs(q, k, left, right, sinks, causal, scale):
    B, S, Hq, D = q.shape
    scale = scale or 1.0 / math.sqrt(D)
    kk = k.double().repeat_interleave(Hq // k.shape[2], dim=2)
    s = torch.einsum("bihd,bjhd->bhij", q.double(), kk) * scale
    s = s.masked_fill(~visible(S, left, right, sinks, causal), -math.inf)
    lse = torch.logsumexp(s, -1)
    return torch.exp(s - lse[..., None]), lse, kk, scale


def attn_fwd(q, k, v, left, right, sinks, causal, scale=None):
    p, lse, _, _ = _probs(q, k, left, right, sinks, causal, scale)
    vv = v.double().repeat_interleave(q.shape[2] // v.shape[2], dim=2)
    return torch.einsum("bhij,bjhd->bihd", p, vv), lse


def attn_bwd(q, k, v, dout, left, right, sinks, causal, scale=None):
    """(dq, dk, dv); dk, dv summed over the query heads of each group."""
    p, _, kk, scale = _probs(q, k, left, right, sinks, causal, scale)
    G = q.shape[2] // k.shape[2]
    vv, do = v.double().repeat_interleave(G, dim=2), dout.double()
    dv = torch.einsum("bhij,bihd->bjhd", p, do)
    dp = torch.einsum("bihd,bjhd->bhij", do, vv)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
    dq = torch.einsum("bhij,bjhd->bihd", ds, kk)
    dk = torch.einsum("bhij,bihd->bjhd", ds, q.double())
    group = lambda t: t.unflatten(2, (k.shape[2], G)).sum(3)
    return dq, group(dk), group(dv)


def decode(q, k, v, lengths, left, sinks, scale=None):
    """The newest T tokens of each sequence over its cache, one row at a time:
    (out, lse), 0 and -infinity for a row that sees nothing."""
    B, T, Hq, D = q.shape
    G, scale = Hq // k.shape[2], scale or 1.0 / math.sqrt(D)
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64)
    for b in range(B):
        for t in range(T):
            pos = int(lengths[b]) - T + t
            if pos < 0:
                continue
            first = 0 if left < 0 else max(0, pos - left)
            keys = list(range(min(sinks, first))) + list(range(first, pos + 1))
            kk, vv = k[b, keys].double(), v[b, keys].double()
            for h in range(Hq):
                s = kk[:, h // G] @ q[b, t, h].double() * scale
                lse[b, h, t] = torch.logsumexp(s, 0)
                out[b, t, h] = torch.softmax(s, 0) @ vv[:, h // G]
    return out, lse
