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
