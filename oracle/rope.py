"""Rotary positions and per-head norms in fp64, from their definitions.

CPU code for the tests; shares nothing with the CUDA path but the meaning of
the frequency table (turns per position as a fraction of 2^64), which it
evaluates with whole-number arithmetic."""
from __future__ import annotations

import numpy as np
import torch


def angles(turns, positions):
    """2 pi * frac(position * turns / 2^64), fp64: turns int64 [pairs],
    positions int64 [B,S] or [B,S,pairs]."""
    t = turns.cpu().numpy().view(np.uint64)
    p = positions.cpu().numpy()
    p = p[..., None] if p.ndim == 2 else p
    with np.errstate(over="ignore"):
        frac = p.astype(np.int64).view(np.uint64) * t  # modulo 2^64
    return torch.from_numpy(frac.view(np.int64).astype(np.float64) * (2 * np.pi / 2.0 ** 64))


def rotate(x, ang, rot_dim, interleaved, magnitude=1.0, transpose=False):
    """x fp64 [B,S,H,D], ang [B,S,rot_dim/2]; the transposed rotation for gradients."""
    c, s = (torch.cos(ang) * magnitude)[:, :, None], (torch.sin(ang) * magnitude)[:, :, None]
    if transpose:
        s = -s
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot_dim:2], x[..., 1:rot_dim:2]
        y[..., 0:rot_dim:2], y[..., 1:rot_dim:2] = a * c - b * s, b * c + a * s
    else:
        h = rot_dim // 2
        a, b = x[..., :h], x[..., h:rot_dim]
        y[..., :h], y[..., h:rot_dim] = a * c - b * s, b * c + a * s
    return y


def norm(x, w, eps):
    """x / sqrt(mean(x^2) + eps) * w over the last dimension."""
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return n if w is None else n * w


def norm_grad(g, x, w, eps):
    """(dx, dw) of norm(x, w) for the incoming gradient g."""
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * r
    gw = g if w is None else g * w
    return r * (gw - n * (gw * n).mean(-1, keepdim=True)), (g * n).flatten(0, 2).sum(0)
