"""Attention over a paged cache with queries that each select one slot of a group, in 64 bits: an output
then shows whether the kernel met that slot, however long the cache is, and the bound on a
right output is a small part of what a missing or wrong slot changes."""
from __future__ import annotations

import numpy as np
import torch

import paged_util as pu


def planes(c, b, n, device):
    """Keys, values and (1/R) sum_r |A_r| (x) |B_r| of the values: [h][n][d_h] float64."""
    kx, vx = c.records(b, np.arange(n))
    s = c.s
    out = (pu.dense(kx, s, s.r_k), pu.dense(vx, s, s.r_v), pu.dense_abs(vx, s, s.r_v))
    return tuple(torch.from_numpy(x).to(device).transpose(0, 1).contiguous() for x in out)


def groups(n, seen=None):
    """First and last slot of what is seen of each 16-slot group of slots 0 .. n - 1."""
    see = np.ones(n, bool) if seen is None else seen
    out = []
    for g in range(0, n, 16):
        s = g + np.nonzero(see[g:g + 16])[0]
        if len(s):
            out.append((s[0], s[-1]))
    return np.array(out)


def select(K, ranges, scale, level=40.0):
    """Queries [len(ranges)][h][d_h] (bf16): in each head the slot of the range with the largest
    key, whose score is `level`."""
    norm = (K * K).sum(-1)                                        # h, n
    slot = torch.stack([lo + norm[:, lo:hi + 1].argmax(-1) for lo, hi in ranges])
    k = K[torch.arange(K.shape[0], device=K.device), slot]        # m, h, d
    return (level / scale * k / (k * k).sum(-1, keepdim=True)).to(torch.bfloat16)


def attention(q, pos, K, V, VA, window, sinks, scale, floor=True, hidden=None):
    """Rows q [m][h][d_h] at positions pos [m]: out, the bound on a kernel's distance from it, and
    the largest weight of each (row, head).

    A weight carries a factor within e^(2 d) of 1, d the error of a score: 3 * 2^-11 sum |q||K|
    scale for the roundings of the query, the key's factors and the key to fp16, 2^-25 of each
    absolutely, and 2^-20 of the score for its fp32 sums.  Weights off by such factors eps move
    sum p V / sum p by sum p eps (V - out) / sum p (1 + eps).  The weight (or the weighted factor)
    and the value are each rounded once or twice by 2^-11 relative, and below fp16's normal range
    by 2^-25 absolutely (never more than the weight itself, which is at most 1); a value's 2^-25
    (`floor`) is a rebuilt one's.  The output is rounded to bf16."""
    z = torch.einsum("mhd,hnd->mhn", q.double(), K) * scale
    s = torch.arange(K.shape[1], device=K.device)
    p = torch.as_tensor(pos, device=K.device)[:, None]
    see = s <= p
    if window:
        see &= (p - s < window) | (s < sinks)
    if hidden is not None:
        see &= ~hidden
    z = z.masked_fill(~see[:, None], -torch.inf)
    w = torch.exp(z - z.amax(-1, keepdim=True))
    l = w.sum(-1, keepdim=True)
    out = torch.einsum("mhn,hnd->mhd", w / l, V)
    qa, ka = q.double().abs() * abs(scale), K.abs()
    size = torch.einsum("mhd,hnd->mhn", qa, ka).masked_fill(~see[:, None], 0.0).amax(-1)
    zmax = z.abs().masked_fill(~see[:, None], 0.0).amax(-1)
    d = 3 * 2.0 ** -11 * size + 2.0 ** -25 * (ka.sum(-1).amax(-1) + qa.sum(-1)) + 2.0 ** -20 * (1 + zmax)
    eps = torch.expm1(2 * d) * torch.exp(2 * d)
    spread = torch.empty_like(out)
    for m in range(len(q)):                                       # sum p |V - out|
        spread[m] = torch.einsum("hn,hnd->hd", w[m] / l[m], (V - out[m][:, None]).abs())
    va = torch.einsum("mhn,hnd->mhd", w / l, VA)
    sub = torch.einsum("mhn,hn->mh", torch.clamp(w, max=2.0 ** -25) / l, VA.amax(-1))
    tol = 2.0 ** -8 * out.abs() + 4 * 2.0 ** -11 * va + eps[..., None] * spread + 2 * sub[..., None]
    if floor:
        tol = tol + 2.0 ** -25
    return out, tol, (w / l).amax(-1)
