"""Paged factor caches for the tests, in 64 bits on the CPU: pools built and read byte by
byte from the layout's definition, the attention over them, and the bound on how far the
GPU's fp16 products may be from it."""
from __future__ import annotations

import dataclasses

import numpy as np
import torch

BYTE = [2 * (t % 8) + t // 8 for t in range(16)]


def f64(x):
    return x.detach().cpu().to(torch.float64).numpy()


@dataclasses.dataclass
class Plane:
    """One plane of a pool: records of R A factors (h1 x d1) and R B factors (h2 x d2)."""
    fmt: str
    n_pages: int
    page: int
    E: int
    a: int                      # elements of the A part

    def empty(self):
        """Every byte a NaN: bf16 0xffff, e4m3 0xff, exponent 0xff."""
        n = self.n_pages * self.page * (self.E * 2 if self.fmt == "bf16" else self.E + 2)
        raw = torch.full((n,), 0xFF, dtype=torch.uint8)
        return raw.view(torch.bfloat16) if self.fmt == "bf16" else raw

    def _view(self, pool):
        if self.fmt == "bf16":
            return pool.view(self.n_pages, self.page // 8, self.E, 8)
        return pool.view(self.n_pages, self.page // 16, self.E + 2, 16)

    def write(self, pool, pages, slots, x):
        """Records x [n][E] (float64 numpy) into slot slots[i] of page pages[i]."""
        v = self._view(pool)
        pages, slots = torch.as_tensor(pages).long(), torch.as_tensor(slots).long()
        if self.fmt == "bf16":
            v[pages, slots // 8, :, slots % 8] = torch.from_numpy(x).to(torch.bfloat16)
        else:
            byte = torch.tensor(BYTE)[slots % 16]
            v[pages, slots // 16, :, byte] = torch.from_numpy(quantise(x, self.a))

    def raw(self, pool, pages, slots):
        v = self._view(pool.cpu())
        pages, slots = torch.as_tensor(pages).long(), torch.as_tensor(slots).long()
        if self.fmt == "bf16":
            return v[pages, slots // 8, :, slots % 8]
        return v[pages, slots // 16, :, torch.tensor(BYTE)[slots % 16]]

    def read(self, pool, pages, slots):
        """The records' values [n][E] in float64."""
        x = self.raw(pool, pages, slots)
        if self.fmt == "bf16":
            return f64(x)
        code = f64(x[:, :self.E].contiguous().view(torch.float8_e4m3fn).float())
        with np.errstate(over="ignore"):
            scale = np.exp2(x[:, self.E:].numpy().astype(np.float64) - 127)
        return np.concatenate([code[:, :self.a] * scale[:, :1], code[:, self.a:] * scale[:, 1:]], 1)


def exponents(x):
    """The smallest e of -64 .. 63 with 448 * 2^e >= every finite |x| of each row."""
    m = np.where(np.isfinite(x), np.abs(x), 0.0).max(1, initial=0.0)
    e = np.full(len(x), -64)
    for i, v in enumerate(m):
        while e[i] < 63 and 448.0 * 2.0 ** float(e[i]) < v:
            e[i] += 1
    return e


def quantise(x, a):
    """Bytes [n][E + 2] of records x [n][E]."""
    parts, exps = [], []
    for p in (x[:, :a], x[:, a:]):
        e = exponents(p)
        y = np.clip(p / np.exp2(e.astype(np.float64))[:, None], -448, 448)
        y = np.where(np.isfinite(p), y, np.nan)
        parts.append(torch.from_numpy(y).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy())
        exps.append((e + 127).astype(np.uint8)[:, None])
    return np.concatenate(parts + exps, 1)


def planes(s, fmt, n_pages, page):
    return (Plane(fmt, n_pages, page, s.e_k, s.r_k * s.h1 * s.d1), Plane(fmt, n_pages, page, s.e_v, s.r_v * s.h1 * s.d1))


def rotate(x, s, pos):
    """Key records x [n][E_K] with B rotated at pos [n], float64."""
    a = s.r_k * s.h1 * s.d1
    y = x.copy()
    b = x[:, a:].reshape(len(x), s.r_k * s.h2, s.d2 // 2, 2)
    ang = np.asarray(pos, np.float64)[:, None] * s.rope_base ** (-2.0 * np.arange(s.d2 // 2) / s.d2)
    c, sn = np.cos(ang)[:, None], np.sin(ang)[:, None]
    y[:, a:] = np.stack([b[..., 0] * c - b[..., 1] * sn, b[..., 0] * sn + b[..., 1] * c], -1).reshape(len(x), -1)
    return y


def dense(x, s, r):
    """[n][h][d_h] of records x [n][E]."""
    n = len(x)
    a = x[:, :r * s.h1 * s.d1].reshape(n, r, s.h1, s.d1)
    b = x[:, r * s.h1 * s.d1:].reshape(n, r, s.h2, s.d2)
    return (np.einsum("nrxi,nryj->nxyij", a, b) / r).reshape(n, s.h, s.dh)


def dense_abs(x, s, r):
    """[n][h][d_h] of (1/R) sum_r |A_r| (x) |B_r|."""
    return dense(np.abs(x), s, r)


def visible(p, n, window, sinks):
    t = np.arange(n)
    see = t <= p
    return see & ((p - t < window) | (t < sinks)) if window else see


class Cache:
    """A pool with the slots below total[b] of each sequence written, every other byte a NaN,
    and a page table whose entries nobody may look at lead outside the pool."""

    def __init__(self, s, fmt, page, total, seed, std=0.7, spare=2, first_seen=None, sinks=0, stride=None):
        self.s, self.fmt, self.page, self.total = s, fmt, page, list(total)
        rng = np.random.default_rng(seed)
        need = [-(-t // page) for t in total]
        self.stride = max(need + [1]) + 1 if stride is None else stride
        n_pages = sum(need) + spare
        order = rng.permutation(n_pages)
        self.kp, self.vp = planes(s, fmt, n_pages, page)
        self.k, self.v = self.kp.empty(), self.vp.empty()
        self.table = torch.full((len(total), self.stride), -7, dtype=torch.int32)
        self.table[:, -1] = 1 << 30
        self.n_pages, at = n_pages, 0
        for b, t in enumerate(total):
            self.table[b, :need[b]] = torch.from_numpy(order[at:at + need[b]].astype(np.int32))
            at += need[b]
            if t == 0:
                continue
            slots = np.arange(t)
            if first_seen is not None:                 # the slots that some row sees
                slots = slots[(slots >= first_seen[b]) | (slots < sinks)]
                for i in range(need[b]):
                    if not ((slots >= i * page) & (slots < (i + 1) * page)).any():
                        self.table[b, i] = -3
            pages = self.table[b].numpy()[slots // page]
            self.kp.write(self.k, pages, slots % page, rng.standard_normal((len(slots), s.e_k)) * std)
            self.vp.write(self.v, pages, slots % page, rng.standard_normal((len(slots), s.e_v)) * std)

    def where(self, b, slots):
        return self.table[b].numpy()[slots // self.page], slots % self.page

    def records(self, b, slots, k=None, v=None):
        pages, inside = self.where(b, slots)
        return (self.kp.read(self.k if k is None else k, pages, inside),
                self.vp.read(self.v if v is None else v, pages, inside))

    def descriptor(self, lib):
        return lib.make_pages(self.page, self.n_pages, self.stride, self.fmt)


def attention(c, b, q, pos, window, sinks, scale, k=None, v=None, factored=False):
    """Rows q [n][h][d_h] (float64) at positions pos [n] of sequence b: out and the bound on the
    GPU's distance from it.

    The kernels round the scaled query, K, V and the weights once to fp16 (2^-11 relative, or
    2^-25 where the result is below fp16's normal range) and the output once to bf16 (2^-8); a
    key that is formed from rounded factors may carry two roundings.  A score is then off by at
    most d = 2^-11 * 3 * sum |q||K| scale + 2^-25 (sum |K| + sum |q| scale) (log2 e times that, in
    base 2), each weight by a factor within e^(2 d), and the rest is linear: the weights' and the
    values' roundings together move an output by at most 2 * 2^-11 * sum p |V|.

    factored: the single-token kernel never forms V.  It rounds each weighted factor p A^V_r to
    fp16 (over an e4m3 pool the weight first), so its error is 2 * 2^-11 * sum_s p sum_r |A_r||B_r|
    / R, where ranks that cancel in V do not cancel: sum p |V| is replaced by that sum."""
    s = c.s
    out = np.zeros((len(q), s.h, s.dh))
    tol = np.zeros_like(out)
    for i, p in enumerate(pos):
        see = visible(p, p + 1, window, sinks)
        slots = np.nonzero(see)[0]
        kx, vx = c.records(b, slots, k, v)
        K, V = dense(kx, s, s.r_k), dense(vx, s, s.r_v)
        z = np.einsum("hd,nhd->hn", q[i], K) * scale
        w = np.exp(z - z.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        out[i] = np.einsum("hn,nhd->hd", w, V)
        size = np.einsum("hd,nhd->hn", np.abs(q[i]), np.abs(K)).max(1) * abs(scale)
        sub = np.abs(K).sum(2).max(0) + np.abs(q[i]).sum(1) * abs(scale)
        d = 3 * 2.0 ** -11 * size + 2.0 ** -25 * sub + 2.0 ** -20 * (1 + np.abs(z).max(1))
        va = np.einsum("hn,nhd->hd", w, dense_abs(vx, s, s.r_v) if factored else np.abs(V))
        tol[i] = (2.0 ** -8 * np.abs(out[i]) + va * (np.expm1(2 * d) + 4 * 2.0 ** -11)[:, None]
                  + 2.0 ** -25 * (1 + len(slots) * np.abs(V).max((0, 2)))[:, None])
    return out, tol


def assert_within(got, want, tol, what=""):
    got = f64(got)
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    over = np.abs(got - want) - tol
    i = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert over.size == 0 or over[i] <= 0, f"{what}: at {i} got {got[i]}, want {want[i]} within {tol[i]}"
