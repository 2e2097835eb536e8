"""A cache in 4 bits as plain numpy in fp64: rows to cells and back, written from the layout's
description, entry by entry."""

import numpy as np
import torch

D = 128


def bf16_bits(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float64)).to(torch.bfloat16).view(torch.int16).numpy().astype(np.uint16)


def from_bits(u):
    return torch.from_numpy(np.asarray(u).astype(np.uint16).view(np.int16).copy()).view(torch.bfloat16).double().numpy()


def quantise(x, group):
    """(codes [..., 128], s, z [..., groups]) of fp64 rows."""
    g = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], D // group, group)
    lo, hi = g.min(-1), g.max(-1)
    s = from_bits(bf16_bits((hi - lo) / 15))
    z = from_bits(bf16_bits((hi + lo) / 2 + s / 2))
    with np.errstate(all="ignore"):
        c = np.where(s[..., None] > 0, np.rint((g - z[..., None]) / s[..., None]), 0.0)
    return (np.clip(c, -8, 7) + 8).astype(np.uint8).reshape(x.shape), s, z


BYTE_AT = np.array([8 * (b % 8) + b // 8 for b in range(64)])  # where byte b of a row stands


def put_rows(pool, cells, rows, codes, s, z):
    """Rows into pool [n_cells, cell] (uint8) at (cell, row of the cell)."""
    ng = s.shape[-1]
    b = codes[..., 0::2] | (codes[..., 1::2] << 4)
    for j in range(64):
        pool[cells, 64 * rows + BYTE_AT[j]] = b[..., j]
    for g in range(ng):
        for half, v in ((0, bf16_bits(s[..., g])), (2, bf16_bits(z[..., g]))):
            at = 1024 + 4 * (rows * ng + g) + half
            pool[cells, at] = (v & 255).astype(np.uint8)
            pool[cells, at + 1] = (v >> 8).astype(np.uint8)


def get_rows(pool, cells, rows, group):
    """(codes, s, z) of the rows at (cell, row of the cell) of pool [n_cells, cell]."""
    ng = D // group
    c = np.empty(cells.shape + (D,), np.uint8)
    for j in range(64):
        v = pool[cells, 64 * rows + BYTE_AT[j]]
        c[..., 2 * j], c[..., 2 * j + 1] = v & 15, v >> 4
    s, z = np.empty(cells.shape + (ng,)), np.empty(cells.shape + (ng,))
    for g in range(ng):
        at = 1024 + 4 * (rows * ng + g)
        s[..., g] = from_bits(pool[cells, at].astype(np.uint16) | (pool[cells, at + 1].astype(np.uint16) << 8))
        z[..., g] = from_bits(pool[cells, at + 2].astype(np.uint16) | (pool[cells, at + 3].astype(np.uint16) << 8))
    return c, s, z


def values(c, s, z):
    g = D // s.shape[-1]
    return np.repeat(s, g, -1) * (c.astype(np.float64) - 8) + np.repeat(z, g, -1)


class Cache:
    """A paged cache in both forms: host numpy cells and the rows' values, for one K or V side."""

    def __init__(self, n_blocks, H, bs, group, rng, fill=0xFF):
        self.H, self.bs, self.group = H, bs, group
        self.cell = 1024 + 64 * (D // group)
        # 0xff: every step and centre of a row that nobody wrote is NaN
        self.pool = np.full((n_blocks, H, bs // 16, self.cell), fill, np.uint8)

    def cells(self, e, h, t):
        return (e * self.H + h) * (self.bs // 16) + (t % self.bs) // 16, t % 16

    def put(self, e, h, t, x):
        """Rows x at blocks e, heads h, positions t."""
        cells, rows = self.cells(e, h, t)
        put_rows(self.pool.reshape(-1, self.cell), cells, rows, *quantise(x, self.group))

    def raw(self, e, h, t, pool=None):
        cells, rows = self.cells(e, h, t)
        return get_rows((self.pool if pool is None else pool).reshape(-1, self.cell), cells, rows, self.group)


def attended(L, ns, nl, sel):
    """The list of a request as skv_sparse_attn has it."""
    sink = min(L, ns)
    first = max(sink, L - nl)
    return list(range(sink)) + [int(t) for t in sel] + list(range(first, L))


def attention(q, kv, vv, scale):
    """(out, lse, tolerance of out, of lse) of queries [G, 128] over rows kv, vv = (codes, s, z).

    Tolerances.  A product's terms are exact and its sums have at most 160 fp32 additions,
    truncated (2^-23) on a tensor core, of parts no larger than M = sum_j |q_j| (15 s + 8 s + |z|):
    a logit is off by 160 * 2^-23 scale M, its weight relatively by that much (twice: the maximum's too) and
    2^-20 for the exponent's own roundings.  Weights times steps are fp16 (half a step: 2^-11 of
    weight times 15 s; under 2^-14, half a step of 2^-24 where the largest is 2^7 at least), and the
    sums over n keys in fp32 add n + 64 roundings of 2^-23 of the same parts at the worst; the output
    rounds once more, by 2^-8 of it."""
    k, v = values(*kv), values(*vv)
    rep = lambda a: np.repeat(np.abs(a), D // a.shape[-1], -1)  # noqa: E731
    n = k.shape[0]
    if n == 0:
        return np.zeros((q.shape[0], D)), np.full(q.shape[0], -np.inf), np.zeros((q.shape[0], D)), np.zeros(q.shape[0])
    x = scale * (q @ k.T)
    dx = scale * 160 * 2.0 ** -23 * (np.abs(q) @ (23 * rep(kv[1]) + rep(kv[2])).T)
    m = x.max(-1, keepdims=True)
    p = np.exp(x - m)
    l = p.sum(-1, keepdims=True)
    out = p @ v / l
    part = 15 * rep(vv[1]) + 8 * rep(vv[1]) + rep(vv[2])
    rel = 2 * dx.max(-1, keepdims=True) + 2.0 ** -20 + (n + 64) * 2.0 ** -23
    tol = (p @ (15 * rep(vv[1]))) / l * 2.0 ** -11 + rel * (p @ part) / l + n * 2.0 ** -25 * 2.0 ** -7 * 2 * 15 * vv[1].max()
    return out, (m + np.log(l))[:, 0], tol + 2.0 ** -8 * np.abs(out), rel[:, 0] + 2.0 ** -22 * np.abs(m[:, 0] + np.log(l)[:, 0])
