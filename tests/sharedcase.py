"""Plain 64-bit attention of sequences that share prefixes, on the CPU, and the inputs of its tests
(test infrastructure; shares no code with the library)."""

import math

import numpy as np
import torch

import cachecase as R
import heldcase as H

F64 = torch.float64
W = 2.0 ** -15                          # what two bf16 operands leave of a weight


class SharedCache:
    """A pool that holds a batch's own rows and the prefixes of its groups, in any type; rows of no
    axis are NaN.  k and v: the bf16 pools of the values."""

    def __init__(self, lens, plens, starts, n_kv, hd, page, kind="bf16", seed=0, max_len=None, max_prefix=None, dev="cuda",
                 change=None):
        self.base = R.Cache(list(lens) + list(plens), n_kv, hd, page, seed=seed, dev="cpu",
                            max_len=max(max(lens), max(plens, default=1), max_len or 1, max_prefix or 1))
        b = self.base
        self.batch_size, self.plens, self.starts, self.kind, self.dev = len(lens), list(plens), list(starts), kind, dev
        self.lens, self.n_kv, self.hd, self.page, self.num_pages = list(lens), n_kv, hd, page, b.num_pages
        self.max_len, self.max_prefix = max_len or max(max(lens), 1), max_prefix or max(max(plens, default=1), 1)
        if change:
            change(self, b.k[0], b.v[0])
        (self.kp, self.ks, self.k), (self.vp, self.vs, self.v) = (H.hold(p, kind) for p in (b.k[0], b.v[0]))
        self.kp, self.vp, self.k, self.v = (t.to(dev) for t in (self.kp, self.vp, self.k, self.v))
        if kind != "bf16":
            self.ks, self.vs = self.ks.to(dev), self.vs.to(dev)
        table = torch.from_numpy(b.table_np)
        self.table, self.ptable = table[:len(lens)].contiguous().to(dev), table[len(lens):].contiguous().to(dev)
        ints = lambda x: torch.tensor(x, dtype=torch.int32).to(dev)  # noqa: E731
        self.lengths, self.plengths, self.group_start = ints(self.lens), ints(self.plens), ints(self.starts)

    def kv(self, B):
        return B.make_batch(self.table, self.lengths, self.page, self.num_pages, self.n_kv, self.hd, self.max_len)

    def cache(self, B):
        return B.make_cache(self.kp, self.vp, self.ks, self.vs)

    def values(self, B):
        """The bf16 cache of the same values."""
        return B.make_cache(self.k, self.v)

    def prefix(self, B):
        return B.make_prefix(self.ptable, self.plengths, self.group_start, self.max_prefix) if self.plens else None

    def group_of(self, b):
        return next((g for g in range(len(self.plens)) if self.starts[g] <= b < self.starts[g + 1]), None)

    def at(self, axis, row):
        """Page and slot of a row of sequence `axis`, or of prefix axis - batch."""
        return int(self.base.table_np[axis, row // self.page]), row % self.page

    def rows(self, pool, b, hidden=()):
        """The rows that sequence b's queries meet, prefix first; which of them are not hidden."""
        g = self.group_of(b)
        own = self.base.rows(pool, b)
        if g is None:
            return own
        return torch.cat([self.base.rows(pool, self.batch_size + g), own])


def attention(c, q, starts, words, scale, gone=()):
    """For every query out and lse, and how far fp32 sums and weights of 15 bits may put them off.
    `gone`: (axis, row) pairs that are on bad pages."""
    n_q, heads, hd = q.shape
    q = q.cpu().to(F64)
    group = heads // c.n_kv
    out = torch.full((n_q, heads, hd), float("nan"), dtype=F64)
    lse = torch.full((n_q, heads), float("nan"), dtype=F64)
    out_tol, lse_tol = out.clone(), lse.clone()
    for b in range(c.batch_size):
        lo, hi, length = starts[b], starts[b + 1], c.lens[b]
        if hi == lo:
            continue
        k, v = c.rows(c.k, b), c.rows(c.v, b)
        before = k.shape[0] - length
        seen = torch.cat([torch.ones(hi - lo, before, dtype=torch.bool),
                          R.visible(length, hi - lo, None if words is None else words[lo:hi])], 1)
        for axis, row in gone:
            if axis == b:
                seen[:, before + row] = False
            elif axis == c.batch_size + (c.group_of(b) if before else -1):
                seen[:, row] = False
        for i in range(lo, hi):
            at = seen[i - lo]
            if not at.any():
                out[i], lse[i], out_tol[i], lse_tol[i] = 0, -math.inf, 0, 0
                continue
            kk, vv = (x[at].repeat_interleave(group, 1).transpose(0, 1) for x in (k, v))       # [heads][rows][hd]
            s = (kk @ q[i][:, :, None])[..., 0] * scale
            # a dot product of hd terms, its scaling and the argument of exp, in fp32
            d = ((hd + 2) * R.U_FP32 * (kk.abs() @ q[i].abs()[:, :, None])[..., 0] * abs(scale)).amax(1) + 8 * R.U_FP32 * s.abs().amax(1)
            n = kk.shape[1]
            w = torch.softmax(s, 1)[:, None]
            out[i], lse[i] = (w @ vv)[:, 0], torch.logsumexp(s, 1)
            # the weights' bits, the scores' error (twice: weight and sum), the sums; one rounding
            out_tol[i] = (w @ vv.abs())[:, 0] * (W + 2 * d + (2 * n + 64) * R.U_FP32)[:, None] + R.U_BF16 * 1.01 * out[i].abs() + 1e-30
            lse_tol[i] = d + (2 * n + 64) * R.U_FP32 + 8 * R.U_FP32 * lse[i].abs()
    return out, lse, out_tol, lse_tol


def starts_of(counts):
    return [0] + [int(x) for x in np.cumsum(counts)]
