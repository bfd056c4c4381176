"""Plain 64-bit implementations of the cache calls, on the CPU, and the inputs of their tests
(test infrastructure; shares no code with the library)."""

import math

import numpy as np
import torch

U_BF16, U_FP32 = 2.0 ** -8, 2.0 ** -24          # half a step, relative to the value
F64 = torch.float64


# ------------------------------------------------------------------------------- rotation

def frequencies(rot, theta=500000.0, scaling=0, factor=1.0, orig_len=0, low=0.0, high=0.0,
                mscale=0.0):
    """Angle per position of every pair, and the factor of cos and sin."""
    f, m = [], 1.0
    for j in range(rot // 2):
        w = theta ** (-2.0 * j / rot)
        if scaling == 1:
            w /= factor
        elif scaling == 2:
            w = (theta * factor ** (rot / (rot - 2.0))) ** (-2.0 * j / rot)
        elif scaling == 3:
            turns = orig_len * w / (2 * math.pi)
            if turns < low:
                w /= factor
            elif turns <= high:
                t = (turns - low) / (high - low)
                w = (1 - t) * w / factor + t * w
        elif scaling == 4:
            at = [rot * math.log(orig_len / (2 * math.pi * n)) / (2 * math.log(theta))
                  for n in (high, low)]
            p, q = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
            t = min(max((j - p) / max(q - p, 1e-3), 0.0), 1.0)
            w = t * w / factor + (1 - t) * w
        f.append(w)
    if scaling == 4:
        m = 0.1 * math.log(factor) + 1.0
    return torch.tensor(f, dtype=F64), mscale or m


def rotate(x, positions, rot, layout, transpose=False, **kw):
    """x [rows][heads][head_dim] in 64 bits; also m (|a| + |b|), what errors scale with."""
    x = x.cpu().to(F64)
    f, m = frequencies(rot, **kw)
    a = positions.cpu().to(F64)[:, None] * f
    c, s = (m * torch.cos(a))[:, None], (m * torch.sin(a))[:, None] * (-1 if transpose else 1)
    y, size = x.clone(), torch.zeros_like(x)
    i = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == 0 else (slice(0, rot, 2), slice(1, rot, 2))
    p, q = x[..., i[0]], x[..., i[1]]
    y[..., i[0]], y[..., i[1]] = p * c - q * s, q * c + p * s
    size[..., i[0]] = size[..., i[1]] = m * (p.abs() + q.abs())
    return y, size


# ------------------------------------------------------------------------------- the cache

class Cache:
    """A pool with the pages of a batch scattered over it; every row random, the rows of no
    sequence NaN."""

    def __init__(self, lens, n_kv, hd, page, max_len=None, spare=3, seed=0, dev="cuda", pools=1):
        g = np.random.default_rng(seed)
        self.lens, self.n_kv, self.hd, self.page = list(lens), n_kv, hd, page
        self.max_len = max_len or max(max(lens), 1)
        per = -(-self.max_len // page)
        self.num_pages = len(lens) * per + spare
        order = g.permutation(self.num_pages)[:len(lens) * per].reshape(len(lens), per)
        self.table_np = order.astype(np.int32)
        t = torch.Generator().manual_seed(seed)
        shape = (self.num_pages, page, n_kv, hd)
        self.k, self.v = [], []
        for _ in range(pools):
            for p in (self.k, self.v):
                full = torch.full(shape, float("nan"), dtype=torch.bfloat16)
                for b, n in enumerate(self.lens):
                    for r in range(n):
                        full[order[b, r // page], r % page] = torch.randn(n_kv, hd, generator=t).to(torch.bfloat16)
                p.append(full.to(dev))
        self.table = torch.from_numpy(self.table_np).to(dev)
        self.lengths = torch.tensor(self.lens, dtype=torch.int32, device=dev)

    def rows(self, pool, b, n=None):
        """Rows 0 .. n-1 of sequence b, [n][n_kv][hd] in 64 bits on the CPU."""
        n = self.lens[b] if n is None else n
        r = np.arange(n)
        page = torch.from_numpy(self.table_np[b, r // self.page].astype(np.int64))
        return pool.cpu()[page, torch.from_numpy(r % self.page)].to(F64)

    def batch(self, B, lengths=None):
        return B.make_batch(self.table, self.lengths if lengths is None else lengths, self.page,
                            self.num_pages, self.n_kv, self.hd, self.max_len)


def visible(length, n, words):
    """[n][length]: what each of a sequence's n queries sees; words: their masks or None."""
    seen = torch.ones(n, length, dtype=torch.bool)
    for i in range(n):
        for j in range(n):
            seen[i, length - n + j] = j <= i if words is None else bool(int(words[i]) >> j & 1)
    return seen


def attention(cache, q, starts, words, scale, layer=0):
    """For every query: out, lse and how far fp32 sums and bf16 weights may put them off; a
    hidden row is left out altogether.  Queries of no sequence give NaN."""
    n_q, heads, hd = q.shape
    q = q.cpu().to(F64)
    group = heads // cache.n_kv
    out = torch.full((n_q, heads, hd), float("nan"), dtype=F64)
    lse = torch.full((n_q, heads), float("nan"), dtype=F64)
    out_tol, lse_tol = out.clone(), lse.clone()
    for b in range(len(cache.lens)):
        lo, hi, length = starts[b], starts[b + 1], cache.lens[b]
        if hi == lo:
            continue
        k, v = cache.rows(cache.k[layer], b), cache.rows(cache.v[layer], b)
        seen = visible(length, hi - lo, None if words is None else words[lo:hi])
        for i in range(lo, hi):
            at = seen[i - lo]
            for h in range(heads):
                kk, vv = k[at, h // group], v[at, h // group]
                if kk.shape[0] == 0:
                    out[i, h], lse[i, h], out_tol[i, h], lse_tol[i, h] = 0, -math.inf, 0, 0
                    continue
                s = kk @ q[i, h] * scale
                # a dot product of hd terms, its scaling and the argument of exp, in fp32
                d = float(((hd + 2) * U_FP32 * (kk.abs() @ q[i, h].abs()) * abs(scale)).max()
                          + 8 * U_FP32 * s.abs().max())
                n = kk.shape[0]
                w = torch.softmax(s, 0)
                out[i, h], lse[i, h] = w @ vv, torch.logsumexp(s, 0)
                # the weights' rounding, the scores' error (twice: weight and sum), the sums
                out_tol[i, h] = (w @ vv.abs()) * (U_BF16 + 2 * d + (2 * n + 64) * U_FP32) \
                    + U_BF16 * 1.01 * out[i, h].abs() + 1e-30
                lse_tol[i, h] = d + (2 * n + 64) * U_FP32 + 8 * U_FP32 * lse[i, h].abs()
    return out, lse, out_tol, lse_tol


def weight(cache, q, starts, words, scale, lse, decay, acc, acc_out, layer=0):
    """What acc_out holds after the call, and how far fp32 may put it off."""
    heads, hd = q.shape[1:]
    q, lse = q.cpu().to(F64), lse.cpu().to(F64)
    want = acc_out.cpu().to(F64).clone()
    tol = torch.zeros_like(want)
    group = heads // cache.n_kv
    for b in range(len(cache.lens)):
        lo, hi, length = starts[b], starts[b + 1], cache.lens[b]
        if hi == lo:
            continue
        k = cache.rows(cache.k[layer], b)
        seen = visible(length, hi - lo, None if words is None else words[lo:hi])
        total, off = torch.zeros(length, dtype=F64), torch.zeros(length, dtype=F64)
        for i in range(lo, hi):
            for h in range(heads):
                if lse[i, h] == -math.inf:
                    continue
                at = seen[i - lo]
                kk = k[at, h // group]
                s = kk @ q[i, h] * scale
                d = (hd + 2) * U_FP32 * (kk.abs() @ q[i, h].abs()) * abs(scale) \
                    + 8 * U_FP32 * (s.abs() + lse[i, h].abs())
                w = torch.exp(s - lse[i, h])
                total[at] += w
                off[at] += w * (d + 8 * U_FP32)
        terms = (hi - lo) * heads
        old = decay * acc.cpu().to(F64)[b, :length] if acc is not None else torch.zeros(length, dtype=F64)
        want[b, :length] = old + total
        tol[b, :length] = off + (terms + 4) * U_FP32 * (total + old.abs())
    return want, tol


def evict(lens, acc, positions, n_keep, n_sink, n_recent):
    """Per sequence: the kept rows' places afterwards, [(from, to)] of the moves, the row that
    each place holds."""
    moves, holds = [], []
    for b, n in enumerate(lens):
        if n <= n_keep:
            moves.append([])
            holds.append(list(range(n)))
            continue
        p, a = positions[b], acc[b]
        top = max(int(p[t]) for t in range(n))

        def rank(t):
            safe = int(p[t]) < n_sink or int(p[t]) > top - n_recent
            w = float(a[t])
            return (0 if safe else 2 if w != w else 1, 0.0 if safe or w != w else -w, t)
        kept = sorted(sorted(range(n), key=rank)[:n_keep])
        low = [t for t in kept if t < n_keep]
        holes = sorted(set(range(n_keep)) - set(low))
        high = [t for t in kept if t >= n_keep]
        moves.append(list(zip(high, holes)))
        h = list(range(n_keep))
        for f, t in moves[-1]:
            h[t] = f
        holds.append(h)
    return moves, holds


def trees(counts, seed):
    """A random tree of drafts for each sequence: bit j of a draft's word where j is the draft
    itself or an ancestor."""
    g = np.random.default_rng(seed)
    words = []
    for n in counts:
        t = []
        for i in range(n):
            parent = int(g.integers(-1, i)) if i else -1
            t.append((t[parent] if parent >= 0 else 0) | 1 << i)
        words += t
    return np.array(words, dtype=np.uint64)
