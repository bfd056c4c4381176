"""GPU parity of the cache calls (rotary positions, append, attention of drafted tokens,
attention weight, eviction) against plain 64-bit implementations (cachecase.py), at the
sizes, masks, layouts and values where they can go wrong.  Tolerances count roundings: half a
step of the output's type, one rounding of the weights to bf16, fp32 sums."""

import numpy as np
import pytest
import torch

import cachecase as R
from ridge_map_kv_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _randn(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def _close(got, want, tol, what):
    got = got.detach().cpu().to(torch.float64)
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    over = torch.where(same, torch.zeros_like(tol), (got - want).abs() - tol)
    assert not torch.isnan(over).any(), f"{what}: NaN"
    assert float(over.max() if over.numel() else 0) <= 0, \
        f"{what}: {float(over.max())} over the tolerance at {int(over.argmax())}"


# ------------------------------------------------------------------------------- rotation

SCALINGS = [dict(), dict(scaling=B.RF_ROPE_LINEAR, factor=4.0), dict(scaling=B.RF_ROPE_NTK, factor=4.0),
            dict(scaling=B.RF_ROPE_BANDS, factor=8.0, orig_len=8192, low=1.0, high=4.0),
            dict(scaling=B.RF_ROPE_YARN, factor=8.0, orig_len=4096, low=1.0, high=32.0),
            dict(scaling=B.RF_ROPE_YARN, factor=2.0, orig_len=1024, low=1.0, high=32.0, mscale=0.7),
            dict(theta=10000.0, scaling=B.RF_ROPE_BANDS, factor=32.0, orig_len=100, low=0.5, high=0.6)]


def _rope_tol(want, size, dtype):
    # cos and sin within 2^-21 (an fp32 argument of half a turn at most, times 2 pi, and the
    # functions' own steps), three fp32 operations; one rounding to bf16
    tol = size * 2.0 ** -20 + 1e-30
    return tol + R.U_BF16 * 1.01 * want.abs() if dtype == torch.bfloat16 else tol


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [B.RF_ROPE_HALF, B.RF_ROPE_INTERLEAVED])
@pytest.mark.parametrize("n,heads,hd,rot", [(1, 1, 64, 0), (7, 4, 64, 32), (33, 5, 128, 64), (300, 1, 16, 16),
                                            (5, 40, 128, 0), (3, 2, 256, 256), (9, 3, 96, 48), (2, 3, 80, 80)])
def test_rope(dtype, layout, n, heads, hd, rot):
    for k, kw in enumerate(SCALINGS):
        x = _randn(n + k, n, heads, hd, dtype=dtype)
        pos = torch.randint(-5000, 70000, (n,), generator=torch.Generator().manual_seed(k), dtype=torch.int32)
        rope = B.make_rope(rotary_dim=rot, layout=layout, **kw)
        for transpose in (False, True):
            out = torch.empty_like(x)
            B.ridgefill_rope(rope, x, pos.to(DEV), out, transpose=transpose)
            want, size = R.rotate(x, pos, rot or hd, layout, transpose, **kw)
            _close(out, want, _rope_tol(want, size, dtype), f"{kw} {transpose}")


def test_rope_far_positions_and_zero():
    n = 6
    x = _randn(3, n, 2, 128, dtype=torch.float32)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 9], dtype=torch.int32)
    out = torch.empty_like(x)
    B.ridgefill_rope(B.make_rope(), x, pos.to(DEV), out)
    want, size = R.rotate(x, pos, 128, 0)
    # an fp64 angle of up to 2^31 / (2 pi) turns keeps 2^-23 of a turn: 2^-20 in cos and sin
    _close(out, want, size * 2.0 ** -19, "far")
    assert torch.equal(out[0], x[0])


def test_rope_strided_and_in_place():
    base = _randn(4, 19, 7 * 128 + 24).view(19, -1)
    x = base[:, 8:8 + 3 * 128].unflatten(1, (3, 128))
    pos = torch.arange(100, 119, dtype=torch.int32, device=DEV)
    before = base.clone()
    want, size = R.rotate(x, pos, 64, 0)
    out = torch.full((19, 5, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    rope = B.make_rope(rotary_dim=64)
    B.ridgefill_rope(rope, x, pos, out[:, :3])
    _close(out[:, :3], want, _rope_tol(want, size, torch.bfloat16), "strided")
    assert (out[:, 3:] == 9).all() and torch.equal(base, before)
    B.ridgefill_rope(rope, x, pos, x)
    assert torch.equal(x, out[:, :3])
    assert torch.equal(base[:, :8], before[:, :8]) and torch.equal(base[:, 8 + 384:], before[:, 8 + 384:])


@pytest.mark.parametrize("layout", [0, 1])
def test_rope_gradient(layout):
    # the rotation is linear: the gradient of sum(g * R x) is R^T g, and differences of it along
    # single coordinates are exact up to rounding
    kw = dict(scaling=B.RF_ROPE_YARN, factor=8.0, orig_len=4096, low=1.0, high=32.0)
    x, g = (_randn(s, 11, 3, 64, dtype=torch.float32) for s in (1, 2))
    pos = torch.arange(0, 1100, 100, dtype=torch.int32, device=DEV)
    rope = B.make_rope(rotary_dim=32, layout=layout, **kw)
    y, grad = torch.empty_like(x), torch.empty_like(x)
    B.ridgefill_rope(rope, x, pos, y)
    B.ridgefill_rope(rope, g, pos, grad, transpose=True)
    lhs, rhs = (y.double() * g.double()).sum(), (x.double() * grad.double()).sum()
    size = float((x.double().abs().amax() * 3 * g.double().abs().sum()))
    assert abs(float(lhs - rhs)) <= size * 2.0 ** -20
    for row, head, feature in ((0, 0, 0), (3, 1, 17), (10, 2, 31), (5, 0, 40), (7, 2, 1)):
        x2, y2 = x.clone(), torch.empty_like(x)
        x2[row, head, feature] += 1.0
        B.ridgefill_rope(rope, x2, pos, y2)
        step = float((x2 - x)[row, head, feature])
        diff = float(((y2.double() - y.double()) * g.double()).sum()) / step
        # each output holds a rounding of 2^-24 of values up to 3 |x|max
        tol = 8 * 2.0 ** -24 * 3 * float(x2.abs().max()) * float(g.abs().max()) + 2.0 ** -20 * 3 * float(g.abs().max())
        assert abs(diff - float(grad[row, head, feature])) <= tol


def test_rope_empty():
    x = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    B.ridgefill_rope(B.make_rope(), x, torch.empty(0, dtype=torch.int32, device=DEV), x)


# --------------------------------------------------------------------------------- append

@pytest.mark.parametrize("hd,n_kv,n_q,page,rot,layout", [(128, 8, 32, 16, 0, 0), (64, 2, 4, 4, 32, 1),
                                                         (128, 1, 5, 7, 64, 0), (64, 3, 0, 1, 0, 1),
                                                         (96, 2, 2, 5, 48, 0), (16, 1, 1, 100, 0, 0)])
def test_append(hd, n_kv, n_q, page, rot, layout):
    n, lens = 37, [40, 9, 64]
    cache = R.Cache(lens, n_kv, hd, page, max_len=64, seed=hd + page)
    kw = SCALINGS[4]
    qkv = _randn(hd, n, n_q + 2 * n_kv, hd)
    g = np.random.default_rng(page)
    places = g.permutation(3 * 64)[:n]
    seq_np, rows_np = (places // 64).astype(np.int32), (places % 64).astype(np.int32)
    seq_np[[2, 30]] = -1                                  # padding rows
    pos_np = g.integers(0, 40000, n).astype(np.int32)
    seq, rows, pos = (torch.from_numpy(a).to(DEV) for a in (seq_np, rows_np, pos_np))
    q, k, v = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    for use_pos in (True, False):
        kp, vp = cache.k[0].clone(), cache.v[0].clone()
        q_out = torch.full((n, max(n_q, 1), hd), 5.0, dtype=torch.bfloat16, device=DEV)
        status = torch.full((1,), -1, dtype=torch.int32, device=DEV)
        B.ridgefill_append_rows(B.make_rope(rotary_dim=rot, layout=layout, **kw), cache.batch(B), k, v, rows,
                                kp, vp, status, seq=seq, positions=pos if use_pos else None,
                                q=q if n_q else None, q_out=q_out if n_q else None)
        assert B.ridgefill_read_status(status) == B.RF_OK
        want, size = R.rotate(qkv[:, :n_q + n_kv], pos if use_pos else rows, rot or hd, layout, **kw)
        tol = _rope_tol(want, size, torch.bfloat16)
        real = torch.from_numpy(np.flatnonzero(seq_np >= 0))
        if n_q:
            _close(q_out[real.to(DEV)], want[real, :n_q], tol[real, :n_q], "q")
            assert (q_out[[2, 30]] == 5).all()
        page_of = torch.from_numpy(cache.table_np.astype(np.int64))[seq_np[real], rows_np[real] // page].to(DEV)
        slot = torch.from_numpy(rows_np[real] % page).to(DEV).long()
        _close(kp[page_of, slot], want[real, n_q:], tol[real, n_q:], "k")
        assert torch.equal(vp[page_of, slot], v[real.to(DEV)])
        for new, old in ((kp, cache.k[0]), (vp, cache.v[0])):    # nothing else is touched
            new, old = new.view(torch.int16).clone(), old.view(torch.int16)
            new[page_of, slot] = old[page_of, slot]
            assert torch.equal(new, old)


def test_append_without_rotation_and_in_place_q():
    cache = R.Cache([8], 2, 64, 4, seed=1)
    k, v, q = (_randn(s, 3, h, 64) for s, h in ((1, 2), (2, 2), (3, 6)))
    rows = torch.tensor([7, 0, 4], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    before = q.clone()
    kv = B.make_batch(cache.table, None, 4, cache.num_pages, 2, 64, 8)
    B.ridgefill_append_rows(None, kv, k, v, rows, cache.k[0], cache.v[0], status, q=q, q_out=q)
    assert B.ridgefill_read_status(status) == B.RF_OK
    assert torch.equal(q, before)
    assert torch.equal(cache.rows(cache.k[0], 0)[[7, 0, 4]], k.cpu().double())
    B.ridgefill_append_rows(B.make_rope(), kv, k, v, rows, cache.k[0], cache.v[0], status, q=q, q_out=q)
    want, size = R.rotate(before, rows, 64, 0)
    _close(q, want, _rope_tol(want, size, torch.bfloat16), "q in place")


def test_append_bad_rows_are_flagged_and_skipped():
    cache = R.Cache([16, 16], 1, 64, 4, seed=2)
    cache.table[1, 2] = cache.num_pages                  # a page out of range
    k, v, q = (_randn(s, 6, 1, 64) for s in (1, 2, 3))
    seq = torch.tensor([0, 0, 2, 1, 1, 0], dtype=torch.int32, device=DEV)
    rows = torch.tensor([0, 16, 3, 9, 3, -1], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = torch.empty_like(q)
    old = cache.k[0].clone()
    B.ridgefill_append_rows(B.make_rope(), cache.batch(B), k, v, rows, cache.k[0], cache.v[0], status, seq=seq,
                            q=q, q_out=q_out)
    assert B.ridgefill_read_status(status) == B.RF_E_ROWS
    changed = (cache.k[0].view(torch.int16) != old.view(torch.int16)).flatten(2).any(-1)
    where = {(int(cache.table_np[0, 0]), 0), (int(cache.table_np[1, 0]), 3)}
    assert {tuple(x) for x in changed.nonzero().tolist()} == where
    want, size = R.rotate(q, rows, 64, 0)                # q is rotated all the same
    _close(q_out, want, _rope_tol(want, size, torch.bfloat16), "q")
    B.ridgefill_append_rows(B.make_rope(), cache.batch(B), k[:1], v[:1], rows[:1], cache.k[0], cache.v[0], status)
    assert B.ridgefill_read_status(status) == B.RF_OK    # the word is the last call's


# ------------------------------------------------------------------------------ attention

def _starts(counts):
    return [0] + [int(x) for x in np.cumsum(counts)]


def _case(lens, counts, heads, n_kv, hd, page, seed=0, tree=False, max_q=None, max_len=None, q_scale=1.0):
    cache = R.Cache(lens, n_kv, hd, page, max_len=max_len, seed=seed)
    starts = _starts(counts)
    q = _randn(seed + 7, starts[-1], heads, hd) * q_scale
    words = R.trees(counts, seed) if tree else None
    return cache, q, starts, words, max_q or max(max(counts), 1)


def _mask(words):
    return None if words is None else torch.from_numpy(words.view(np.int64)).to(DEV)


def _attend(cache, q, starts, words, max_q, scale, want_out=True, want_lse=True, n_pad=0, kv=None):
    n, heads, hd = q.shape
    kv = kv or cache.batch(B)
    out = torch.full((n + n_pad, heads, hd), 3.0, dtype=torch.bfloat16, device=DEV) if want_out else None
    lse = torch.full((n + n_pad, heads), 3.0, device=DEV) if want_lse else None
    qp = torch.cat([q, torch.full((n_pad, heads, hd), float("nan"), dtype=q.dtype, device=DEV)])
    if words is not None and n_pad:
        words = np.concatenate([words, np.zeros(n_pad, np.uint64)])
    ws = torch.full((B.ridgefill_tree_attention_workspace_bytes(kv, heads, max_q),), 0xff, dtype=torch.uint8, device=DEV)
    B.ridgefill_tree_attention(kv, cache.k[0], cache.v[0] if want_out else None, qp,
                               torch.tensor(starts, dtype=torch.int32, device=DEV), max_q, scale, out, ws, lse=lse,
                               tree_mask=_mask(words))
    return out, lse, B.ridgefill_read_status(ws)


ATTEND = [  # lens, counts, heads, n_kv, hd, page, tree
    ([1], [1], 1, 1, 64, 1, False),
    ([29], [1], 4, 2, 64, 4, False),
    ([1, 2, 31, 32, 33], [1, 1, 1, 1, 1], 8, 2, 128, 16, False),
    ([64, 63, 65, 0, 127], [3, 0, 64, 0, 5], 4, 2, 64, 16, True),
    ([70, 200], [64, 64], 8, 2, 128, 16, True),
    ([300, 5, 129], [7, 5, 1], 10, 2, 128, 12, False),
    ([511, 4], [17, 4], 6, 1, 64, 100, True),
    ([1000], [48], 16, 1, 128, 3, True),
    ([2051, 700], [2, 1], 5, 5, 128, 32, False),
    ([257, 300], [20, 33], 3, 3, 64, 8, True),
    ([90], [64], 40, 2, 128, 16, False),
    ([9001, 150], [1, 1], 2, 1, 128, 16, False),
    ([6000, 20, 4100], [9, 3, 12], 2, 2, 64, 20, True),
]


@pytest.mark.parametrize("lens,counts,heads,n_kv,hd,page,tree", ATTEND)
def test_attention(lens, counts, heads, n_kv, hd, page, tree):
    cache, q, starts, words, max_q = _case(lens, counts, heads, n_kv, hd, page, seed=len(lens) + hd + page, tree=tree)
    scale = hd ** -0.5
    out, lse, st = _attend(cache, q, starts, words, max_q, scale, n_pad=3)
    assert st == B.RF_OK
    want, wl, ot, lt = R.attention(cache, q, starts, words, scale)
    n = q.shape[0]
    _close(out[:n], want, ot, "out")
    _close(lse[:n], wl, lt, "lse")
    assert (out[n:] == 3).all() and (lse[n:] == 3).all()       # padded queries stay as they were
    only, _, _ = _attend(cache, q, starts, words, max_q, scale, want_lse=False)
    assert torch.equal(only, out[:n])
    _, only, _ = _attend(cache, q, starts, words, max_q, scale, want_out=False)
    _close(only, wl, lt, "lse alone")


@pytest.mark.parametrize("max_q", [1, 13, 64])
def test_attention_bound_larger_than_the_counts(max_q):
    cache, q, starts, words, _ = _case([77, 500], [1, 1], 8, 2, 128, 16, seed=5, max_len=4000)
    out, lse, st = _attend(cache, q, starts, words, max_q, 0.09)
    want, wl, ot, lt = R.attention(cache, q, starts, words, 0.09)
    assert st == B.RF_OK
    _close(out, want, ot, "out")
    _close(lse, wl, lt, "lse")


def test_attention_large_scores_and_negative_scale():
    # scores of hundreds: the running maximum has to carry them
    for scale in (4.0, -2.0, 0.0):
        cache, q, starts, words, max_q = _case([400], [6], 4, 2, 64, 16, seed=9, tree=True, q_scale=4.0)
        out, lse, st = _attend(cache, q, starts, words, max_q, scale)
        want, wl, ot, lt = R.attention(cache, q, starts, words, scale)
        assert st == B.RF_OK
        _close(out, want, ot, f"out {scale}")
        _close(lse, wl, lt, f"lse {scale}")


@pytest.mark.parametrize("hd,page,counts,ctx", [(64, 4, 5, 0), (128, 16, 20, 44), (128, 5, 64, 3), (64, 16, 9, 130)])
def test_attention_masks_with_empty_rows(hd, page, counts, ctx):
    cache, q, starts, words, max_q = _case([ctx + counts], [counts], 4, 2, hd, page, seed=ctx + 1, tree=True)
    words[0] = 0                                         # sees only what came before
    words[counts // 2] = np.uint64(1) << np.uint64(counts - 1)   # a later draft, not itself
    words[counts - 1] = np.uint64(2 ** 64 - 1)           # bits past the drafts mean nothing
    out, lse, st = _attend(cache, q, starts, words, max_q, 0.1)
    want, wl, ot, lt = R.attention(cache, q, starts, words, 0.1)
    assert st == B.RF_OK
    _close(out, want, ot, "out")
    _close(lse, wl, lt, "lse")
    if ctx == 0:
        assert (out[0] == 0).all() and (lse[0] == -float("inf")).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_hidden_rows_may_hold_anything(bad, hd):
    counts, ctx = 24, 50
    cache, q, starts, words, max_q = _case([ctx + counts], [counts], 6, 2, hd, 8, seed=3, tree=True)
    hidden = [3, 10, 23]                                  # drafts that only they themselves see
    for i in range(counts):
        for j in hidden:
            if i != j:
                words[i] &= ~(np.uint64(1) << np.uint64(j))
    want, wl, ot, lt = R.attention(cache, q, starts, words, 0.1)
    for j in hidden:
        t = ctx + j
        page = int(cache.table_np[0, t // 8])
        cache.k[0][page, t % 8] = bad
        cache.v[0][page, t % 8] = bad
    out, lse, st = _attend(cache, q, starts, words, max_q, 0.1)
    assert st == B.RF_OK
    others = [i for i in range(counts) if i not in hidden]
    _close(out[others], want[others], ot[others], "out")
    _close(lse[others], wl[others], lt[others], "lse")
    if bad != bad:
        assert torch.isnan(out[hidden]).all() and torch.isnan(lse[hidden]).all()


def test_attention_visible_infinite_value():
    # an infinite value reaches exactly the queries that see its row
    cache, q, starts, words, max_q = _case([40], [8], 2, 1, 64, 16, seed=4, tree=True)
    j = 2
    t = 32 + j
    cache.v[0][int(cache.table_np[0, t // 16]), t % 16, 0, 5] = float("inf")
    out, _, _ = _attend(cache, q, starts, words, max_q, 0.1)
    sees = [bool(int(w) >> j & 1) for w in words]
    for i in range(8):
        assert torch.isinf(out[i, :, 5]).all() == sees[i]
        assert torch.isfinite(out[i, :, :5]).all() and torch.isfinite(out[i, :, 6:]).all()


def test_attention_scores_of_minus_infinity():
    cache, q, starts, words, max_q = _case([5], [1], 1, 1, 64, 4, seed=6)
    cache.k[0][..., 0] = torch.where(torch.isnan(cache.k[0][..., 0]), cache.k[0][..., 0], -float("inf"))
    q[..., 0] = 1.0
    out, lse, st = _attend(cache, q, starts, words, max_q, 0.1)
    assert st == B.RF_OK and (out == 0).all() and (lse == -float("inf")).all()


def test_attention_strided_q_and_out():
    cache, _, starts, words, max_q = _case([90, 33], [4, 2], 4, 2, 128, 16, seed=8)
    wide = _randn(1, 6, 9, 128)
    q = wide[:, 2:6]
    kv = cache.batch(B)
    out = torch.full((6, 7, 128), 2.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(B.ridgefill_tree_attention_workspace_bytes(kv, 4, max_q), dtype=torch.uint8, device=DEV)
    B.ridgefill_tree_attention(kv, cache.k[0], cache.v[0], q, torch.tensor(starts, dtype=torch.int32, device=DEV), max_q,
                               0.1, out[:, 1:5], ws)
    want, _, ot, _ = R.attention(cache, q, starts, words, 0.1)
    _close(out[:, 1:5], want, ot, "strided")
    assert (out[:, 0] == 2).all() and (out[:, 5:] == 2).all()


def test_attention_bad_sequences_are_flagged_and_skipped():
    lens, counts = [50, 50, 50, 50], [2, 2, 2, 2]
    cache, q, starts, words, max_q = _case(lens, counts, 4, 2, 64, 16, seed=11)
    ref, ref_lse, _ = _attend(cache, q, starts, words, max_q, 0.1)
    for lengths, st_q in (([50, 51, 50, 50], starts), ([50, -1, 50, 50], starts), ([50, 1, 50, 50], starts)):
        kv = cache.batch(B, torch.tensor(lengths, dtype=torch.int32, device=DEV))
        out, lse, st = _attend(cache, q, st_q, words, max_q, 0.1, kv=kv)
        assert st == B.RF_E_ROWS
        assert (out[2:4] == 3).all() and (lse[2:4] == 3).all()
        for i in (0, 1, 4, 5, 6, 7):
            assert torch.equal(out[i], ref[i]) and torch.equal(lse[i], ref_lse[i])
    out, lse, st = _attend(cache, q, [0, 2, 5, 6, 9], words, 2, 0.1)     # 3 > max_q; past the end
    assert st == B.RF_E_ROWS
    assert torch.equal(out[:2], ref[:2]) and (out[2:5] == 3).all() and (out[6:] == 3).all()
    out, lse, st = _attend(cache, q, starts, words, max_q, 0.1)
    assert st == B.RF_OK


@pytest.mark.parametrize("hd,entry", [(64, -1), (128, 1 << 20)])
def test_attention_bad_pages_are_taken_as_not_there(hd, entry):
    cache, q, starts, words, max_q = _case([200], [3], 4, 2, hd, 16, seed=12)
    whole = R.Cache([200], 2, hd, 16, seed=12)
    cache.table[0, 5] = entry
    out, lse, st = _attend(cache, q, starts, words, max_q, 0.1)
    assert st == B.RF_E_ROWS
    k, v = whole.rows(whole.k[0], 0), whole.rows(whole.v[0], 0)
    there = torch.ones(3, 200, dtype=torch.bool)
    there[:, 80:96] = False
    for i in range(3):
        there[i, 198 + i:] = False
        for h in range(4):
            s = k[there[i], h // 2] @ q[i, h].cpu().double() * 0.1
            want = torch.softmax(s, 0) @ v[there[i], h // 2]
            tol = (torch.softmax(s, 0) @ v[there[i], h // 2].abs()) * (R.U_BF16 + 2.0 ** -13) + R.U_BF16 * 1.01 * want.abs()
            assert ((out[i, h].cpu().double() - want).abs() <= tol).all()


def test_attention_offsets_past_32_bits():
    # a pool of over 2^32 bytes, the sequence on its last pages
    n_kv, hd, page = 8, 128, 16
    num_pages = (1 << 32) // (page * n_kv * hd * 2) + 40
    small = R.Cache([500], n_kv, hd, page, seed=13)
    pools = []
    table = torch.arange(num_pages - 1, num_pages - 1 - 32, -1, dtype=torch.int32, device=DEV)[None].contiguous()
    for src in (small.k[0], small.v[0]):
        pool = torch.empty(num_pages, page, n_kv, hd, dtype=torch.bfloat16, device=DEV)
        pool[table[0].long()] = src[small.table[0].long()]
        pools.append(pool)
    kv = B.make_batch(table, small.lengths, page, num_pages, n_kv, hd, 500)
    q = _randn(1, 5, 16, hd)
    starts = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    ref, ref_lse, _ = _attend(small, q, [0, 5], None, 5, 0.1)
    out, lse = torch.empty_like(ref), torch.empty_like(ref_lse)
    ws = torch.empty(B.ridgefill_tree_attention_workspace_bytes(kv, 16, 5), dtype=torch.uint8, device=DEV)
    B.ridgefill_tree_attention(kv, pools[0], pools[1], q, starts, 5, 0.1, out, ws, lse=lse)
    assert B.ridgefill_read_status(ws) == B.RF_OK
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    wws = torch.empty(B.ridgefill_attention_weight_workspace_bytes(kv, 16, 5), dtype=torch.uint8, device=DEV)
    a, b = torch.zeros(1, 500, device=DEV), torch.zeros(1, 500, device=DEV)
    B.ridgefill_attention_weight(kv, pools[0], q, starts, 5, 0.1, lse, a, wws)
    skv = small.batch(B)
    B.ridgefill_attention_weight(skv, small.k[0], q, starts, 5, 0.1, lse, b, wws)
    assert torch.equal(a, b)
    rows = torch.tensor([3, 499], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    new = _randn(2, 2, n_kv, hd)
    B.ridgefill_append_rows(None, kv, new, new, rows, pools[0], pools[1], status)
    assert torch.equal(pools[1][table[0, 0], 3], new[0]) and torch.equal(pools[1][table[0, 31], 3], new[1])
    # and an eviction that moves its last row to its first place
    acc = torch.ones(1, 500, device=DEV)
    acc[0, 0] = 0
    pos = torch.arange(500, dtype=torch.int32, device=DEV)[None].contiguous()
    ews = torch.empty(B.ridgefill_evict_workspace_bytes(kv, 499), dtype=torch.uint8, device=DEV)
    B.ridgefill_evict_rows(kv, B.make_pools(pools[:1], pools[1:]), acc, pos, 499, acc, pos, small.lengths, ews)
    assert B.ridgefill_read_status(ews) == B.RF_OK
    assert torch.equal(pools[0][table[0, 0], 0], new[1]) and int(pos[0, 0]) == 499


# --------------------------------------------------------------------------------- weight

@pytest.mark.parametrize("lens,counts,heads,n_kv,hd,page,tree", ATTEND)
def test_weight(lens, counts, heads, n_kv, hd, page, tree):
    cache, q, starts, words, max_q = _case(lens, counts, heads, n_kv, hd, page, seed=len(lens) + hd + page, tree=tree)
    scale = hd ** -0.5
    _, lse, _ = _attend(cache, q, starts, words, max_q, scale)
    kv = cache.batch(B)
    ws = torch.full((B.ridgefill_attention_weight_workspace_bytes(kv, heads, max_q),), 0xff, dtype=torch.uint8, device=DEV)
    start = torch.tensor(starts, dtype=torch.int32, device=DEV)
    acc0 = torch.rand(len(lens), cache.max_len + 5, generator=torch.Generator().manual_seed(1)).to(DEV)
    for acc, decay in ((acc0, 0.75), (None, 1.0), (acc0, 1.0)):
        out = torch.full_like(acc0, -7.0)
        B.ridgefill_attention_weight(kv, cache.k[0], q, start, max_q, scale, lse, out, ws, acc=acc, decay=decay,
                                     tree_mask=_mask(words))
        assert B.ridgefill_read_status(ws) == B.RF_OK
        want, tol = R.weight(cache, q, starts, words, scale, lse, decay, acc, torch.full_like(acc0, -7.0))
        _close(out, want, tol, f"decay {decay}")
        again = torch.full_like(acc0, -7.0)
        B.ridgefill_attention_weight(kv, cache.k[0], q, start, max_q, scale, lse, again, ws, acc=acc, decay=decay,
                                     tree_mask=_mask(words))
        assert torch.equal(again, out)                   # the same sums in the same order
    inplace = acc0.clone()
    B.ridgefill_attention_weight(kv, cache.k[0], q, start, max_q, scale, lse, inplace, ws, acc=inplace,
                                 tree_mask=_mask(words))
    inside = torch.arange(acc0.shape[1], device=DEV)[None] < cache.lengths[:, None]
    inside &= (start[1:] > start[:-1])[:, None]
    assert torch.equal(torch.where(inside, inplace, out), out)


def test_weight_of_empty_rows_and_hidden_values():
    cache, q, starts, words, max_q = _case([8], [8], 2, 1, 64, 4, seed=2, tree=True)
    words[0] = 0
    for i in range(8):
        words[i] &= ~np.uint64(1 << 5)                    # nobody sees draft 5
    cache.k[0][int(cache.table_np[0, 1]), 1] = float("nan")
    _, lse, _ = _attend(cache, q, starts, words, max_q, 0.1)
    kv = cache.batch(B)
    ws = torch.empty(B.ridgefill_attention_weight_workspace_bytes(kv, 2, max_q), dtype=torch.uint8, device=DEV)
    out = torch.empty(1, 8, device=DEV)
    B.ridgefill_attention_weight(kv, cache.k[0], q, torch.tensor(starts, dtype=torch.int32, device=DEV), max_q, 0.1, lse,
                                 out, ws, tree_mask=_mask(words))
    assert float(out[0, 5]) == 0 and torch.isfinite(out).all()
    # every other query spreads a weight of one over the rows it sees, for each head
    seeing = sum(1 for w in words if int(w))
    assert abs(float(out.double().sum()) - 2 * seeing) <= 2 * seeing * 2.0 ** -18


def test_weight_bad_sequences():
    cache, q, starts, words, max_q = _case([50, 50], [2, 2], 4, 2, 64, 16, seed=3)
    _, lse, _ = _attend(cache, q, starts, words, max_q, 0.1)
    kv = cache.batch(B, torch.tensor([51, 50], dtype=torch.int32, device=DEV))
    ws = torch.empty(B.ridgefill_attention_weight_workspace_bytes(kv, 4, max_q), dtype=torch.uint8, device=DEV)
    out = torch.full((2, 50), -7.0, device=DEV)
    start = torch.tensor(starts, dtype=torch.int32, device=DEV)
    B.ridgefill_attention_weight(kv, cache.k[0], q, start, max_q, 0.1, lse, out, ws)
    assert B.ridgefill_read_status(ws) == B.RF_E_ROWS
    assert (out[0] == -7).all() and (out[1] >= 0).all()
    cache.table[1, 1] = -3
    B.ridgefill_attention_weight(cache.batch(B), cache.k[0], q, start, max_q, 0.1, lse, out, ws)
    assert B.ridgefill_read_status(ws) == B.RF_E_ROWS
    assert (out[1, 16:32] == 0).all() and (out[1, :16] > 0).all()


# ------------------------------------------------------------------------------- eviction

def _evict(cache, acc, pos, keep, sink, recent, in_place=False, pools=None, lengths=None):
    kv = cache.batch(B) if lengths is None else cache.batch(B, lengths)
    ws = torch.full((B.ridgefill_evict_workspace_bytes(kv, keep),), 0xff, dtype=torch.uint8, device=DEV)
    a, p = acc.to(DEV), pos.to(DEV)
    if in_place:
        ao, po, lo = a, p, kv._keep[1]
    else:
        ao, po, lo = torch.full_like(a, -7.0), torch.full_like(p, -7), torch.full_like(cache.lengths, -7)
    layers = B.make_pools(*(pools or (cache.k, cache.v)))
    B.ridgefill_evict_rows(kv, layers, a, p, keep, ao, po, lo, ws, n_sink=sink, n_recent=recent)
    return ao.cpu(), po.cpu(), lo.cpu(), B.ridgefill_read_status(ws)


def _check_evict(cache, acc, pos, keep, sink, recent, in_place=False, status=B.RF_OK):
    lens = list(cache.lens)
    moves, holds = R.evict(lens, acc.numpy(), pos.numpy(), keep, sink, recent)
    old = [(cache.rows(p, b), p.clone()) for p in cache.k + cache.v for b in range(len(lens))]
    ao, po, lo, st = _evict(cache, acc, pos, keep, sink, recent, in_place)
    assert st == status
    for b, n in enumerate(lens):
        m = min(n, keep)
        assert int(lo[b]) == m
        assert torch.equal(ao[b, :m].view(torch.int32), acc[b, holds[b]].view(torch.int32))
        assert torch.equal(po[b, :m], pos[b, holds[b]])
        assert (ao[b, m:n] == 0).all()
        rest = acc[b, n:] if in_place else torch.full_like(acc[b, n:], -7.0)
        assert torch.equal(ao[b, n:].view(torch.int32), rest.view(torch.int32))
        assert torch.equal(po[b, m:], pos[b, m:] if in_place else torch.full_like(pos[b, m:], -7))
    i = 0
    for p in cache.k + cache.v:
        for b, n in enumerate(lens):
            rows, before = old[i]
            i += 1
            m = min(n, keep)
            assert torch.equal(cache.rows(p, b, m), rows[holds[b]])
        new, want = p.view(torch.int16).clone(), before.view(torch.int16)
        for b in range(len(lens)):                       # only the free places are written
            for _, t in moves[b]:
                at = int(cache.table_np[b, t // cache.page]), t % cache.page
                new[at] = want[at]
        assert torch.equal(new, want)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,page,n_kv,hd,keep,sink,recent", [
    ([20, 7, 0, 8, 64], 4, 2, 64, 8, 2, 3), ([1500, 1030], 16, 1, 128, 1024, 4, 100),
    ([70], 7, 3, 64, 69, 0, 0), ([33, 40], 1, 1, 16, 1, 0, 1), ([130], 100, 2, 128, 0, 0, 0),
    ([5, 6], 4, 1, 64, 200, 1, 1), ([3000], 12, 1, 64, 1500, 0, 0), ([40], 8, 1, 64, 10, 30, 30)])
def test_evict(lens, page, n_kv, hd, keep, sink, recent, in_place):
    cache = R.Cache(lens, n_kv, hd, page, seed=sum(lens), pools=2)
    g = torch.Generator().manual_seed(keep)
    shape = (len(lens), cache.max_len + 3)
    acc = torch.randint(0, 12, shape, generator=g).float() / 4       # many ties
    pos = torch.stack([torch.randperm(shape[1], generator=g) for _ in lens]).to(torch.int32)
    _check_evict(cache, acc, pos, keep, sink, recent, in_place)


def test_evict_special_weights():
    cache = R.Cache([64], 1, 64, 8, seed=1)
    acc = torch.linspace(-1, 1, 64)[None].contiguous()
    acc[0, 3], acc[0, 60], acc[0, 9], acc[0, 11] = float("inf"), float("inf"), -float("inf"), -0.0
    acc[0, 13], acc[0, 50] = 0.0, -1e-42
    pos = torch.arange(64, dtype=torch.int32)[None].contiguous()
    _check_evict(cache, acc, pos, 30, 1, 2)
    cache = R.Cache([64], 1, 64, 8, seed=1)
    acc[0, [5, 40, 63]] = float("nan")                    # the last one is protected all the same
    _check_evict(cache, acc, pos, 62, 1, 2, status=B.RF_E_INVALID)


def test_evict_all_equal_keeps_the_lowest_rows():
    cache = R.Cache([5000], 1, 16, 16, seed=2)
    acc = torch.full((1, 5000), 0.25)
    pos = torch.arange(5000, dtype=torch.int32)[None].contiguous()
    _check_evict(cache, acc, pos, 1234, 0, 0)


def test_evict_many_pools():
    cache = R.Cache([50], 1, 64, 8, seed=3, pools=70)     # more pools than one launch takes
    acc = torch.rand(1, 50, generator=torch.Generator().manual_seed(0))
    pos = torch.arange(50, dtype=torch.int32)[None].contiguous()
    _check_evict(cache, acc, pos, 20, 2, 4)


def test_evict_without_layers():
    cache = R.Cache([50], 1, 64, 8, seed=3)
    acc = torch.rand(1, 50, generator=torch.Generator().manual_seed(0))
    pos = torch.arange(50, dtype=torch.int32)[None].contiguous()
    ao, po, lo, st = _evict(cache, acc, pos, 20, 2, 4, pools=([], []))
    _, holds = R.evict([50], acc.numpy(), pos.numpy(), 20, 2, 4)
    assert st == B.RF_OK and torch.equal(po[0, :20], pos[0, holds[0]]) and int(lo[0]) == 20


def test_evict_bad_lengths_and_pages():
    cache = R.Cache([40, 40], 1, 64, 8, seed=4)
    acc = torch.rand(2, 40, generator=torch.Generator().manual_seed(0))
    pos = torch.arange(40, dtype=torch.int32).repeat(2, 1).contiguous()
    old = cache.k[0].clone()
    ao, po, lo, st = _evict(cache, acc, pos, 20, 0, 0, lengths=torch.tensor([41, -1], dtype=torch.int32, device=DEV))
    assert st == B.RF_E_ROWS
    assert (ao == -7).all() and (po == -7).all() and (lo == -7).all()
    assert torch.equal(cache.k[0].view(torch.int16), old.view(torch.int16))
    cache.table[0, 4] = -1                                # rows 32..39 of sequence 0
    ao, po, lo, st = _evict(cache, acc, pos, 20, 0, 0)
    assert st == B.RF_E_ROWS and lo.tolist() == [20, 20]
    moves, _ = R.evict([40, 40], acc.numpy(), pos.numpy(), 20, 0, 0)
    changed = {tuple(x) for x in (cache.k[0].view(torch.int16) != old.view(torch.int16)).flatten(2).any(-1).nonzero().tolist()}
    assert changed == {(int(cache.table_np[b, t // 8]), t % 8) for b in (0, 1) for f, t in moves[b] if b or f < 32}


# ----------------------------------------------------------------- graphs, streams, devices

def test_captured_step_replays_with_new_lengths():
    """One serving step (append, attention, weight, eviction) captured once; each replay, with
    new rows and lengths and eager work between, equals the eager step."""
    lens = [70, 33]
    n_kv, heads, hd, page, keep = 2, 8, 128, 16, 64
    cache = R.Cache(lens, n_kv, hd, page, max_len=96, seed=5)
    max_len = 96
    kv = cache.batch(B)
    qkv = _randn(1, 2, heads + 2 * n_kv, hd)
    rows, seq = torch.zeros(2, dtype=torch.int32, device=DEV), torch.arange(2, dtype=torch.int32, device=DEV)
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out, out = torch.empty(2, heads, hd, dtype=torch.bfloat16, device=DEV), torch.empty(2, heads, hd, dtype=torch.bfloat16, device=DEV)
    lse, acc = torch.empty(2, heads, device=DEV), torch.zeros(2, max_len, device=DEV)
    pos = torch.zeros(2, max_len, dtype=torch.int32, device=DEV)
    rope, layers = B.make_rope(), B.make_pools(cache.k, cache.v)
    ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in (
        B.ridgefill_tree_attention_workspace_bytes(kv, heads, 1), B.ridgefill_attention_weight_workspace_bytes(kv, heads, 1),
        B.ridgefill_evict_workspace_bytes(kv, keep))]

    def step():
        B.ridgefill_append_rows(rope, kv, qkv[:, heads:heads + n_kv], qkv[:, heads + n_kv:], rows, cache.k[0], cache.v[0],
                                status, seq=seq, q=qkv[:, :heads], q_out=q_out)
        B.ridgefill_tree_attention(kv, cache.k[0], cache.v[0], q_out, start, 1, 0.1, out, ws[0], lse=lse)
        B.ridgefill_attention_weight(kv, cache.k[0], q_out, start, 1, 0.1, lse, acc, ws[1], acc=acc, decay=0.9)
        B.ridgefill_evict_rows(kv, layers, acc, pos, keep, acc, pos, cache.lengths, ws[2], n_sink=2, n_recent=8)

    state = [cache.k[0], cache.v[0], acc, pos, cache.lengths, out, lse]
    first = [t.clone() for t in state]

    def setup(i):
        for t, f in zip(state, first):
            t.copy_(f)
        qkv.copy_(_randn(20 + i, 2, heads + 2 * n_kv, hd))
        cache.lengths.copy_(torch.tensor([lens[0] - i, lens[1] + 0 * i], dtype=torch.int32))
        rows.copy_(cache.lengths - 1)
        acc.copy_(torch.rand(2, max_len, generator=torch.Generator().manual_seed(i)))
        pos.copy_(torch.arange(max_len, dtype=torch.int32).repeat(2, 1))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        setup(0)
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    torch.cuda.synchronize()
    other = torch.randn(1 << 18, device=DEV)
    for i in range(4):
        setup(i)
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in state]
        other.mul_(1.5).add_(0.25)
        setup(i)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for w in ws:
            assert B.ridgefill_read_status(w) == B.RF_OK
        assert B.ridgefill_read_status(status) == B.RF_OK
        for a, b in zip(state, want):
            assert torch.equal(a.view(torch.int16) if a.dtype == torch.bfloat16 else a,
                               b.view(torch.int16) if b.dtype == torch.bfloat16 else b), i
    del graph


def test_captured_eviction_of_a_long_cache():
    # more keys than a launch's LDS unasked
    n = 20000
    cache = R.Cache([n], 1, 16, 100, seed=7)
    acc0 = torch.rand(1, n, generator=torch.Generator().manual_seed(0))
    pos0 = torch.randperm(n, generator=torch.Generator().manual_seed(1))[None].to(torch.int32)
    acc, pos, kv = acc0.to(DEV), pos0.to(DEV), cache.batch(B)
    pools, layers = (cache.k[0].clone(), cache.v[0].clone()), B.make_pools(cache.k, cache.v)
    ws = torch.empty(B.ridgefill_evict_workspace_bytes(kv, 9000), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        B.ridgefill_evict_rows(kv, layers, acc, pos, 9000, acc, pos, cache.lengths, ws, n_sink=3, n_recent=10)
    moves, holds = R.evict([n], acc0.numpy(), pos0.numpy(), 9000, 3, 10)
    want = R.Cache.rows(cache, pools[0], 0)[holds[0]]
    for _ in range(2):
        acc.copy_(acc0)
        pos.copy_(pos0)
        cache.lengths.fill_(n)
        cache.k[0].copy_(pools[0])
        cache.v[0].copy_(pools[1])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert B.ridgefill_read_status(ws) == B.RF_OK and int(cache.lengths) == 9000
        assert pos[0, :9000].tolist() == pos0[0, holds[0]].tolist()
        assert torch.equal(cache.rows(cache.k[0], 0, 9000), want)
    del graph


@pytest.mark.parametrize("n", [32768, 33000, 70001])
def test_evict_long(n):
    # as many rows as LDS holds, and more: the order is kept in pieces
    g = torch.Generator().manual_seed(n)
    acc = torch.randint(0, 300, (1, n), generator=g).float()
    pos = torch.arange(n, dtype=torch.int32)[None].contiguous()
    _check_evict(R.Cache([n], 1, 16, 64, seed=1), acc, pos, n // 3, 4, 64)


def test_nothing_to_do():
    cache = R.Cache([40, 9], 2, 64, 16, seed=1)
    kv = cache.batch(B)
    q, lse = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV), torch.empty(0, 4, device=DEV)
    start, acc = torch.zeros(3, dtype=torch.int32, device=DEV), torch.full((2, 40), 2.0, device=DEV)
    ws = torch.empty(B.ridgefill_tree_attention_workspace_bytes(kv, 4, 8), dtype=torch.uint8, device=DEV)
    B.ridgefill_tree_attention(kv, cache.k[0], cache.v[0], q, start, 8, 0.1, torch.empty_like(q), ws, lse=lse)
    assert B.ridgefill_read_status(ws) == B.RF_OK
    ws = torch.empty(B.ridgefill_attention_weight_workspace_bytes(kv, 4, 8), dtype=torch.uint8, device=DEV)
    B.ridgefill_attention_weight(kv, cache.k[0], q, start, 8, 0.1, lse, acc, ws, acc=acc, decay=0.5)
    assert B.ridgefill_read_status(ws) == B.RF_OK and (acc == 2).all()
    status = torch.full((1,), -1, dtype=torch.int32, device=DEV)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    B.ridgefill_append_rows(B.make_rope(), kv, none, none, torch.empty(0, dtype=torch.int32, device=DEV), cache.k[0],
                            cache.v[0], status)
    assert B.ridgefill_read_status(status) == B.RF_OK


def test_many_sequences_of_all_lengths():
    # more sequences than lanes, split unevenly, some without queries
    lens = [int(x) for x in np.random.default_rng(5).integers(0, 700, 150)]
    counts = [min(n, (3 * b) % 4) for b, n in enumerate(lens)]
    cache, q, starts, words, _ = _case(lens, counts, 2, 1, 64, 16, seed=15, tree=True, max_q=5)
    for max_q in (5, 12):                                 # both kernels
        out, lse, st = _attend(cache, q, starts, words, max_q, 0.1, n_pad=1)
        assert st == B.RF_OK
        want, wl, ot, lt = R.attention(cache, q, starts, words, 0.1)
        n = q.shape[0]
        _close(out[:n], want, ot, "out")
        _close(lse[:n], wl, lt, "lse")
        kv = cache.batch(B)
        ws = torch.empty(B.ridgefill_attention_weight_workspace_bytes(kv, 2, max_q), dtype=torch.uint8, device=DEV)
        acc = torch.full((150, cache.max_len), -7.0, device=DEV)
        B.ridgefill_attention_weight(kv, cache.k[0], q, torch.tensor(starts, dtype=torch.int32, device=DEV), max_q, 0.1,
                                     lse[:n].contiguous(), acc, ws, tree_mask=_mask(words))
        assert B.ridgefill_read_status(ws) == B.RF_OK
        want, tol = R.weight(cache, q, starts, words, 0.1, lse[:n], 1.0, None, torch.full_like(acc, -7.0))
        _close(acc, want, tol, "weight")


def test_two_calls_on_two_streams():
    a, b = (_case([2000, 300], [4, 9], 8, 2, 128, 16, seed=s, tree=True) for s in (21, 22))
    want = [_attend(*c[:4], c[4], 0.1)[0] for c in (a, b)]
    got, keep = [], []
    torch.cuda.synchronize()
    for c in (a, b):
        s = torch.cuda.Stream()
        kv = c[0].batch(B)
        ws = torch.empty(B.ridgefill_tree_attention_workspace_bytes(kv, 8, c[4]), dtype=torch.uint8, device=DEV)
        start, mask, out = torch.tensor(c[2], dtype=torch.int32, device=DEV), _mask(c[3]), torch.empty_like(c[1])
        torch.cuda.synchronize()
        keep.append((s, kv, ws, start, mask))
        got.append(out)
    for _ in range(5):
        for c, out, (s, kv, ws, start, mask) in zip((a, b), got, keep):
            B.ridgefill_tree_attention(kv, c[0].k[0], c[0].v[0], c[1], start, c[4], 0.1, out, ws, tree_mask=mask, stream=s)
    torch.cuda.synchronize()
    for out, w in zip(got, want):
        assert torch.equal(out, w)


@pytest.mark.parametrize("heads,runs", [(2, 2 ** 17), (32, 2 ** 20)])
def test_longest_cache(heads, runs):
    # 2^30 rows: one page of 2^16, over and over.  runs: how many additions follow one another in one
    # lane (2^30 rows over 1,024 parts of 16 lanes; over 256 parts of two waves, a lane half of each).
    page, times = 2 ** 16, 2 ** 14
    cache = R.Cache([page], 1, 64, page, spare=0, seed=3)
    cache.v[0].add_(1.0)
    q = _randn(2, 1, heads, 64)
    table = torch.zeros(1, times, dtype=torch.int32, device=DEV)
    table.fill_(int(cache.table_np[0, 0]))
    length = torch.tensor([page * times], dtype=torch.int32, device=DEV)
    kv = B.make_batch(table, length, page, 1, 1, 64)
    start = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(1, heads, device=DEV)
    ws = torch.empty(B.ridgefill_tree_attention_workspace_bytes(kv, heads, 1), dtype=torch.uint8, device=DEV)
    B.ridgefill_tree_attention(kv, cache.k[0], cache.v[0], q, start, 1, 0.1, out, ws, lse=lse)
    assert B.ridgefill_read_status(ws) == B.RF_OK
    want, wl, ot, lt = R.attention(cache, q, [0, 1], None, 0.1)
    # the oracle counts one addition a row of the page
    more = 2 * (runs - page) * R.U_FP32 if runs > page else 0.0
    _close(out, want, ot + more * (1 + want.abs()) * 2, "out")
    _close(lse, wl + np.log(times), lt + more + 8 * R.U_FP32 * np.log(times), "lse")


def test_longest_weight():
    page, times = 2 ** 16, 2 ** 13
    cache = R.Cache([page], 1, 64, page, spare=0, seed=4)
    q, lse = _randn(2, 1, 2, 64), torch.full((1, 2), 3.0, device=DEV)
    table = torch.zeros(1, times, dtype=torch.int32, device=DEV)
    table.fill_(int(cache.table_np[0, 0]))
    length = torch.tensor([page * times], dtype=torch.int32, device=DEV)
    kv = B.make_batch(table, length, page, 1, 1, 64)
    acc = torch.full((1, page * times), -1.0, device=DEV)
    ws = torch.empty(B.ridgefill_attention_weight_workspace_bytes(kv, 2, 1), dtype=torch.uint8, device=DEV)
    B.ridgefill_attention_weight(kv, cache.k[0], q, torch.tensor([0, 1], dtype=torch.int32, device=DEV), 1, 0.1, lse, acc, ws)
    assert B.ridgefill_read_status(ws) == B.RF_OK
    acc = acc.view(times, page)
    want, tol = R.weight(cache, q, [0, 1], None, 0.1, lse, 1.0, None, acc[:1].clone())
    _close(acc[:1], want, tol, "weight")
    assert bool((acc == acc[:1]).all())


def test_another_stream():
    cache, q, starts, words, max_q = _case([3000], [5], 8, 2, 128, 16, seed=6, tree=True)
    ref, ref_lse, _ = _attend(cache, q, starts, words, max_q, 0.1)
    kv, side = cache.batch(B), torch.cuda.Stream()
    ws = torch.empty(B.ridgefill_tree_attention_workspace_bytes(kv, 8, max_q), dtype=torch.uint8, device=DEV)
    out, lse, start, mask = torch.empty_like(ref), torch.empty_like(ref_lse), torch.tensor(starts, dtype=torch.int32, device=DEV), _mask(words)
    torch.cuda.synchronize()
    B.ridgefill_tree_attention(kv, cache.k[0], cache.v[0], q, start, max_q, 0.1, out, ws, lse=lse, tree_mask=mask, stream=side)
    assert B.ridgefill_read_status(ws, stream=side) == B.RF_OK
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


# ------------------------------------------------------------------------- the run together

def test_fill_append_attend_select_and_evict_together():
    """A prompt filled by the library, its exact and tail rows appended, drafts attended, the
    weights of the last tokens ranked by the row selection, the cache cut, and the attention
    after the cut equal to attention over the kept rows."""
    from fillcase import Case, build_inputs, run_fill
    import oracle
    N, T, d, n_kv, hd, heads, page = 260, 40, 512, 2, 128, 8, 16
    exact = np.arange(3, N - T, 9)
    case = Case(d=d, n_layers=1, n_kv=n_kv, hd=hd, N=N, T=T, exact=exact, page_size=page, seed=30)
    inp = build_inputs(case)
    filled, _, _ = oracle.partition(N, T, exact)
    assert run_fill(case, inp, filled) == B.RF_OK
    layer = inp["layers"][0]
    kp, vp = layer["k_pages"], layer["v_pages"]
    rest = np.setdiff1d(np.arange(N), filled).astype(np.int32)          # exact and tail rows
    k, v, q = _randn(1, len(rest), n_kv, hd), _randn(2, len(rest), n_kv, hd), _randn(3, len(rest), heads, hd)
    lengths = torch.tensor([N], dtype=torch.int32, device=DEV)
    table = inp["table"][None, :].contiguous()
    kv = B.make_batch(table, lengths, page, inp["num_pages"], n_kv, hd, N)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = torch.empty_like(q)
    rope = B.make_rope(theta=case.theta)
    B.ridgefill_append_rows(rope, kv, k, v, torch.from_numpy(rest).to(DEV), kp, vp, status, q=q, q_out=q_out)
    assert B.ridgefill_read_status(status) == B.RF_OK

    class View(R.Cache):
        def __init__(self, n):
            self.lens, self.n_kv, self.hd, self.page, self.max_len = [n], n_kv, hd, page, N
            self.table_np, self.k, self.v = table.cpu().numpy(), [kp], [vp]
    last = q_out[-32:].contiguous()                       # the last 32 tokens of the prompt
    start = torch.tensor([0, 32], dtype=torch.int32, device=DEV)
    ws = torch.empty(B.ridgefill_tree_attention_workspace_bytes(kv, heads, 32), dtype=torch.uint8, device=DEV)
    wws = torch.empty(B.ridgefill_attention_weight_workspace_bytes(kv, heads, 32), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(last), torch.empty(32, heads, device=DEV)
    scale = hd ** -0.5
    B.ridgefill_tree_attention(kv, kp, vp, last, start, 32, scale, out, ws, lse=lse)
    want, wl, ot, lt = R.attention(View(N), last, [0, 32], None, scale)
    _close(out, want, ot, "out")
    _close(lse, wl, lt, "lse")
    acc = torch.zeros(1, N, device=DEV)
    B.ridgefill_attention_weight(kv, kp, last, start, 32, scale, lse, acc, wws)
    want, tol = R.weight(View(N), last, [0, 32], None, scale, lse, 1.0, None, acc)
    _close(acc, want, tol, "weights")
    P, keep_rows = N - T, 22                               # the weights are selection scores
    sws = torch.empty(B.ridgefill_select_workspace_bytes(P), dtype=torch.uint8, device=DEV)
    chosen = torch.empty(P, dtype=torch.uint8, device=DEV)
    left = torch.empty(P - keep_rows, dtype=torch.int32, device=DEV)
    B.ridgefill_select_rows(acc[0, :P].contiguous(), keep_rows, left, sws, exact_mask=chosen)
    assert B.ridgefill_read_status(sws) == B.RF_OK
    assert sorted(np.flatnonzero(chosen.cpu().numpy())) == sorted(oracle.select_exact(acc[0, :P].cpu().double().numpy(), keep_rows))
    keep = 150
    pos = torch.arange(N, dtype=torch.int32, device=DEV)[None].contiguous()
    ews = torch.empty(B.ridgefill_evict_workspace_bytes(kv, keep), dtype=torch.uint8, device=DEV)
    _, holds = R.evict([N], acc.cpu().numpy(), pos.cpu().numpy(), keep, 4, 32)
    before = View(N).rows(kp, 0)
    B.ridgefill_evict_rows(kv, [layer], acc, pos, keep, acc, pos, lengths, ews, n_sink=4, n_recent=32)
    assert B.ridgefill_read_status(ews) == B.RF_OK
    assert pos[0, :keep].tolist() == holds[0] and int(lengths) == keep
    assert torch.equal(View(keep).rows(kp, 0), before[holds[0]])
    # a tree of drafts goes behind the kept rows, at its own positions, and sees them all
    drafts = 5
    words = R.trees([drafts], 3)
    nk, nv, nq = _randn(4, drafts, n_kv, hd), _randn(5, drafts, n_kv, hd), _randn(6, drafts, heads, hd)
    depth = torch.tensor([N + bin(int(w)).count("1") - 1 for w in words], dtype=torch.int32, device=DEV)
    B.ridgefill_append_rows(rope, kv, nk, nv, torch.arange(keep, keep + drafts, dtype=torch.int32, device=DEV), kp, vp,
                            status, positions=depth, q=nq, q_out=nq)
    lengths += drafts
    start = torch.tensor([0, drafts], dtype=torch.int32, device=DEV)
    out = torch.empty_like(nq)
    B.ridgefill_tree_attention(kv, kp, vp, nq, start, drafts, scale, out, ws, tree_mask=_mask(words))
    assert B.ridgefill_read_status(ws) == B.RF_OK
    want, _, ot, _ = R.attention(View(keep + drafts), nq, [0, drafts], words, scale)
    _close(out, want, ot, "after the cut")
