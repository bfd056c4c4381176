"""GPU parity of the attention over caches of 16 and 8 bits and of sequences that share prefixes,
against a plain 64-bit implementation (sharedcase.py), by kernel form: up to 16, 128 or 256 query rows
of a key head, for a sequence's own rows and for its prefix's, whole or split."""

import math

import numpy as np
import pytest
import torch

import cachecase as R
import heldcase as H
import sharedcase as S
from test_gpu_cache import _close, _mask, _randn
from ridge_map_kv_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"

# own lengths, queries, prefix lengths, group starts, heads, n_kv, hd, page, trees
CASES = {
    "one token each, prefix in registers": ([9, 4, 1], [1, 1, 1], [29], [0, 3], 4, 2, 64, 4, False),
    "one token each, prefix split": ([40, 7], [1, 1], [700], [0, 2], 8, 2, 128, 16, False),
    "three prefixes, one empty, two sequences without": ([5, 30, 64, 65, 2, 9], [1, 2, 1, 3, 1, 2], [65, 0, 300], [0, 2, 3, 4], 4, 2, 64, 5, True),
    "groups without sequences or queries": ([20, 33, 8], [0, 2, 0], [10, 40, 50, 7], [0, 1, 1, 3, 3], 2, 2, 128, 16, True),
    "128 rows of a prefix, tokens in registers": ([3, 17, 100, 9, 31, 60, 2, 8, 77, 40], [1] * 10, [200], [0, 10], 8, 1, 64, 7, False),
    "128 rows of both": ([25, 40, 33], [20, 7, 15], [150], [0, 3], 4, 2, 128, 16, True),
    "256 rows of a prefix, 128 own": ([40, 30, 25, 33, 60, 20, 48, 30], [24, 20, 24, 8, 24, 20, 16, 24], [333], [0, 8], 4, 2, 64, 16, True),
    "256 rows of both, blocks": ([70, 64, 90], [64, 64, 40], [129], [0, 3], 10, 2, 128, 12, True),
    "blocks of 16 rows of a prefix": ([3] * 12, [1] * 12, [31], [0, 12], 5, 1, 128, 16, False),
    "a prefix of one row": ([2, 1], [1, 1], [1], [0, 2], 3, 3, 64, 1, False),
    "no prefix, one token": ([1, 300, 33, 0], [1, 1, 1, 0], [], [0], 8, 2, 128, 16, False),
    "no prefix, split": ([900, 70], [1, 1], [], [0], 4, 1, 64, 9, False),
    "no prefix, 128 rows": ([90, 20], [30, 17], [], [0], 4, 1, 64, 16, True),
    "no prefix, 128 rows, split": ([400, 129], [30, 64], [], [0], 4, 2, 128, 16, True),
    "no prefix, 256 rows": ([64, 100, 70], [64, 40, 11], [], [0], 16, 4, 128, 3, True),
    "no prefix, 320 rows, split": ([300], [64], [], [0], 10, 2, 128, 100, True),
    "four key heads a workgroup, split": ([900, 70, 3], [1, 1, 1], [], [0], 8, 4, 128, 16, False),
    "eight key heads, prefix in registers": ([20, 9], [2, 1], [700], [0, 2], 16, 8, 64, 16, True),
    "more parts than four waves join": ([20000], [1], [], [0], 4, 4, 64, 16, False),
    "many rows of many parts": ([64] * 9, [64] * 9, [2600], [0, 9], 4, 1, 64, 16, True),
    "more rows of a workgroup than slots looked up at a time": ([5000] + [1] * 31, [48] + [1] * 31, [], [0], 24, 8, 64, 16, True),
    "key heads that are no power of two": ([50, 20, 9, 30], [3, 1, 2, 9], [90, 200], [0, 2, 4], 6, 3, 128, 16, True),
}


def _make(case, kind, seed=0, **kw):
    lens, counts, plens, groups, heads, n_kv, hd, page, tree = case
    c = S.SharedCache(lens, plens, groups, n_kv, hd, page, kind, seed, **kw)
    starts = S.starts_of(counts)
    q = _randn(seed + 7, starts[-1], heads, hd)
    return c, q, starts, R.trees(counts, seed) if tree else None, max(max(counts), 1)


def _attend(c, q, starts, words, max_q, scale, cache=None, want_out=True, want_lse=True, n_pad=0, prefix=True, kv=None):
    n, heads, hd = q.shape
    kv = kv or c.kv(B)
    pre = (c.prefix(B) if prefix is True else prefix) or None
    out = torch.full((n + n_pad, heads, hd), 3.0, dtype=torch.bfloat16, device=DEV) if want_out else None
    lse = torch.full((n + n_pad, heads), 3.0, device=DEV) if want_lse else None
    qp = torch.cat([q, torch.full((n_pad, heads, hd), float("nan"), dtype=q.dtype, device=DEV)])
    if words is not None and n_pad:
        words = np.concatenate([words, np.zeros(n_pad, np.uint64)])
    need = B.ridgefill_cache_attention_workspace_bytes(kv, heads, max_q, n + n_pad, pre)
    ws = torch.full((need + 4096,), 0xff, dtype=torch.uint8, device=DEV)
    B.ridgefill_cache_attention(kv, cache or c.cache(B), qp, torch.tensor(starts, dtype=torch.int32, device=DEV), max_q, scale, out,
                                ws[:need], prefix=pre, lse=lse, tree_mask=_mask(words))
    assert (ws[need:] == 0xff).all()                      # nothing behind the workspace is touched
    return out, lse, B.ridgefill_read_status(ws)


def _check(c, q, starts, words, max_q, scale, out, lse, gone=(), which=None):
    want, wl, ot, lt = S.attention(c, q, starts, words, scale, gone)
    which = list(range(q.shape[0])) if which is None else which
    if out is not None:
        _close(out[which], want[which], ot[which], "out")
    _close(lse[which], wl[which], lt[which], "lse")


@pytest.mark.parametrize("kind", H.KINDS)
@pytest.mark.parametrize("name", CASES)
def test_cache_attention(name, kind):
    c, q, starts, words, max_q = _make(CASES[name], kind, seed=len(name))
    scale, n = c.hd ** -0.5, q.shape[0]
    out, lse, st = _attend(c, q, starts, words, max_q, scale, n_pad=3)
    assert st == B.RF_OK
    _check(c, q, starts, words, max_q, scale, out[:n], lse[:n])
    assert (out[n:] == 3).all() and (lse[n:] == 3).all()   # padded queries stay as they were
    again, lse2, _ = _attend(c, q, starts, words, max_q, scale, n_pad=3)
    assert torch.equal(again, out) and torch.equal(lse2, lse)
    only, _, _ = _attend(c, q, starts, words, max_q, scale, want_lse=False, n_pad=3)
    assert torch.equal(only, out)
    _, only, st = _attend(c, q, starts, words, max_q, scale, want_out=False, cache=B.make_cache(c.kp, None, c.ks))
    assert st == B.RF_OK
    _check(c, q, starts, words, max_q, scale, None, only)


@pytest.mark.parametrize("kind", ["fp8", "int8"])
@pytest.mark.parametrize("name", CASES)
def test_codes_give_what_their_values_give(name, kind):
    # the same operands of the same products: kernels of more than 16 query rows give the same bits, those of up to
    # 16 cut the rows into other parts, so that each may be off by its own tolerance
    c, q, starts, words, max_q = _make(CASES[name], kind, seed=2)
    got = _attend(c, q, starts, words, max_q, 0.1)
    want = _attend(c, q, starts, words, max_q, 0.1, cache=c.values(B))
    group = q.shape[1] // c.n_kv
    if max_q * group > 16 and (not c.plens or starts[-1] * group > 64):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    else:
        _, _, ot, lt = S.attention(c, q, starts, words, 0.1)
        _close(got[0], want[0].cpu().double(), 2 * ot, "out")
        _close(got[1], want[1].cpu().double(), 2 * lt, "lse")


@pytest.mark.parametrize("name", [n for n in CASES if n.startswith("no prefix")])
def test_bf16_without_prefix_is_tree_attention(name):
    c, q, starts, words, max_q = _make(CASES[name], "bf16", seed=3)
    out, lse, st = _attend(c, q, starts, words, max_q, 0.1)
    kv, out2, lse2 = c.kv(B), torch.full_like(out, 3.0), torch.full_like(lse, 3.0)
    ws = torch.empty(B.ridgefill_tree_attention_workspace_bytes(kv, q.shape[1], max_q), dtype=torch.uint8, device=DEV)
    B.ridgefill_tree_attention(kv, c.kp, c.vp, q, torch.tensor(starts, dtype=torch.int32, device=DEV), max_q, 0.1, out2, ws, lse=lse2,
                               tree_mask=_mask(words))
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", H.KINDS)
@pytest.mark.parametrize("name", ["one token each, prefix in registers", "128 rows of both", "256 rows of a prefix, 128 own"])
def test_large_scores_negative_scale_and_scale_zero(name, kind):
    for scale in (4.0, -2.0, 0.0):
        c, q, starts, words, max_q = _make(CASES[name], kind, seed=9)
        q = q * 4
        out, lse, st = _attend(c, q, starts, words, max_q, scale)
        assert st == B.RF_OK
        _check(c, q, starts, words, max_q, scale, out, lse)


@pytest.mark.parametrize("kind", H.KINDS)
@pytest.mark.parametrize("plen", [0, 70])
@pytest.mark.parametrize("hd,page,counts", [(64, 4, 5), (128, 16, 20), (128, 5, 64), (64, 16, 3)])
def test_masks_that_leave_nothing_of_a_sequence(kind, plen, hd, page, counts):
    # own rows: the drafts alone, one of which sees none of them
    case = ([counts, counts], [counts, counts], [plen], [0, 1], 4, 2, hd, page, True)
    c, q, starts, words, max_q = _make(case, kind, seed=counts)
    for b in range(2):
        words[b * counts] = 0
        words[b * counts + counts // 2] = np.uint64(1) << np.uint64(counts - 1)
        words[b * counts + counts - 1] = np.uint64(2 ** 64 - 1)
    out, lse, st = _attend(c, q, starts, words, max_q, 0.1)
    assert st == B.RF_OK
    _check(c, q, starts, words, max_q, 0.1, out, lse)
    for b in range(2):
        empty = b == 1 or plen == 0
        assert bool((lse[b * counts] == -math.inf).all()) == empty and bool((out[b * counts] == 0).all()) == empty


@pytest.mark.parametrize("kind", H.KINDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("hd,counts", [(64, 3), (128, 24), (64, 60), (128, 2), (128, 50)])
def test_rows_that_a_query_does_not_see(kind, bad, hd, counts):
    # drafts that only they themselves see, and another group's prefix, may hold anything
    case = ([40 + counts, 12 + counts], [counts, counts], [90, 33], [0, 1, 2], 6, 2, hd, 8, True)
    hidden = [counts - 1] if counts < 4 else [1, counts // 2, counts - 1]

    def change(c, k, v):
        for p in (k, v):
            for j in hidden:
                p[c.base.table_np[0, (40 + j) // 8], (40 + j) % 8] = bad
            for r in (0, 5, 32):
                p[c.base.table_np[3, r // 8], r % 8] = bad
    c, q, starts, words, max_q = _make(case, kind, seed=3, change=change)
    for i in range(counts):
        for j in hidden:
            if i != j:
                words[i] &= ~(np.uint64(1) << np.uint64(j))
    out, lse, st = _attend(c, q, starts, words, max_q, 0.1)
    assert st == B.RF_OK
    clean, *_ = _make(case, kind, seed=3)
    others = [i for i in range(counts) if i not in hidden]
    _check(clean, q, starts, words, max_q, 0.1, out, lse, which=others)
    if bad != bad or (kind != "bf16" and math.isinf(bad)):
        assert torch.isnan(out[hidden]).all() and torch.isnan(lse[hidden]).all()
        assert torch.isnan(out[counts:]).all() and torch.isnan(lse[counts:]).all()       # the second group sees its prefix


@pytest.mark.parametrize("name", ["one token each, prefix in registers", "128 rows of a prefix, tokens in registers",
                                  "256 rows of a prefix, 128 own"])
def test_infinite_values_of_a_prefix(name):
    def change(c, k, v):
        v[c.base.table_np[c.batch_size, 3 // c.page], 3 % c.page, :, 5] = float("inf")
        v[c.base.table_np[c.batch_size, 20 // c.page], 20 % c.page, :, 9] = -float("inf")
    c, q, starts, words, max_q = _make(CASES[name], "bf16", seed=4, change=change)
    out, _, st = _attend(c, q, starts, words, max_q, 0.1)
    assert st == B.RF_OK
    assert (out[..., 5] == float("inf")).all() and (out[..., 9] == -float("inf")).all()
    rest = torch.ones(c.hd, dtype=torch.bool)
    rest[[5, 9]] = False
    assert torch.isfinite(out[..., rest.to(DEV)]).all()


# -------------------------------------------------------------- bounds, lists, bad lists and pages

def test_bounds_larger_than_what_there_is():
    # host bounds on lengths, queries and prefixes far above the real ones
    for kind in H.KINDS:
        for name in ("three prefixes, one empty, two sequences without", "128 rows of both", "no prefix, one token"):
            for max_q in (24, 64):
                c, q, starts, words, _ = _make(CASES[name], kind, seed=5, max_len=3000, max_prefix=9000)
                out, lse, st = _attend(c, q, starts, words, max_q, 0.09, n_pad=150)
                assert st == B.RF_OK
                n = q.shape[0]
                _check(c, q, starts, words, max_q, 0.09, out[:n], lse[:n])
                assert (out[n:] == 3).all()


@pytest.mark.parametrize("kind", H.KINDS)
def test_no_queries(kind):
    c, q, starts, words, _ = _make(([5, 9], [0, 0], [40], [0, 2], 4, 2, 64, 16, False), kind)
    for max_q in (1, 20):
        out, lse, st = _attend(c, q, starts, words, max_q, 0.1, n_pad=2)
        assert st == B.RF_OK and (out == 3).all() and (lse == 3).all()
        kv, pre = c.kv(B), c.prefix(B)
        ws = torch.empty(B.ridgefill_cache_attention_workspace_bytes(kv, 4, max_q, 0, pre), dtype=torch.uint8, device=DEV)
        B.ridgefill_cache_attention(kv, c.cache(B), q, torch.tensor(starts, dtype=torch.int32, device=DEV), max_q, 0.1, q, ws, prefix=pre)
        assert B.ridgefill_read_status(ws) == B.RF_OK


@pytest.mark.parametrize("batch,groups", [(150, 3), (200, 100), (70, 70)])
def test_many_sequences_and_groups(batch, groups):
    g = np.random.default_rng(batch)
    lens = [int(x) for x in g.integers(2, 40, batch)]
    counts = [int(x) for x in g.integers(0, 3, batch)]
    plens = [int(x) for x in g.integers(0, 300, groups)]
    cuts = np.sort(g.integers(3, batch - 1, groups + 1))
    c, q, starts, words, max_q = _make((lens, counts, plens, [int(x) for x in cuts], 4, 2, 64, 16, False), "fp8", seed=1)
    out, lse, st = _attend(c, q, starts, words, max_q, 0.125)
    assert st == B.RF_OK
    _check(c, q, starts, words, max_q, 0.125, out, lse)


@pytest.mark.parametrize("groups,order,kind", [(64, True, "fp8"), (65, True, "bf16"), (4500, True, "int8"), (4500, False, "bf16")])
def test_groups_by_the_thousands(groups, order, kind):
    # some without sequences, queries or rows; and with two that begin too early
    g = np.random.default_rng(groups)
    batch = groups + 20
    lens = [int(x) for x in g.integers(1, 4, batch)]
    counts = [int(x) for x in g.integers(0, 2, batch)]
    plens = [int(x) for x in g.integers(0, 7, groups)]
    cuts = [int(x) for x in np.sort(g.integers(0, batch + 1, groups + 1))]
    gone = []
    if not order:
        for i in (2000, 4200):
            cuts[i] = cuts[i - 100]
        for b in range(batch):
            i = next((i for i in range(groups) if cuts[i] <= b < cuts[i + 1]), None)
            gone += [b] * (i in (2000, 4200))
        assert gone
    c, q, starts, words, max_q = _make((lens, counts, plens, cuts, 2, 1, 64, 4, False), kind, seed=3)
    out, lse, st = _attend(c, q, starts, words, max_q, 0.125)
    assert st == (B.RF_OK if order else B.RF_E_ROWS)
    skipped = [i for b in gone for i in range(starts[b], starts[b + 1])]
    _check(c, q, starts, words, max_q, 0.125, out, lse, which=[i for i in range(q.shape[0]) if i not in skipped])
    assert (out[skipped] == 3).all() and (lse[skipped] == 3).all()


def _status_case(kind="fp8"):
    case = ([20, 30, 40, 9], [2, 1, 2, 1], [50, 80], [0, 2, 4], 4, 2, 64, 8, False)
    return _make(case, kind, seed=6)


@pytest.mark.parametrize("change", [dict(plens=[-1, 80]), dict(plens=[2000, 80]), dict(starts=[0, 5, 4]), dict(starts=[-1, 2, 4]),
                                    dict(starts=[1, 0, 4])])
def test_bad_groups_are_flagged_and_skipped(change):
    c, q, starts, words, max_q = _status_case()
    good, lse_good, _ = _attend(c, q, starts, words, max_q, 0.1)
    if "plens" in change:
        c.plengths = torch.tensor(change["plens"], dtype=torch.int32, device=DEV)
        keep, gone = [3, 4, 5], [0, 1, 2]
    else:
        c.group_start = torch.tensor(change["starts"], dtype=torch.int32, device=DEV)
        keep, gone = {(0, 5, 4): ([], [0, 1, 2, 3, 4, 5]), (-1, 2, 4): ([3, 4, 5], [0, 1, 2]), (1, 0, 4): (None, [])}[tuple(change["starts"])]
    out, lse, st = _attend(c, q, starts, words, max_q, 0.1)
    assert st == B.RF_E_ROWS
    if keep is None:                                      # no first group; all four have the second's prefix
        c.starts = [0, 0, 4]
        _check(c, q, starts, words, max_q, 0.1, out, lse)
    else:
        assert torch.equal(out[keep], good[keep]) and torch.equal(lse[keep], lse_good[keep])
    assert (out[gone] == 3).all() and (lse[gone] == 3).all()


def test_bad_sequences_among_good_ones():
    # a length out of range; too many queries for max_q; the others answer as ever
    c, q, starts, words, max_q = _status_case("int8")
    good, _, _ = _attend(c, q, starts, words, max_q, 0.1)
    c.lengths[1] = c.max_len + 1
    out, lse, st = _attend(c, q, starts, words, max_q, 0.1)
    assert st == B.RF_E_ROWS
    assert (out[2] == 3).all() and (lse[2] == 3).all()
    rest = [0, 1, 3, 4, 5]
    # the same numbers: other parts than before may have been taken
    want, _, ot, _ = S.attention(c, q, starts, words, 0.1)
    _close(out[rest], want[rest], ot[rest], "others")
    c.lengths[1] = 30
    wrong = [0, 1, 3, 2, 6]                               # sequence 2 runs backwards
    out, lse, st = _attend(c, q, wrong, words, 4, 0.1)
    assert st == B.RF_E_ROWS and (out[2:6] == out[2:6]).all()
    wrong = [0, 2, 3, 5, 70]                              # past the queries
    out, lse, st = _attend(c, q, wrong, words, 64, 0.1)
    assert st == B.RF_E_ROWS and (out[3:] == 3).all()
    _check(c, q, starts, words, max_q, 0.1, out, lse, which=[0, 1, 2])
    wrong = [4, 6, 0, 1, 2]                               # queries that leave their group's
    out, lse, st = _attend(c, q, wrong, words, 6, 0.1)
    assert st == B.RF_E_ROWS


# own lengths, queries, prefix lengths, group starts that fall and rise again, heads, n_kv, and the sequences that
# have no answer: those whose first group begins before an earlier one ends
UNORDERED = {
    "the same two again and again": ([20, 30, 9], [1, 1, 1], [40] * 6, [0, 2, 0, 2, 0, 2, 3], 8, 2, []),
    "all but one again and again, 128 rows": ([12 + i for i in range(64)], [8] * 64, [128 - i for i in range(16)], [0, 63] * 8 + [64], 32, 8, []),
    "256 rows, again and again": ([70, 80, 66, 64], [64, 40, 64, 60], [200, 90, 130, 70, 20], [0, 3, 0, 3, 0, 4], 10, 2, [3]),
    "the second begins in the first": ([20, 30, 9, 15, 8, 50], [1, 2, 1, 3, 1, 2], [40, 33, 70], [0, 4, 2, 6], 4, 2, [4, 5]),
    "one of 130 begins at the first": ([3 + i % 40 for i in range(130)], [1 + i % 2 for i in range(130)], [i % 90 for i in range(130)],
                                       list(range(70)) + [0] + list(range(71, 131)), 4, 2, [69, 70]),
    "one of 130 takes a hundred": ([3 + i % 40 for i in range(130)], [1 + i % 2 for i in range(130)], [i % 90 + 1 for i in range(130)],
                                   list(range(20)) + [120] + list(range(21, 131)), 4, 2, []),
}


@pytest.mark.parametrize("kind", H.KINDS)
@pytest.mark.parametrize("name", UNORDERED)
def test_groups_out_of_order(name, kind):
    lens, counts, plens, groups, heads, n_kv, gone = UNORDERED[name]
    c, q, starts, words, max_q = _make((lens, counts, plens, groups, heads, n_kv, 64, 16, False), kind, seed=len(name))
    out, lse, st = _attend(c, q, starts, words, max_q, 0.1)
    assert st == B.RF_E_ROWS
    skipped = [i for b in gone for i in range(starts[b], starts[b + 1])]
    _check(c, q, starts, words, max_q, 0.1, out, lse, which=[i for i in range(q.shape[0]) if i not in skipped])
    assert (out[skipped] == 3).all() and (lse[skipped] == 3).all()


@pytest.mark.parametrize("kind", H.KINDS)
@pytest.mark.parametrize("heads,n,batch", [(64, 64, 200), (8, 5, 90), (16, 1, 150)])
def test_queries_that_run_backwards_between_groups(kind, heads, n, batch):
    # every other sequence has all the queries, and a group of its own: they are the first one's
    c, _, _, _, _ = _make(([70] * batch, [1] * batch, [100 - i % 30 for i in range(batch)], list(range(batch + 1)), heads, 8, 64, 16, False), kind, seed=n)
    q = _randn(n, n, heads, 64)
    out, lse, st = _attend(c, q, [0, n] * (batch // 2) + [0], None, 64, 0.1)
    assert st == B.RF_E_ROWS
    _check(c, q, [0] + [n] * batch, None, 64, 0.1, out, lse)


def test_outputs_beside_sequences_that_run_backwards():
    c, q, _, words, _ = _status_case("int8")
    for wrong, right in (([0, 1, 3, 2, 6], [0, 1, 3, 3, 3]),     # the last one has queries from before its group's
                         ([4, 6, 0, 1, 2], [0, 0, 0, 1, 2])):    # the first group's end before they begin
        out, lse, st = _attend(c, q, wrong, words, 6, 0.1)
        assert st == B.RF_E_ROWS
        _check(c, q, right, words, 6, 0.1, out, lse, which=list(range(right[-1])))
        assert (out[right[-1]:] == 3).all() and (lse[right[-1]:] == 3).all()


@pytest.mark.parametrize("kind", H.KINDS)
@pytest.mark.parametrize("name", ["one token each, prefix split", "128 rows of both"])
def test_rows_on_bad_pages_are_not_there(name, kind):
    c, q, starts, words, max_q = _make(CASES[name], kind, seed=8)
    c.ptable[0, 2], c.ptable[0, 5], c.table[1, 0] = -1, c.num_pages, c.num_pages + 7
    gone = [(c.batch_size, r) for p in (2, 5) for r in range(p * c.page, (p + 1) * c.page)] + [(1, r) for r in range(min(c.page, c.lens[1]))]
    out, lse, st = _attend(c, q, starts, words, max_q, 0.1)
    assert st == B.RF_E_ROWS
    _check(c, q, starts, words, max_q, 0.1, out, lse, gone=gone)
    c.ptable[0, 2], c.ptable[0, 5], c.table[1, 0] = (int(c.base.table_np[a, p]) for a, p in ((c.batch_size, 2), (c.batch_size, 5), (1, 0)))
    out, lse, st = _attend(c, q, starts, words, max_q, 0.1)
    assert st == B.RF_OK                                  # the word is the last call's
    _check(c, q, starts, words, max_q, 0.1, out, lse)


def test_prefix_pages_may_be_those_of_a_sequence():
    # a sequence alone, and the same rows as a prefix of it: the same numbers
    lens = [300]
    c, q, starts, words, max_q = _make((lens, [1], [], [0], 4, 2, 64, 16, False), "fp8", seed=1)
    whole, lse, _ = _attend(c, q, starts, words, max_q, 0.125)
    want, wl, ot, lt = S.attention(c, q, starts, words, 0.125)
    kv = B.make_batch(c.table[:, 16:].contiguous(), torch.tensor([44], dtype=torch.int32, device=DEV), 16, c.num_pages, 2, 64, 48)
    pre = B.make_prefix(c.table[:, :16].contiguous(), torch.tensor([256], dtype=torch.int32, device=DEV),
                        torch.tensor([0, 1], dtype=torch.int32, device=DEV), 256)
    out, lse2, st = _attend(c, q, starts, words, max_q, 0.125, prefix=pre, kv=kv)
    assert st == B.RF_OK
    _close(out, want, ot, "out")
    _close(lse2, wl, lt, "lse")


# --------------------------------------------------------------------------- strides, graphs, streams

@pytest.mark.parametrize("kind", H.KINDS)
def test_strided_queries_and_outputs(kind):
    c, _, starts, words, max_q = _make(CASES["128 rows of both"], kind, seed=4)
    n, heads, hd = starts[-1], 4, 128
    base = _randn(3, n, heads + 4, hd)
    q = base[:, :heads]
    out = torch.full((n, heads + 1, hd), 3.0, dtype=torch.bfloat16, device=DEV)
    kv, pre = c.kv(B), c.prefix(B)
    ws = torch.empty(B.ridgefill_cache_attention_workspace_bytes(kv, heads, max_q, n, pre), dtype=torch.uint8, device=DEV)
    B.ridgefill_cache_attention(kv, c.cache(B), q, torch.tensor(starts, dtype=torch.int32, device=DEV), max_q, 0.1, out[:, :heads], ws,
                                prefix=pre, tree_mask=_mask(words))
    want, _, ot, _ = S.attention(c, q.contiguous(), starts, words, 0.1)
    _close(out[:, :heads], want, ot, "out")
    assert (out[:, heads] == 3).all()


@pytest.mark.parametrize("filled", [40, 64])
def test_graph_replays_with_new_lengths_and_groups(filled):
    # a step: norm, rotation and append of new tokens, then attention; captured once, replayed with other
    # lengths, groups and inputs, with eager work and synchronisation between.  With 40 rows filled a longer
    # sequence meets the pool's NaN: the same bits all the same
    heads, n_kv, hd, page, batch = 8, 2, 64, 16, 6
    c, _, _, _, _ = _make(([filled] * batch, [1] * batch, [100, 333] if filled == 40 else [400, 400], [0, 3, 6], heads, n_kv, hd, page, False),
                          "fp8", seed=2, max_len=64, max_prefix=400)
    kv, cache, pre = c.kv(B), c.cache(B), c.prefix(B)
    x = torch.zeros(batch, heads + 2 * n_kv, hd, dtype=torch.bfloat16, device=DEV)
    q, k, v = x[:, :heads], x[:, heads:heads + n_kv], x[:, heads + n_kv:]
    rows, seq = torch.zeros(batch, dtype=torch.int32, device=DEV), torch.arange(batch, dtype=torch.int32, device=DEV)
    qw = (torch.rand(hd) + 0.5).bfloat16().to(DEV)
    norm, rope = B.make_head_norm(qw, qw), B.make_rope()
    start = torch.arange(batch + 1, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(B.ridgefill_cache_attention_workspace_bytes(kv, heads, 1, batch, pre), dtype=torch.uint8, device=DEV)
    q_out, out = torch.empty(batch, heads, hd, dtype=torch.bfloat16, device=DEV), torch.empty(batch, heads, hd, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(batch, heads, device=DEV)

    def step():
        B.ridgefill_append_cache(rope, norm, kv, cache, k, v, rows, status, seq=seq, q=q, q_out=q_out)
        B.ridgefill_cache_attention(kv, cache, q_out, start, 1, 0.125, out, ws, prefix=pre, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator().manual_seed(1)
    for i, (lens, plens, groups) in enumerate((([41] * 6, [100, 333], [0, 3, 6]), ([1, 64, 33, 2, 40, 17], [399, 1], [0, 5, 5]),
                                               ([42] * 6, [0, 64], [1, 2, 6]), ([41] * 6, [100, 333], [0, 3, 6]))):
        x.copy_(torch.randn(x.shape, generator=g).bfloat16())
        c.lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        rows.copy_(torch.tensor(lens, dtype=torch.int32) - 1)
        c.plengths.copy_(torch.tensor(plens, dtype=torch.int32))
        c.group_start.copy_(torch.tensor(groups, dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone(), q_out.clone()
        assert B.ridgefill_read_status(ws) == B.RF_OK and B.ridgefill_read_status(status) == B.RF_OK
        out.zero_()
        step()
        for a, b in zip(got, (out, lse, q_out)):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16)), i
        assert filled == 40 or torch.isfinite(out).all()


def test_backward_replays_in_a_graph():
    n, hq, hk, hd = 700, 6, 2, 64
    q, k, gq, gk = (_randn(i, n, h, hd) for i, h in enumerate((hq, hk, hq, hk)))
    w = (torch.rand(hd) + 0.5).bfloat16().to(DEV)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    norm, rope = B.make_head_norm(w, w), B.make_rope()
    outs = [torch.empty_like(q), torch.empty_like(k), torch.empty(hd, device=DEV), torch.empty(hd, device=DEV)]
    ws = torch.empty(B.ridgefill_norm_rope_grad_workspace_bytes(n, hq, hk, hd), dtype=torch.uint8, device=DEV)

    def step():
        B.ridgefill_norm_rope_grad(rope, norm, pos, ws, q, gq, outs[0], outs[2], k, gk, outs[1], outs[3])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        gq.copy_(_randn(20 + i, n, hq, hd))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        step()
        for a, b in zip(got, outs):
            assert torch.equal(a, b)


def test_two_streams_with_their_own_workspaces():
    names = ["256 rows of a prefix, 128 own", "one token each, prefix split"]
    cases = [_make(CASES[n], k, seed=5) for n, k in zip(names, ("int8", "fp8"))]
    want = [_attend(*case, 0.1) for case in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    done = []
    for _ in range(5):
        for (c, q, starts, words, max_q), s in zip(cases, streams):
            kv, pre, cache = c.kv(B), c.prefix(B), c.cache(B)
            with torch.cuda.stream(s):
                st, mask = torch.tensor(starts, dtype=torch.int32, device=DEV), _mask(words)
                ws = torch.empty(B.ridgefill_cache_attention_workspace_bytes(kv, q.shape[1], max_q, q.shape[0], pre), dtype=torch.uint8, device=DEV)
                out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
                B.ridgefill_cache_attention(kv, cache, q, st, max_q, 0.1, out, ws, prefix=pre, lse=lse, tree_mask=mask)
            done.append((out, lse, ws, mask, st))
    torch.cuda.synchronize()
    for i, (out, lse, *_) in enumerate(done):
        assert torch.equal(out, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])


@pytest.mark.parametrize("kind", ["fp8", "int8", "bf16"])
def test_offsets_past_32_bits(kind):
    # pools of more than 2^32 bytes (codes) and elements (bf16), their last pages in use
    page, n_kv, hd = 1 << 15, 8, 128
    num_pages = 140
    lens, plen = [200, 90], 3000
    dtype = H.KINDS[kind]
    kp, vp = (torch.zeros(num_pages, page, n_kv, hd, dtype=torch.uint8 if kind != "bf16" else torch.bfloat16, device=DEV).view(dtype)
              for _ in range(2))
    ks, vs = (None if kind == "bf16" else torch.zeros(num_pages, page, n_kv, hd // 32, dtype=torch.uint8, device=DEV) for _ in range(2))
    table = torch.tensor([[139], [138]], dtype=torch.int32, device=DEV)
    ptable = torch.tensor([[137]], dtype=torch.int32, device=DEV)
    cache = B.make_cache(kp, vp, ks, vs)
    every = B.make_batch(torch.cat([table, ptable]), None, page, num_pages, n_kv, hd, page)
    n = sum(lens) + plen
    k, v = (_randn(s, n, n_kv, hd) for s in (1, 2))
    seq = torch.cat([torch.full((m,), i, dtype=torch.int32) for i, m in enumerate(lens + [plen])]).to(DEV)
    rows = torch.cat([torch.arange(m, dtype=torch.int32) for m in lens + [plen]]).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.ridgefill_append_cache(None, None, every, cache, k, v, rows, status, seq=seq)
    assert B.ridgefill_read_status(status) == B.RF_OK
    k_out, v_out = torch.empty_like(k), torch.empty_like(v)
    B.ridgefill_read_rows(every, cache, rows, status, seq=seq, k_out=k_out, v_out=v_out)
    for got, x in ((k_out, k), (v_out, v)):
        assert torch.equal(got.cpu().double(), H.held(x, kind)[0])
    kv = B.make_batch(table, torch.tensor(lens, dtype=torch.int32, device=DEV), page, num_pages, n_kv, hd, 256)
    pre = B.make_prefix(ptable, torch.tensor([plen], dtype=torch.int32, device=DEV), torch.tensor([0, 2], dtype=torch.int32, device=DEV), plen)
    for heads, counts in ((8, [1, 1]), (32, [20, 3])):
        start = torch.tensor(S.starts_of(counts), dtype=torch.int32, device=DEV)
        q = _randn(5, sum(counts), heads, hd)
        max_q = max(counts)
        ws = torch.empty(B.ridgefill_cache_attention_workspace_bytes(kv, heads, max_q, q.shape[0], pre), dtype=torch.uint8, device=DEV)
        out = torch.empty_like(q)
        B.ridgefill_cache_attention(kv, cache, q, start, max_q, 0.088, out, ws, prefix=pre)
        assert B.ridgefill_read_status(ws) == B.RF_OK
        # the first token of each sequence, in 64 bits, over the rows that came back
        for b, (m, at) in enumerate(zip(lens, (0, lens[0]))):
            own = m - counts[b] + 1
            kk, vv = (torch.cat([t[sum(lens):], t[at:at + own]]).double().repeat_interleave(heads // n_kv, 1).transpose(0, 1) for t in (k_out, v_out))
            qq = q[int(start[b])].double()
            w = torch.softmax((kk @ qq[:, :, None])[..., 0] * 0.088, 1)[:, None]
            want, size = (w @ vv)[:, 0], (w @ vv.abs())[:, 0]
            _close(out[int(start[b])], want.cpu(), (size * 2.0 ** -12 + R.U_BF16 * 1.01 * want.abs()).cpu(), f"{heads} {b}")
