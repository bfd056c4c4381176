"""GPU tests of the cache calls by kernel: each of the attention's forms (up to 16, up to 128, up
to 256 query rows of a key head, whole or split caches) and of the weight's, at what they could
get wrong."""

import copy
import math

import numpy as np
import pytest
import torch

import cachecase as R
from test_gpu_cache import _attend, _case, _close, _evict

from ridge_map_kv_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"

# lens, counts, heads, n_kv, hd, page, tree: query rows of a key head, and whether the cache is split
FORMS = {
    "16 rows, whole": ([40, 21, 1], [1, 4, 1], 8, 2, 128, 16, False),
    "16 rows, split": ([700, 90], [8, 3], 4, 2, 64, 5, True),
    "128 rows, whole": ([45, 80], [20, 7], 4, 1, 64, 4, True),
    "128 rows, split": ([150, 129], [30, 64], 4, 2, 128, 16, True),
    "256 rows, whole": ([64, 70, 100], [64, 11, 40], 16, 4, 128, 16, True),
    "256 rows, split": ([300, 6], [64, 6], 3, 1, 64, 100, False),
    "320 rows, split": ([200], [64], 10, 2, 128, 12, True),
}


@pytest.mark.parametrize("form", FORMS)
def test_weights_of_the_values_keep_15_bits(form):
    # the product with V takes each weight as two bf16 operands: an eighth bit cut off leaves less than
    # 2^-7 of it, which loses at most half a step of bf16, 2^-8 of itself
    lens, counts, heads, n_kv, hd, page, tree = FORMS[form]
    cache, q, starts, words, max_q = _case(lens, counts, heads, n_kv, hd, page, seed=31, tree=tree)
    out, _, st = _attend(cache, q, starts, words, max_q, hd ** -0.5)
    assert st == B.RF_OK
    want, _, tol, _ = R.attention(cache, q, starts, words, hd ** -0.5)
    size = copy.copy(cache)                               # sums of the weights times |v|
    size.v = [cache.v[0].abs()]
    size = R.attention(size, q, starts, words, hd ** -0.5)[0]
    _close(out, want, tol - size * (R.U_BF16 - 2.0 ** -15), form)


@pytest.mark.parametrize("scale", [0.0, 0.1])
@pytest.mark.parametrize("form", FORMS)
def test_infinite_value_that_all_see(form, scale):
    # with a scale of 0 all weights are 1, which one bf16 operand holds whole
    lens, counts, heads, n_kv, hd, page, tree = FORMS[form]
    lens = [n + 64 for n in lens]                         # its step has no drafts
    cache, q, starts, words, max_q = _case(lens, counts, heads, n_kv, hd, page, seed=32, tree=tree)
    for b in range(len(lens)):
        cache.v[0][int(cache.table_np[b, 3 // page]), 3 % page, :, 5] = float("inf")
        cache.v[0][int(cache.table_np[b, 1 // page]), 1 % page, :, 9] = -float("inf")
    out, _, st = _attend(cache, q, starts, words, max_q, scale)
    assert st == B.RF_OK
    assert (out[..., 5] == float("inf")).all() and (out[..., 9] == -float("inf")).all()
    rest = torch.ones(hd, dtype=torch.bool)
    rest[[5, 9]] = False
    assert torch.isfinite(out[..., rest.to(DEV)]).all()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page", [4, 0])
def test_evict_rows_on_bad_pages_keep_their_places(in_place, page):
    # page 4 of 5 holds sources of moves (rows 32 .. 39), page 0 destinations (rows 0 .. 7)
    lens, keep = [40, 40], 20
    cache = R.Cache(lens, 1, 64, 8, seed=4)
    acc = torch.rand(2, 40, generator=torch.Generator().manual_seed(0))
    pos = torch.stack([torch.randperm(40, generator=torch.Generator().manual_seed(b)) for b in (1, 2)]).to(torch.int32)
    old = [p.clone() for p in (cache.k[0], cache.v[0])]
    cache.table[0, page] = cache.num_pages
    ao, po, lo, st = _evict(cache, acc, pos, keep, 0, 0, in_place)
    assert st == B.RF_E_ROWS and lo.tolist() == [keep, keep]
    moves, _ = R.evict(lens, acc.numpy(), pos.numpy(), keep, 0, 0)
    lost = [m for m in moves[0] if page in (m[0] // 8, m[1] // 8)]
    assert lost and len(lost) < len(moves[0])
    for b in range(2):
        holds = list(range(keep))
        for f, t in moves[b]:
            if b or (f, t) not in lost:
                holds[t] = f
        assert torch.equal(ao[b, :keep], acc[b, holds]) and torch.equal(po[b, :keep], pos[b, holds])
        assert (ao[b, keep:] == 0).all()
        for pool, was in zip((cache.k[0], cache.v[0]), old):     # what every place holds is what it says
            was = cache.rows(was, b)[holds]
            there = [t for t in range(keep) if b or t // 8 != page]
            assert torch.equal(cache.rows(pool, b, keep)[there], was[there])


def test_sums_of_a_long_cache_in_one_workgroup():
    # as many sequences as parts are wanted: each is one workgroup's for each key head.  Equal scores have
    # weights of 1, 48 million for each of a query's two lanes, and values of 1 have means of 1
    page, times, n_kv, batch = 2 ** 16, 3 * 2 ** 9, 8, 32
    rows = page * times
    pool = torch.ones(1, page, n_kv, 64, dtype=torch.bfloat16, device=DEV)
    lengths = torch.zeros(batch, dtype=torch.int32, device=DEV)
    lengths[0] = rows
    kv = B.make_batch(torch.zeros(batch, times, dtype=torch.int32, device=DEV), lengths, page, 1, n_kv, 64)
    q = torch.ones(34, 4 * n_kv, 64, dtype=torch.bfloat16, device=DEV)
    start = torch.tensor([0] + [34] * batch, dtype=torch.int32, device=DEV)
    ws = torch.empty(B.ridgefill_tree_attention_workspace_bytes(kv, 4 * n_kv, 34), dtype=torch.uint8, device=DEV)
    assert ws.numel() == 256                              # no parts to join
    out, lse = torch.empty_like(q), torch.empty(34, 4 * n_kv, device=DEV)
    B.ridgefill_tree_attention(kv, pool, pool, q, start, 34, 0.0, out, ws, lse=lse)
    assert B.ridgefill_read_status(ws) == B.RF_OK
    # chains of a step's sums of 32 and of products of 16 rows are whole numbers below 2^29: exact
    want = torch.tensor([math.log(rows - 33 + i) for i in range(34)], dtype=torch.float64)[:, None]
    assert float((lse.cpu().double() - want).abs().max()) <= 8 * R.U_FP32 * math.log(rows)
    assert float((out.float() - 1).abs().max()) <= R.U_BF16


def test_a_single_row_of_any_stride():
    # one token taken out of rows of an odd length, rotated in place and elsewhere
    base = torch.randn(4, 387, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    row = lambda t: t.as_strided((1, 3, 128), (387, 128, 1))  # noqa: E731
    x, pos = row(base), torch.tensor([77], dtype=torch.int32, device=DEV)
    want, out, rest = torch.empty(1, 3, 128, dtype=torch.bfloat16, device=DEV), torch.zeros_like(base), base.clone()
    B.ridgefill_rope(B.make_rope(), x.contiguous(), pos, want)
    B.ridgefill_rope(B.make_rope(), x, pos, row(out))
    B.ridgefill_rope(B.make_rope(), x, pos, x)
    rest[0, :384] = want.view(-1)
    assert torch.equal(out[0, :384], want.view(-1)) and not out[0, 384:].any() and torch.equal(base, rest)


def test_no_part_of_a_long_cache_is_lost():
    # 2^28 rows in 256 parts: one page over and over in the first half, another in the second, so that
    # what is left out of either shows in out, and in lse by its share
    page, times, heads = 2 ** 14, 2 ** 14, 32
    cache = R.Cache([2 * page], 1, 64, page, spare=0, seed=5)
    cache.v[0][int(cache.table_np[0, 1])].add_(1.0)
    q = torch.randn(1, heads, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    table = cache.table.repeat_interleave(times // 2, 1).contiguous()
    length = torch.tensor([page * times], dtype=torch.int32, device=DEV)
    kv = B.make_batch(table, length, page, 2, 1, 64)
    start = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(1, heads, device=DEV)
    ws = torch.empty(B.ridgefill_tree_attention_workspace_bytes(kv, heads, 1), dtype=torch.uint8, device=DEV)
    B.ridgefill_tree_attention(kv, cache.k[0], cache.v[0], q, start, 1, 0.1, out, ws, lse=lse)
    assert B.ridgefill_read_status(ws) == B.RF_OK
    want, wl, ot, lt = R.attention(cache, q, [0, 1], None, 0.1)
    size = copy.copy(cache)
    size.v = [cache.v[0].abs()]
    size = R.attention(size, q, [0, 1], None, 0.1)[0]
    # additions that follow one another in a lane: one a step of 64 rows, 2^14 of them, and two products
    # of 16 rows for each half of a step, 2^16; the oracle's tolerance counts 2^16 for its 2^15 rows
    old = (2 * 2 ** 15 + 64) * R.U_FP32
    sums, products = (2 ** 14 + 512) * R.U_FP32, (2 ** 16 + 512) * R.U_FP32
    _close(lse, wl + math.log(times // 2), lt - old + sums + 16 * R.U_FP32 * math.log(times), "lse")
    _close(out, want, ot + size * (2.0 ** -15 - R.U_BF16 + sums + products - old), "out")
    assert float((lt - old + sums).max()) < 2e-3


# ------------------------------------------------------- what each form does with what is wrong or hidden

FEW = [f for f in FORMS if f != "16 rows, whole"]          # that one is every other test's
LONG_TABLES = {                                           # over 4,096 entries: cleared and reported, not scanned
    "16 rows, long tables": ([30, 70, 1, 90] * 10, [1, 3, 0, 2] * 10, 4, 2, 64, 1, True),
    "128 rows, long tables": ([30, 70, 64, 99] * 10, [10, 3, 0, 20] * 10, 4, 2, 64, 1, True),
}
ALL = {**FORMS, **LONG_TABLES}


def _plain(cache, q, starts, words, scale, gone=()):
    """out, lse and their tolerances in 64 bits; rows (sequence, row) in `gone` are not there."""
    n_q, heads, hd = q.shape
    q, group = q.cpu().double(), heads // cache.n_kv
    out, lse = torch.zeros(n_q, heads, hd, dtype=R.F64), torch.full((n_q, heads), -math.inf, dtype=R.F64)
    ot, lt = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(len(cache.lens)):
        lo, hi = starts[b], starts[b + 1]
        if lo == hi:
            continue
        k, v = cache.rows(cache.k[0], b), cache.rows(cache.v[0], b)
        seen = R.visible(cache.lens[b], hi - lo, None if words is None else words[lo:hi])
        seen[:, [r for s, r in gone if s == b]] = False
        for i in range(lo, hi):
            at = seen[i - lo]
            n = int(at.sum())
            for h in range(heads if n else 0):
                kk, vv = k[at, h // group], v[at, h // group]
                s = kk @ q[i, h] * scale
                w = torch.softmax(s, 0)
                out[i, h], lse[i, h] = w @ vv, torch.logsumexp(s, 0)
                # the scores' dot product, scaling and exponential in fp32; the weights to 2^-15; the sums
                d = float((hd + 2) * R.U_FP32 * (kk.abs() @ q[i, h].abs()).max() * abs(scale) + 8 * R.U_FP32 * s.abs().max())
                ot[i, h] = (w @ vv.abs()) * (2.0 ** -15 + 2 * d + (2 * n + 64) * R.U_FP32) \
                    + R.U_BF16 * 1.01 * out[i, h].abs() + 1e-30
                lt[i, h] = d + (2 * n + 64) * R.U_FP32 + 8 * R.U_FP32 * lse[i, h].abs()
    return out, lse, ot, lt


def _form(form, seed, more=0):
    lens, counts, heads, n_kv, hd, page, tree = ALL[form]
    long = dict(max_len=120) if form in LONG_TABLES else {}
    cache, q, starts, words, max_q = _case([n + more for n in lens], counts, heads, n_kv, hd, page, seed=seed, tree=tree, **long)
    return cache, q, starts, words, max_q


@pytest.mark.parametrize("scale", [-0.2, 0.0])
@pytest.mark.parametrize("form", FEW)
def test_negative_scale_and_none(form, scale):
    cache, q, starts, words, max_q = _form(form, 41)
    out, lse, st = _attend(cache, q, starts, words, max_q, scale)
    want, wl, ot, lt = _plain(cache, q, starts, words, scale)
    assert st == B.RF_OK
    _close(out, want, ot, "out")
    _close(lse, wl, lt, "lse")


@pytest.mark.parametrize("wrong", ["too long", "negative", "fewer rows than queries", "queries past the end"])
@pytest.mark.parametrize("form", ALL)
def test_bad_sequences_in_each_form(form, wrong):
    cache, q, starts, words, max_q = _form(form, 42)
    ref, ref_lse, st = _attend(cache, q, starts, words, max_q, 0.1)
    assert st == B.RF_OK
    lens, starts = list(cache.lens), list(starts)
    b = 0 if wrong != "queries past the end" else len(lens) - 1
    if wrong == "queries past the end":
        while starts[b] == starts[b + 1]:
            b -= 1
        starts[b + 1:] = [starts[b + 1] + 1] * (len(starts) - b - 1)
    else:
        lens[b] = {"too long": cache.max_len + 1, "negative": -1, "fewer rows than queries": starts[b + 1] - starts[b] - 1}[wrong]
    kv = cache.batch(B, torch.tensor(lens, dtype=torch.int32, device=DEV))
    out, lse, st = _attend(cache, q, starts, words, max_q, 0.1, kv=kv)
    assert st == B.RF_E_ROWS
    mine = torch.zeros(q.shape[0], dtype=torch.bool)
    mine[starts[b]:starts[b + 1]] = True
    mine = mine.to(DEV)
    assert (out[mine] == 3).all() and (lse[mine] == 3).all()
    want, wl, ot, lt = _plain(cache, q, _starts_of(form), words, 0.1)
    _close(out[~mine], want[~mine.cpu()], ot[~mine.cpu()], "the others")
    _close(lse[~mine], wl[~mine.cpu()], lt[~mine.cpu()], "the others")
    again, again_lse, st = _attend(cache, q, _starts_of(form), words, max_q, 0.1)
    assert st == B.RF_OK and torch.equal(again, ref) and torch.equal(again_lse, ref_lse)


def _starts_of(form):
    starts = [0]
    for n in ALL[form][1]:
        starts.append(starts[-1] + n)
    return starts


@pytest.mark.parametrize("entry", [-1, 1 << 20])
@pytest.mark.parametrize("form", ALL)
def test_bad_pages_in_each_form(form, entry):
    # the first page of sequence 0, and the one that holds the last sequence's last row but one
    cache, q, starts, words, max_q = _form(form, 43)
    last = max(b for b in range(len(cache.lens)) if starts[b] < starts[b + 1])
    bad = {(0, 0), (last, max(cache.lens[last] - 2, 0) // cache.page)}
    gone = [(b, r) for b, p in bad for r in range(cache.lens[b]) if r // cache.page == p]
    want, wl, ot, lt = _plain(cache, q, starts, words, 0.1, gone)
    for b, p in bad:
        cache.table[b, p] = entry
    out, lse, st = _attend(cache, q, starts, words, max_q, 0.1)
    assert st == B.RF_E_ROWS
    _close(out, want, ot, "out")
    _close(lse, wl, lt, "lse")
    _, alone, st = _attend(cache, q, starts, words, max_q, 0.1, want_out=False)
    assert st == B.RF_E_ROWS
    _close(alone, wl, lt, "lse alone")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("form", ["16 rows, split", "128 rows, split", "256 rows, whole", "320 rows, split"])
def test_hidden_rows_in_each_form(form, bad):
    cache, q, starts, words, max_q = _form(form, 44)
    hidden = []
    for b in range(len(cache.lens)):
        n, lo = starts[b + 1] - starts[b], starts[b]
        for j in {0, n // 3, n - 1} if n > 2 else ():
            hidden.append((b, j))
            for i in range(n):
                if i != j:
                    words[lo + i] &= ~(1 << j) & (2 ** 64 - 1)
    want, wl, ot, lt = _plain(cache, q, starts, words, 0.1)
    for b, j in hidden:
        t = cache.lens[b] - (starts[b + 1] - starts[b]) + j
        cache.k[0][int(cache.table_np[b, t // cache.page]), t % cache.page] = bad
        cache.v[0][int(cache.table_np[b, t // cache.page]), t % cache.page] = bad
    out, lse, st = _attend(cache, q, starts, words, max_q, 0.1)
    assert st == B.RF_OK
    own = {starts[b] + j for b, j in hidden}
    others = [i for i in range(q.shape[0]) if i not in own]
    _close(out[others], want[others], ot[others], "out")
    _close(lse[others], wl[others], lt[others], "lse")
    if bad != bad:
        assert torch.isnan(out[sorted(own)]).all() and torch.isnan(lse[sorted(own)]).all()


@pytest.mark.parametrize("form", ["16 rows, split", "128 rows, whole", "128 rows, split", "256 rows, whole", "320 rows, split"])
def test_infinite_value_of_a_draft(form):
    # it reaches the queries that see it, and of their features only its own
    cache, q, starts, words, max_q = _form(form, 45)
    want, _, ot, _ = _plain(cache, q, starts, words, 0.1)
    sees = torch.zeros(q.shape[0], dtype=torch.bool)
    for b in range(len(cache.lens)):
        n = starts[b + 1] - starts[b]
        j, t = min(2, n - 1), cache.lens[b] - n + min(2, n - 1)
        cache.v[0][int(cache.table_np[b, t // cache.page]), t % cache.page, :, 37] = float("inf")
        for i in range(n):
            sees[starts[b] + i] = bool(int(words[starts[b] + i]) >> j & 1)
    out, _, st = _attend(cache, q, starts, words, max_q, 0.1)
    assert st == B.RF_OK
    assert (out[sees.to(DEV)][..., 37] == float("inf")).all()
    out, finite = out.cpu(), torch.arange(q.shape[2]) != 37
    _close(out[:, :, finite], want[:, :, finite], ot[:, :, finite], "the other features")
    _close(out[~sees], want[~sees], ot[~sees], "those who do not see it")


@pytest.mark.parametrize("form", ["16 rows, split", "128 rows, split", "256 rows, whole", "256 rows, split"])
def test_infinite_scores(form):
    # a key that is infinite in one feature: scores of +inf make out and lse NaN, those of -inf add nothing
    cache, q, starts, words, max_q = _form(form, 46, more=64)
    q[..., 7] = torch.where(q[..., 7] == 0, torch.ones_like(q[..., 7]), q[..., 7])
    gone = [(b, 3) for b in range(len(cache.lens))]
    want, wl, ot, lt = _plain(cache, q, starts, words, 0.1, gone)
    for b in range(len(cache.lens)):
        cache.k[0][int(cache.table_np[b, 3 // cache.page]), 3 % cache.page, :, 7] = float("inf")
    out, lse, st = _attend(cache, q, starts, words, max_q, 0.1)
    assert st == B.RF_OK
    up = (q[..., 7] > 0).cpu()
    out, lse = out.cpu(), lse.cpu()
    assert torch.isnan(out[up]).all() and torch.isnan(lse[up]).all()
    _close(out[~up], want[~up], ot[~up], "out")
    _close(lse[~up], wl[~up], lt[~up], "lse")


@pytest.mark.parametrize("heads,count", [(16, 30), (32, 64)])
def test_offsets_past_32_bits_of_the_forms_through_lds(heads, count):
    n_kv, hd, page, rows = 8, 128, 16, 500
    num_pages = (1 << 32) // (page * n_kv * hd * 2) + 40
    small = R.Cache([rows], n_kv, hd, page, seed=13)
    table = torch.arange(num_pages - 1, num_pages - 1 - 32, -1, dtype=torch.int32, device=DEV)[None].contiguous()
    pools = []
    for src in (small.k[0], small.v[0]):
        pools.append(torch.empty(num_pages, page, n_kv, hd, dtype=torch.bfloat16, device=DEV))
        pools[-1][table[0].long()] = src[small.table[0].long()]
    kv = B.make_batch(table, small.lengths, page, num_pages, n_kv, hd, rows)
    q = torch.randn(count, heads, hd, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    start = torch.tensor([0, count], dtype=torch.int32, device=DEV)
    ref, ref_lse, _ = _attend(small, q, [0, count], None, count, 0.1)
    out, lse = torch.empty_like(ref), torch.empty_like(ref_lse)
    ws = torch.empty(B.ridgefill_tree_attention_workspace_bytes(kv, heads, count), dtype=torch.uint8, device=DEV)
    B.ridgefill_tree_attention(kv, pools[0], pools[1], q, start, count, 0.1, out, ws, lse=lse)
    assert B.ridgefill_read_status(ws) == B.RF_OK and torch.equal(out, ref) and torch.equal(lse, ref_lse)
    ws = torch.empty(B.ridgefill_attention_weight_workspace_bytes(kv, heads, count), dtype=torch.uint8, device=DEV)
    a, b = torch.zeros(1, rows, device=DEV), torch.zeros(1, rows, device=DEV)
    B.ridgefill_attention_weight(kv, pools[0], q, start, count, 0.1, lse, a, ws)
    B.ridgefill_attention_weight(small.batch(B), small.k[0], q, start, count, 0.1, lse, b, ws)
    assert torch.equal(a, b)


def test_a_tail_as_windows_that_share_a_block_table():
    # 150 last rows of one sequence: windows of 64 queries, each a sequence that ends with its own rows
    heads, n_kv, hd, page, rows, tail = 8, 2, 64, 16, 300, 150
    cache, q, _, _, _ = _case([rows], [tail], heads, n_kv, hd, page, seed=47)
    ends = [rows - tail + 22, rows - 64, rows]
    starts = [0, 22, 86, 150]
    kv = B.make_batch(cache.table.repeat(3, 1), torch.tensor(ends, dtype=torch.int32, device=DEV), page, cache.num_pages, n_kv, hd,
                      rows)
    out, lse, st = _attend(cache, q, starts, None, 64, 0.1, kv=kv)
    assert st == B.RF_OK
    for i in (0, 21, 22, 85, 86, 149):
        one = copy.copy(cache)
        one.lens = [rows - tail + i + 1]
        want, wl, ot, lt = _plain(one, q[i:i + 1], [0, 1], None, 0.1)
        _close(out[i:i + 1], want, ot, f"row {i}")
        _close(lse[i:i + 1], wl, lt, f"row {i}")


# ------------------------------------------------------------------- the weight of more than 64 query rows

WINDOWS = {  # lens, counts, heads, n_kv, hd, page, tree
    "one block": ([700, 90, 40], [20, 18, 33], 8, 2, 64, 16, True),
    "two blocks": ([300], [64], 10, 2, 128, 12, False),
    "several splits": ([1300, 5], [64, 5], 6, 3, 64, 100, True),
    "64 rows": ([300, 70], [16, 9], 8, 2, 128, 16, True),
    "32 rows, long tables": ([30, 70, 1, 90] * 10, [2, 3, 0, 8] * 10, 4, 1, 64, 1, True),
}


def _weigh(cache, q, starts, words, max_q, scale, lse, kv=None):
    kv = kv or cache.batch(B)
    ws = torch.full((B.ridgefill_attention_weight_workspace_bytes(kv, q.shape[1], max_q),), 0xff, dtype=torch.uint8, device=DEV)
    acc = torch.full((len(cache.lens), cache.max_len), -7.0, device=DEV)
    mask = None if words is None else torch.from_numpy(words.view("int64")).to(DEV)
    B.ridgefill_attention_weight(kv, cache.k[0], q, torch.tensor(starts, dtype=torch.int32, device=DEV), max_q, scale, lse, acc, ws,
                                 tree_mask=mask)
    return acc, B.ridgefill_read_status(ws)


def _window(form, seed):
    lens, counts, heads, n_kv, hd, page, tree = WINDOWS[form]
    long = dict(max_len=120) if "long tables" in form else {}
    cache, q, starts, words, max_q = _case(lens, counts, heads, n_kv, hd, page, seed=seed, tree=tree, **long)
    lse = torch.rand(q.shape[0], heads, generator=torch.Generator().manual_seed(seed)).to(DEV) + 5.0
    return cache, q, starts, words, max_q, lse


@pytest.mark.parametrize("scale", [0.1, -0.2, 0.0])
@pytest.mark.parametrize("form", WINDOWS)
def test_weight_of_each_form(form, scale):
    cache, q, starts, words, max_q, lse = _window(form, 51)
    lse[3, 1] = -float("inf")                             # gives nothing
    acc, st = _weigh(cache, q, starts, words, max_q, scale, lse)
    assert st == B.RF_OK
    want, tol = R.weight(cache, q, starts, words, scale, lse, 1.0, None, torch.full_like(acc, -7.0))
    _close(acc, want, tol, form)


@pytest.mark.parametrize("form", WINDOWS)
def test_weight_of_hidden_rows_and_bad_pages(form):
    cache, q, starts, words, max_q, lse = _window(form, 52)
    hidden = {}
    for b in range(len(cache.lens)):
        n = starts[b + 1] - starts[b]
        if n > 4 and words is not None:
            hidden[b] = cache.lens[b] - n + 3
            for i in range(n):
                words[starts[b] + i] &= ~(1 << 3) & (2 ** 64 - 1)
    want, tol = R.weight(cache, q, starts, words, 0.1, lse, 1.0, None, torch.full((len(cache.lens), cache.max_len), -7.0))
    for k, (b, t) in enumerate(hidden.items()):           # nobody sees it
        cache.k[0][int(cache.table_np[b, t // cache.page]), t % cache.page] = (float("nan"), float("inf"))[k % 2]
    acc, st = _weigh(cache, q, starts, words, max_q, 0.1, lse)
    assert st == B.RF_OK
    _close(acc, want, tol, form)
    assert all(float(acc[b, t]) == 0 for b, t in hidden.items())
    page = 20 // cache.page if cache.lens[0] > 20 else 0
    cache.table[0, page] = cache.num_pages
    acc, st = _weigh(cache, q, starts, words, max_q, 0.1, lse)
    assert st == B.RF_E_ROWS
    gone = [t for t in range(cache.lens[0]) if t // cache.page == page]
    want[0, gone] = 0
    _close(acc, want, tol, form)


@pytest.mark.parametrize("form", WINDOWS)
def test_weight_of_bad_sequences(form):
    cache, q, starts, words, max_q, lse = _window(form, 53)
    want, tol = R.weight(cache, q, starts, words, 0.1, lse, 1.0, None, torch.full((len(cache.lens), cache.max_len), -7.0))
    want[0] = -7.0
    for n in (cache.max_len + 1, -1, starts[1] - 1):
        lens = torch.tensor([n] + cache.lens[1:], dtype=torch.int32, device=DEV)
        acc, st = _weigh(cache, q, starts, words, max_q, 0.1, lse, cache.batch(B, lens))
        assert st == B.RF_E_ROWS
        _close(acc, want, tol, form)
    _, st = _weigh(cache, q, starts, words, max_q, 0.1, lse)
    assert st == B.RF_OK


# ------------------------------------------------------------------------------------ append of many rows

@pytest.mark.parametrize("n,n_kv,hd,heads", [(4096, 1, 64, 0), (4097, 1, 64, 0), (9001, 2, 64, 3), (5000, 8, 128, 32)])
def test_append_many_rows(n, n_kv, hd, heads):
    # looked over by one workgroup or reported by all: the same rows, the same status
    page, g = 16, np.random.default_rng(n)
    per = -(-n // page)
    table = torch.from_numpy(g.permutation(2 * per)[:per].astype(np.int32))[None].to(DEV)
    kv = B.make_batch(table, None, page, 2 * per, n_kv, hd, n)
    qkv = torch.randn(n, heads + 2 * n_kv, hd, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16).to(DEV)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + n_kv], qkv[:, heads + n_kv:]
    rows_np = g.permutation(n).astype(np.int32)
    status = torch.full((1,), -1, dtype=torch.int32, device=DEV)
    for bad in ([], [n - 1], [0, n // 2]):
        rows_bad = rows_np.copy()
        rows_bad[bad] = n
        seq_np = np.zeros(n, np.int32)
        seq_np[3] = -1                                    # padding is no error
        kp, vp = (torch.zeros(2 * per, page, n_kv, hd, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        q_out = torch.zeros(n, heads, hd, dtype=torch.bfloat16, device=DEV) if heads else None
        B.ridgefill_append_rows(None, kv, k, v, torch.from_numpy(rows_bad).to(DEV), kp, vp, status,
                                seq=torch.from_numpy(seq_np).to(DEV), q=q if heads else None, q_out=q_out)
        assert B.ridgefill_read_status(status) == (B.RF_E_ROWS if bad else B.RF_OK)
        real = np.setdiff1d(np.arange(n), bad + [3])
        at = table[0].long()[torch.from_numpy(rows_np[real] // page).to(DEV).long()], torch.from_numpy(rows_np[real] % page).to(DEV).long()
        real = torch.from_numpy(real).to(DEV)
        for pool, x in ((kp, k), (vp, v)):
            assert torch.equal(pool[at], x[real])
            pool[at] = 0
            assert not pool.any()
        if heads:
            assert not q_out[3].any()
            q_out[3] = q[3]
            assert torch.equal(q_out, q)
