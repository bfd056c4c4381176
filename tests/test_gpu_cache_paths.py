"""GPU tests of the cache calls by kernel: each of the attention's forms (up to 16, up to 128, up
to 256 query rows of a key head, whole or split caches) and of the weight's, at what they could
get wrong."""

import copy
import math

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
