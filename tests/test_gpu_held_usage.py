"""The calls on caches of 16 and 8 bits as they are used together: a prompt that the library fills, held in
8 bits as the prefix of several answers; and on streams other than the current one."""

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


@pytest.mark.parametrize("kind", H.KINDS)
def test_fill_append_hold_and_answer_together(kind):
    from fillcase import Case, build_inputs, run_fill
    import oracle
    N, T, d, n_kv, hd, heads, page = 260, 40, 512, 2, 128, 8, 16
    exact = np.arange(3, N - T, 9)
    case = Case(d=d, n_layers=1, n_kv=n_kv, hd=hd, N=N, T=T, exact=exact, page_size=page, seed=31)
    inp = build_inputs(case)
    filled, _, _ = oracle.partition(N, T, exact)
    assert run_fill(case, inp, filled) == B.RF_OK
    layer = inp["layers"][0]
    rope, scale = B.make_rope(theta=case.theta), hd ** -0.5
    g = torch.Generator().manual_seed(5)
    qw, kw = ((torch.rand(hd, generator=g) + 0.5).bfloat16().to(DEV) for _ in range(2))
    norm = B.make_head_norm(qw, kw, 1e-6)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    # the exact and the tail rows into the 16-bit pools that the fill wrote, with the layer's head norms
    kv = B.make_batch(inp["table"][None].contiguous(), None, page, inp["num_pages"], n_kv, hd, N)
    cache16 = B.make_cache(layer["k_pages"], layer["v_pages"])
    rest = torch.from_numpy(np.setdiff1d(np.arange(N), filled).astype(np.int32)).to(DEV)
    n = rest.shape[0]
    q_out = torch.empty(n, heads, hd, dtype=torch.bfloat16, device=DEV)
    B.ridgefill_append_cache(rope, norm, kv, cache16, _randn(1, n, n_kv, hd), _randn(2, n, n_kv, hd), rest, status,
                             q=_randn(3, n, heads, hd), q_out=q_out)
    assert B.ridgefill_read_status(status) == B.RF_OK

    # the whole prompt back, and into the pools of the answers, as their prefix
    every = torch.arange(N, dtype=torch.int32, device=DEV)
    k16, v16 = (torch.empty(N, n_kv, hd, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    B.ridgefill_read_rows(kv, cache16, every, status, k_out=k16, v_out=v16)
    pages, own_pages, counts = -(-N // page), 2, [5, 3, 1]
    batch, num_pages = len(counts), pages + len(counts) * own_pages
    order = np.random.default_rng(7).permutation(num_pages).astype(np.int32)
    ptable, table = order[None, :pages].copy(), order[pages:].reshape(batch, own_pages)
    kp, vp, ks, vs = H.pools(num_pages, page, n_kv, hd, kind, fill=0x55)
    cache = B.make_cache(kp, vp, ks, vs)
    prompt = B.make_batch(torch.from_numpy(ptable).to(DEV), None, page, num_pages, n_kv, hd, N)
    B.ridgefill_append_cache(None, None, prompt, cache, k16, v16, every, status)
    assert B.ridgefill_read_status(status) == B.RF_OK

    # each answer's drafts, a tree, at the positions behind the prompt, and their attention
    words = R.trees(counts, 4)
    depth = torch.tensor([N + bin(int(w)).count("1") - 1 for w in words], dtype=torch.int32, device=DEV)
    rows = torch.tensor([i for c in counts for i in range(c)], dtype=torch.int32, device=DEV)
    seq = torch.tensor([b for b, c in enumerate(counts) for _ in range(c)], dtype=torch.int32, device=DEV)
    lengths = torch.tensor(counts, dtype=torch.int32, device=DEV)
    answers = B.make_batch(torch.from_numpy(table).to(DEV), lengths, page, num_pages, n_kv, hd, own_pages * page)
    total = sum(counts)
    q = _randn(6, total, heads, hd)
    B.ridgefill_append_cache(rope, norm, answers, cache, _randn(7, total, n_kv, hd), _randn(8, total, n_kv, hd), rows, status,
                             seq=seq, positions=depth, q=q, q_out=q)
    prefix = B.make_prefix(prompt._keep[0], torch.tensor([N], dtype=torch.int32, device=DEV),
                           torch.tensor([0, batch], dtype=torch.int32, device=DEV), N)
    starts = S.starts_of(counts)
    out, lse = torch.empty_like(q), torch.empty(total, heads, device=DEV)
    ws = torch.empty(B.ridgefill_cache_attention_workspace_bytes(answers, heads, max(counts), total, prefix), dtype=torch.uint8,
                     device=DEV)
    B.ridgefill_cache_attention(answers, cache, q, torch.tensor(starts, dtype=torch.int32, device=DEV), max(counts), scale, out, ws,
                                prefix=prefix, lse=lse, tree_mask=_mask(words))
    assert B.ridgefill_read_status(status) == B.RF_OK and B.ridgefill_read_status(ws) == B.RF_OK

    def of_rows(pool, scales, tab, count):
        at = np.arange(count)
        page_of, slot = torch.from_numpy(tab[at // page].astype(np.int64)), torch.from_numpy(at % page)
        codes = pool.cpu().view(torch.uint8)[page_of, slot].view(pool.dtype)
        return H.values(codes, None if scales is None else scales.cpu()[page_of, slot])

    # the prefix holds what the fill and the append wrote, by the format's rule
    assert torch.equal(of_rows(kp, ks, ptable[0], N), H.held(k16, kind)[0])
    assert torch.equal(of_rows(vp, vs, ptable[0], N), H.held(v16, kind)[0])

    class View:
        batch_size, lens, k, v = batch, counts, (kp, ks), (vp, vs)

        def __init__(self):
            self.n_kv = n_kv

        def group_of(self, b):
            return 0

        def rows(self, pool, b):
            return torch.cat([of_rows(*pool, ptable[0], N), of_rows(*pool, table[b], counts[b])])
    want, wl, ot, lt = S.attention(View(), q, starts, words, scale)
    _close(out, want, ot, "out")
    _close(lse, wl, lt, "lse")


def test_another_stream():
    # all calls on a stream given to them, with inputs that the current stream made
    n, heads, n_kv, hd, page = 300, 4, 2, 64, 16
    w = (torch.rand(hd, generator=torch.Generator().manual_seed(1)) + 0.5).bfloat16().to(DEV)
    norm, rope = B.make_head_norm(w, w), B.make_rope()
    q, k, v, gq, gk = (_randn(i, n, h, hd) for i, h in enumerate((heads, n_kv, n_kv, heads, n_kv)))
    rows = torch.arange(n, dtype=torch.int32, device=DEV)
    table = torch.arange(-(-n // page), dtype=torch.int32, device=DEV)[None].contiguous()
    length, start = torch.tensor([n], dtype=torch.int32, device=DEV), torch.tensor([0, 9], dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()

    def all_calls(stream):
        kv = B.make_batch(table, length, page, table.shape[1], n_kv, hd, n)
        pools = H.pools(table.shape[1], page, n_kv, hd, "fp8")
        cache = B.make_cache(*pools)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        outs = [torch.zeros_like(t) for t in (q, k, q, k, q, k, k, q[:9])]
        dws = [torch.zeros(hd, device=DEV) for _ in range(2)]
        gws = torch.empty(B.ridgefill_norm_rope_grad_workspace_bytes(n, heads, n_kv, hd), dtype=torch.uint8, device=DEV)
        ws = torch.empty(B.ridgefill_cache_attention_workspace_bytes(kv, heads, 9, 9), dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        B.ridgefill_norm_rope(rope, norm, rows, q=q, q_out=outs[0], k=k, k_out=outs[1], stream=stream)
        B.ridgefill_norm_rope_grad(rope, norm, rows, gws, q, gq, outs[2], dws[0], k, gk, outs[3], dws[1], stream=stream)
        B.ridgefill_append_cache(rope, norm, kv, cache, k, v, rows, status, q=q, q_out=outs[4], stream=stream)
        B.ridgefill_read_rows(kv, cache, rows, status, k_out=outs[5], v_out=outs[6], stream=stream)
        B.ridgefill_cache_attention(kv, cache, outs[4][-9:], start, 9, 0.125, outs[7], ws, stream=stream)
        assert B.ridgefill_read_status(status, stream=stream) == B.RF_OK and B.ridgefill_read_status(ws, stream=stream) == B.RF_OK
        torch.cuda.synchronize()
        return outs + dws + [p.view(torch.uint8) for p in pools]
    for a, b in zip(all_calls(None), all_calls(side)):
        assert torch.equal(a, b) and a.any()


def test_two_graphs_with_one_workspace():
    # attention of two calls, plain and after a prefix, captured with one workspace and replayed in turn
    heads, n_kv, hd = 8, 2, 64
    cases = [S.SharedCache([700, 33, 250], [], [0], n_kv, hd, 16, "int8", 1), S.SharedCache([40, 9, 64, 30], [300, 77], [0, 2, 4], n_kv, hd, 16, "fp8", 2)]
    counts = [[1, 1, 1], [20, 9, 17, 30]]
    calls = []
    for c, n in zip(cases, counts):
        starts = torch.tensor(S.starts_of(n), dtype=torch.int32, device=DEV)
        q = _randn(9, sum(n), heads, hd)
        calls.append((c.kv(B), c.cache(B), q, starts, max(n), c.prefix(B), torch.empty_like(q), torch.empty(sum(n), heads, device=DEV)))
    need = max(B.ridgefill_cache_attention_workspace_bytes(kv, heads, mq, q.shape[0], pre) for kv, _, q, _, mq, pre, _, _ in calls)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)

    def run(i):
        kv, cache, q, starts, max_q, pre, out, lse = calls[i]
        B.ridgefill_cache_attention(kv, cache, q, starts, max_q, 0.125, out, ws, prefix=pre, lse=lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = []
    with torch.cuda.stream(side):
        for i in range(2):
            run(i)
            want.append((calls[i][6].clone(), calls[i][7].clone()))
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in calls]
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            run(i)
    for i in (0, 1, 1, 0, 0, 1):
        calls[i][6].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert B.ridgefill_read_status(ws) == B.RF_OK
        assert torch.equal(calls[i][6], want[i][0]) and torch.equal(calls[i][7], want[i][1])
        run(1 - i)                                        # eager work of the other call between
        assert torch.equal(calls[1 - i][6], want[1 - i][0])
