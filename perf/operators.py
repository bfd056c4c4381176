"""The operators around the paged cache, as cases to measure: rotary positions, appending
rotated rows, attention of drafted tokens, accumulated attention weight and eviction.

`own = False` computes their plain form with elementary torch operations in 32 bits (angles
in 64); `own = True` makes the calls of ridge_map_kv_amd.binding.  `exact` is the same from
the definitions in 64 bits.  Shapes are those of ridge_map_kv_amd.configs: 32 query and 8
key heads of 128 over a 32,768-row prompt (hidden size 4096), 40 query heads over 65,536
rows (hidden size 5120), and the tiny shape with 2 key heads of 64 and pages of 4.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
HALF, INTERLEAVED = 0, 1
PLAIN, LINEAR, NTK, BANDS, YARN = range(5)


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a few rows of the tiny shape: what a single decode step of a small model rotates
        dict(name="rope_smallest", op="rope", n=7, heads=4, hd=64, rot=64, layout=HALF, scaling=PLAIN,
             f32=False, transpose=False),
        # gradient of a long fp32 activation through a scaled, interleaved, partial rotation
        dict(name="rope_grad_fp32", op="rope", n=8191, heads=32, hd=128, rot=64, layout=INTERLEAVED,
             scaling=YARN, f32=True, transpose=True),
        # one generated token of each of 16 sequences into their caches
        dict(name="append_decode", op="append", n=16, batch=16, heads=32, n_kv=8, hd=128, page=16,
             max_len=2048, rot=128, layout=HALF, scaling=PLAIN),
        # the 4,096 tail rows of a 32,768-row prompt, written after its fill
        dict(name="append_tail", op="append", n=4096, batch=1, heads=32, n_kv=8, hd=128, page=16,
             max_len=32768, rot=128, layout=HALF, scaling=BANDS),
        # one token of the tiny shape: latency only
        dict(name="attend_one_small", op="attend", batch=1, max_q=1, heads=4, n_kv=2, hd=64, page=4,
             max_len=29, tree=False, ragged=False),
        # ordinary decoding: 16 sequences of different lengths, one token each
        dict(name="attend_decode", op="attend", batch=16, max_q=1, heads=32, n_kv=8, hd=128, page=16,
             max_len=16384, tree=False, ragged=True),
        # drafted trees of up to 48 tokens on 4 sequences
        dict(name="attend_tree", op="attend", batch=4, max_q=48, heads=32, n_kv=8, hd=128, page=16,
             max_len=32768, tree=True, ragged=True),
        # one tree of 64 drafts over the longest prompt
        dict(name="attend_tree_long", op="attend", batch=1, max_q=64, heads=40, n_kv=8, hd=128, page=16,
             max_len=65536, tree=True, ragged=False),
        # running weights kept along with decoding
        dict(name="weight_decode", op="weight", batch=16, max_q=1, heads=32, n_kv=8, hd=128, page=16,
             max_len=16384, tree=False, ragged=True, decay=0.95),
        # the attention that a prompt's last 64 tokens pay to its rows: scores for row selection
        dict(name="weight_window", op="weight", batch=1, max_q=64, heads=32, n_kv=8, hd=128, page=16,
             max_len=32768, tree=False, ragged=False, decay=0.0),
        # a cache held at 4,096 rows, shortened after every 64 tokens
        dict(name="evict_step", op="evict", batch=8, layers=4, n_kv=8, hd=128, page=16, max_len=4160,
             keep=4096, sink=4, recent=64, ragged=False),
        # a 32,768-row cache cut to half
        dict(name="evict_half", op="evict", batch=1, layers=4, n_kv=8, hd=128, page=16, max_len=32768,
             keep=16384, sink=4, recent=512, ragged=False),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: sizes spread over their logarithm, odd ones among them, never more work
    than the largest listed case of its kind."""
    kind = rng.choice(["rope", "append", "attend", "attend", "weight", "evict"])
    most = max(_cost(c) for c in listed() if c["op"] == kind)
    while True:
        hd, page = rng.choice([64, 128, 128]), rng.choice([4, 12, 16, 16, 32, 100])
        n_kv = rng.choice([1, 2, 4, 8, 8])
        heads = n_kv * rng.choice([1, 2, 4, 4, 5, 8])
        if kind == "rope":
            c = dict(n=_spread(rng, 1, 16384), heads=heads, hd=hd, rot=rng.choice([hd, hd, hd // 2, 32]),
                     layout=rng.choice([HALF, INTERLEAVED]), scaling=rng.choice([PLAIN, LINEAR, NTK, BANDS, YARN]),
                     f32=rng.random() < 0.5, transpose=rng.random() < 0.5)
        elif kind == "append":
            batch = _spread(rng, 1, 64)
            c = dict(n=_spread(rng, 1, 8192), batch=batch, heads=heads, n_kv=n_kv, hd=hd, page=page,
                     max_len=0, rot=rng.choice([hd, hd // 2]), layout=rng.choice([HALF, INTERLEAVED]),
                     scaling=rng.choice([PLAIN, LINEAR, NTK, BANDS, YARN]))
            c["max_len"] = -(-c["n"] // batch) + _spread(rng, 1, 8192)
        elif kind == "evict":
            max_len = _spread(rng, 8, 32768)
            keep = max(1, int(max_len * rng.choice([0.25, 0.5, 0.9, 0.98])))
            c = dict(batch=_spread(rng, 1, 16), layers=rng.choice([1, 2, 4]), n_kv=n_kv, hd=hd, page=page,
                     max_len=max_len, keep=keep, sink=min(keep // 4, 4), recent=min(keep // 4, 128),
                     ragged=rng.random() < 0.5)
        else:
            c = dict(batch=_spread(rng, 1, 32), max_q=_spread(rng, 1, 64), heads=heads, n_kv=n_kv, hd=hd,
                     page=page, max_len=0, tree=rng.random() < 0.5, ragged=rng.random() < 0.5)
            c["max_len"] = c["max_q"] + _spread(rng, 1, 65536)
            if kind == "weight":
                c["decay"] = rng.choice([0.0, 0.9, 1.0])
        c["op"] = kind
        if _cost(c) <= most and _plain_values(c) <= 3.2e8:
            return c


def _plain_values(c):
    """Values that the plain form holds at once (scores, or the gathered rows)."""
    if c["op"] in ("attend", "weight"):
        return c["batch"] * c["max_len"] * max(c["max_q"] * c["heads"], 2 * c["n_kv"] * c["hd"])
    if c["op"] == "append":
        return c["batch"] * c["max_len"] * c["n_kv"] * c["hd"]
    if c["op"] == "evict":
        return c["batch"] * c["max_len"] * c["n_kv"] * c["hd"] * c["layers"]
    return c["n"] * c["heads"] * c["hd"]


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def _mean_len(c):
    return 0.75 * c["max_len"] if c["ragged"] else c["max_len"]


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    c = case
    if c["op"] == "rope":
        n = c["n"] * c["heads"] * c["hd"]
        return dict(bytes=2 * n * (4 if c["f32"] else 2) + 4 * c["n"], flops=3 * n)
    if c["op"] == "append":
        row = (c["heads"] + 2 * c["n_kv"]) * c["hd"]
        return dict(bytes=c["n"] * (4 * row + 12), flops=3 * c["n"] * row)
    if c["op"] == "evict":
        rows = c["batch"] * _mean_len(c)
        share = min(1.0, c["keep"] / _mean_len(c))
        moves = rows * share * (1 - share)
        return dict(bytes=16 * rows + moves * c["layers"] * 8 * c["n_kv"] * c["hd"], flops=rows)
    rows = c["batch"] * _mean_len(c)
    nq = c["batch"] * (0.75 * c["max_q"] if c["ragged"] and c["max_q"] > 1 else c["max_q"])
    q = nq * c["heads"] * c["hd"] * 2
    dots = 2.0 * (nq / c["batch"]) * c["heads"] * c["hd"] * rows
    if c["op"] == "attend":
        return dict(bytes=rows * c["n_kv"] * c["hd"] * 4 + 2 * q, flops=2 * dots)
    return dict(bytes=rows * (c["n_kv"] * c["hd"] * 2 + 8) + q, flops=dots)


# ------------------------------------------------------------------------------- the inputs

ORIG_LEN = 8192                       # trained context length of the scaled rotations
ROPE = {PLAIN: dict(factor=1.0, low=0.0, high=0.0), LINEAR: dict(factor=4.0, low=0.0, high=0.0),
        NTK: dict(factor=4.0, low=0.0, high=0.0), BANDS: dict(factor=8.0, low=1.0, high=4.0),
        YARN: dict(factor=8.0, low=1.0, high=32.0)}
THETA = 500000.0


def _rope(c):
    """The descriptor of the rotation, as the binding takes it."""
    return dict(theta=THETA, rotary_dim=c["rot"], layout=c["layout"], scaling=c["scaling"],
                orig_len=ORIG_LEN, mscale=0.0, **ROPE[c["scaling"]])


def _lengths(c, lo):
    """Sequence lengths, from `lo` upward: all max_len, or between half of it and all of it."""
    if not c["ragged"]:
        return [c["max_len"]] * c["batch"]
    r = np.random.RandomState(c["batch"] * 7919 + c["max_len"])
    return [max(min(lo, c["max_len"]), int(x)) for x in r.randint((c["max_len"] + 1) // 2, c["max_len"] + 1, c["batch"])]


def _tables(c, g):
    """Every sequence's pages, scattered over the pool."""
    per = -(-c["max_len"] // c["page"])
    pages = c["batch"] * per
    return torch.randperm(pages, generator=g, device=DEV).to(torch.int32).view(c["batch"], per), pages


def _bf(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(c=c)
    if c["op"] == "rope":
        s["x"] = torch.randn(c["n"], c["heads"], c["hd"], generator=g, device=DEV,
                             dtype=torch.float32 if c["f32"] else torch.bfloat16)
        s["pos"] = torch.randint(0, 65536, (c["n"],), generator=g, device=DEV, dtype=torch.int32)
        s["out"] = torch.empty_like(s["x"])
    elif c["op"] == "append":
        # q, k and v of a row lie side by side, as a fused projection leaves them
        s["qkv"] = _bf(g, c["n"], c["heads"] + 2 * c["n_kv"], c["hd"])
        s["table"], s["pages"] = _tables(c, g)
        s["seq"] = torch.arange(c["n"], device=DEV, dtype=torch.int32) % c["batch"]
        # the last rows of every sequence, in order
        s["rows"] = (c["max_len"] - 1 - torch.arange(c["n"], device=DEV, dtype=torch.int32) // c["batch"]).to(torch.int32)
        s["kp"] = torch.zeros(s["pages"], c["page"], c["n_kv"], c["hd"], device=DEV, dtype=torch.bfloat16)
        s["vp"] = torch.zeros_like(s["kp"])
        s["q_out"] = torch.empty(c["n"], c["heads"], c["hd"], device=DEV, dtype=torch.bfloat16)
        s["status"] = torch.zeros(1, device=DEV, dtype=torch.int32)
        s["len"] = torch.full((c["batch"],), c["max_len"], device=DEV, dtype=torch.int32)
    elif c["op"] == "evict":
        s["table"], s["pages"] = _tables(c, g)
        s["len"] = torch.tensor(_lengths(c, 1), device=DEV, dtype=torch.int32)
        s["pools"] = [_bf(g, s["pages"], c["page"], c["n_kv"], c["hd"]) for _ in range(2 * c["layers"])]
        # heavy-tailed weights, as accumulated attention is, in eighths so that some tie
        w = torch.rand(c["batch"], c["max_len"], generator=g, device=DEV)
        s["acc"] = (0.5 / (w + 1e-3)).mul_(64).round_().div_(64)
        s["pos"] = torch.arange(c["max_len"], device=DEV, dtype=torch.int32).repeat(c["batch"], 1).contiguous()
        s["acc_out"], s["pos_out"] = torch.zeros_like(s["acc"]), torch.zeros_like(s["pos"])
        s["len_out"] = torch.zeros_like(s["len"])
    else:
        s["table"], s["pages"] = _tables(c, g)
        lens = _lengths(c, c["max_q"])
        if c["ragged"]:
            nq = [max(1, c["max_q"] - (5 * b) % max(1, c["max_q"] // 2)) for b in range(c["batch"])]
        else:
            nq = [c["max_q"]] * c["batch"]
        nq = [min(a, b) for a, b in zip(nq, lens)]
        s["len"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
        s["start"] = torch.tensor([0] + list(np.cumsum(nq)), device=DEV, dtype=torch.int32)
        s["nq"] = n = int(sum(nq))
        s["kp"] = _bf(g, s["pages"], c["page"], c["n_kv"], c["hd"])
        # a few rows that most queries attend to, as real caches have
        s["kp"][:, 0].mul_(1.0 + 2.0 * (torch.rand(s["pages"], 1, 1, generator=g, device=DEV) < 0.1))
        s["q"] = _bf(g, n, c["heads"], c["hd"])
        s["scale"] = c["hd"] ** -0.5
        s["mask"] = _trees(nq, seed) if c["tree"] else None
        if c["op"] == "attend":
            s["vp"] = _bf(g, s["pages"], c["page"], c["n_kv"], c["hd"])
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(n, c["heads"], device=DEV)
        else:
            s["lse"] = _lse(s)
            s["acc0"] = torch.rand(c["batch"], c["max_len"], generator=g, device=DEV)
            s["acc_out"] = torch.zeros_like(s["acc0"])
    if own:                                   # what a serving program keeps: workspace and descriptors
        from ridge_map_kv_amd import binding as B
        if c["op"] in ("rope", "append"):
            s["rope"] = B.make_rope(**_rope(c))
        if c["op"] != "rope":
            s["kv"] = B.make_batch(s["table"], s["len"], c["page"], s["pages"], c["n_kv"], c["hd"], c["max_len"])
        if c["op"] == "attend":
            n = B.ridgefill_tree_attention_workspace_bytes(s["kv"], c["heads"], c["max_q"])
        elif c["op"] == "weight":
            n = B.ridgefill_attention_weight_workspace_bytes(s["kv"], c["heads"], c["max_q"])
        elif c["op"] == "evict":
            n = B.ridgefill_evict_workspace_bytes(s["kv"], c["keep"])
            s["layers"] = B.make_pools(s["pools"][0::2], s["pools"][1::2])
        else:
            n = 256
        s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    return s


def _trees(nq, seed):
    """One random tree of drafts a sequence: bit j of a draft's word where draft j is the draft
    itself or one of its ancestors."""
    r = np.random.RandomState(seed % (1 << 31))
    words = []
    for n in nq:
        tree = []
        for i in range(n):
            parent = int(r.randint(max(-1, i - 6), i)) if i else -1
            tree.append((tree[parent] if parent >= 0 else 0) | (1 << i))
        words += tree
    return torch.from_numpy(np.array(words, dtype=np.uint64).view(np.int64)).to(DEV)


# --------------------------------------------------------------------------------- one pass

def run(s):
    c = s["c"]
    return (_run_own if own else _run_plain)(s, c)


def _run_own(s, c):
    from ridge_map_kv_amd import binding as B
    if c["op"] == "rope":
        B.ridgefill_rope(s["rope"], s["x"], s["pos"], s["out"], transpose=c["transpose"])
        return s["out"]
    if c["op"] == "append":
        h, n_kv = c["heads"], c["n_kv"]
        q, k, v = s["qkv"][:, :h], s["qkv"][:, h:h + n_kv], s["qkv"][:, h + n_kv:]
        B.ridgefill_append_rows(s["rope"], s["kv"], k, v, s["rows"], s["kp"], s["vp"], s["status"],
                                seq=s["seq"], q=q, q_out=s["q_out"])
        return [s["q_out"], s["kp"], s["vp"]]
    if c["op"] == "attend":
        B.ridgefill_tree_attention(s["kv"], s["kp"], s["vp"], s["q"], s["start"], c["max_q"], s["scale"],
                                   s["out"], s["ws"], lse=s["lse"], tree_mask=s["mask"])
        return [s["out"], s["lse"]]
    if c["op"] == "weight":
        B.ridgefill_attention_weight(s["kv"], s["kp"], s["q"], s["start"], c["max_q"], s["scale"], s["lse"],
                                     s["acc_out"], s["ws"], acc=s["acc0"] if c["decay"] else None,
                                     decay=c["decay"], tree_mask=s["mask"])
        return s["acc_out"]
    B.ridgefill_evict_rows(s["kv"], s["layers"], s["acc"], s["pos"], c["keep"], s["acc_out"], s["pos_out"],
                           s["len_out"], s["ws"], n_sink=c["sink"], n_recent=c["recent"])
    return [s["acc_out"], s["pos_out"], s["len_out"], s["pools"]]


def _run_plain(s, c):
    if c["op"] == "rope":
        cos, sin = _angles(c, s["pos"])
        s["out"].copy_(_rotate(s["x"], cos, -sin if c["transpose"] else sin, c))
        return s["out"]
    if c["op"] == "append":
        h, n_kv = c["heads"], c["n_kv"]
        cos, sin = _angles(c, s["rows"])
        qk = _rotate(s["qkv"][:, :h + n_kv], cos, sin, c)
        s["q_out"].copy_(qk[:, :h])
        page = s["table"][s["seq"].long(), (s["rows"] // c["page"]).long()].long()
        slot = page * c["page"] + s["rows"] % c["page"]
        s["kp"].view(-1, n_kv, c["hd"])[slot] = qk[:, h:].to(torch.bfloat16)
        s["vp"].view(-1, n_kv, c["hd"])[slot] = s["qkv"][:, h + n_kv:]
        return [s["q_out"], s["kp"], s["vp"]]
    if c["op"] == "evict":
        return _evict_plain(s, c)
    seq, i = _of_query(s)
    score = _scores(s, c)                                        # [batch, n_kv, max_q * group, max_len]
    group = c["heads"] // c["n_kv"]
    if c["op"] == "attend":
        m = score.amax(-1, keepdim=True)
        p = torch.exp(score - torch.where(torch.isinf(m), torch.zeros_like(m), m))
        total = p.sum(-1, keepdim=True)
        v = _gathered(s["vp"], s, c)
        o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
        o = o.view(c["batch"], c["n_kv"], c["max_q"], group, c["hd"]).permute(0, 2, 1, 3, 4)
        lse = (m + torch.log(total)).view(c["batch"], c["n_kv"], c["max_q"], group).permute(0, 2, 1, 3)
        s["out"].copy_(o[seq, i].reshape(s["out"].shape))
        s["lse"].copy_(lse[seq, i].reshape(s["lse"].shape))
        return [s["out"], s["lse"]]
    lse = torch.zeros(c["batch"], c["max_q"], c["heads"], device=DEV)
    lse[seq, i] = s["lse"]
    lse = lse.view(c["batch"], c["max_q"], c["n_kv"], group).transpose(1, 2).reshape(c["batch"], c["n_kv"], -1, 1)
    w = torch.exp(score - lse).sum((1, 2))
    inside = torch.arange(c["max_len"], device=DEV)[None] < s["len"][:, None]
    s["acc_out"].copy_(torch.where(inside, c["decay"] * s["acc0"] + w, s["acc_out"]))
    return s["acc_out"]


def _angles(c, pos):
    """cos and sin of every row and pair, from 64-bit angles, times the rotation's factor."""
    r, k = c["rot"], ROPE[c["scaling"]]
    j = torch.arange(r // 2, device=DEV, dtype=torch.float64)
    theta = THETA * k["factor"] ** (r / (r - 2)) if c["scaling"] == NTK else THETA
    f, m = theta ** (-2 * j / r), 1.0
    if c["scaling"] == LINEAR:
        f = f / k["factor"]
    elif c["scaling"] == BANDS:
        turns = ORIG_LEN * f / (2 * math.pi)
        t = ((turns - k["low"]) / (k["high"] - k["low"])).clamp(0, 1)
        f = (1 - t) * f / k["factor"] + t * f
    elif c["scaling"] == YARN:
        at = lambda turns: r * math.log(ORIG_LEN / (2 * math.pi * turns)) / (2 * math.log(THETA))  # noqa: E731
        lo, hi = max(math.floor(at(k["high"])), 0), min(math.ceil(at(k["low"])), r - 1)
        t = ((j - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f / k["factor"] * t + f * (1 - t)
        m = 0.1 * math.log(k["factor"]) + 1
    a = pos.double()[:, None] * f
    return (m * torch.cos(a)).float()[:, None], (m * torch.sin(a)).float()[:, None]


def _rotate(x, cos, sin, c):
    x, r = x.float(), c["rot"]
    if c["layout"] == HALF:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def _of_query(s):
    """Sequence of every query, and its place among that sequence's queries."""
    t = torch.arange(s["nq"], device=DEV)
    seq = torch.searchsorted(s["start"].long(), t, right=True) - 1
    return seq, t - s["start"].long()[seq]


def _gathered(pool, s, c):
    """The cached rows of every sequence, in order: [batch, n_kv, max_len, hd] in 32 bits."""
    t = torch.arange(c["max_len"], device=DEV)
    slot = s["table"].long()[:, t // c["page"]] * c["page"] + t % c["page"]
    return pool.view(-1, c["n_kv"], c["hd"])[slot].permute(0, 2, 1, 3).float().contiguous()


def _scores(s, c):
    """scale * q.k, with -inf where a query does not see a row."""
    batch, max_q, n_kv, hd = c["batch"], c["max_q"], c["n_kv"], c["hd"]
    group = c["heads"] // n_kv
    seq, i = _of_query(s)
    q = torch.zeros(batch, max_q, c["heads"], hd, device=DEV)
    q[seq, i] = s["q"].float()
    q = q.view(batch, max_q, n_kv, group, hd).transpose(1, 2).reshape(batch, n_kv, max_q * group, hd)
    score = torch.matmul(q * s["scale"], _gathered(s["kp"], s, c).transpose(-1, -2))
    t = torch.arange(c["max_len"], device=DEV)
    n = s["start"][1:] - s["start"][:-1]
    ctx = (s["len"] - n).long()
    draft = t[None, :] - ctx[:, None]                            # [batch, max_len]
    if s["mask"] is None:
        seen = draft[:, None] <= torch.arange(max_q, device=DEV)[None, :, None]
    else:
        word = torch.zeros(batch, max_q, dtype=torch.int64, device=DEV)
        word[seq, i] = s["mask"]
        bit = (word[:, :, None] >> draft.clamp(0, 63)[:, None]) & 1
        seen = (draft < 0)[:, None] | (bit == 1)
    there = torch.arange(max_q, device=DEV)[None, :, None] < n[:, None, None]
    seen = seen & (t[None, :] < s["len"][:, None])[:, None] & there
    seen = seen[:, None, :, None].expand(batch, 1, max_q, group, c["max_len"]).reshape(batch, 1, max_q * group, -1)
    return torch.where(seen, score, torch.full((), -math.inf, device=DEV))


def _lse(s):
    """The log-sum-exp that the attention before hands on."""
    c = s["c"]
    seq, i = _of_query(s)
    lse = torch.logsumexp(_scores(s, c), -1).view(c["batch"], c["n_kv"], c["max_q"], -1).transpose(1, 2)
    return lse[seq, i].reshape(s["nq"], c["heads"]).contiguous()


def _evict_plain(s, c):
    """Kept rows: the protected ones, then those of largest weight, ties to the lower slot."""
    keep, batch, max_len = c["keep"], c["batch"], c["max_len"]
    t = torch.arange(max_len, device=DEV)
    inside = t[None] < s["len"][:, None]
    newest = torch.where(inside, s["pos"], torch.full_like(s["pos"], -1)).amax(1, keepdim=True)
    safe = (s["pos"] < c["sink"]) | (s["pos"] > newest - c["recent"])
    rank = torch.where(safe, torch.full_like(s["acc"], math.inf), s["acc"])
    rank = torch.where(inside, rank, torch.full_like(rank, -math.inf))
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices
    kept = torch.zeros_like(inside).scatter_(1, order[:, :keep], torch.ones_like(inside)[:, :keep]) & inside
    length = s["len"].clamp(max=keep)
    # slot of every kept row afterwards: its own, or the free slot of the same rank below `length`
    low = t[None] < length[:, None]
    hole, mover = low & ~kept, kept & ~low
    of_hole = torch.where(hole, hole.cumsum(1) - 1, torch.full_like(order, max_len))
    place = torch.full((batch, max_len + 1), -1, device=DEV, dtype=torch.int64)
    place.scatter_(1, of_hole, t[None].expand(batch, -1))
    to = torch.where(mover, place.gather(1, (mover.cumsum(1) - 1).clamp(min=0)), t[None].expand(batch, -1))
    b, src = torch.nonzero(mover, as_tuple=True)
    dst = to[b, src]
    s["acc_out"].copy_(torch.where(inside & ~low, torch.zeros_like(s["acc"]), torch.where(inside, s["acc"], s["acc_out"])))
    s["pos_out"].copy_(torch.where(low, s["pos"], s["pos_out"]))
    s["acc_out"][b, dst], s["pos_out"][b, dst] = s["acc"][b, src], s["pos"][b, src]
    s["len_out"].copy_(length)
    table = s["table"].long()
    old = table[b, src // c["page"]] * c["page"] + src % c["page"]
    new = table[b, dst // c["page"]] * c["page"] + dst % c["page"]
    pools = [p.view(-1, c["n_kv"] * c["hd"]) for p in s["pools"]]
    for p in pools:
        p[new] = p[old]
    return [s["acc_out"], s["pos_out"], s["len_out"], s["pools"]]


# ---------------------------------------------------------------------- the exact answers

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = s["c"]
    if c["op"] == "rope":
        return _exact_turn(s["x"], s["pos"], c, -1.0 if c["transpose"] else 1.0)
    if c["op"] == "append":
        h, n_kv = c["heads"], c["n_kv"]
        q = _exact_turn(s["qkv"][:, :h], s["rows"], c, 1.0)
        k = _exact_turn(s["qkv"][:, h:h + n_kv], s["rows"], c, 1.0)
        kp, vp = s["kp"].double(), s["vp"].double()
        at = s["table"][s["seq"].long(), (s["rows"] // c["page"]).long()].long(), (s["rows"] % c["page"]).long()
        kp[at], vp[at] = k, s["qkv"][:, h + n_kv:].double()
        return [q, kp, vp]
    if c["op"] == "evict":
        return None                           # nothing is computed: values are moved, whole numbers chosen
    return _exact_attention(s, c)


def _exact_turn(x, pos, c, sign):
    """The rotation as a product of complex numbers."""
    r, k = c["rot"], ROPE[c["scaling"]]
    s, lo, hi = k["factor"], k["low"], k["high"]
    f, m = [], 1.0
    for j in range(r // 2):
        w = THETA ** (-2.0 * j / r)
        if c["scaling"] == LINEAR:
            w /= s
        elif c["scaling"] == NTK:
            w = (THETA * s ** (r / (r - 2.0))) ** (-2.0 * j / r)
        elif c["scaling"] == BANDS:
            length = 2 * math.pi / w
            if length > ORIG_LEN / lo:
                w /= s
            elif length >= ORIG_LEN / hi:
                t = (ORIG_LEN / length - lo) / (hi - lo)
                w = (1 - t) * w / s + t * w
        elif c["scaling"] == YARN:
            a = max(0, math.floor(r * math.log(ORIG_LEN / (hi * 2 * math.pi)) / (2 * math.log(THETA))))
            e = min(r - 1, math.ceil(r * math.log(ORIG_LEN / (lo * 2 * math.pi)) / (2 * math.log(THETA))))
            t = min(1.0, max(0.0, (j - a) / max(e - a, 1e-3)))
            w = w / s * t + w * (1 - t)
        f.append(w)
    if c["scaling"] == YARN:
        m = 1.0 + 0.1 * math.log(s)
    turn = torch.polar(torch.full((1,), m, device=DEV, dtype=torch.float64),
                       sign * torch.outer(pos.double(), torch.tensor(f, device=DEV, dtype=torch.float64)))[:, None]
    y = x.double().clone()
    h = r // 2
    at = (slice(0, h), slice(h, r)) if c["layout"] == HALF else (slice(0, r, 2), slice(1, r, 2))
    z = torch.complex(y[..., at[0]].contiguous(), y[..., at[1]].contiguous()) * turn
    y[..., at[0]], y[..., at[1]] = z.real, z.imag
    return y


def _exact_attention(s, c):
    """Sequence by sequence and head by head."""
    group, start, lens = c["heads"] // c["n_kv"], s["start"].tolist(), s["len"].tolist()
    out = torch.zeros(s["nq"], c["heads"], c["hd"], device=DEV, dtype=torch.float64)
    lse = torch.zeros(s["nq"], c["heads"], device=DEV, dtype=torch.float64)
    acc = None if c["op"] == "attend" else s["acc_out"].double()
    for b in range(c["batch"]):
        n, length = start[b + 1] - start[b], lens[b]
        if n == 0:
            continue
        if acc is not None:
            acc[b, :length] = s["acc0"][b, :length].double() * c["decay"]
        pages = s["table"][b].long()
        keys = s["kp"][pages].flatten(0, 1)[:length]
        seen = torch.ones(n, length, dtype=torch.bool, device=DEV)
        if s["mask"] is None:
            seen[:, length - n:] = torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
        else:
            words = [w & ((1 << 64) - 1) for w in s["mask"][start[b]:start[b + 1]].tolist()]
            seen[:, length - n:] = torch.tensor([[bool(w >> j & 1) for j in range(n)] for w in words], device=DEV)
        for h in range(c["heads"]):
            x = s["q"][start[b]:start[b + 1], h].double() @ keys[:, h // group].double().t() * s["scale"]
            x = x.masked_fill(~seen, -math.inf)
            if c["op"] == "attend":
                lse[start[b]:start[b + 1], h] = torch.logsumexp(x, 1)
                values = s["vp"][pages][:, :, h // group].flatten(0, 1)[:length]
                out[start[b]:start[b + 1], h] = torch.softmax(x, 1) @ values.double()
            else:
                acc[b, :length] += torch.exp(x - s["lse"][start[b]:start[b + 1], h].double()[:, None]).sum(0)
    return [out, lse] if acc is None else acc
