"""More operators around the paged cache, as cases to measure: norms of queries and keys with
their rotation (and the gradient), caches held in 8 bits as they are written and read back, and
attention over such caches for sequences that share long prefixes.

`own = False` computes their plain form with elementary torch operations in 32 bits (angles in
64); `own = True` makes the calls of ridge_map_kv_amd.binding.  `exact` is the same from the
definitions in 64 bits.  Shapes are those of ridge_map_kv_amd.configs: 32 query and 8 key heads
of 128 over a 32,768-row prompt (hidden size 4096), 40 query heads over 65,536 rows (hidden size
5120), and the tiny shape with 2 key heads of 64 and pages of 4.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
HALF, INTERLEAVED = 0, 1
PLAIN, LINEAR, NTK, BANDS, YARN = range(5)
BLOCK = 32                             # features that share a scale in 8 bits
LARGEST = dict(fp8=448.0, int8=127.0)  # of a code


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a few rows of the tiny shape: what a single decode step of a small model normalises
        dict(name="norm_smallest", op="norm", n=7, heads=4, n_kv=2, hd=64, rot=64, layout=HALF, scaling=PLAIN,
             f32=False, grad=False),
        # q and k of a long prompt's exact rows, beside their projection
        dict(name="norm_prompt", op="norm", n=8191, heads=32, n_kv=8, hd=128, rot=128, layout=HALF, scaling=BANDS,
             f32=False, grad=False),
        # a training step's way back through them, in fp32
        dict(name="norm_grad_fp32", op="norm", n=4097, heads=32, n_kv=8, hd=128, rot=64, layout=INTERLEAVED,
             scaling=YARN, f32=True, grad=True),
        # and in bf16
        dict(name="norm_grad_bf16", op="norm", n=8192, heads=40, n_kv=8, hd=128, rot=128, layout=HALF,
             scaling=PLAIN, f32=False, grad=True),
        # one generated token of each of 16 sequences into fp8 caches
        dict(name="append_decode_fp8", op="append", n=16, batch=16, heads=32, n_kv=8, hd=128, page=16,
             max_len=2048, rot=128, layout=HALF, scaling=PLAIN, type="fp8", norm=True),
        # the 4,096 tail rows of a 32,768-row prompt into an int8 cache, and their values back
        dict(name="append_tail_int8", op="append", n=4096, batch=1, heads=32, n_kv=8, hd=128, page=16,
             max_len=32768, rot=128, layout=HALF, scaling=BANDS, type="int8", norm=True),
        # two sequences of the tiny shape after one prefix: latency only
        dict(name="attend_small", op="attend", type="fp8", batch=2, groups=1, alone=0, prefix=29, max_q=1, heads=4,
             n_kv=2, hd=64, page=4, max_len=9, tree=False, ragged=False),
        # ordinary decoding over fp8 caches: 16 sequences of different lengths, one token each
        dict(name="attend_decode_fp8", op="attend", type="fp8", batch=16, groups=0, alone=16, prefix=0, max_q=1,
             heads=32, n_kv=8, hd=128, page=16, max_len=16384, tree=False, ragged=True),
        # drafted trees of up to 48 tokens on 4 int8 caches
        dict(name="attend_tree_int8", op="attend", type="int8", batch=4, groups=0, alone=4, prefix=0, max_q=48,
             heads=32, n_kv=8, hd=128, page=16, max_len=32768, tree=True, ragged=True),
        # 64 answers of different lengths over one 32,768-row prompt, in bf16 as the fill wrote it
        dict(name="prefix_decode", op="attend", type="bf16", batch=64, groups=1, alone=0, prefix=32768, max_q=1,
             heads=32, n_kv=8, hd=128, page=16, max_len=512, tree=False, ragged=True),
        # 48 sequences on 4 prompts of different lengths, five of them on none, in fp8
        dict(name="prefix_groups_fp8", op="attend", type="fp8", batch=48, groups=4, alone=5, prefix=16384, max_q=4,
             heads=32, n_kv=8, hd=128, page=16, max_len=2048, tree=False, ragged=True),
        # trees of 24 drafts for 8 answers over the longest prompt, in int8
        dict(name="prefix_tree_int8", op="attend", type="int8", batch=8, groups=1, alone=0, prefix=65536, max_q=24,
             heads=40, n_kv=8, hd=128, page=16, max_len=1024, tree=True, ragged=False),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: sizes spread over their logarithm, odd ones among them, never more work
    than the largest listed case of its kind."""
    kind = rng.choice(["norm", "norm", "append", "attend", "attend", "attend"])
    most = max(_cost(c) for c in listed() if c["op"] == kind)
    while True:
        hd, page = rng.choice([64, 128, 128]), rng.choice([4, 12, 16, 16, 32, 100])
        n_kv = rng.choice([1, 2, 4, 8, 8])
        heads = n_kv * rng.choice([1, 2, 4, 4, 5, 8])
        turn = dict(rot=rng.choice([hd, hd, hd // 2]), layout=rng.choice([HALF, INTERLEAVED]),
                    scaling=rng.choice([PLAIN, LINEAR, NTK, BANDS, YARN]))
        if kind == "norm":
            c = dict(n=_spread(rng, 1, 16384), heads=heads, n_kv=n_kv, hd=hd, f32=rng.random() < 0.4,
                     grad=rng.random() < 0.5, **turn)
        elif kind == "append":
            batch = _spread(rng, 1, 64)
            c = dict(n=_spread(rng, 1, 8192), batch=batch, heads=heads, n_kv=n_kv, hd=hd, page=page, max_len=0,
                     type=rng.choice(["bf16", "fp8", "int8"]), norm=rng.random() < 0.7, **turn)
            c["max_len"] = -(-c["n"] // batch) + _spread(rng, 1, 8192)
        else:
            batch, max_q = _spread(rng, 1, 96), rng.choice([1, 1, 1, _spread(rng, 2, 64)])
            groups = rng.choice([0, 1, 1, _spread(rng, 2, 8)])
            groups = min(groups, batch)
            c = dict(type=rng.choice(["bf16", "fp8", "int8"]), batch=batch, groups=groups, alone=0, prefix=0,
                     max_q=max_q, heads=heads, n_kv=n_kv, hd=hd, page=page,
                     max_len=max_q + _spread(rng, 1, 2048 if groups else 32768), tree=rng.random() < 0.5,
                     ragged=rng.random() < 0.7)
            if groups:
                c["prefix"] = _spread(rng, 1, 65536)
                c["alone"] = rng.choice([0, 0, (batch - groups) // 4])
            else:
                c["alone"] = batch
        c["op"] = kind
        if _cost(c) <= most and _plain_values(c) <= 5.5e8:
            return c


def _plain_values(c):
    """Values that the plain form holds at once (scores, or the gathered rows)."""
    if c["op"] == "attend":
        rows = c["batch"] * c["max_len"] * max(c["max_q"] * c["heads"], 2 * c["n_kv"] * c["hd"])
        # of the prefixes: every group as large as the largest
        shared = c["batch"] - c["alone"]
        return max(rows, c["prefix"] * max(c["groups"], 1) * max(shared * c["max_q"] * c["heads"], 2 * c["n_kv"] * c["hd"]))
    if c["op"] == "append":
        return c["batch"] * c["max_len"] * c["n_kv"] * c["hd"]
    return c["n"] * (c["heads"] + c["n_kv"]) * c["hd"] * (3 if c["grad"] else 1)


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def _value_bytes(kind):
    return 2.0 if kind == "bf16" else 1.0 + 1.0 / BLOCK


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    c = case
    if c["op"] == "norm":
        n = c["n"] * (c["heads"] + c["n_kv"]) * c["hd"]
        size = 4 if c["f32"] else 2
        return dict(bytes=(3 if c["grad"] else 2) * n * size + 4 * c["n"], flops=(16 if c["grad"] else 7) * n)
    if c["op"] == "append":
        q, kv = c["n"] * c["heads"] * c["hd"], c["n"] * 2 * c["n_kv"] * c["hd"]
        held = _value_bytes(c["type"])
        return dict(bytes=4 * q + kv * (2 + held + held + 2) + 12 * c["n"], flops=7 * q + 9 * kv)
    lens, nq, plens, sizes = _sequences(c)
    row = 2 * c["n_kv"] * c["hd"] * _value_bytes(c["type"])
    pairs, at = sum(n * m for n, m in zip(lens, nq)), 0
    for g, size in enumerate(sizes):
        pairs += plens[g] * sum(nq[at:at + size])
        at += size
    return dict(bytes=(sum(lens) + sum(plens)) * row + 4 * sum(nq) * c["heads"] * c["hd"],
                flops=4.0 * c["heads"] * c["hd"] * pairs)


# ------------------------------------------------------------------------------- the inputs

ORIG_LEN = 8192                       # trained context length of the scaled rotations
ROPE = {PLAIN: dict(factor=1.0, low=0.0, high=0.0), LINEAR: dict(factor=4.0, low=0.0, high=0.0),
        NTK: dict(factor=4.0, low=0.0, high=0.0), BANDS: dict(factor=8.0, low=1.0, high=4.0),
        YARN: dict(factor=8.0, low=1.0, high=32.0)}
THETA = 500000.0
EPS = 1e-6


def _rope(c):
    """The descriptor of the rotation, as the binding takes it."""
    return dict(theta=THETA, rotary_dim=c["rot"], layout=c["layout"], scaling=c["scaling"],
                orig_len=ORIG_LEN, mscale=0.0, **ROPE[c["scaling"]])


def _sequences(c):
    """Own lengths and query counts of the sequences, lengths of the prefixes and how many
    sequences each has, of a case alone."""
    r = np.random.RandomState(c["batch"] * 7919 + c["max_len"] + c["prefix"])
    lens, nq, plens = [c["max_len"]] * c["batch"], [c["max_q"]] * c["batch"], [c["prefix"]] * c["groups"]
    if c["ragged"]:
        nq = [max(1, c["max_q"] - (5 * b) % max(1, c["max_q"] // 2)) for b in range(c["batch"])]
        lens = [max(n, int(x)) for n, x in zip(nq, r.randint((c["max_len"] + 1) // 2, c["max_len"] + 1, c["batch"]))]
        plens = [int(x) for x in r.randint((c["prefix"] + 1) // 2, c["prefix"] + 1, c["groups"])] if c["prefix"] else plens
    shared = c["batch"] - c["alone"]
    sizes = [(shared * (g + 1)) // c["groups"] - (shared * g) // c["groups"] for g in range(c["groups"])]
    if c["ragged"] and c["groups"] > 1 and sizes[0] > 1:
        moved = sizes[0] // 2                                    # groups of different sizes
        sizes = [sizes[0] - moved] + sizes[1:-1] + [sizes[-1] + moved]
    return lens, nq, plens, sizes


def _tables(batch, max_len, page, pages, first=0):
    """Pages of `batch` axes of max_len rows: entries first .. of a shuffled pool."""
    per = -(-max_len // page)
    return pages[first:first + batch * per].view(batch, per), first + batch * per


def _bf(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _pool(g, shape, kind, peaks=False):
    """A pool of rows, in bf16 or as codes with the scales of their blocks."""
    x = _bf(g, *shape)
    if peaks:                      # a few rows that most queries attend to, as real caches have
        x[:, 0].mul_(1.0 + 2.0 * (torch.rand(shape[0], 1, 1, generator=g, device=DEV) < 0.1))
    if kind == "bf16":
        return x, None
    codes = torch.empty(shape, dtype=torch.float8_e4m3fn if kind == "fp8" else torch.int8, device=DEV)
    scales = torch.empty(*shape[:-1], shape[-1] // BLOCK, dtype=torch.uint8, device=DEV)
    for i in range(0, shape[0], 4096):
        code, e = _code(x[i:i + 4096].float(), kind)
        codes[i:i + 4096] = code.to(codes.dtype)
        scales[i:i + 4096] = (e + 127).to(torch.uint8)
    return codes, scales


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(c=c)
    if c["op"] == "norm":
        dtype = torch.float32 if c["f32"] else torch.bfloat16
        h, n_kv, hd = c["heads"], c["n_kv"], c["hd"]
        # q, k and v of a row lie side by side, as a fused projection leaves them; rows and heads of
        # different sizes
        qkv = torch.randn(c["n"], h + 2 * n_kv, hd, generator=g, device=DEV)
        qkv *= torch.exp(torch.randn(c["n"], h + 2 * n_kv, 1, generator=g, device=DEV))
        s["qkv"] = qkv.to(dtype)
        s["qw"], s["kw"] = (torch.randn(hd, generator=g, device=DEV).mul_(0.2).add_(1).to(dtype) for _ in range(2))
        s["pos"] = torch.randint(0, 65536, (c["n"],), generator=g, device=DEV, dtype=torch.int32)
        make = lambda heads: torch.empty(c["n"], heads, hd, device=DEV, dtype=dtype)  # noqa: E731
        s["q_out"], s["k_out"] = make(h), make(n_kv)
        if c["grad"]:
            s["gq"], s["gk"] = (torch.randn(c["n"], x, hd, generator=g, device=DEV).to(dtype) for x in (h, n_kv))
            s["qw_grad"], s["kw_grad"] = (torch.empty(hd, device=DEV) for _ in range(2))
    elif c["op"] == "append":
        h, n_kv, hd = c["heads"], c["n_kv"], c["hd"]
        s["qkv"] = _bf(g, c["n"], h + 2 * n_kv, hd) * torch.exp(torch.randn(c["n"], h + 2 * n_kv, 1, generator=g, device=DEV)).bfloat16()
        s["qw"], s["kw"] = (torch.randn(hd, generator=g, device=DEV).mul_(0.2).add_(1).bfloat16() for _ in range(2))
        s["pages"] = c["batch"] * -(-c["max_len"] // c["page"])
        order = torch.randperm(s["pages"], generator=g, device=DEV).to(torch.int32)
        s["table"], _ = _tables(c["batch"], c["max_len"], c["page"], order)
        s["seq"] = torch.arange(c["n"], device=DEV, dtype=torch.int32) % c["batch"]
        # the last rows of every sequence, in order
        s["rows"] = (c["max_len"] - 1 - torch.arange(c["n"], device=DEV, dtype=torch.int32) // c["batch"]).to(torch.int32)
        shape = (s["pages"], c["page"], n_kv, hd)
        kinds = dict(bf16=torch.bfloat16, fp8=torch.float8_e4m3fn, int8=torch.int8)
        s["kp"], s["vp"] = (torch.zeros(shape, device=DEV, dtype=torch.uint8 if c["type"] != "bf16" else torch.bfloat16).view(kinds[c["type"]])
                            for _ in range(2))
        s["ks"], s["vs"] = (None if c["type"] == "bf16" else torch.zeros(*shape[:3], hd // BLOCK, device=DEV, dtype=torch.uint8)
                            for _ in range(2))
        s["q_out"] = torch.empty(c["n"], h, hd, device=DEV, dtype=torch.bfloat16)
        s["k_out"], s["v_out"] = (torch.empty(c["n"], n_kv, hd, device=DEV, dtype=torch.bfloat16) for _ in range(2))
        s["status"] = torch.zeros(1, device=DEV, dtype=torch.int32)
        s["len"] = torch.full((c["batch"],), c["max_len"], device=DEV, dtype=torch.int32)
    else:
        lens, nq, plens, sizes = _sequences(c)
        page, per_group = c["page"], -(-c["prefix"] // c["page"])
        s["pages"] = c["batch"] * -(-c["max_len"] // page) + c["groups"] * per_group
        order = torch.randperm(s["pages"], generator=g, device=DEV).to(torch.int32)
        s["table"], used = _tables(c["batch"], c["max_len"], page, order)
        ints = lambda v: torch.tensor(v, device=DEV, dtype=torch.int32)  # noqa: E731
        s["len"], s["start"] = ints(lens), ints([0] + list(np.cumsum(nq)))
        s["nq"] = n = int(sum(nq))
        if c["groups"]:
            s["ptable"], _ = _tables(c["groups"], c["prefix"], page, order, used)
            first = [0] + [int(x) for x in np.cumsum(sizes)]
            s["plen"], s["group"] = ints(plens), ints(first)
            s["most"] = max(sum(nq[a:b]) for a, b in zip(first, first[1:]))      # queries of one group
        shape = (s["pages"], page, c["n_kv"], c["hd"])
        s["kp"], s["ks"] = _pool(g, shape, c["type"], peaks=True)
        s["vp"], s["vs"] = _pool(g, shape, c["type"])
        s["q"] = _bf(g, n, c["heads"], c["hd"])
        s["scale"] = c["hd"] ** -0.5
        s["mask"] = _trees(nq, seed) if c["tree"] else None
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(n, c["heads"], device=DEV)
    if own:                                   # what a serving program keeps: workspace and descriptors
        from ridge_map_kv_amd import binding as B
        n = 256
        if c["op"] != "attend":
            s["rope"] = B.make_rope(**_rope(c))
            s["norm"] = B.make_head_norm(s["qw"], s["kw"], EPS) if c.get("norm", True) else None
        if c["op"] == "norm":
            if c["grad"]:
                n = B.ridgefill_norm_rope_grad_workspace_bytes(c["n"], c["heads"], c["n_kv"], c["hd"])
        else:
            s["kv"] = B.make_batch(s["table"], s["len"], c["page"], s["pages"], c["n_kv"], c["hd"], c["max_len"])
            s["cache"] = B.make_cache(s["kp"], s["vp"], s["ks"], s["vs"])
        if c["op"] == "attend":
            s["prefix"] = B.make_prefix(s["ptable"], s["plen"], s["group"], c["prefix"]) if c["groups"] else None
            n = B.ridgefill_cache_attention_workspace_bytes(s["kv"], c["heads"], c["max_q"], s["nq"], s["prefix"])
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
    if c["op"] == "attend":
        B.ridgefill_cache_attention(s["kv"], s["cache"], s["q"], s["start"], c["max_q"], s["scale"], s["out"],
                                    s["ws"], prefix=s["prefix"], lse=s["lse"], tree_mask=s["mask"])
        return [s["out"], s["lse"]]
    h, n_kv = c["heads"], c["n_kv"]
    q, k, v = s["qkv"][:, :h], s["qkv"][:, h:h + n_kv], s["qkv"][:, h + n_kv:]
    if c["op"] == "append":
        B.ridgefill_append_cache(s["rope"], s["norm"], s["kv"], s["cache"], k, v, s["rows"], s["status"],
                                 seq=s["seq"], q=q, q_out=s["q_out"])
        B.ridgefill_read_rows(s["kv"], s["cache"], s["rows"], s["status"], seq=s["seq"], k_out=s["k_out"],
                              v_out=s["v_out"])
        return [s["q_out"], s["k_out"], s["v_out"]]
    if c["grad"]:
        B.ridgefill_norm_rope_grad(s["rope"], s["norm"], s["pos"], s["ws"], q=q, gq=s["gq"], q_grad=s["q_out"],
                                   qw_grad=s["qw_grad"], k=k, gk=s["gk"], k_grad=s["k_out"], kw_grad=s["kw_grad"])
        return [s["q_out"], s["k_out"], s["qw_grad"], s["kw_grad"]]
    B.ridgefill_norm_rope(s["rope"], s["norm"], s["pos"], q=q, q_out=s["q_out"], k=k, k_out=s["k_out"])
    return [s["q_out"], s["k_out"]]


def _run_plain(s, c):
    if c["op"] == "attend":
        return _attend_plain(s, c)
    h, n_kv = c["heads"], c["n_kv"]
    q, k, v = s["qkv"][:, :h].float(), s["qkv"][:, h:h + n_kv].float(), s["qkv"][:, h + n_kv:].float()
    if c["op"] == "append":
        cos, sin = _angles(c, s["rows"])
        if c["norm"]:
            q, k = _normed(q) * s["qw"].float(), _normed(k) * s["kw"].float()
        s["q_out"].copy_(_rotate(q, cos, sin, c))
        slot = s["table"][s["seq"].long(), (s["rows"] // c["page"]).long()].long() * c["page"] + s["rows"] % c["page"]
        k = _rotate(k, cos, sin, c)
        _write(s["kp"], s["ks"], slot, k, c)
        _write(s["vp"], s["vs"], slot, v, c)
        s["k_out"].copy_(_read(s["kp"], s["ks"], slot, c))
        s["v_out"].copy_(_read(s["vp"], s["vs"], slot, c))
        return [s["q_out"], s["k_out"], s["v_out"]]
    cos, sin = _angles(c, s["pos"])
    if not c["grad"]:
        s["q_out"].copy_(_rotate(_normed(q) * s["qw"].float(), cos, sin, c))
        s["k_out"].copy_(_rotate(_normed(k) * s["kw"].float(), cos, sin, c))
        return [s["q_out"], s["k_out"]]
    dq, dqw = _norm_grad(q, s["qw"].float(), _rotate(s["gq"].float(), cos, -sin, c))
    dk, dkw = _norm_grad(k, s["kw"].float(), _rotate(s["gk"].float(), cos, -sin, c))
    s["q_out"].copy_(dq)
    s["k_out"].copy_(dk)
    s["qw_grad"].copy_(dqw)
    s["kw_grad"].copy_(dkw)
    return [s["q_out"], s["k_out"], s["qw_grad"], s["kw_grad"]]


def _normed(x):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)


def _norm_grad(x, w, g):
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh, wg = x * r, w * g
    return r * (wg - xh * (wg * xh).mean(-1, keepdim=True)), (g * xh).sum((0, 1))


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
    r = c["rot"]
    if c["layout"] == HALF:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def _power(e):
    """2^e of whole numbers, exactly: the exponent's bits of a number in 32 bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _code(x, kind):
    """Codes of x (as the values of the type) and the exponents of their blocks' scales."""
    b = x.unflatten(-1, (-1, BLOCK))
    mant, e = torch.frexp(b.abs().amax(-1))                      # in [0.5, 1) 2^e
    top, bits = torch.frexp(torch.tensor(LARGEST[kind]))
    e = (e - int(bits) + (mant > float(top)).int()).clamp(-110, 118)
    y = b * _power(-e)[..., None]
    y = y.to(torch.float8_e4m3fn).float() if kind == "fp8" else torch.round(y)
    return y.flatten(-2), e


def _write(pool, scales, slot, x, c):
    if c["type"] == "bf16":
        pool.view(-1, c["n_kv"], c["hd"])[slot] = x.to(torch.bfloat16)
        return
    code, e = _code(x, c["type"])
    pool.view(torch.uint8).view(-1, c["n_kv"], c["hd"])[slot] = code.to(pool.dtype).view(torch.uint8)
    scales.view(-1, c["n_kv"], c["hd"] // BLOCK)[slot] = (e + 127).to(torch.uint8)


def _read(pool, scales, slot, c):
    """Rows of a pool in 32 bits."""
    if c["type"] == "bf16":
        return pool.view(-1, c["n_kv"], c["hd"])[slot].float()
    code = pool.view(torch.uint8).view(-1, c["n_kv"], c["hd"])[slot].view(pool.dtype).float()
    e = scales.view(-1, c["n_kv"], c["hd"] // BLOCK)[slot].int() - 127
    return (code.unflatten(-1, (-1, BLOCK)) * _power(e)[..., None]).flatten(-2)


def _gathered(pool, scales, table, max_len, c):
    """The cached rows of every axis of a table, in order: [axes, n_kv, max_len, hd] in 32 bits."""
    t = torch.arange(max_len, device=DEV)
    slot = table.long()[:, t // c["page"]] * c["page"] + t % c["page"]
    return _read(pool, scales, slot, c).permute(0, 2, 1, 3).contiguous()


def _softmax_parts(score, v):
    """Largest score, sum of exponentials about it, and their product with the values."""
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    return m, p.sum(-1, keepdim=True), torch.matmul(p, v)


def _attend_plain(s, c):
    batch, max_q, n_kv, hd, heads = c["batch"], c["max_q"], c["n_kv"], c["hd"], c["heads"]
    group, nothing = heads // n_kv, torch.full((), -math.inf, device=DEV)
    at = torch.arange(s["nq"], device=DEV)
    start = s["start"].long()
    seq = torch.searchsorted(start, at, right=True) - 1
    i = at - start[seq]
    # every sequence's own rows
    q = torch.zeros(batch, max_q, heads, hd, device=DEV)
    q[seq, i] = s["q"].float()
    q = q.view(batch, max_q, n_kv, group, hd).transpose(1, 2).reshape(batch, n_kv, max_q * group, hd)
    score = torch.matmul(q * s["scale"], _gathered(s["kp"], s["ks"], s["table"], c["max_len"], c).transpose(-1, -2))
    t = torch.arange(c["max_len"], device=DEV)
    n = start[1:] - start[:-1]
    draft = t[None, :] - (s["len"] - n)[:, None]
    if s["mask"] is None:
        seen = draft[:, None] <= torch.arange(max_q, device=DEV)[None, :, None]
    else:
        word = torch.zeros(batch, max_q, dtype=torch.int64, device=DEV)
        word[seq, i] = s["mask"]
        seen = (draft < 0)[:, None] | (((word[:, :, None] >> draft.clamp(0, 63)[:, None]) & 1) == 1)
    seen = seen & (t[None, :] < s["len"][:, None])[:, None]
    seen = seen[:, None, :, None].expand(batch, 1, max_q, group, c["max_len"]).reshape(batch, 1, max_q * group, -1)
    m, total, o = _softmax_parts(torch.where(seen, score, nothing), _gathered(s["vp"], s["vs"], s["table"], c["max_len"], c))
    of_query = lambda x: x.view(batch, n_kv, max_q, group, -1).transpose(1, 2)[seq, i]  # noqa: E731
    m, total, o = of_query(m), of_query(total), of_query(o)      # [nq, n_kv, group, 1 or hd]
    if c["groups"]:
        first = s["group"].long()
        of = torch.searchsorted(first, seq, right=True) - 1
        has, of = of < c["groups"], of.clamp(max=c["groups"] - 1)
        place = (at - start[first[of]]).clamp(0, s["most"] - 1)
        q = torch.zeros(c["groups"], s["most"], heads, hd, device=DEV)
        q[of[has], place[has]] = s["q"][has].float()
        q = q.view(c["groups"], s["most"], n_kv, group, hd).transpose(1, 2).reshape(c["groups"], n_kv, -1, hd)
        score = torch.matmul(q * s["scale"], _gathered(s["kp"], s["ks"], s["ptable"], c["prefix"], c).transpose(-1, -2))
        there = torch.arange(c["prefix"], device=DEV)[None] < s["plen"][:, None]
        score = torch.where(there[:, None, None], score, nothing)
        pm, ptotal, po = _softmax_parts(score, _gathered(s["vp"], s["vs"], s["ptable"], c["prefix"], c))
        of_group = lambda x: x.view(c["groups"], n_kv, s["most"], group, -1).transpose(1, 2)[of, place]  # noqa: E731
        pm = torch.where(has[:, None, None, None], of_group(pm), nothing)
        both = torch.maximum(m, pm)
        a, b = torch.exp(m - both), torch.exp(pm - both)
        m, total, o = both, total * a + of_group(ptotal) * b, o * a + of_group(po) * b
    s["out"].copy_((o / total).reshape(s["out"].shape))
    s["lse"].copy_((m + torch.log(total)).reshape(s["lse"].shape))
    return [s["out"], s["lse"]]


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
    if c["op"] == "attend":
        return _exact_attention(s, c)
    h, n_kv = c["heads"], c["n_kv"]
    parts = [(s["qkv"][:, :h].double(), s["qw"].double()), (s["qkv"][:, h:h + n_kv].double(), s["kw"].double())]
    pos = s["rows"] if c["op"] == "append" else s["pos"]
    if c["op"] == "append":
        turned = [_exact_norm_turn(x, w if c["norm"] else None, pos, c) for x, w in parts]
        return [turned[0], _exact_held(turned[1], c["type"]), _exact_held(s["qkv"][:, h + n_kv:].double(), c["type"])]
    if not c["grad"]:
        return [_exact_norm_turn(x, w, pos, c) for x, w in parts]
    dx, dw = [], []
    for (x, w), g in zip(parts, (s["gq"], s["gk"])):             # the gradient by the chain rule
        x.requires_grad_(True)
        w.requires_grad_(True)
        (_exact_norm_turn(x, w, pos, c) * g.double()).sum().backward()
        dx.append(x.grad)
        dw.append(w.grad)
    return dx + dw


def _exact_norm_turn(x, w, pos, c):
    """Norm of every head, then the rotation as a product of complex numbers."""
    if w is not None:
        x = w * x * torch.rsqrt(x.square().sum(-1, keepdim=True) / c["hd"] + EPS)
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
                       torch.outer(pos.double(), torch.tensor(f, device=DEV, dtype=torch.float64)))[:, None]
    if c["layout"] == HALF:
        z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * turn
        return torch.cat([z.real, z.imag, x[..., r:]], -1)
    z = torch.view_as_complex(x[..., :r].contiguous().unflatten(-1, (-1, 2))) * turn
    return torch.cat([torch.view_as_real(z).flatten(-2), x[..., r:]], -1)


def _exact_held(x, kind):
    """What a cache of this type holds of x."""
    if kind == "bf16":
        return x
    powers = torch.tensor([2.0 ** i for i in range(-256, 256)], dtype=torch.float64, device=DEV)
    b = x.unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    e = (torch.searchsorted(LARGEST[kind] * powers, top) - 256).clamp(-110, 118)     # smallest that holds it
    scale = powers[e + 256]
    y = b / scale
    if kind == "int8":
        return (torch.round(y) * scale).flatten(-2)
    above = torch.searchsorted(powers, y.abs(), right=True) - 257                    # its leading bit
    fine = powers[above.clamp(min=-6) - 3 + 256]
    return (torch.round(y / fine) * fine * scale).flatten(-2)


def _exact_values(pool, scales, pages, length, kh, kind):
    """The first `length` rows of an axis of pages, one key head, in 64 bits."""
    rows = pool.view(torch.uint8)[pages][:, :, kh].flatten(0, 1)[:length] if kind != "bf16" else \
        pool[pages][:, :, kh].flatten(0, 1)[:length]
    if kind == "bf16":
        return rows.double()
    powers = torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64, device=DEV)
    scale = powers[scales[pages][:, :, kh].flatten(0, 1)[:length].long()]
    return rows.view(pool.dtype).float().double() * scale.repeat_interleave(BLOCK, -1)


def _exact_attention(s, c):
    """Sequence by sequence and head by head, over one concatenated axis of rows."""
    group, start, lens = c["heads"] // c["n_kv"], s["start"].tolist(), s["len"].tolist()
    out = torch.zeros(s["nq"], c["heads"], c["hd"], device=DEV, dtype=torch.float64)
    lse = torch.zeros(s["nq"], c["heads"], device=DEV, dtype=torch.float64)
    first = s["group"].tolist() if c["groups"] else [0]
    for kh in range(c["n_kv"]):
        held, kept = None, None                    # the prefix of one group at a time
        for b in range(c["batch"]):
            lo, hi, length = start[b], start[b + 1], lens[b]
            n = hi - lo
            k = _exact_values(s["kp"], s["ks"], s["table"][b].long(), length, kh, c["type"])
            v = _exact_values(s["vp"], s["vs"], s["table"][b].long(), length, kh, c["type"])
            seen = torch.ones(n, length, dtype=torch.bool, device=DEV)
            if s["mask"] is None:
                seen[:, length - n:] = torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
            else:
                words = [w & ((1 << 64) - 1) for w in s["mask"][lo:hi].tolist()]
                seen[:, length - n:] = torch.tensor([[bool(w >> j & 1) for j in range(n)] for w in words], device=DEV)
            g = sum(x <= b for x in first) - 1
            if g < c["groups"]:
                if held != g:
                    pages, rows = s["ptable"][g].long(), int(s["plen"][g])
                    kept = [_exact_values(s["kp"], s["ks"], pages, rows, kh, c["type"]),
                            _exact_values(s["vp"], s["vs"], pages, rows, kh, c["type"])]
                    held = g
                k, v = torch.cat([kept[0], k]), torch.cat([kept[1], v])
                seen = torch.cat([torch.ones(n, kept[0].shape[0], dtype=torch.bool, device=DEV), seen], 1)
            x = s["q"][lo:hi, kh * group:(kh + 1) * group].double() @ k.t() * s["scale"]
            x = x.masked_fill(~seen[:, None], -math.inf)
            lse[lo:hi, kh * group:(kh + 1) * group] = torch.logsumexp(x, -1)
            out[lo:hi, kh * group:(kh + 1) * group] = torch.softmax(x, -1) @ v
    return [out, lse]
