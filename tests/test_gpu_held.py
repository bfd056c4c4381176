"""GPU parity of the head norms with their rotation (forward and backward), of the append to caches
of 16 and 8 bits and of reading them back, against plain 64-bit implementations (heldcase.py).
Tolerances count roundings: half a step of what is written, fp32 sums, cos and sin within 2^-20."""

import numpy as np
import pytest
import torch

import cachecase as R
import heldcase as H
from test_gpu_cache import SCALINGS, _close, _randn
from ridge_map_kv_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64


def _rounded(want, off, dtype):
    half = R.U_BF16 if dtype == torch.bfloat16 else R.U_FP32
    return off + half * (want.abs() + off) + 1e-38


def _weights(hd, dtype, seed):
    return tuple((1 + 0.3 * torch.randn(hd, generator=torch.Generator().manual_seed(seed + i))).to(dtype).to(DEV) for i in range(2))


def _positions(n, seed=0):
    return torch.randint(-5000, 70000, (n,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)


SIZES = [(1, 1, 1, 64, 0), (7, 4, 2, 64, 32), (33, 5, 1, 128, 64), (300, 1, 0, 16, 16), (5, 32, 8, 128, 0),
         (3, 0, 2, 256, 256), (9, 3, 3, 96, 48), (2, 3, 1, 80, 80), (70, 6, 2, 48, 16), (64, 40, 8, 128, 128)]


# ---------------------------------------------------------------------------------- norms

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [B.RF_ROPE_HALF, B.RF_ROPE_INTERLEAVED])
@pytest.mark.parametrize("n,hq,hk,hd,rot", SIZES)
def test_norm_rope(dtype, layout, n, hq, hk, hd, rot):
    qw, kw = _weights(hd, dtype, hd)
    for i, scaling in enumerate(SCALINGS[::2]):
        q, k = (_randn(n + i + s, n, h, hd, dtype=dtype) * 2.0 ** s if h else None for s, h in ((0, hq), (3, hk)))
        pos = _positions(n, i)
        rope = B.make_rope(rotary_dim=rot, layout=layout, **scaling)
        for weights in ((qw, kw), (qw, None), (None, kw), None):
            norm = None if weights is None else B.make_head_norm(*weights, 1e-5)
            outs = [None if t is None else torch.empty_like(t) for t in (q, k)]
            B.ridgefill_norm_rope(rope, norm, pos.to(DEV), q, outs[0], k, outs[1])
            for t, out, w in zip((q, k), outs, weights or (None, None)):
                if t is not None:
                    want, off = H.norm_rope(t, w, 1e-5, pos, rot or hd, layout, **scaling)
                    _close(out, want, _rounded(want, off, dtype), f"{scaling} {w is not None}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_without_rotation_and_rotation_without_norm(dtype):
    q = _randn(1, 19, 6, 128, dtype=dtype)
    qw, _ = _weights(128, dtype, 3)
    out, again = torch.empty_like(q), torch.empty_like(q)
    B.ridgefill_norm_rope(None, B.make_head_norm(qw, None, 0.0), None, q, out)
    want, off = H.normed(q, qw, 0.0)
    _close(out, want, _rounded(want, off, dtype), "norm alone")
    pos = _positions(19).to(DEV)
    rope = B.make_rope(rotary_dim=64)
    B.ridgefill_norm_rope(rope, None, pos, q, out)
    B.ridgefill_rope(rope, q, pos, again)
    assert torch.equal(out, again)                     # the rotation alone is ridgefill_rope's
    B.ridgefill_norm_rope(None, None, None, q, out)
    assert torch.equal(out, q)


def test_norm_strided_and_in_place():
    # q, k and v of a row side by side, as a fused projection leaves them
    base = _randn(4, 29, (6 + 2 + 2) * 64 + 8).view(29, -1)
    q, k = base[:, :384].unflatten(1, (6, 64)), base[:, 384:512].unflatten(1, (2, 64))
    qw, kw = _weights(64, torch.bfloat16, 5)
    pos, before = _positions(29), base.clone()
    rope, norm = B.make_rope(), B.make_head_norm(qw, kw)
    out_q, out_k = torch.full((29, 7, 64), 9.0, dtype=torch.bfloat16, device=DEV), torch.empty(29, 2, 64, dtype=torch.bfloat16, device=DEV)
    B.ridgefill_norm_rope(rope, norm, pos.to(DEV), q, out_q[:, :6], k, out_k)
    want, off = H.norm_rope(q, qw, 1e-6, pos, 64, 0)
    _close(out_q[:, :6], want, _rounded(want, off, torch.bfloat16), "q")
    assert (out_q[:, 6] == 9).all() and torch.equal(base, before)
    B.ridgefill_norm_rope(rope, norm, pos.to(DEV), q, q, k, k)
    assert torch.equal(q, out_q[:, :6]) and torch.equal(k, out_k)
    assert torch.equal(base[:, 512:], before[:, 512:])


def test_norm_of_zeros_infinities_and_large_values():
    q = torch.zeros(6, 1, 64, device=DEV)
    q[1, 0, 5] = float("inf")
    q[2, 0, 5] = float("nan")
    q[3] = 2.0 ** 59
    q[4] = 2.0 ** -70
    q[5, 0, 0] = 1.0
    w = torch.ones(64, device=DEV)
    out = torch.empty_like(q)
    B.ridgefill_norm_rope(None, B.make_head_norm(w, None, 1e-6), None, q, out)
    assert (out[0] == 0).all()
    assert torch.isnan(out[1, 0, 5]) and (out[1, 0, :5] == 0).all()      # infinite times 0
    assert torch.isnan(out[2]).all()
    _close(out[3:], *(lambda y: (y[0], y[1] + 1e-38))(H.normed(q[3:], w, 1e-6)), "sizes")
    B.ridgefill_norm_rope(None, B.make_head_norm(w, None, 0.0), None, q[:1], out[:1])
    assert torch.isnan(out[0]).all()


def _grads(rope, norm, pos, q, gq, k, gk, dtype, hd, want_w=True, in_place=False):
    n = (gq if gq is not None else gk).shape[0]
    ws = torch.full((B.ridgefill_norm_rope_grad_workspace_bytes(n, 0 if gq is None else gq.shape[1], 0 if gk is None else gk.shape[1], hd),),
                    0xff, dtype=torch.uint8, device=DEV)
    outs = [None if g is None else g.clone() if in_place else torch.empty_like(g) for g in (gq, gk)]
    dws = [torch.full((hd,), 7.0, device=DEV) if want_w and g is not None else None for g in (gq, gk)]
    B.ridgefill_norm_rope_grad(rope, norm, pos, ws, q, outs[0] if in_place else gq, outs[0], dws[0],
                               k, outs[1] if in_place else gk, outs[1], dws[1])
    return outs, dws


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [B.RF_ROPE_HALF, B.RF_ROPE_INTERLEAVED])
@pytest.mark.parametrize("n,hq,hk,hd,rot", SIZES + [(1500, 3, 2, 64, 64), (2049, 2, 1, 128, 0)])
def test_norm_rope_grad(dtype, layout, n, hq, hk, hd, rot):
    qw, kw = _weights(hd, dtype, hd + 1)
    scaling = SCALINGS[4] if rot else SCALINGS[0]
    q, k, gq, gk = (_randn(n + s, n, h, hd, dtype=dtype) * 2.0 ** s if h else None
                    for s, h in ((0, hq), (3, hk), (1, hq), (2, hk)))
    pos = _positions(n, 9)
    rope = B.make_rope(rotary_dim=rot, layout=layout, **scaling)
    for weights in ((qw, kw), (qw, None), (None, kw), None):
        norm = None if weights is None else B.make_head_norm(*weights, 1e-5)
        outs, dws = _grads(rope, norm, pos.to(DEV), q, gq, k, gk, dtype, hd)
        for t, g, out, dw, w in zip((q, k), (gq, gk), outs, dws, weights or (None, None)):
            if g is None:
                continue
            dx, want, off, w_off = H.norm_rope_grad(t, w, 1e-5, g, pos, rot or hd, layout, **scaling)
            _close(out, dx, _rounded(dx, off, dtype), "x")
            if w is None:
                assert (dw == 7).all()                 # no weight, no gradient
            else:
                _close(dw, want, w_off + R.U_FP32 * want.abs(), "w")
        again, dws2 = _grads(rope, norm, pos.to(DEV), q, gq, k, gk, dtype, hd, in_place=True)
        for a, b in zip(outs + dws, again + dws2):     # in place, and the same bits again
            assert a is None or torch.equal(a, b)
        alone, _ = _grads(rope, norm, pos.to(DEV), q, gq, k, gk, dtype, hd, want_w=False)
        for a, b in zip(outs, alone):
            assert a is None or torch.equal(a, b)


def test_norm_rope_grad_of_differences():
    n, h, hd, eps, step = 5, 3, 64, 1e-5, 2.0 ** -5
    q, gq = _randn(1, n, h, hd, dtype=torch.float32), _randn(2, n, h, hd, dtype=torch.float32)
    qw, _ = _weights(hd, torch.float32, 2)
    pos = _positions(n, 1)
    rope = B.make_rope(rotary_dim=32)
    (dx, _), (dw, _) = _grads(rope, B.make_head_norm(qw, None, eps), pos.to(DEV), q, gq, None, None, torch.float32, hd)
    dx64, dw64, dx_off, dw_off = H.norm_rope_grad(q, qw, eps, gq, pos, 32, 0)
    g = gq.cpu().to(F64)

    def run(x, w):
        out = torch.empty_like(x)
        B.ridgefill_norm_rope(rope, B.make_head_norm(w, None, eps), pos.to(DEV), x, out)
        want, off = H.norm_rope(x, w, eps, pos, 32, 0)
        off = _rounded(want, off, torch.float32)
        return float((out.cpu().to(F64) * g).sum()), float((want * g).sum()), float((off * g.abs()).sum())

    def difference(change):
        (a, a64, ea), (b, b64, eb) = (run(*change(s)) for s in (step, -step))
        return (a - b) / (2 * step), (a64 - b64) / (2 * step), (ea + eb) / (2 * step)

    for row, head, feature in ((0, 0, 0), (1, 2, 17), (4, 1, 31), (2, 0, 40), (3, 2, 63)):
        def change(s):
            x = q.clone()
            x[row, head, feature] += s
            return x, qw
        moved = float(change(step)[0][row, head, feature] - change(-step)[0][row, head, feature]) / (2 * step)
        got, want, off = (v / moved for v in difference(change))
        # the difference's own distance from the derivative, in 64 bits
        off += abs(want - float(dx64[row, head, feature]))
        assert abs(got - float(dx[row, head, feature])) <= off + float(dx_off[row, head, feature]) * 1.01
    for feature in (0, 20, 63):
        def change(s):
            w = qw.clone()
            w[feature] += s
            return q, w
        moved = float(change(step)[1][feature] - change(-step)[1][feature]) / (2 * step)
        got, want, off = (v / moved for v in difference(change))
        off += abs(want - float(dw64[feature]))
        assert abs(got - float(dw[feature])) <= off + float(dw_off[feature]) * 1.01


@pytest.mark.parametrize("layout", [B.RF_ROPE_HALF, B.RF_ROPE_INTERLEAVED])
def test_turns_of_normed_fp32_rows_are_as_near_as_their_rounding(layout):
    # 1 at one feature alone: r is 8, and y is 8 cos p and 8 sin p, exactly as the kernel holds them.  At positions
    # near half a turn, where the sine is below 2^-3 and its last place 2^-27: within four of those and its rounding,
    # 3.4e-8; the rounding of the angle to fp32 alone would put it up to pi 2^-25 = 9.4e-8 off
    p = np.arange(70000)
    turn = p / (2 * np.pi)
    p = p[np.abs(2 * (turn - np.rint(turn))) > 0.97]
    n, other, tol = len(p), 32 if layout == B.RF_ROPE_HALF else 1, 4.5 * 2.0 ** -27
    assert n > 1000 and np.abs(np.sin(p)).max() < 2.0 ** -3
    pos = torch.from_numpy(p.astype(np.int32)).to(DEV)
    w, rope = torch.ones(64, device=DEV), B.make_rope(layout=layout)
    norm = B.make_head_norm(w, w, 0.0)
    cos, sin = torch.from_numpy(np.cos(p)), torch.from_numpy(np.sin(p))
    x, g = torch.zeros(n, 1, 64, device=DEV), torch.zeros(n, 1, 64, device=DEV)
    x[:, :, 0] = 1
    q, k = torch.empty_like(x), torch.empty_like(x)
    B.ridgefill_norm_rope(rope, norm, pos, x, q, x, k)
    for y in (q, k):
        y = y.cpu().to(F64)[:, 0] / 8
        assert float((y[:, 0] - cos).abs().max()) <= 4.5 * 2.0 ** -24 and float((y[:, other] - sin).abs().max()) <= tol
    # backward: the row's norm lies in a feature that the gradient does not touch, so that dx is 8 g
    x.zero_()
    x[:, :, 63] = 1
    g[:, :, 0] = 1
    (dq, dk), _ = _grads(rope, norm, pos, x, g, x, g, torch.float32, 64)
    for y in (dq, dk):
        y = y.cpu().to(F64)[:, 0] / 8
        assert float((y[:, 0] - cos).abs().max()) <= 4.5 * 2.0 ** -24 and float((y[:, other] + sin).abs().max()) <= tol


def test_root_of_the_mean_is_within_half_a_place():
    # rows of v = 1 + k / 1024, 1 and zeros: the mean of squares is (v^2 + 1) / 64, exact in fp32 (at most 23 bits), and
    # what a weight of 1 makes of the 1 is the root itself; second-order terms of its correction are below 2^-20
    k = np.arange(1024)
    x = torch.zeros(1024, 1, 64, device=DEV)
    x[:, 0, 3], x[:, 0, 40] = torch.from_numpy((1 + k / 1024).astype(np.float32)).to(DEV), 1
    out = torch.empty_like(x)
    B.ridgefill_norm_rope(None, B.make_head_norm(torch.ones(64, device=DEV), None, 0.0), None, x, out)
    want = (((1 + k / 1024) ** 2 + 1) / 64) ** -0.5
    got = out[:, 0, 40].cpu().numpy()
    assert np.abs(got - want).max() > 0 and (np.abs(got - want) <= (0.5 + 2.0 ** -10) * np.spacing(got)).all()


def test_norm_empty():
    q = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    pos = torch.empty(0, dtype=torch.int32, device=DEV)
    qw, _ = _weights(64, torch.bfloat16, 1)
    norm = B.make_head_norm(qw, None)
    B.ridgefill_norm_rope(B.make_rope(), norm, pos, q, q)
    _, (dw, _) = _grads(B.make_rope(), norm, pos, q, q, None, None, torch.bfloat16, 64)
    assert (dw == 0).all()                             # the sum over no rows


# ---------------------------------------------------------------------------------- caches

def _place(seq, rows, table, page):
    page_of = torch.from_numpy(table.astype(np.int64))[seq, rows // page]
    return page_of.to(DEV), torch.from_numpy((rows % page).astype(np.int64)).to(DEV)


def _check_held(got, scales, want, off, kind, what):
    """Values of a cache against what went in: half a step of the type, of a scale that is the
    rule's for a largest value within the error."""
    if kind == "bf16":
        return _close(got, want, _rounded(want, off, torch.bfloat16), what)
    b, t = want.unflatten(-1, (-1, 32)), off.unflatten(-1, (-1, 32))
    lo, hi = (H.exponents((b.abs() + s * t).clamp(min=0).amax(-1).numpy(), kind) + 127 for s in (-1, 1))
    byte = scales.cpu().numpy().astype(np.int64)
    assert ((lo <= byte) & (byte <= hi)).all(), what
    step = torch.from_numpy(2.0 ** (byte - 127.0))[..., None].expand(b.shape).flatten(-2)
    if kind == "int8":
        tol = 0.5 * step + off
    else:
        tol = torch.maximum((want.abs() + off) * 2.0 ** -4, step * 2.0 ** -10) + off
    _close(got, want, tol * (1 + 2.0 ** -40), what)


HOLD = [(128, 8, 32, 16, 0, 0), (64, 2, 4, 4, 32, 1), (128, 1, 5, 7, 64, 0), (64, 3, 0, 1, 0, 1), (96, 2, 2, 5, 48, 0),
        (32, 1, 1, 100, 0, 0), (256, 2, 3, 3, 64, 1), (160, 1, 2, 16, 160, 0), (192, 2, 1, 8, 16, 1)]


@pytest.mark.parametrize("kind", H.KINDS)
@pytest.mark.parametrize("hd,n_kv,n_q,page,rot,layout", HOLD)
def test_append_cache_and_read_back(kind, hd, n_kv, n_q, page, rot, layout):
    n, batch, max_len = 37, 3, 64
    num_pages = batch * -(-max_len // page) + 2
    g = np.random.default_rng(page + hd)
    table_np = g.permutation(num_pages)[:num_pages - 2].reshape(batch, -1).astype(np.int32)
    scaling = SCALINGS[4]
    qkv = _randn(hd, n, n_q + 2 * n_kv, hd) * torch.exp2(_randn(hd + 1, n, n_q + 2 * n_kv, 1) * 4)
    places = g.permutation(batch * max_len)[:n]
    seq_np, rows_np = (places // max_len).astype(np.int32), (places % max_len).astype(np.int32)
    seq_np[[2, 30]] = -1                                  # padding rows
    real = np.flatnonzero(seq_np >= 0)
    pos = torch.from_numpy(g.integers(0, 40000, n).astype(np.int32))
    seq, rows = torch.from_numpy(seq_np).to(DEV), torch.from_numpy(rows_np).to(DEV)
    q, k, v = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    qw, kw = _weights(hd, torch.bfloat16, 1)
    kv = B.make_batch(torch.from_numpy(table_np).to(DEV), None, page, num_pages, n_kv, hd, max_len)
    status = torch.full((1,), -1, dtype=torch.int32, device=DEV)
    for weights, use_pos, turn in (((qw, kw), True, True), ((None, kw), False, True), (None, True, True), ((qw, kw), True, False)):
        kp, vp, ks, vs = H.pools(num_pages, page, n_kv, hd, kind, fill=0x55)
        cache = B.make_cache(kp, vp, ks, vs)
        norm = None if weights is None else B.make_head_norm(*weights, 1e-5)
        q_out = torch.full((n, max(n_q, 1), hd), 5.0, dtype=torch.bfloat16, device=DEV)
        rope = B.make_rope(rotary_dim=rot, layout=layout, **scaling) if turn else None
        B.ridgefill_append_cache(rope, norm, kv, cache, k, v, rows, status, seq=seq, positions=pos.to(DEV) if use_pos else None,
                                 q=q if n_q else None, q_out=q_out if n_q else None)
        assert B.ridgefill_read_status(status) == B.RF_OK
        at = pos if use_pos else rows.cpu()
        turned = (rot or hd) if turn else 0
        page_of, slot = _place(seq_np[real], rows_np[real], table_np, page)
        if n_q:
            want, off = H.norm_rope(q, weights[0] if weights else None, 1e-5, at, turned, layout, **scaling)
            _close(q_out[real], want[real], _rounded(want, off, torch.bfloat16)[real], "q")
            assert (q_out[[2, 30]] == 5).all()
        want, off = H.norm_rope(k, weights[1] if weights else None, 1e-5, at, turned, layout, **scaling)
        held = [H.values(p[page_of, slot] if p.dtype != torch.float8_e4m3fn else p.view(torch.uint8)[page_of, slot].view(p.dtype),
                         None if s is None else s[page_of, slot]) for p, s in ((kp, ks), (vp, vs))]
        _check_held(held[0], None if ks is None else ks[page_of, slot], want[real], off[real], kind, "k")
        exact, scale = H.held(v[real], kind)              # v comes as it is: its codes are the rule's
        assert torch.equal(held[1], exact)
        assert scale is None or torch.equal(vs[page_of, slot].cpu(), scale)
        for pool in (kp, vp, ks, vs):                     # nothing else is touched
            if pool is not None:
                rest = pool.view(torch.uint8).clone()
                rest[page_of, slot] = 0x55
                assert (rest == 0x55).all()
        # and back, whole and in strides, in both types
        for dtype in (torch.bfloat16, torch.float32):
            wide = torch.full((n, 2 * n_kv + 1, hd), 3.0, dtype=dtype, device=DEV)
            k_out, v_out = wide[:, :n_kv], wide[:, n_kv:2 * n_kv]
            B.ridgefill_read_rows(kv, cache, rows, status, seq=seq, k_out=k_out, v_out=v_out)
            assert B.ridgefill_read_status(status) == B.RF_OK
            assert torch.equal(k_out[real].cpu().to(F64), held[0]) and torch.equal(v_out[real].cpu().to(F64), held[1])
            assert (wide[[2, 30]] == 3).all() and (wide[:, 2 * n_kv] == 3).all()
            only = torch.empty(n, n_kv, hd, dtype=dtype, device=DEV)
            B.ridgefill_read_rows(kv, cache, rows, status, seq=seq, v_out=only)
            assert torch.equal(only[real], v_out[real])
            B.ridgefill_read_rows(kv, cache, rows, status, seq=seq, k_out=only)
            assert torch.equal(only[real], k_out[real])


def test_append_cache_without_norm_is_append_rows():
    cache = R.Cache([40, 9], 2, 128, 16, max_len=64, seed=3)
    qkv = _randn(1, 20, 8, 128)
    rows = torch.arange(20, dtype=torch.int32, device=DEV) * 3
    rope = B.make_rope(rotary_dim=64)
    outs = []
    for new in (False, True):
        kp, vp, q_out = cache.k[0].clone(), cache.v[0].clone(), torch.empty(20, 4, 128, dtype=torch.bfloat16, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        if new:
            B.ridgefill_append_cache(rope, None, cache.batch(B), B.make_cache(kp, vp), qkv[:, 4:6], qkv[:, 6:], rows, status,
                                     q=qkv[:, :4], q_out=q_out)
        else:
            B.ridgefill_append_rows(rope, cache.batch(B), qkv[:, 4:6], qkv[:, 6:], rows, kp, vp, status, q=qkv[:, :4], q_out=q_out)
        assert B.ridgefill_read_status(status) == B.RF_OK
        outs.append([t.view(torch.int16) for t in (kp, vp, q_out)])
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_what_8_bits_hold(kind):
    # magnitudes over the whole range of bf16, at and next to the scales' borders; ties; blocks of zeros,
    # of one value, with infinities and NaN
    most = H.MOST[kind]
    g = torch.Generator().manual_seed(3)
    x = torch.randn(64, 1, 128, generator=g) * torch.exp2(torch.randint(-126, 120, (64, 1, 128), generator=g).float())
    x[8:24] = torch.randn(16, 1, 128, generator=g) * torch.exp2(torch.randint(-12, 12, (16, 1, 1), generator=g).float())
    for i, top in enumerate((most, most * 1.01, most / 2, most * 0.99, 1.0, 2.0 ** -126, 2.0 ** 127, 3.3e38)):
        x[i] = torch.linspace(-1, 1, 128) * top
    x[24, 0, :32] = 0
    x[24, 0, 32:64] = torch.tensor([most] + [0.5 + 0.25 * j for j in range(31)])      # ties of whole and of eighths
    x[25, 0, 5], x[25, 0, 40], x[25, 0, 127] = float("inf"), float("nan"), -float("inf")
    x[26] = 0
    x[26, 0, 64] = 2.0 ** -133                            # the smallest of bf16
    x[27] = -0.0
    x = x.bfloat16().to(DEV)
    kv = B.make_batch(torch.arange(4, dtype=torch.int32, device=DEV).view(1, 4), None, 16, 4, 1, 128)
    kp, vp, ks, vs = H.pools(4, 16, 1, 128, kind, fill=0x55)
    cache, rows = B.make_cache(kp, vp, ks, vs), torch.arange(64, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.ridgefill_append_cache(None, None, kv, cache, x, x.flip(0), rows, status)
    assert B.ridgefill_read_status(status) == B.RF_OK
    want, scale = H.held(x, kind)
    assert torch.equal(ks.view(64, 1, 4).cpu(), scale)
    k_out, v_out = torch.empty_like(x), torch.empty(64, 1, 128, device=DEV)
    B.ridgefill_read_rows(kv, cache, rows, status, k_out=k_out)
    B.ridgefill_read_rows(kv, cache, rows.flip(0), status, v_out=v_out)
    for got in (k_out, v_out):
        got = got.cpu().to(F64)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    assert torch.isnan(want[25, 0, :64]).all() and torch.isfinite(want[25, 0, 64:96]).all()
    # values that a cache has held are held as they are
    B.ridgefill_append_cache(None, None, kv, cache, k_out, k_out, rows, status)
    again = torch.empty_like(x)
    B.ridgefill_read_rows(kv, cache, rows, status, k_out=again)
    same = (again == k_out) | (torch.isnan(again) & torch.isnan(k_out))
    assert same.all()


@pytest.mark.parametrize("kind", H.KINDS)
def test_bad_rows_of_append_and_read(kind):
    table = torch.tensor([[2, 0, 5, 1], [7, 9, -1, 4]], dtype=torch.int32, device=DEV)       # 9 and -1 are no pages of 8
    kv = B.make_batch(table, None, 4, 8, 1, 64, 16)
    k, v, q = (_randn(s, 8, 1, 64) for s in (1, 2, 3))
    seq = torch.tensor([0, 0, 2, 1, 1, 0, 1, -1], dtype=torch.int32, device=DEV)
    rows = torch.tensor([0, 16, 3, 9, 3, -1, 5, 100], dtype=torch.int32, device=DEV)
    kp, vp, ks, vs = H.pools(8, 4, 1, 64, kind, fill=0x55)
    cache, status, q_out = B.make_cache(kp, vp, ks, vs), torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros_like(q)
    B.ridgefill_append_cache(None, None, kv, cache, k, v, rows, status, seq=seq, q=q, q_out=q_out)
    assert B.ridgefill_read_status(status) == B.RF_E_ROWS
    changed = (kp.view(torch.uint8) != 0x55).flatten(2).any(-1).nonzero().tolist()
    assert sorted(map(tuple, changed)) == [(2, 0), (7, 3)]
    assert torch.equal(q_out[:7], q[:7]) and (q_out[7] == 0).all()
    out = torch.full_like(k, 3.0)
    B.ridgefill_read_rows(kv, cache, rows, status, seq=seq, k_out=out)
    assert B.ridgefill_read_status(status) == B.RF_E_ROWS
    good = torch.tensor([0, 4], device=DEV)
    want = H.held(k[good], kind)[0]
    assert torch.equal(out[good].cpu().to(F64), want)
    rest = torch.ones(8, dtype=torch.bool, device=DEV)
    rest[good] = False
    assert (out[rest] == 3).all()
    B.ridgefill_read_rows(kv, cache, rows[:1].repeat(5), status, seq=seq[:1].repeat(5), k_out=out[:5])   # one row many times
    assert B.ridgefill_read_status(status) == B.RF_OK
    assert (out[:5] == out[0]).all()
    B.ridgefill_read_rows(kv, cache, rows[:0], status, k_out=out[:0])
    assert B.ridgefill_read_status(status) == B.RF_OK


@pytest.mark.parametrize("n,n_kv", [(5000, 1), (4097, 2), (9000, 1)])
def test_many_short_rows_of_append_and_read(n, n_kv):
    # rows so many and short that the workgroups report, not one that looks them over
    num_pages, page = -(-n // 16), 16
    table = torch.randperm(num_pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(1, -1)
    kv = B.make_batch(table.to(DEV), None, page, num_pages, n_kv, 64, n)
    k, v = (_randn(s, n, n_kv, 64) for s in (1, 2))
    rows = torch.randperm(n, generator=torch.Generator().manual_seed(2)).to(torch.int32).to(DEV)
    kp, vp, ks, vs = H.pools(num_pages, page, n_kv, 64, "int8")
    cache, status = B.make_cache(kp, vp, ks, vs), torch.full((1,), -1, dtype=torch.int32, device=DEV)
    B.ridgefill_append_cache(None, None, kv, cache, k, v, rows, status)
    assert B.ridgefill_read_status(status) == B.RF_OK
    k_out, v_out = torch.empty_like(k), torch.empty_like(v)
    B.ridgefill_read_rows(kv, cache, rows, status, k_out=k_out, v_out=v_out)
    assert B.ridgefill_read_status(status) == B.RF_OK
    assert torch.equal(k_out.cpu().to(F64), H.held(k, "int8")[0]) and torch.equal(v_out.cpu().to(F64), H.held(v, "int8")[0])
    rows[n - 1] = n
    for call in (lambda: B.ridgefill_append_cache(None, None, kv, cache, k, v, rows, status),
                 lambda: B.ridgefill_read_rows(kv, cache, rows, status, k_out=k_out)):
        call()
        assert B.ridgefill_read_status(status) == B.RF_E_ROWS


# ---------------------------------------------------------------------------------- many rows
# Enough rows that workgroups take several at a time, or block after block of them, with a rest in the last.

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,hq,hk,hd,rot", [(4099, 40, 8, 128, 0), (65601, 2, 1, 64, 32)])
def test_norm_rope_of_many_rows(dtype, n, hq, hk, hd, rot):
    qw, kw = _weights(hd, dtype, 4)
    q, k = _randn(1, n, hq, hd, dtype=dtype), _randn(2, n, hk, hd, dtype=dtype) * 8
    pos, rope = _positions(n, 3), B.make_rope(rotary_dim=rot)
    outs = [torch.full_like(t, 9.0) for t in (q, k)]
    B.ridgefill_norm_rope(rope, B.make_head_norm(qw, kw, 1e-5), pos.to(DEV), q, outs[0], k, outs[1])
    for t, out, w in zip((q, k), outs, (qw, kw)):
        want, off = H.norm_rope(t, w, 1e-5, pos, rot or hd, 0)
        _close(out, want, _rounded(want, off, dtype), "many rows")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,hq,hk,hd,rot", [(1601, 40, 8, 128, 64), (25001, 2, 1, 64, 0)])
def test_norm_rope_grad_of_many_rows(dtype, n, hq, hk, hd, rot):
    qw, kw = _weights(hd, dtype, 5)
    q, k, gq, gk = (_randn(s, n, h, hd, dtype=dtype) for s, h in ((1, hq), (2, hk), (3, hq), (4, hk)))
    pos, rope = _positions(n, 6), B.make_rope(rotary_dim=rot)
    outs, dws = _grads(rope, B.make_head_norm(qw, kw, 1e-5), pos.to(DEV), q, gq, k, gk, dtype, hd)
    for t, g, out, dw, w in zip((q, k), (gq, gk), outs, dws, (qw, kw)):
        dx, want, off, _ = H.norm_rope_grad(t, w, 1e-5, g, pos, rot or hd, 0)
        _close(out, dx, _rounded(dx, off, dtype), "x")
        # A weight's sum: a thread adds the heads of its place, at most nine of these sizes; then 64 lanes by pairs, four
        # waves, and of at most 768 workgroups twelve rows and 64 sums: below 96 additions one after another,
        # each of which errs by half a place of no more than the sum of the magnitudes, which are within
        # those of the rotated gradient (cos and sin 2^-20), the row's sum of squares and a few products
        x, gy = t.cpu().to(F64), g.cpu().to(F64)
        size = R.rotate(gy, pos, rot or hd, 0, True)[1]
        size[..., rot or hd:] = gy[..., rot or hd:].abs()
        xh = (x * (x.square().mean(-1, keepdim=True) + float(np.float32(1e-5))) ** -0.5).abs()
        tol = (size * xh).sum((0, 1)) * (2.0 ** -20 + (hd / 2 + 8 + 96) * R.U_FP32)
        _close(dw, want, tol, "w")


@pytest.mark.parametrize("kind", H.KINDS)
def test_append_of_many_rows(kind):
    n, n_q, n_kv, hd, page, max_len = 4099, 32, 8, 128, 16, 2100
    per = -(-max_len // page)
    g = np.random.default_rng(8)
    table_np = g.permutation(2 * per + 1)[:2 * per].reshape(2, per).astype(np.int32)
    places = g.permutation(2 * max_len)[:n]
    seq_np, rows_np = (places // max_len).astype(np.int32), (places % max_len).astype(np.int32)
    qkv = _randn(9, n, n_q + 2 * n_kv, hd)
    q, k, v = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    qw, kw = _weights(hd, torch.bfloat16, 7)
    kv = B.make_batch(torch.from_numpy(table_np).to(DEV), None, page, 2 * per + 1, n_kv, hd, max_len)
    status = torch.full((1,), -1, dtype=torch.int32, device=DEV)
    kp, vp, ks, vs = H.pools(2 * per + 1, page, n_kv, hd, kind)
    seq, rows, q_out = torch.from_numpy(seq_np).to(DEV), torch.from_numpy(rows_np).to(DEV), torch.full((n, n_q, hd), 9.0, dtype=torch.bfloat16, device=DEV)
    cache = B.make_cache(kp, vp, ks, vs)
    B.ridgefill_append_cache(B.make_rope(), B.make_head_norm(qw, kw, 1e-5), kv, cache, k, v, rows, status, seq=seq, q=q, q_out=q_out)
    assert B.ridgefill_read_status(status) == B.RF_OK
    at = torch.from_numpy(rows_np)
    want, off = H.norm_rope(q, qw, 1e-5, at, hd, 0)
    _close(q_out, want, _rounded(want, off, torch.bfloat16), "q")
    k_out, v_out = torch.empty(n, n_kv, hd, device=DEV), torch.empty(n, n_kv, hd, device=DEV)
    B.ridgefill_read_rows(kv, cache, rows, status, seq=seq, k_out=k_out, v_out=v_out)
    assert B.ridgefill_read_status(status) == B.RF_OK
    want, off = H.norm_rope(k, kw, 1e-5, at, hd, 0)
    page_of, slot = _place(seq_np, rows_np, table_np, page)
    _check_held(k_out.cpu().to(F64), None if ks is None else ks[page_of, slot], want, off, kind, "k")
    assert torch.equal(v_out.cpu().to(F64), H.held(v, kind)[0])
