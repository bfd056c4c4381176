"""CPU checks of the head norms' calls and of the caches in 16 and 8 bits: invalid arguments are
refused on the host, with a status and a text, before anything is enqueued; size queries; the
binding's own checks; and the plain 64-bit gradient that the GPU tests compare with, against
differences."""

import ctypes as C

import pytest
import torch

import heldcase as H
from test_cache_refusals import BAD_KV, FAKE, _kv, _refused
from ridge_map_kv_amd import binding as B


def _norm(q_w=FAKE, k_w=FAKE, eps=1e-6, reserved=0):
    return B.rf_head_norm(q_w, k_w, eps, reserved)


BAD_NORM_SHAPE = [dict(q_w=FAKE + 8), dict(k_w=FAKE + 2)]
BAD_NORM = [dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(reserved=1)]


def _forward(norm=None, kind=0, n=4, hd=64, pos=FAKE, q=FAKE, hq=2, qs=128, qo=FAKE + 65536, qos=128, k=FAKE, hk=1, ks=64,
             ko=FAKE + 65536, kos=64, rope=True, **kw):
    r = B.make_rope(**kw)
    return B.lib().ridgefill_norm_rope(C.byref(r) if rope else None, C.byref(norm or _norm()), kind, n, hd, pos, q, hq, qs, qo, qos,
                                       k, hk, ks, ko, kos, None)


def _backward(norm=None, kind=0, n=4, hd=64, pos=FAKE, q=FAKE, hq=2, qs=128, gq=FAKE, gqs=128, qg=FAKE + 65536, qgs=128, qw=FAKE,
              k=FAKE, hk=1, ks=64, gk=FAKE, gks=64, kg=FAKE + 65536, kgs=64, kw_=FAKE + 1024, ws=FAKE, ws_bytes=1 << 20, **kw):
    r = B.make_rope(**kw)
    return B.lib().ridgefill_norm_rope_grad(C.byref(r), C.byref(norm or _norm()), kind, n, hd, pos, q, hq, qs, gq, gqs, qg, qgs, qw,
                                            k, hk, ks, gk, gks, kg, kgs, kw_, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [_forward, _backward])
def test_norm_refusals(call):
    for kw in (dict(hd=40), dict(hd=272), dict(hd=0), dict(hq=-1), dict(hq=5000), dict(hk=5000), dict(hq=0, hk=0), dict(n=-1),
               dict(n=(1 << 23) + 1), dict(qs=120), dict(ks=56), dict(qs=132), dict(kind=1, qs=130), dict(q=FAKE + 8),
               dict(k=FAKE + 4), dict(pos=FAKE + 2), dict(rotary_dim=128), dict(rotary_dim=8)):
        _refused(call(**kw), B.RF_E_SHAPE)
    for kw in (dict(kind=2), dict(q=None), dict(k=None), dict(hq=0), dict(hk=0), dict(pos=None), dict(theta=0.5), dict(layout=3)):
        _refused(call(**kw), B.RF_E_INVALID)
    for kw in BAD_NORM_SHAPE:
        _refused(call(norm=_norm(**kw)), B.RF_E_SHAPE)
    for kw in BAD_NORM:
        _refused(call(norm=_norm(**kw)), B.RF_E_INVALID)


def test_forward_refusals():
    for kw in (dict(qos=120), dict(kos=65), dict(qo=FAKE + 8), dict(ko=FAKE + 2)):
        _refused(_forward(**kw), B.RF_E_SHAPE)
    for kw in (dict(qo=None), dict(ko=None), dict(qo=FAKE, qos=136), dict(ko=FAKE, kos=72)):
        _refused(_forward(**kw), B.RF_E_INVALID)
    assert _forward(n=0, q=None, qo=None, k=None, ko=None, pos=None) == B.RF_OK


def test_backward_refusals():
    for kw in (dict(gqs=120), dict(gks=65), dict(qgs=120), dict(kgs=65), dict(gq=FAKE + 8), dict(gk=FAKE + 2), dict(qg=FAKE + 4),
               dict(kg=FAKE + 8), dict(qw=FAKE + 2), dict(kw_=FAKE + 1)):
        _refused(_backward(**kw), B.RF_E_SHAPE)
    for kw in (dict(gq=None), dict(gk=None), dict(qg=None), dict(kg=None), dict(qg=FAKE, qgs=136), dict(kg=FAKE, kgs=72),
               dict(ws=None), dict(hk=0, k=None, gk=None, kg=None), dict(kw_=FAKE)):        # the last: one gradient for two weights
        _refused(_backward(**kw), B.RF_E_INVALID)
    need = B.ridgefill_norm_rope_grad_workspace_bytes(4, 2, 1, 64)
    for kw in (dict(ws=FAKE + 64), dict(ws_bytes=need - 1)):
        _refused(_backward(**kw), B.RF_E_WORKSPACE)


def test_norm_workspace():
    size = B.ridgefill_norm_rope_grad_workspace_bytes
    assert size(4, 2, 1, 64) > 0 and size(0, 2, 1, 64) > 0
    assert size(1 << 23, 32, 8, 128) == size(1 << 14, 40, 8, 128)      # bounded by the workgroups
    for bad in ((-1, 2, 1, 64), ((1 << 23) + 1, 2, 1, 64), (4, 0, 0, 64), (4, 5000, 0, 64), (4, 2, -1, 64), (4, 2, 1, 40),
                (1 << 40, 2, 1, 64), (4, 1 << 33, 1, 64)):
        assert size(*bad) == 0


def _cache(kind=0, reserved=0, kp=FAKE, vp=FAKE, ks=None, vs=None):
    return B.rf_cache(kind, reserved, kp, vp, ks, vs)


def _append(kv=None, cache=None, norm=None, q=FAKE, heads=4, qs=256, qo=FAKE + 65536, qos=256, k=FAKE, ks=128, v=FAKE, vs=128, n=3,
            seq=FAKE, rows=FAKE, pos=None, status=FAKE, **kw):
    r = B.make_rope(**kw)
    return B.lib().ridgefill_append_cache(C.byref(r), C.byref(norm or _norm()), C.byref(kv or _kv()), C.byref(cache or _cache()), q,
                                          heads, qs, qo, qos, k, ks, v, vs, n, seq, rows, pos, status, None)


def _read(kv=None, cache=None, n=3, seq=FAKE, rows=FAKE, kind=0, ko=FAKE, kos=128, vo=FAKE, vos=128, status=FAKE):
    return B.lib().ridgefill_read_rows(C.byref(kv or _kv()), C.byref(cache or _cache()), n, seq, rows, kind, ko, kos, vo, vos,
                                       status, None)


HELD = dict(kind=B.RF_CACHE_FP8, ks=FAKE, vs=FAKE)


@pytest.mark.parametrize("call", [_append, _read])
def test_cache_refusals(call):
    for kw in BAD_KV + [dict(head_dim=8), dict(head_dim=72), dict(head_dim=512)]:
        _refused(call(kv=_kv(**kw)), B.RF_E_SHAPE)
    wide = dict(heads=1, qs=80, qos=80, ks=160, vs=160) if call is _append else dict(kos=160, vos=160)
    for hd in (80, 16, 48):                               # blocks of 32 features
        _refused(call(kv=_kv(head_dim=hd), cache=_cache(**HELD), **wide), B.RF_E_SHAPE)
    for kw in (dict(kind=3), dict(kind=-1), dict(reserved=1), dict(kp=None), dict(vp=None), dict(ks=FAKE), dict(vs=FAKE),
               dict(kind=1), dict(kind=2, ks=FAKE), dict(kind=2, vs=FAKE)):
        _refused(call(cache=_cache(**kw)), B.RF_E_INVALID)
    for kw in (dict(kp=FAKE + 8), dict(vp=FAKE + 2), dict(HELD, ks=FAKE + 4), dict(HELD, vs=FAKE + 1)):
        _refused(call(cache=_cache(**kw)), B.RF_E_SHAPE)
    for kw in (dict(n=-1), dict(n=(1 << 23) + 1), dict(rows=FAKE + 2), dict(seq=FAKE + 1)):
        _refused(call(**kw), B.RF_E_SHAPE)
    for kw in (dict(rows=None), dict(status=None), dict(status=FAKE + 2), dict(kv=_kv(block_tables=None))):
        _refused(call(**kw), B.RF_E_INVALID)


def test_append_cache_refusals():
    for kw in (dict(ks=120), dict(vs=129), dict(qs=248), dict(qos=260), dict(heads=-1), dict(heads=5000), dict(q=FAKE + 8),
               dict(k=FAKE + 2), dict(pos=FAKE + 2), dict(rotary_dim=128)):
        _refused(_append(**kw), B.RF_E_SHAPE)
    for kw in (dict(q=None), dict(qo=None), dict(heads=0), dict(k=None), dict(v=None), dict(qo=FAKE, qos=264), dict(theta=0.5)):
        _refused(_append(**kw), B.RF_E_INVALID)
    for kw in BAD_NORM_SHAPE:
        _refused(_append(norm=_norm(**kw)), B.RF_E_SHAPE)
    for kw in BAD_NORM:
        _refused(_append(norm=_norm(**kw)), B.RF_E_INVALID)


def test_read_rows_refusals():
    for kw in (dict(kos=120), dict(vos=129), dict(ko=FAKE + 8), dict(vo=FAKE + 2), dict(kind=1, kos=130),
               dict(kv=_kv(n_kv_heads=256, head_dim=256, page_size=1, max_len=8), n=1 << 19, kos=65536, vos=65536)):
        _refused(_read(**kw), B.RF_E_SHAPE)
    for kw in (dict(kind=2), dict(ko=None, vo=None)):
        _refused(_read(**kw), B.RF_E_INVALID)


def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def _i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def test_binding_refusals():
    kv = B.make_batch(_i32(2, 8), _i32(2), 16, 20, 2, 64, 100)
    codes, scales = torch.zeros(20, 16, 2, 64, dtype=torch.int8), torch.zeros(20, 16, 2, 2, dtype=torch.uint8)
    good, held = B.make_cache(_bf(20, 16, 2, 64), _bf(20, 16, 2, 64)), B.make_cache(codes, codes, scales, scales)
    assert good.type == B.RF_CACHE_BF16 and held.type == B.RF_CACHE_INT8
    assert B.make_cache(codes.view(torch.float8_e4m3fn), None, scales).type == B.RF_CACHE_FP8
    k, rows, status = _bf(3, 2, 64), _i32(3), _i32(1)
    w = _bf(64)
    for call, text in (
            (lambda: B.make_cache(torch.zeros(2, 2, 2, 64), None), "bfloat16"),
            (lambda: B.make_cache(codes, codes), "k_scales"), (lambda: B.make_cache(codes, codes, scales), "v_scales"),
            (lambda: B.make_cache(_bf(20, 16, 2, 64), None, scales), "k_scales"),
            (lambda: B.make_cache(codes, codes, scales, scales[:, :, :, :1].contiguous()), "v_scales"),
            (lambda: B.make_cache(codes, codes[:10], scales, scales), "v_pages"),
            (lambda: B.make_cache(codes[:, :, :, ::2], None, scales), "k_pages"),
            (lambda: B.make_head_norm(torch.zeros(2, 64)), "q_w"), (lambda: B.make_head_norm(None, _bf(128)[::2]), "k_w"),
            (lambda: B.ridgefill_append_cache(None, None, kv, B.make_cache(_bf(19, 16, 2, 64), _bf(19, 16, 2, 64)), k, k, rows, status), "pools"),
            (lambda: B.ridgefill_append_cache(None, None, kv, B.make_cache(_bf(20, 16, 2, 64), None), k, k, rows, status), "v_pages"),
            (lambda: B.ridgefill_append_cache(None, B.make_head_norm(torch.zeros(64)), kv, good, k, k, rows, status), "q_w"),
            (lambda: B.ridgefill_append_cache(None, B.make_head_norm(None, _bf(32)), kv, good, k, k, rows, status), "k_w"),
            (lambda: B.ridgefill_append_cache(None, None, kv, held, k.float(), k, rows, status), "k "),
            (lambda: B.ridgefill_append_cache(None, None, kv, held, k, k, rows, status, q=k), "q_out"),
            (lambda: B.ridgefill_append_cache(None, None, kv, held, k, k, rows.long(), status), "rows"),
            (lambda: B.ridgefill_append_cache(None, None, kv, held, k, k, rows, torch.zeros(1, dtype=torch.int64)), "status"),
            (lambda: B.ridgefill_read_rows(kv, held, rows, status), "neither"),
            (lambda: B.ridgefill_read_rows(kv, held, rows, status, k_out=_bf(3, 1, 64)), "heads"),
            (lambda: B.ridgefill_read_rows(kv, held, rows, status, k_out=k, v_out=k.float()), "v_out"),
            (lambda: B.ridgefill_read_rows(kv, B.make_cache(codes, None, scales), rows, status, v_out=k), "v_pages"),
            (lambda: B.ridgefill_norm_rope(None, None, None), "neither"),
            (lambda: B.ridgefill_norm_rope(None, None, None, q=k), "q_out"),
            (lambda: B.ridgefill_norm_rope(None, B.make_head_norm(torch.zeros(64)), None, q=k, q_out=k), "q_w"),
            (lambda: B.ridgefill_norm_rope(None, None, None, q=k, q_out=_bf(3, 1, 64)), "heads"),
            (lambda: B.ridgefill_norm_rope(None, None, None, q=k, q_out=k, k=_bf(4, 1, 64), k_out=_bf(4, 1, 64)), "k "),
            (lambda: B.ridgefill_norm_rope(B.make_rope(), None, rows.long(), q=k, q_out=k), "positions"),
            (lambda: B.ridgefill_norm_rope_grad(None, None, None, status), "neither"),
            (lambda: B.ridgefill_norm_rope_grad(None, B.make_head_norm(w), None, status, gq=k, q_grad=k), "needs q"),
            (lambda: B.ridgefill_norm_rope_grad(None, B.make_head_norm(w), None, status, q=k, gq=k, q_grad=k, qw_grad=_bf(64)), "qw_grad"),
            (lambda: B.ridgefill_norm_rope_grad(None, None, None, status, gq=k, q_grad=k, k=k), "k: "),
            (lambda: B.ridgefill_norm_rope_grad(None, None, None, status, gq=k, q_grad=_bf(3, 1, 64)), "heads")):
        with pytest.raises(ValueError, match=text):
            call()


def test_plain_gradient():
    # of the tests' own formula, by differentiation in 64 bits
    g = torch.Generator().manual_seed(1)
    x, gy = (torch.randn(4, 3, 32, generator=g, dtype=torch.float64) for _ in range(2))
    w = torch.randn(32, generator=g, dtype=torch.float64).requires_grad_(True)
    x.requires_grad_(True)
    r = (x.square().mean(-1, keepdim=True) + 2.0 ** -10) ** -0.5
    (w * r * x * gy).sum().backward()
    dx, dw, _, _ = H.norm_rope_grad(x, w, 2.0 ** -10, gy, None, 0, 0)
    assert torch.allclose(dx, x.grad, rtol=1e-12, atol=1e-12) and torch.allclose(dw, w.grad, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_plain_blocks(kind):
    # the rule's exponent is the smallest that holds the block; a code is no further than half a step
    g = torch.Generator().manual_seed(2)
    x = (torch.randn(50, 64, generator=g) * torch.exp2(torch.randint(-20, 20, (50, 1), generator=g).float())).bfloat16()
    want, scale = H.held(x, kind)
    top = x.double().unflatten(-1, (-1, 32)).abs().amax(-1)
    f = 2.0 ** (scale.double() - 127)
    assert (top <= H.MOST[kind] * f).all() and (top > H.MOST[kind] * f / 2).all()
    if kind == "fp8":                                     # the type's own rounding
        code = (x.float().unflatten(-1, (-1, 32)) / f[..., None].float()).to(torch.float8_e4m3fn).double()
        assert torch.equal((code * f[..., None]).flatten(-2), want)
    else:
        assert ((want - x.double()).abs().unflatten(-1, (-1, 32)) <= 0.5 * f[..., None]).all()


# ------------------------------------------------------------------------------ attention

def _prefix(tables=FAKE, lengths=FAKE, starts=FAKE, stride=8, groups=2, max_len=100):
    return B.rf_prefix(tables, lengths, starts, stride, groups, max_len)


def _attend(kv=None, prefix=None, cache=None, q=FAKE, heads=4, qs=256, start=FAKE, n=3, max_q=2, mask=None, scale=0.1, out=FAKE,
            os_=256, lse=FAKE, ws=FAKE, ws_bytes=1 << 30):
    return B.lib().ridgefill_cache_attention(C.byref(kv or _kv()), C.byref(prefix) if prefix else None, C.byref(cache or _cache()), q,
                                             heads, qs, start, n, max_q, mask, scale, out, os_, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("shared", [False, True])
def test_attention_refusals(shared):
    pre = dict(prefix=_prefix()) if shared else {}
    for kw in BAD_KV + [dict(head_dim=32), dict(head_dim=96), dict(head_dim=256)]:
        _refused(_attend(kv=_kv(**kw), **pre), B.RF_E_SHAPE)
    for kw in (dict(kind=3), dict(reserved=1), dict(kp=None), dict(vp=None), dict(ks=FAKE), dict(vs=FAKE), dict(kind=1),
               dict(kind=2, ks=FAKE), dict(kind=2, vs=FAKE)):
        _refused(_attend(cache=_cache(**kw), **pre), B.RF_E_INVALID)
    for kw in (dict(kp=FAKE + 8), dict(vp=FAKE + 2), dict(HELD, ks=FAKE + 4), dict(HELD, vs=FAKE + 1)):
        _refused(_attend(cache=_cache(**kw), **pre), B.RF_E_SHAPE)
    for kw in (dict(heads=0), dict(heads=3), dict(heads=4098), dict(max_q=0), dict(max_q=65), dict(n=-1), dict(n=1 << 31), dict(qs=248),
               dict(qs=260), dict(q=FAKE + 8), dict(start=FAKE + 2), dict(mask=FAKE + 4), dict(lse=FAKE + 2), dict(os_=248), dict(os_=257),
               dict(out=FAKE + 8), dict(kv=_kv(lengths=FAKE + 2)), dict(kv=_kv(batch=1 << 14), heads=4096, qs=1 << 18, os_=1 << 18)):
        _refused(_attend(**kw, **pre), B.RF_E_SHAPE)
    for kw in (dict(q=None), dict(start=None), dict(scale=float("nan")), dict(scale=float("inf")), dict(ws=None), dict(out=None, lse=None),
               dict(kv=_kv(lengths=None)), dict(kv=_kv(block_tables=None))):
        _refused(_attend(**kw, **pre), B.RF_E_INVALID)
    for kw in (dict(ws=FAKE + 64), dict(ws_bytes=255)):
        _refused(_attend(**kw, **pre), B.RF_E_WORKSPACE)


def test_prefix_refusals():
    for kw in (dict(groups=0), dict(groups=65536), dict(max_len=0), dict(max_len=(1 << 30) + 1, stride=1 << 27), dict(stride=6),
               dict(tables=FAKE + 2), dict(lengths=FAKE + 1), dict(starts=FAKE + 2)):
        _refused(_attend(prefix=_prefix(**kw)), B.RF_E_SHAPE)
    for kw in (dict(tables=None), dict(lengths=None), dict(starts=None)):
        _refused(_attend(prefix=_prefix(**kw)), B.RF_E_INVALID)
    # many groups of many key heads; many queries
    _refused(_attend(prefix=_prefix(groups=1 << 15), kv=_kv(n_kv_heads=256), heads=256, qs=1 << 14, os_=1 << 14), B.RF_E_SHAPE)
    _refused(_attend(prefix=_prefix(), kv=_kv(batch=1 << 13), heads=4096, max_q=2, qs=1 << 18, os_=1 << 18, ws_bytes=1 << 60), B.RF_E_SHAPE)
    need = B.ridgefill_cache_attention_workspace_bytes(_kv(), 4, 2, 3, _prefix())
    _refused(_attend(prefix=_prefix(), ws_bytes=need - 1), B.RF_E_WORKSPACE)


def test_attention_workspace():
    size = B.ridgefill_cache_attention_workspace_bytes
    assert size(_kv(), 4, 2, 3) >= B.ridgefill_tree_attention_workspace_bytes(_kv(), 4, 2) > 0
    assert size(_kv(), 4, 2, 3, _prefix()) > size(_kv(), 4, 2, 3)
    # more queries than the sequences can have need no more
    assert size(_kv(), 4, 2, 1 << 30, _prefix()) == size(_kv(), 4, 2, 4, _prefix())
    for args in ((4, 2, -1), (4, 65, 3), (3, 2, 3), (4, 2, 1 << 31), (1 << 33, 2, 3), (4, 1 << 32, 3)):
        assert size(_kv(), *args) == 0 and size(_kv(), *args, _prefix()) == 0
    assert size(_kv(), 4, 2, 3, _prefix(groups=0)) == 0 and size(_kv(head_dim=96), 4, 2, 3) == 0


def test_attention_binding_refusals():
    kv = B.make_batch(_i32(2, 8), _i32(2), 16, 20, 2, 64, 100)
    pool, q, ws = _bf(20, 16, 2, 64), _bf(3, 4, 64), torch.zeros(1 << 20, dtype=torch.uint8)
    cache = B.make_cache(pool, pool)
    ok = B.make_prefix(_i32(2, 8), _i32(2), _i32(3), 100)
    assert ok.groups == 2 and ok.table_stride == 8
    call = lambda **kw: B.ridgefill_cache_attention(kv, kw.pop("cache", cache), kw.pop("q", q), kw.pop("start", _i32(3)), kw.pop("max_q", 2),  # noqa: E731
                                                    0.1, kw.pop("out", q), kw.pop("ws", ws), **kw)
    for bad, text in ((lambda: B.make_prefix(_i32(2, 8), _i32(3), _i32(3), 100), "lengths"),
                      (lambda: B.make_prefix(_i32(2, 8), _i32(2), _i32(2), 100), "group_start"),
                      (lambda: B.make_prefix(_i32(2, 16)[:, ::2], _i32(2), _i32(3), 100), "block table"),
                      (lambda: B.make_prefix(_i32(2, 8).long(), _i32(2), _i32(3), 100), "block_tables"),
                      (lambda: B.make_prefix(_i32(2, 8), _i32(2), _i32(3), 1 << 32), "32 bits"),
                      (lambda: call(prefix=B.make_prefix(_i32(2, 8), _i32(2), _i32(3), 129)), "129"),
                      (lambda: call(max_q=1 << 32), "32 bits"), (lambda: call(cache=B.make_cache(pool, None)), "v_pages"),
                      (lambda: call(cache=B.make_cache(pool[:10], pool[:10])), "pools"), (lambda: call(out=_bf(3, 2, 64)), "heads"),
                      (lambda: call(start=_i32(4)), "q_start"), (lambda: call(lse=torch.zeros(3, 2)), "lse"),
                      (lambda: call(tree_mask=_i32(3)), "tree_mask"), (lambda: call(q=q.float()), "q "),
                      (lambda: call(ws=ws[::2]), "workspace"), (lambda: call(prefix=ok), "GPU memory")):
        with pytest.raises(ValueError, match=text):
            bad()
