"""CPU checks of the cache calls: every invalid argument is refused on the host, with a status
and a text, before anything is enqueued; size queries; the binding's own checks of tensors; and
the plain 64-bit rotation that the GPU tests compare with, against complex products."""

import ctypes as C

import numpy as np
import pytest
import torch

import cachecase as R
from ridge_map_kv_amd import binding as B

FAKE = 1 << 20                                           # aligned, never read: the call is refused


def _kv(**kw):
    v = dict(block_tables=FAKE, lengths=FAKE, table_stride=8, batch=2, max_len=100, page_size=16,
             num_pages=20, n_kv_heads=2, head_dim=64)
    v.update(kw)
    return B.rf_paged_batch(*[v[n] for n, _ in B.rf_paged_batch._fields_])


BAD_KV = [dict(batch=0), dict(batch=65536), dict(max_len=0), dict(page_size=0), dict(num_pages=0),
          dict(table_stride=6), dict(num_pages=1 << 28), dict(max_len=(1 << 30) + 1, table_stride=1 << 28),
          dict(batch=60000, max_len=1 << 22, table_stride=1 << 20), dict(n_kv_heads=0), dict(n_kv_heads=257)]


def _refused(status, want):
    assert status == want, (status, want)
    assert B.lib().ridgefill_last_error()


def _rope(x=FAKE, kind=0, n=4, heads=2, hd=64, xs=128, pos=FAKE, out=FAKE + 65536, os_=128, tr=0, rope=None, **kw):
    r = B.make_rope(**kw) if rope is None else rope
    return B.lib().ridgefill_rope(C.byref(r), x, kind, n, heads, hd, xs, pos, out, os_, tr, None)


def test_rope_refusals():
    for kw in (dict(rotary_dim=8), dict(rotary_dim=80), dict(rotary_dim=-16), dict(rotary_dim=24), dict(hd=40),
               dict(hd=272), dict(hd=0), dict(heads=0), dict(heads=5000), dict(n=-1), dict(n=(1 << 23) + 1), dict(xs=120), dict(os_=127),
               dict(xs=132), dict(kind=1, xs=130), dict(x=FAKE + 8), dict(out=FAKE + 2), dict(pos=FAKE + 1)):
        _refused(_rope(**kw), B.RF_E_SHAPE)
    for kw in (dict(layout=2), dict(layout=-1), dict(scaling=5), dict(scaling=-1), dict(theta=1.0), dict(theta=float("nan")),
               dict(theta=float("inf")), dict(mscale=-1.0), dict(mscale=float("nan")), dict(scaling=1, factor=0.5),
               dict(scaling=2, factor=float("inf")), dict(scaling=3, factor=2.0), dict(scaling=3, factor=2.0, orig_len=10, low=2.0, high=2.0),
               dict(scaling=4, factor=2.0, orig_len=10, low=0.0, high=2.0), dict(scaling=4, factor=2.0, orig_len=0, low=1.0, high=2.0),
               dict(kind=2), dict(tr=2), dict(x=None), dict(pos=None), dict(out=None), dict(out=FAKE, os_=136)):
        _refused(_rope(**kw), B.RF_E_INVALID)
    _refused(B.lib().ridgefill_rope(None, FAKE, 0, 1, 1, 64, 64, FAKE, FAKE, 64, 0, None), B.RF_E_INVALID)
    assert _rope(n=0, x=None, pos=None, out=None) == B.RF_OK


def _append(kv=None, q=FAKE, heads=4, qs=256, qo=FAKE + 65536, qos=256, k=FAKE, ks=128, v=FAKE, vs=128, n=3, seq=FAKE,
            rows=FAKE, pos=None, kp=FAKE, vp=FAKE, status=FAKE, rope=True, **kw):
    r = B.make_rope(**kw)
    return B.lib().ridgefill_append_rows(C.byref(r) if rope else None, C.byref(kv or _kv()), q, heads, qs, qo, qos, k, ks,
                                         v, vs, n, seq, rows, pos, kp, vp, status, None)


def test_append_refusals():
    for kw in BAD_KV + [dict(head_dim=8), dict(head_dim=72), dict(head_dim=512)]:
        _refused(_append(kv=_kv(**kw)), B.RF_E_SHAPE)
    for kw in (dict(ks=120), dict(vs=129), dict(qs=248), dict(qos=260), dict(n=-1), dict(n=(1 << 23) + 1), dict(heads=-1), dict(heads=5000),
               dict(q=FAKE + 8), dict(k=FAKE + 2), dict(vp=FAKE + 4), dict(rows=FAKE + 2), dict(seq=FAKE + 1),
               dict(pos=FAKE + 2), dict(rotary_dim=128)):
        _refused(_append(**kw), B.RF_E_SHAPE)
    for kw in (dict(q=None), dict(qo=None), dict(heads=0), dict(q=None, qo=None), dict(k=None), dict(v=None),
               dict(rows=None), dict(kp=None), dict(vp=None), dict(status=None), dict(status=FAKE + 2),
               dict(kv=_kv(block_tables=None)), dict(q=FAKE, qo=FAKE, qos=264), dict(theta=0.5)):
        _refused(_append(**kw), B.RF_E_INVALID)
    _refused(B.lib().ridgefill_append_rows(None, None, None, 0, 0, None, 0, FAKE, 128, FAKE, 128, 1, None, FAKE, None, FAKE,
                                           FAKE, FAKE, None), B.RF_E_INVALID)


def _attend(kv=None, kp=FAKE, vp=FAKE, q=FAKE, heads=4, qs=256, start=FAKE, n=3, max_q=2, mask=None, scale=0.1, out=FAKE,
            os_=256, lse=FAKE, ws=FAKE, ws_bytes=1 << 30):
    return B.lib().ridgefill_tree_attention(C.byref(kv or _kv()), kp, vp, q, heads, qs, start, n, max_q, mask, scale, out,
                                            os_, lse, ws, ws_bytes, None)


def _weight(kv=None, kp=FAKE, q=FAKE, heads=4, qs=256, start=FAKE, n=3, max_q=2, mask=None, scale=0.1, lse=FAKE, decay=0.5,
            acc=FAKE, out=FAKE, stride=100, ws=FAKE, ws_bytes=1 << 30):
    return B.lib().ridgefill_attention_weight(C.byref(kv or _kv()), kp, q, heads, qs, start, n, max_q, mask, scale, lse, decay,
                                              acc, out, stride, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [_attend, _weight])
def test_query_refusals(call):
    for kw in BAD_KV + [dict(head_dim=32), dict(head_dim=96), dict(head_dim=256)]:
        _refused(call(kv=_kv(**kw)), B.RF_E_SHAPE)
    for kw in (dict(heads=0), dict(heads=3), dict(heads=4098), dict(max_q=0), dict(max_q=65), dict(n=-1), dict(qs=248),
               dict(qs=260), dict(q=FAKE + 8), dict(start=FAKE + 2), dict(mask=FAKE + 4), dict(kp=FAKE + 8),
               dict(lse=FAKE + 2), dict(kv=_kv(lengths=FAKE + 2)),
               dict(kv=_kv(batch=1 << 14), heads=4096, qs=1 << 18, os_=1 << 18) if call is _attend
               else dict(kv=_kv(batch=1 << 14), heads=4096, qs=1 << 18)):
        _refused(call(**kw), B.RF_E_SHAPE)
    for kw in (dict(q=None), dict(start=None), dict(kp=None), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(ws=None), dict(kv=_kv(lengths=None)), dict(kv=_kv(block_tables=None))):
        _refused(call(**kw), B.RF_E_INVALID)
    for kw in (dict(ws=FAKE + 64), dict(ws_bytes=255)):
        _refused(call(**kw), B.RF_E_WORKSPACE)


def test_attention_refusals():
    for kw in (dict(out=None, lse=None), dict(vp=None)):
        _refused(_attend(**kw), B.RF_E_INVALID)
    for kw in (dict(os_=248), dict(os_=257), dict(out=FAKE + 8), dict(vp=FAKE + 8)):
        _refused(_attend(**kw), B.RF_E_SHAPE)


def test_weight_refusals():
    for kw in (dict(lse=None), dict(out=None), dict(decay=float("nan"))):
        _refused(_weight(**kw), B.RF_E_INVALID)
    many = dict(batch=1 << 15, max_len=(1 << 14) + 1, table_stride=1 << 14)
    assert B.ridgefill_attention_weight_workspace_bytes(_kv(**many), 4, 2) == 0
    for kw in (dict(stride=99), dict(acc=FAKE + 1), dict(out=FAKE + 2), dict(kv=_kv(**many), stride=1 << 15)):
        _refused(_weight(**kw), B.RF_E_SHAPE)


def _evict(kv=None, layers="ok", n_layers=1, acc=FAKE, pos=FAKE, stride=100, keep=10, sink=1, recent=1, ao=FAKE, po=FAKE,
           lo=FAKE, ws=FAKE, ws_bytes=1 << 30, pools=(FAKE, FAKE)):
    arr = (B.rf_layer * 1)()
    arr[0].k_pages, arr[0].v_pages = pools
    return B.lib().ridgefill_evict_rows(C.byref(kv or _kv()), arr if layers else None, n_layers, acc, pos, stride, keep, sink,
                                        recent, ao, po, lo, ws, ws_bytes, None)


def test_evict_refusals():
    for kw in BAD_KV:
        _refused(_evict(kv=_kv(**kw)), B.RF_E_SHAPE)
    for kw in (dict(stride=99), dict(n_layers=-1), dict(n_layers=1025), dict(acc=FAKE + 2), dict(lo=FAKE + 1),
               dict(pools=(FAKE, FAKE + 8))):
        _refused(_evict(**kw), B.RF_E_SHAPE)
    for kw in (dict(keep=-1), dict(sink=-1), dict(recent=-1), dict(acc=None), dict(pos=None), dict(ao=None), dict(po=None),
               dict(lo=None), dict(layers=None), dict(pools=(None, FAKE)), dict(ws=None)):
        _refused(_evict(**kw), B.RF_E_INVALID)
    for kw in (dict(ws=FAKE + 8), dict(ws_bytes=B.ridgefill_evict_workspace_bytes(_kv(), 10) - 1)):
        _refused(_evict(**kw), B.RF_E_WORKSPACE)


def test_workspace_queries():
    kv = _kv()
    for f in (B.ridgefill_tree_attention_workspace_bytes, B.ridgefill_attention_weight_workspace_bytes):
        assert f(kv, 4, 2) >= 256
        assert f(kv, 3, 2) == 0 and f(kv, 4, 65) == 0 and f(kv, 4, 0) == 0
        assert f(_kv(batch=0), 4, 2) == 0 and f(_kv(head_dim=96), 4, 2) == 0
        n = f(_kv(max_len=60000, table_stride=4000), 64, 64)
        assert _refusable(n)
    assert B.ridgefill_evict_workspace_bytes(kv, 10) >= 256
    assert B.ridgefill_evict_workspace_bytes(kv, -1) == 0
    assert B.ridgefill_evict_workspace_bytes(_kv(page_size=0), 3) == 0


def _refusable(n):
    return 256 <= n < 1 << 36


def test_binding_checks_tensors():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    rope = B.make_rope()
    kv = B.make_batch(i32(2, 8), i32(2), 16, 20, 2, 64, 100)
    k, pool, ws = bf(3, 2, 64), bf(20, 16, 2, 64), torch.zeros(512, dtype=torch.uint8)
    bad = [
        lambda: B.make_batch(i32(2, 8).long(), i32(2), 16, 20, 2, 64),
        lambda: B.make_batch(i32(2, 8), i32(3), 16, 20, 2, 64),
        lambda: B.make_batch(i32(2, 8), i32(2), 16, 20, 2, 64, 129),
        lambda: B.make_batch(i32(2, 16)[:, ::2], i32(2), 16, 20, 2, 64),
        lambda: B.make_pools([pool], []),
        lambda: B.ridgefill_rope(rope, k.half(), i32(3), k),
        lambda: B.ridgefill_rope(rope, k, i32(4), k),
        lambda: B.ridgefill_rope(rope, k, i32(3).long(), k),
        lambda: B.ridgefill_rope(rope, k, i32(3), k.float()),
        lambda: B.ridgefill_rope(rope, k.transpose(0, 1), i32(2), k),
        lambda: B.ridgefill_rope(rope, k, i32(3), bf(3, 1, 64)),
        lambda: B.ridgefill_rope(rope, k, i32(3), k),                        # not GPU memory
        lambda: B.ridgefill_append_rows(rope, kv, bf(3, 1, 64), k, i32(3), pool, pool, i32(1)),
        lambda: B.ridgefill_append_rows(rope, kv, k, k, i32(3), bf(20, 16, 2, 128), pool, i32(1)),
        lambda: B.ridgefill_append_rows(rope, kv, k, k, i32(3), pool, pool, i32(1), seq=i32(2)),
        lambda: B.ridgefill_append_rows(rope, kv, k, k, i32(3), pool, pool, i32(1), positions=i32(3).long()),
        lambda: B.ridgefill_append_rows(rope, kv, k, k, i32(3), pool, pool, i32(1), q_out=k),
        lambda: B.ridgefill_append_rows(rope, kv, k, k, i32(3), pool, pool, i32(1), q=k, q_out=bf(3, 1, 64)),
        lambda: B.ridgefill_append_rows(rope, kv, k, k, i32(3), pool, pool, i32(1).long()),
        lambda: B.ridgefill_append_rows(rope, kv, k, k, i32(3), pool, pool, i32(1)),
        lambda: B.ridgefill_tree_attention(kv, pool, pool, k, i32(2), 2, 0.1, k, ws),
        lambda: B.ridgefill_tree_attention(kv, pool, pool, k, i32(3), 2, 0.1, k, ws, lse=torch.zeros(3, 3)),
        lambda: B.ridgefill_tree_attention(kv, pool, pool, k, i32(3), 2, 0.1, k, ws, tree_mask=i32(3)),
        lambda: B.ridgefill_tree_attention(kv, pool, pool, k, i32(3), 2, 0.1, bf(3, 4, 64), ws),
        lambda: B.ridgefill_tree_attention(kv, pool, pool, bf(3, 2, 128), i32(3), 2, 0.1, k, ws),
        lambda: B.ridgefill_tree_attention(kv, pool, pool, k, i32(3), 2, 0.1, k, ws),
        lambda: B.ridgefill_tree_attention(B.make_batch(i32(2, 8), None, 16, 20, 2, 64), pool, pool, k, i32(3), 2, 0.1, k, ws),
        lambda: B.ridgefill_attention_weight(kv, pool, k, i32(3), 2, 0.1, torch.zeros(3, 2), torch.zeros(1, 100), ws),
        lambda: B.ridgefill_attention_weight(kv, pool, k, i32(3), 2, 0.1, torch.zeros(3, 2), torch.zeros(2, 100), ws,
                                             acc=torch.zeros(2, 101)),
        lambda: B.ridgefill_attention_weight(kv, pool, k, i32(3), 2, 0.1, torch.zeros(3, 2).double(), torch.zeros(2, 100), ws),
        lambda: B.ridgefill_evict_rows(kv, B.make_pools([bf(20, 16, 2, 128)], [pool]), torch.zeros(2, 100), i32(2, 100), 5,
                                       torch.zeros(2, 100), i32(2, 100), i32(2), ws),
        lambda: B.ridgefill_evict_rows(kv, B.make_pools([pool], [pool]), torch.zeros(2, 100), i32(2, 99), 5,
                                       torch.zeros(2, 100), i32(2, 100), i32(2), ws),
        lambda: B.ridgefill_evict_rows(kv, B.make_pools([pool], [pool]), torch.zeros(2, 100), i32(2, 100), 5,
                                       torch.zeros(2, 100), i32(2, 100), i32(3), ws),
    ]
    for k_, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            raise AssertionError(f"call {k_} was not refused")


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("kw", [dict(), dict(scaling=4, factor=8.0, orig_len=4096, low=1.0, high=32.0),
                                dict(scaling=3, factor=8.0, orig_len=8192, low=1.0, high=4.0)])
def test_plain_rotation_is_a_product_of_complex_numbers(layout, kw):
    x = torch.randn(5, 2, 64, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    pos = torch.tensor([0, 1, 77, 4095, 100000], dtype=torch.int32)
    y, _ = R.rotate(x, pos, 48, layout, **kw)
    f, m = R.frequencies(48, **kw)
    z = np.exp(1j * np.outer(pos.numpy().astype(np.float64), f.numpy()))[:, None] * m
    at = (slice(0, 24), slice(24, 48)) if layout == 0 else (slice(0, 48, 2), slice(1, 48, 2))
    w = (x[..., at[0]].numpy() + 1j * x[..., at[1]].numpy()) * z
    assert np.allclose(y[..., at[0]].numpy(), w.real, atol=1e-12) and np.allclose(y[..., at[1]].numpy(), w.imag, atol=1e-12)
    assert torch.equal(y[..., 48:], x[..., 48:])
    back, _ = R.rotate(y, pos, 48, layout, transpose=True, **kw)
    assert np.allclose(back[..., :48].numpy() / m ** 2, x[..., :48].numpy(), atol=1e-12)
