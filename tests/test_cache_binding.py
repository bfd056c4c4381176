"""CPU tests of what the binding's cache calls hand to the C side: integers past 32 bits, which ctypes
would cut off, tensors that are missing, and the strides of single rows."""

import pytest
import torch

from ridge_map_kv_amd import binding as B


def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def _i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


PAST = [1 << 32, (1 << 32) + 2, -(1 << 32) + 2, 1 << 31, (1 << 64) + 1]


@pytest.fixture
def kv():
    return B.make_batch(_i32(2, 8), _i32(2), 16, 20, 2, 64, 100)


@pytest.mark.parametrize("n", PAST)
def test_integers_past_32_bits_are_refused(kv, n):
    pool, k, ws = _bf(20, 16, 2, 64), _bf(3, 2, 64), torch.zeros(512, dtype=torch.uint8)
    acc, pos, lse = torch.zeros(2, 100), _i32(2, 100), torch.zeros(3, 2)
    # 2^32 rows to keep would be none: the whole cache cut off
    evict = lambda **kw: B.ridgefill_evict_rows(kv, B.make_pools([pool], [pool]), acc, pos, kw.pop("n_keep", 5), acc, pos,  # noqa: E731
                                                _i32(2), ws, **kw)
    for call in (lambda: evict(n_keep=n), lambda: evict(n_sink=n), lambda: evict(n_recent=n),
                 lambda: B.ridgefill_tree_attention(kv, pool, pool, k, _i32(3), n, 0.1, k, ws),
                 lambda: B.ridgefill_attention_weight(kv, pool, k, _i32(3), n, 0.1, lse, acc, ws),
                 lambda: B.make_rope(rotary_dim=n), lambda: B.make_rope(orig_len=n),
                 lambda: B.make_rope(scaling=n), lambda: B.make_rope(layout=n),
                 lambda: B.make_batch(_i32(2, 8), None, 16, n, 2, 64), lambda: B.make_batch(_i32(2, 8), None, n, 1, 2, 64),
                 lambda: B.make_batch(_i32(2, 8), None, 16, 20, n, 64), lambda: B.make_batch(_i32(2, 8), None, 16, 20, 2, n),
                 lambda: B.make_batch(_i32(2, 8), None, 16, 20, 2, 64, n)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
    assert B.ridgefill_evict_workspace_bytes(kv, n) == 0
    for size in (B.ridgefill_tree_attention_workspace_bytes, B.ridgefill_attention_weight_workspace_bytes):
        assert size(kv, 2, 1) > 0 and size(kv, 2, n) == 0 and size(kv, n, 1) == 0


def test_missing_tensors_are_refused(kv):
    pool, k, ws = _bf(20, 16, 2, 64), _bf(3, 2, 64), torch.zeros(512, dtype=torch.uint8)
    for call, text in ((lambda: B.ridgefill_append_rows(None, kv, k, k, _i32(3), pool, pool, _i32(1), q=k), "q_out"),
                       (lambda: B.ridgefill_tree_attention(kv, pool, None, k, _i32(3), 2, 0.1, k, ws), "v_pages"),
                       (lambda: B.ridgefill_attention_weight(kv, pool, k, _i32(3), 2, 0.1, None, torch.zeros(2, 100), ws), "lse")):
        with pytest.raises(ValueError, match=text):
            call()


def test_a_single_row_has_no_stride():
    for base in (_bf(4, 387), _bf(4, 1000)):
        row = base.as_strided((1, 3, 128), (base.shape[1], 128, 1))
        assert B._rows_of("x", row, torch.bfloat16, base.device, 128) == 384
        assert B._rows_of("x", base[:, :384].unflatten(1, (3, 128)), torch.bfloat16, base.device, 128) == base.shape[1]
