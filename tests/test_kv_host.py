"""The host side of the 8-bit cache operators, without a GPU: what the C entry points refuse before any launch (the
pointers are never dereferenced)."""
from __future__ import annotations

import ctypes

import entropy_coding_gb300 as zc
from entropy_coding_gb300 import kv

P = 0x10000


def _cache(**kw):
    f = dict(d_k=P, d_v=P, d_k_scale=P, d_v_scale=P, block_stride=2 * 16 * 32, scale_stride=2, n_blocks=4, kv_heads=2,
             block_tokens=16, head_dim=32)
    f.update(kw)
    return kv._Cache(**f)


def _batch(**kw):
    f = dict(d_table=P, table_stride=3, d_cu=P, d_lens=P, n_seqs=2, total_tokens=6, max_tokens=3, table_width=3)
    f.update(kw)
    return kv._Batch(**f)


def _rows(data=P, token=64, head=32):
    return kv._Rows(data, token, head)


def _call(name, cache=None, batch=None, dtype=zc.BF16, k=None, v=None, status=P):
    ref = lambda x: ctypes.byref(x) if x is not None else None  # noqa: E731
    f = getattr(zc.lib(), name)
    return f(ref(cache or _cache()), ref(batch or _batch()), dtype, ref(k or _rows()), ref(v or _rows()), status, None)


def _attend(cache=None, batch=None, dtype=zc.BF16, heads=4, q=None, out=None, lse=None, scale=0.1, flags=1, window=0, ws=P, ws_bytes=1 << 30, status=P):
    return zc.lib().zc_kv_attend(ctypes.byref(cache or _cache()), ctypes.byref(batch or _batch()), dtype, heads,
                                 ctypes.byref(q or _rows(token=128)), ctypes.byref(out or _rows(token=128)), lse, scale,
                                 flags, window, ws, ws_bytes, status, None)


BAD_CACHES = [dict(d_k=None), dict(d_v_scale=None), dict(d_k=P + 8), dict(d_k_scale=P + 2), dict(head_dim=0),
              dict(head_dim=24), dict(head_dim=144, block_stride=1 << 20), dict(block_tokens=0), dict(block_tokens=24),
              dict(block_tokens=272, block_stride=1 << 20), dict(kv_heads=0), dict(n_blocks=0),
              dict(block_stride=1023), dict(block_stride=1024 + 8), dict(block_stride=2 ** 62), dict(scale_stride=1)]
BAD_BATCHES = [dict(d_table=None), dict(d_cu=None), dict(d_lens=None), dict(d_cu=P + 1), dict(table_width=0),
               dict(table_stride=2), dict(max_tokens=0), dict(max_tokens=7), dict(max_tokens=2), dict(n_seqs=0),
               dict(total_tokens=2 ** 31, max_tokens=2 ** 31)]
BAD_ROWS = [dict(data=None), dict(data=P + 8), dict(token=65), dict(head=36)]


def test_bad_caches_batches_and_rows_are_refused():
    for name in ("zc_kv_write", "zc_kv_read"):
        for kw in BAD_CACHES:
            assert _call(name, cache=_cache(**kw)) == zc.EINVAL, kw
        for kw in BAD_BATCHES:
            assert _call(name, batch=_batch(**kw)) == zc.EINVAL, kw
        for kw in BAD_ROWS:
            assert _call(name, k=_rows(**kw)) == zc.EINVAL and _call(name, v=_rows(**kw)) == zc.EINVAL, kw
        for dt in (zc.U8, zc.U16, zc.U32, 0, 9):
            assert _call(name, dtype=dt) == zc.EINVAL
        assert _call(name, status=None) == zc.EINVAL
    for kw in BAD_CACHES:
        assert _attend(cache=_cache(**kw)) == zc.EINVAL, kw
    for kw in BAD_BATCHES:
        assert _attend(batch=_batch(**kw)) == zc.EINVAL, kw
    for kw in BAD_ROWS:
        assert _attend(q=_rows(**kw)) == zc.EINVAL and _attend(out=_rows(**kw)) == zc.EINVAL, kw


def test_attend_refuses_its_own_arguments():
    for dt in (zc.FP32, zc.U8, 0):
        assert _attend(dtype=dt) == zc.EINVAL
    for heads in (0, 3, 65538):
        assert _attend(heads=heads) == zc.EINVAL
    for scale in (float("nan"), float("inf"), 1e30):
        assert _attend(scale=scale) == zc.EINVAL
    assert _attend(ws=None) == zc.EINVAL and _attend(ws=P + 8) == zc.EINVAL and _attend(ws_bytes=1000) == zc.ECAPACITY
    assert _attend(flags=2) == zc.EINVAL and _attend(lse=P + 2) == zc.EINVAL and _attend(status=None) == zc.EINVAL


def test_workspace_size_of_valid_arguments_only():
    size = lambda c, b, h: zc.lib().zc_kv_attend_workspace_size(ctypes.byref(c), ctypes.byref(b), h)  # noqa: E731
    assert size(_cache(), _batch(), 4) > 0
    for kw in BAD_CACHES:
        assert size(_cache(**kw), _batch(), 4) == 0, kw
    for kw in BAD_BATCHES:
        assert size(_cache(), _batch(**kw), 4) == 0, kw
    assert size(_cache(), _batch(), 3) == 0 and size(_cache(), _batch(), 0) == 0


def test_a_batch_without_tokens_launches_nothing():
    none = dict(total_tokens=0, max_tokens=0)
    for name in ("zc_kv_write", "zc_kv_read"):
        assert _call(name, batch=_batch(**none)) == zc.OK
    assert _attend(batch=_batch(**none)) == zc.OK
    assert _attend(batch=_batch(n_seqs=0, d_table=None, d_cu=None, d_lens=None, **none)) == zc.OK
