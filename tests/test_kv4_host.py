"""The host side of the 4-bit cache and of the rotation, without a GPU: what the C entry points and the Python layer refuse
before any launch (the pointers are never dereferenced), the kept fractions of a turn, and the oracle itself."""
from __future__ import annotations

import ctypes
import decimal
import math

import numpy as np
import pytest
import torch

import entropy_coding_gb300 as zc
from entropy_coding_gb300 import kv

from kv4_reference import CODES, SCALES, numbers, pack, quantise, scale_of

P = 0x10000


def _cache(**kw):
    f = dict(d_k=P, d_v=P, d_k_scale=P, d_v_scale=P, block_stride=2 * 16 * 16, scale_stride=2 * 16 * 2, n_blocks=4, kv_heads=2,
             block_tokens=16, head_dim=32)
    f.update(kw)
    return kv._Cache(**f)


def _batch(**kw):
    f = dict(d_table=P, table_stride=3, d_cu=P, d_lens=P, n_seqs=2, total_tokens=6, max_tokens=3, table_width=3)
    f.update(kw)
    return kv._Batch(**f)


def _rows(data=P, token=64, head=32):
    return kv._Rows(data, token, head)


ref = ctypes.byref


def _move(name, cache=None, batch=None, dtype=zc.BF16, k=None, v=None, status=P):
    return getattr(zc.lib(), name)(ref(cache or _cache()), ref(batch or _batch()), dtype, ref(k or _rows()), ref(v or _rows()), status, None)


def _attend(cache=None, batch=None, dtype=zc.BF16, heads=4, q=None, out=None, lse=None, scale=0.1, flags=1, window=0, ws=P, ws_bytes=1 << 30, status=P):
    return zc.lib().zc_kv4_attend(ref(cache or _cache()), ref(batch or _batch()), dtype, heads, ref(q or _rows(token=128)),
                                  ref(out or _rows(token=128)), lse, scale, flags, window, ws, ws_bytes, status, None)


BAD_CACHES = [dict(d_k=None), dict(d_v_scale=None), dict(d_k=P + 8), dict(d_k_scale=P + 4), dict(head_dim=0),
              dict(head_dim=24), dict(head_dim=144, block_stride=1 << 20), dict(block_tokens=0), dict(block_tokens=24),
              dict(block_tokens=272, block_stride=1 << 20), dict(kv_heads=0), dict(n_blocks=0), dict(block_stride=496),
              dict(block_stride=512 + 8), dict(block_stride=2 ** 62), dict(scale_stride=48), dict(scale_stride=72),
              dict(scale_stride=2 ** 62), dict(head_dim=48, scale_stride=96)]
BAD_BATCHES = [dict(d_table=None), dict(d_cu=None), dict(d_lens=None), dict(d_cu=P + 1), dict(table_width=0),
               dict(table_stride=2), dict(max_tokens=0), dict(max_tokens=7), dict(max_tokens=2), dict(n_seqs=0),
               dict(total_tokens=2 ** 31, max_tokens=2 ** 31)]
BAD_ROWS = [dict(data=None), dict(data=P + 8), dict(token=65), dict(head=36)]


def test_bad_caches_batches_and_rows_are_refused():
    for name in ("zc_kv4_write", "zc_kv4_read"):
        for kw in BAD_CACHES:
            assert _move(name, cache=_cache(**kw)) == zc.EINVAL, kw
        for kw in BAD_BATCHES:
            assert _move(name, batch=_batch(**kw)) == zc.EINVAL, kw
        for kw in BAD_ROWS:
            assert _move(name, k=_rows(**kw)) == zc.EINVAL and _move(name, v=_rows(**kw)) == zc.EINVAL, kw
        for dt in (zc.U8, zc.U16, zc.U32, 0, 9):
            assert _move(name, dtype=dt) == zc.EINVAL
        assert _move(name, status=None) == zc.EINVAL
    for kw in BAD_CACHES:
        assert _attend(cache=_cache(**kw)) == zc.EINVAL, kw
    for kw in BAD_BATCHES:
        assert _attend(batch=_batch(**kw)) == zc.EINVAL, kw
    for kw in BAD_ROWS:
        assert _attend(q=_rows(**kw)) == zc.EINVAL and _attend(out=_rows(**kw)) == zc.EINVAL, kw


def test_attend_refuses_its_own_arguments():
    for kw in ([dict(dtype=d) for d in (zc.FP32, zc.U8, 0)] + [dict(heads=h) for h in (0, 3, 65538)] +
               [dict(scale=s) for s in (math.nan, math.inf, 1e30)] + [dict(ws=None), dict(ws=P + 8), dict(flags=2), dict(lse=P + 2), dict(status=None)]):
        assert _attend(**kw) == zc.EINVAL, kw
    assert _attend(ws_bytes=1000) == zc.ECAPACITY


def test_workspace_sizes_of_valid_arguments_only():
    L = zc.lib()

    def sizes(c, b, h):
        return [f(ref(c), ref(b), h) for f in (L.zc_kv4_attend_counter_bytes, L.zc_kv4_attend_workspace_size)]

    for batch in (_batch(), _batch(total_tokens=600, max_tokens=300)):
        counters, size = sizes(_cache(), batch, 4)
        assert 0 < counters < size and counters % 256 == 0
    for kw in BAD_CACHES:
        assert sizes(_cache(**kw), _batch(), 4) == [0, 0], kw
    for kw in BAD_BATCHES:
        assert sizes(_cache(), _batch(**kw), 4) == [0, 0], kw
    assert sizes(_cache(), _batch(), 3) == [0, 0] and sizes(_cache(), _batch(), 0) == [0, 0]


def _rotate(batch=None, turns=P, rot=32, flags=0, qw=None, kw=None, wd=0, eps=1e-6, dtype=zc.BF16, dim=32, heads=4, kv_heads=2,
            rows=None, status=P):
    r = kv._Rotation(turns, rot, flags, qw, kw, wd, eps)
    rows = rows or [_rows(token=128), _rows(), _rows(token=128), _rows()]
    return zc.lib().zc_kv_rotate(ref(batch or _batch()), ref(r), dtype, dim, heads, kv_heads, *map(ref, rows), status, None)


def test_rotate_refuses_bad_arguments():
    for kw in [dict(turns=None), dict(turns=P + 4), dict(rot=8), dict(rot=48), dict(rot=24), dict(flags=1), dict(flags=4), dict(dim=0),
               dict(dim=40, rot=16), dict(dim=144), dict(heads=0), dict(heads=65536), dict(kv_heads=0), dict(dtype=zc.U16), dict(status=None),
               dict(qw=P, wd=zc.FP16), dict(qw=P, wd=0), dict(kw=P + 2, wd=zc.FP32), dict(qw=P + 1, wd=zc.BF16), dict(qw=P, wd=zc.BF16, eps=0.0),
               dict(qw=P, wd=zc.BF16, eps=-1.0), dict(qw=P, wd=zc.BF16, eps=math.nan), dict(qw=P, wd=zc.BF16, eps=math.inf),
               dict(batch=_batch(total_tokens=2 ** 26, max_tokens=2 ** 26), heads=64)]:
        assert _rotate(**kw) == zc.EINVAL, kw
    for kw in BAD_BATCHES:
        assert _rotate(batch=_batch(**kw)) == zc.EINVAL, kw
    good = [_rows(token=128), _rows(), _rows(token=128), _rows()]
    for i in range(4):
        for kw in BAD_ROWS:
            assert _rotate(rows=good[:i] + [_rows(**kw)] + good[i + 1:]) == zc.EINVAL, (i, kw)


def test_batches_without_tokens_launch_nothing():
    none = dict(total_tokens=0, max_tokens=0)
    assert _move("zc_kv4_write", batch=_batch(**none)) == _move("zc_kv4_read", batch=_batch(**none)) == zc.OK
    assert _attend(batch=_batch(**none)) == _rotate(batch=_batch(**none)) == zc.OK


def _refused(match, call):
    with pytest.raises(zc.ZcError, match=match) as e:
        call()
    assert e.value.status == zc.EINVAL


def test_layouts_that_the_python_layer_refuses():
    u8 = dict(dtype=torch.uint8)
    k, s = torch.zeros(4, 2, 16, 48, **u8), torch.zeros(4, 2, 16, 5, **u8)  # 80 columns
    _refused("CUDA", lambda: zc.KV4Cache(k, k, s, s))  # (all of its layout is right)
    _refused("uint8", lambda: zc.KV4Cache(k, k, s.float(), s))
    _refused("uint8", lambda: zc.KV4Cache(k, k, s[0], s[0]))
    _refused("same sizes", lambda: zc.KV4Cache(k, k[:3], s, s))
    _refused("same sizes", lambda: zc.KV4Cache(k, k, s, s[:3]))
    _refused("scales are", lambda: zc.KV4Cache(k, k, s[:3], s[:3]))
    _refused("scales are", lambda: zc.KV4Cache(k[..., :40], k[..., :40], s, s))
    _refused("contiguous", lambda: zc.KV4Cache(k.transpose(1, 2), k.transpose(1, 2), *[s.transpose(1, 2)] * 2))
    _refused("contiguous", lambda: zc.KV4Cache(k, k, *[torch.zeros(4, 2, 16, 6, **u8)[..., :5]] * 2))
    for dim in (0, 24, 144):
        _refused("head_dim", lambda: zc.KV4Cache.empty(4, 2, dim, 16, "cpu"))
    _refused("blocks overlap", lambda: zc.KV4Cache(*[k[:1].expand(4, 2, 16, 48)] * 2, s, s))
    _refused("scales of blocks overlap", lambda: zc.KV4Cache(k, k, *[s[:1].expand(4, 2, 16, 5)] * 2))


def test_frequencies_that_are_refused():
    for bad in ([1.0] * 7, [1.0] * 72, [1.0] * 7 + [math.nan], [1.0] * 7 + [math.inf], [2.0 ** 20] * 8):
        _refused("frequencies", lambda: zc.KVRotation(bad, device="cpu"))
    r = zc.KVRotation(torch.ones(16), interleaved=True, device="cpu")
    assert r.rot_dim == 32 and r.interleaved and r.turns.dtype == torch.int64


def test_fractions_of_a_turn_hold_at_any_position():
    """The low 64 bits of position times fraction are the angle's fraction of a turn, to position / 2^65 of one."""
    with decimal.localcontext(decimal.Context(prec=80)):
        tau = 2 * decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
        for f in (1.0, 500000.0 ** -0.99, 10000.0 ** -0.5, 0.1, 123.456, -0.7, 2.0 ** -40):
            u = kv.fraction_of_turn(f)
            for p in (0, 1, 131071, 10 ** 9, 2 ** 30 - 1):
                turn = decimal.Decimal(p) * decimal.Decimal(f) / tau % 1
                off = abs(decimal.Decimal((u * p) % 2 ** 64) / 2 ** 64 - (turn + 1) % 1)
                assert min(off, 1 - off) <= decimal.Decimal(p + 1) / 2 ** 65, (f, p)


def test_the_oracles_scales_are_halves_and_its_codes_nearest():
    half = (np.arange(0xE3, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(SCALES, half) and np.isnan(scale_of(np.array([0xFF]))).all() and SCALES[-1] == 10240.0 and SCALES[1] == 2.0 ** -17
    rng = np.random.default_rng(0)
    x = rng.standard_normal((300, 64)) * np.exp2(rng.integers(-20, 20, (300, 1)))
    code, byte = quantise(x)
    y = numbers(pack(code), byte)
    s = np.repeat(SCALES[byte], 16, -1)
    # no other code of the scale is nearer, and no other scale nearer to a sixth of the largest
    best = np.abs(np.abs(x)[..., None] - CODES * s[..., None]).min(-1)
    assert np.allclose(np.abs(x - y), best, rtol=1e-12, atol=0)
    a = np.abs(x).reshape(300, 4, 16).max(-1)
    assert (np.abs(SCALES[byte] - a / 6) <= np.abs(SCALES[1:] - a[..., None] / 6).min(-1) * (1 + 1e-12)).all()
