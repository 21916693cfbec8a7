"""Arguments of the 8-bit cache's Python layer that are checked before any pointer is taken; no GPU."""
from __future__ import annotations

import ctypes
import types

import pytest
import torch

import entropy_coding_gb300 as zc
from entropy_coding_gb300 import kv


def _codes(n=4, h=2, b=16, d=32):
    return torch.zeros(n, h, b, d, dtype=torch.uint8)


def _refused(match, call):
    with pytest.raises(zc.ZcError, match=match) as e:
        call()
    assert e.value.status == zc.EINVAL


def test_blocks_or_scales_that_overlap_are_refused():
    """An expanded tensor has the storage of one block; stepping through it leaves that storage."""
    k, s = _codes(), torch.ones(4, 2)
    _refused("blocks overlap", lambda: zc.KVCache(_codes(1).expand(4, 2, 16, 32), _codes(1).expand(4, 2, 16, 32), s, s))
    _refused("scales of blocks overlap", lambda: zc.KVCache(k, k, torch.ones(2).expand(4, 2), torch.ones(2).expand(4, 2)))
    one = torch.ones(5)
    _refused("scales of blocks overlap", lambda: zc.KVCache(k, k, one.as_strided((4, 2), (1, 1)), one.as_strided((4, 2), (1, 1))))


def test_the_distance_of_slices():
    table = torch.zeros(3, 6, dtype=torch.int32)
    assert kv._outer(table, 6, "rows") == 6 and kv._outer(table[:, :4], 4, "rows") == 6
    assert kv._outer(table[:1].expand(1, 6), 6, "rows") == 6 and kv._outer(table[:0], 6, "rows") == 6
    _refused("rows overlap", lambda: kv._outer(table[0].expand(64, 6), 6, "rows"))
    _refused("rows overlap", lambda: kv._outer(table.view(-1).as_strided((4, 6), (4, 1)), 6, "rows"))


class _Device:
    """torch.cuda.device, without a GPU."""
    now = 0

    def __init__(self, index):
        self.index = index

    def __enter__(self):
        self.was, _Device.now = _Device.now, self.index

    def __exit__(self, *_):
        _Device.now = self.was


@pytest.fixture
def two_devices(monkeypatch):
    """The layer with fakes of the entry points and of two devices, the first of them current; the calls' devices."""
    seen = []

    def entry(*args):
        seen.append(_Device.now)
        return 0

    monkeypatch.setattr(kv, "_entries", lambda: (entry, entry, entry))
    monkeypatch.setattr(kv, "_current_device", lambda: _Device.now, raising=False)
    monkeypatch.setattr(kv, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "device", _Device)
    return seen


def _on_device(index):
    """A cache and a batch that say they are on that device (their tensors are the host's)."""
    cache, batch = object.__new__(kv.KVCache), object.__new__(kv.KVBatch)
    cache.__dict__.update(_many=True, _streams={0}, kv_heads=2, head_dim=32, device=torch.device("cpu"), _index=index, _ref=0, _status=0)
    batch.__dict__.update(total_tokens=3, _index=index, _ref=0, _ws={})
    batch._workspace = lambda *_: [0, 0, None, 0]
    return cache, batch


def _calls(cache, batch):
    x, q = torch.zeros(3, 2, 32).half(), torch.zeros(3, 4, 32).half()
    yield lambda: zc.kv_write(cache, batch, x, x)
    yield lambda: zc.kv_read_into(cache, batch, x, x)
    yield lambda: zc.kv_read(cache, batch)
    yield lambda: zc.kv_attend_into(cache, batch, q, q.clone())
    yield lambda: zc.kv_attend(cache, batch, q)


@pytest.mark.parametrize("index", [0, 1])
def test_a_call_runs_on_the_caches_device(two_devices, index):
    for call in _calls(*_on_device(index)):
        call()
    assert two_devices == [index] * 5 and _Device.now == 0


def test_a_batch_of_another_device_is_refused(two_devices):
    for call in _calls(_on_device(1)[0], _on_device(0)[1]):
        _refused("another device", call)
    assert not two_devices


def test_a_batch_on_two_devices_is_refused():
    def t(index):  # as much of a tensor as is looked at before the refusal
        return types.SimpleNamespace(dtype=torch.int32, is_cuda=True, device=torch.device("cuda", index), numel=lambda: 2)

    for where in ((1, 0, 0), (0, 1, 0), (0, 0, 1)):
        _refused("one device", lambda: zc.KVBatch(*map(t, where), 2, 1))


def test_counter_bytes_are_part_of_the_workspace():
    def sizes(heads=4, tokens=6, most=3, **kw):
        c = kv._Cache(**{**dict(d_k=1 << 16, d_v=1 << 16, d_k_scale=1 << 16, d_v_scale=1 << 16, block_stride=1024, scale_stride=2,
                                n_blocks=4, kv_heads=2, block_tokens=16, head_dim=32), **kw})
        b = kv._Batch(d_table=1 << 16, table_stride=3, d_cu=1 << 16, d_lens=1 << 16, n_seqs=2, total_tokens=tokens, max_tokens=most,
                      table_width=3)
        return [f(ctypes.byref(c), ctypes.byref(b), heads)
                for f in (zc.lib().zc_kv_attend_counter_bytes, zc.lib().zc_kv_attend_workspace_size)]

    for args in (dict(), dict(tokens=600, most=300), dict(heads=64), dict(heads=2, tokens=2, most=1)):
        counters, size = sizes(**args)
        assert 0 < counters < size and counters % 256 == 0
    assert sizes(heads=3) == [0, 0] and sizes(head_dim=24) == [0, 0] and sizes(most=7) == [0, 0]
