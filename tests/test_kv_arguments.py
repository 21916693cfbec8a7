"""Arguments of the 8-bit cache's Python layer that are checked before any pointer is taken; no GPU."""
from __future__ import annotations

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
