"""Counts that fall, where two sequences of a batch claim the same rows: written they are one or the other
sequence's, reported, and what belongs to neither is left alone."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import entropy_coding_gb300 as zc  # noqa: E402

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("seqs", [40, 130])
def test_rows_that_two_sequences_claim(seqs):
    """The first sequence and the last claim all rows, at positions that the other's length does not reach: the
    table's entries there name a block of someone else."""
    total, width, block = 64, 8, 16
    cu = [0, total] + [total] * (seqs - 3) + [0, total]  # the last but one falls
    lens = [total] + [0] * (seqs - 2) + [2 * total]
    cache = zc.KV4Cache.empty(1 + 2 * width, 1, 32, block)
    table = torch.zeros(seqs, width, dtype=torch.int32, device=DEV)
    table[0, : total // block] = 1 + torch.arange(total // block, device=DEV).int()               # and block 0 beyond its length
    table[-1, total // block:] = 1 + width + torch.arange(total // block, device=DEV).int()       # and block 0 before its new tokens
    batch = zc.KVBatch(table, torch.tensor(cu, dtype=torch.int32, device=DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), total, total)
    x = torch.randn(total, 1, 32, device=DEV).half()
    for _ in range(200):
        zc.kv_write(cache, batch, x, x)
    with pytest.raises(zc.ZcError) as e:
        cache.check()
    assert e.value.status == zc.EFORMAT
    assert not cache.k[0].any() and not cache.v[0].any() and not cache.k_scale[0].any() and not cache.v_scale[0].any()
