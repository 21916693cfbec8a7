"""The 8-bit key/value cache on the GPU at the edges of what its calls take: layouts, counts, streams and states that
the ordinary tests do not reach."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import entropy_coding_gb300 as zc  # noqa: E402

DEV = torch.device("cuda:0")


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cache(n, hkv, dim, block, seed=0):
    """A cache of random numbers of magnitude about one."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    cache = zc.KVCache.empty(n, hkv, dim, block, DEV)
    batch = zc.KVBatch(torch.arange(n, dtype=torch.int32, device=DEV).view(1, n), _i32([0, n * block]), _i32([n * block]),
                       n * block, n * block)
    zc.kv_write(cache, batch, *(torch.randn(n * block, hkv, dim, generator=g, device=DEV).bfloat16() for _ in range(2)))
    cache.check()
    return cache


def test_an_expanded_block_table_is_refused():
    """One row for several sequences (samples of one prompt): its storage ends after the first. Nothing is launched."""
    row = _i32([0, 1, 2, 3, 4, 5])
    with pytest.raises(zc.ZcError, match="rows of the table overlap") as e:
        zc.KVBatch(row.expand(64, 6), torch.arange(65, dtype=torch.int32, device=DEV), torch.full_like(row[:1], 90).repeat(64), 64, 1)
    assert e.value.status == zc.EINVAL
    cache = _cache(6, 2, 64, 16)
    q = torch.randn(64, 4, 64, device=DEV).half()
    cu, lens = torch.arange(65, dtype=torch.int32, device=DEV), _i32([90] * 64)
    whole = zc.KVBatch(row.expand(64, 6).contiguous(), cu, lens, 64, 1)
    out, _ = zc.kv_attend(cache, whole, q)
    one = zc.KVBatch(row.expand(1, 6), cu[:2], lens[:1], 1, 1)  # a single row is no overlap
    assert torch.allclose(zc.kv_attend(cache, one, q[:1])[0], out[:1], atol=2 ** -8)
    cache.check()
