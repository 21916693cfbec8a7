"""The cache's calls through ctypes, as where the module of its calls on torch tensors cannot be built, give the same bits."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import entropy_coding_gb300 as zc  # noqa: E402
from entropy_coding_gb300 import kv  # noqa: E402


@pytest.mark.parametrize("kind", [zc.KVCache, zc.KV4Cache])
def test_calls_without_the_module(kind, monkeypatch):
    dev = torch.device("cuda:0")
    x = torch.randn(90, 8, 64, generator=torch.Generator(device=dev).manual_seed(1), device=dev).half()
    weight = torch.rand(64, device=dev)
    outs = []
    kind.empty(1, 1, 64, 16)
    for module in (kv._torch, False):
        monkeypatch.setattr(kv, "_torch", module)
        cache = kind.empty(8, 2, 64, 16)
        assert (cache._quick is None) == (module is False)
        batch = zc.KVBatch(torch.arange(8, dtype=torch.int32, device=dev).view(2, 4), torch.tensor([0, 40, 90], dtype=torch.int32, device=dev),
                           torch.tensor([60, 50], dtype=torch.int32, device=dev), 90, 50)
        rotation = zc.KVRotation([10.0 ** -i for i in range(16)])
        q, k = zc.kv_rotate(cache, batch, rotation, x[:, :4], x[:, 4:6], weight, weight)
        zc.kv_write(cache, batch, k, x[:, 6:])
        outs.append([q, k, *zc.kv_read(cache, batch), *zc.kv_attend(cache, batch, q, causal=False)])
        cache.check()
    assert all(torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip(*outs))
