"""Calls of several threads of Python at once, each on a stream of its own, over one cache."""
from __future__ import annotations

import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import entropy_coding_gb300 as zc  # noqa: E402

DEV = torch.device("cuda:0")
SEQS, LEN, THREADS, STEPS = 3, 200, 4, 25


@pytest.mark.parametrize("kind", [zc.KVCache, zc.KV4Cache])
def test_threads_with_streams_of_their_own(kind):
    g = torch.Generator(device=DEV).manual_seed(5)
    width = LEN // 16 + 1
    cache = kind.empty(THREADS * SEQS * width, 2, 64, 16)
    rotation = zc.KVRotation([100.0 ** (-i / 32) for i in range(32)])
    table = torch.arange(THREADS * SEQS * width, dtype=torch.int32, device=DEV).view(THREADS, SEQS, width)
    x = torch.randn(THREADS, SEQS * LEN, 8, 64, generator=g, device=DEV).half()
    torch.cuda.synchronize()

    def work(t, steps):
        """Prompts, and after them one token a step; every output of it."""
        outs = []
        for step in range(steps):
            new, lens = (LEN - STEPS, LEN - STEPS) if step == 0 else (1, LEN - STEPS + step)
            cu = torch.arange(SEQS + 1, dtype=torch.int32, device=DEV) * new
            batch = zc.KVBatch(table[t], cu, torch.full((SEQS,), lens, dtype=torch.int32, device=DEV), SEQS * new, new)
            rows = x[t, step * SEQS: step * SEQS + SEQS * new]
            q, k = zc.kv_rotate(cache, batch, rotation, rows[:, :4], rows[:, 4:6])
            zc.kv_write(cache, batch, k, rows[:, 6:])
            outs += [q, *zc.kv_attend(cache, batch, q), *zc.kv_read(cache, batch)]
        return outs

    want = [work(t, STEPS) for t in range(THREADS)]
    torch.cuda.synchronize()
    got, errors = [None] * THREADS, []

    def run(t):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[t] = work(t, STEPS)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(t,)) for t in range(THREADS)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    cache.check()
    for t in range(THREADS):
        assert all(torch.equal(a, b) for a, b in zip(got[t], want[t]))
