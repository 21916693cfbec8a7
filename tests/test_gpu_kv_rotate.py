"""Norms of queries and keys and the rotation by their positions, on the GPU, against their definition in 64 bits.

The tolerance, before the one rounding to the type: a float32 sum of up to 128 squares is within 20 steps of 2^-24 (16 one
after another in a lane, three across lanes), of which the root takes half; the reciprocal root's own error is 2^-22, two
products more 2^-23: 2^-20 of a normed number. Sine and cosine: an angle within an eighth of a turn, rounded to 24 bits, and
two units of sincospif: 2^-22 each; a turned number adds two products: 2^-21 of |a| + |b|. Together 2^-19 (|a| + |b|)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import entropy_coding_gb300 as zc  # noqa: E402

from kv4_reference import rotate  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _batch(news, lens):
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    return zc.KVBatch(torch.zeros(len(lens), 8, dtype=torch.int32, device=DEV), torch.from_numpy(cu).to(DEV),
                      torch.tensor(lens, dtype=torch.int32, device=DEV), int(cu[-1]), int(max(news)))


def _positions(news, lens):
    return [n - m + i for n, m in zip(lens, news) for i in range(m)]


def _frequencies(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def _check(got, x, positions, frequencies, interleaved, weight, eps, dtype):
    x64 = x.double().cpu().numpy()
    w = None if weight is None else weight.double().cpu().numpy()
    want = rotate(x64, positions, frequencies, interleaved, w, eps)
    plain = rotate(x64, positions, [], interleaved, w, eps)
    size = np.abs(plain).copy()
    half = len(frequencies)
    if half:
        a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
        both = size[..., a] + size[..., b]
        size[..., a] = size[..., b] = both
    if weight is None:
        size[..., 2 * half:] = 0.0  # neither normed nor turned: the input
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(want))
    tol = 2.0 ** -19 * size
    with np.errstate(invalid="ignore", over="ignore"):
        low, high = (torch.from_numpy(want + d).to(DT[dtype]).double().numpy() for d in (-tol, tol))
        bad = ~np.isnan(want) & ((g < low) | (g > high))
    assert not bad.any(), (g[bad][:8], low[bad][:8], high[bad][:8])


CASES = [  # dtype, heads, kv heads, dim, rot, interleaved, norm, lens, new
    ("bf16", 32, 8, 128, 128, False, "own", [100, 4000, 1, 7], [1, 1, 1, 1]),
    ("bf16", 32, 8, 128, 128, False, "own", [700], [700]),
    ("fp16", 12, 6, 80, 32, True, None, [131072, 100000], [33, 5]),
    ("fp32", 5, 1, 64, 64, False, "fp32", [70, 0, 9], [70, 0, 3]),
    ("bf16", 8, 8, 96, 96, True, "fp32", [50, 60], [50, 2]),
    ("fp16", 7, 1, 112, 112, False, "own", [37], [37]),
    ("bf16", 3, 2, 16, 16, False, "own", [300], [300]),
    ("bf16", 1, 1, 16, 0, False, "own", [9, 5], [9, 5]),
    ("fp32", 2, 2, 32, 16, True, "own", [2 ** 30 - 1, 3], [5, 3]),
    ("fp16", 71, 1, 48, 48, True, "fp32", [129, 1], [129, 1]),
    ("bf16", 4, 4, 128, 64, False, "q", [200], [100]),
    ("fp16", 4, 2, 80, 80, False, "k", [200, 2], [100, 2]),
    ("bf16", 300, 60, 128, 128, False, "own", [6], [6]),
    ("bf16", 4, 1, 64, 64, False, "own", [33] * 700, [1] * 500 + [3] * 200),
    ("fp32", 2, 1, 128, 0, False, None, [12], [12]),
]


def _weights(norm, dim, dtype, g):
    if norm is None:
        return None, None
    t = torch.float32 if norm == "fp32" else DT[dtype]
    wq, wk = ((1.0 + 0.3 * torch.randn(dim, generator=g, device=DEV)).to(t) for _ in range(2))
    return (None if norm == "k" else wq), (None if norm == "q" else wk)


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("dtype,heads,kv_heads,dim,rot,interleaved,norm,lens,news", CASES)
def test_rotate_matches_its_definition(dtype, heads, kv_heads, dim, rot, interleaved, norm, lens, news, fused):
    g = torch.Generator(device=DEV).manual_seed(3)
    T = sum(news)
    cache = zc.KVCache.empty(1, kv_heads, dim, 16)
    batch = _batch(news, lens)
    rotation = zc.KVRotation(_frequencies(rot), interleaved=interleaved)
    x = torch.randn(T, heads + kv_heads, dim, generator=g, device=DEV) * torch.exp2(torch.randint(-4, 5, (T, 1, 1), generator=g, device=DEV).float())
    x = x.to(DT[dtype])
    q, k = x[:, :heads], x[:, heads:]
    if not fused:
        q, k = q.contiguous(), k.transpose(0, 1).contiguous().transpose(0, 1)
    wq, wk = _weights(norm, dim, dtype, g)
    q2, k2 = zc.kv_rotate(cache, batch, rotation, q, k, wq, wk, eps=1e-5)
    cache.check()
    assert q2.is_contiguous() and k2.is_contiguous() and q2.dtype == q.dtype
    for got, y, w in ((q2, q, wq), (k2, k, wk)):
        _check(got, y, _positions(news, lens), _frequencies(rot), interleaved, w, float(np.float32(1e-5)), dtype)
    # into the inputs themselves, and into other layouts: the same bits
    zc.kv_rotate_into(cache, batch, rotation, q, k, q, k, wq, wk, eps=1e-5)
    assert torch.equal(q, q2) and torch.equal(k, k2)
    both = x.clone()
    if fused:
        assert torch.equal(x[:, :heads], q2) and torch.equal(x[:, heads:], k2)
    out = torch.full((heads + kv_heads, T, dim), 7.0, device=DEV, dtype=DT[dtype]).transpose(0, 1)
    both[:, :heads], both[:, heads:] = q2, k2
    zc.kv_rotate_into(cache, batch, zc.KVRotation([]), q2, k2, out[:, :heads], out[:, heads:])
    assert torch.equal(out, both)  # nothing to do: the inputs
    cache.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32", "fp16"])
def test_norms_of_rows_near_the_ends_of_the_types_range(dtype):
    """Squares that float32 cannot hold, rows of zeros, of infinities and NaN, an eps that matters or hardly does."""
    big = 60000.0 if dtype == "fp16" else 1e38
    small = 2.0 ** -20 if dtype == "fp16" else 1e-30
    g = torch.Generator(device=DEV).manual_seed(1)
    dim, rows = 64, 12
    x = torch.randn(rows, 1, dim, generator=g, device=DEV)
    x[0], x[1], x[2], x[3] = x[0] * big / 8, x[1] * small, 0.0, 0.0
    x[3, 0, 5] = big
    x[4, 0, 7], x[5, 0, 9] = float("inf"), float("nan")
    x[6] = x[6] * 1e18 if dtype != "fp16" else x[6]
    x[7] = x[7] * 1e-18 if dtype != "fp16" else x[7]
    x[8], x[9] = x[8] * 1e-22 if dtype != "fp16" else x[8] * 2.0 ** -18, 0.0
    x[9, 0, 0] = small
    x = x.to(DT[dtype])
    w = torch.ones(dim, device=DEV) * 0.5
    cache, batch = zc.KVCache.empty(1, 1, dim, 16), _batch([rows], [rows])
    for eps in (1e-6, 1e-30, 1e-38, 3.0):
        q, k = zc.kv_rotate(cache, batch, zc.KVRotation([]), x, x, w, w, eps=eps)
        _check(q, x, range(rows), [], False, w, float(np.float32(eps)), dtype)
        assert torch.equal(q.nan_to_num(3.0), k.nan_to_num(3.0))


def test_infinities_stay_in_their_pairs():
    x = torch.ones(4, 1, 32, device=DEV)
    x[1, 0, 3], x[2, 0, 25] = float("inf"), float("nan")
    cache, batch = zc.KVCache.empty(1, 1, 32, 16), _batch([4], [4])
    q, _ = zc.kv_rotate(cache, batch, zc.KVRotation(_frequencies(16)), x, x)
    ok = torch.isfinite(q[:, 0])
    assert not ok[1, [3, 11]].any() and ok[1].sum() == 30 and not ok[2, 25] and ok[2].sum() == 31 and ok[[0, 3]].all()


def test_rows_behind_the_last_sequence_and_of_wrong_counts_stay_as_they_were():
    cache = zc.KVCache.empty(1, 1, 32, 16)
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    rotation = zc.KVRotation(_frequencies(32))
    x = torch.randn(9, 1, 32, device=DEV).half()
    for cu, lens, touched, bad in (([0, 2, 5], [8, 3], range(0, 5), False), ([1, 2, 5], [8, 3], range(1, 5), False),
                                   ([0, 4, 2], [8, 9], range(0, 4), True), ([0, 2, 5], [1, 3], range(2, 5), True),
                                   ([0, 2, 11], [8, 20], range(0, 2), True), ([0, 2, 5], [-1, 3], range(2, 5), True),
                                   ([0, 9, 9], [9, 5], (), True)):
        batch = zc.KVBatch(t([[0], [0]]), t(cu), t(lens), 9, 6)
        q, k = torch.full_like(x, 5.0), torch.full_like(x, 6.0)
        zc.kv_rotate_into(cache, batch, rotation, x, x, q, k)
        if bad:
            with pytest.raises(zc.ZcError) as e:
                cache.check()
            assert e.value.status == zc.EFORMAT
        cache.check()
        rest = [i for i in range(9) if i not in touched]
        assert (q[rest] == 5.0).all() and (k[rest] == 6.0).all() and not (q[list(touched)] == 5.0).all(-1).any()


def test_a_captured_call_follows_the_lengths_and_streams_keep_their_order():
    cache = zc.KV4Cache.empty(4, 2, 64, 16)
    batch = _batch([1, 1], [5, 90])
    rotation = zc.KVRotation(_frequencies(64))
    x = torch.randn(2, 2, 64, device=DEV).bfloat16()
    w = torch.rand(64, device=DEV)
    q, k = torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    zc.kv_rotate_into(cache, batch, rotation, x, x, q, k, w, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        zc.kv_rotate_into(cache, batch, rotation, x, x, q, k, w, w)
    for _ in range(5):
        batch.lens.add_(7)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        a, b = zc.kv_rotate(cache, batch, zc.KVRotation(_frequencies(64)), x, x, w, w, stream=side)
        c, d = zc.kv_rotate(cache, batch, rotation, x, x, w, w, stream=side.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(a, q) and torch.equal(b, k) and torch.equal(c, q) and torch.equal(d, k)
    cache.check()


def test_arguments_that_the_host_refuses():
    cache = zc.KVCache.empty(1, 2, 32, 16)
    batch = _batch([2, 1], [9, 4])
    r = zc.KVRotation(_frequencies(32))
    q, k, w = torch.zeros(3, 4, 32, device=DEV).half(), torch.zeros(3, 2, 32, device=DEV).half(), torch.ones(32, device=DEV)
    for i, call in enumerate([
            lambda: zc.kv_rotate(cache, batch, r, q, k[:, :1]), lambda: zc.kv_rotate(cache, batch, r, q[:2], k),
            lambda: zc.kv_rotate(cache, batch, r, q.float(), k), lambda: zc.kv_rotate(cache, batch, r, q.double(), k.double()),
            lambda: zc.kv_rotate(cache, batch, r, q, k.cpu()), lambda: zc.kv_rotate(cache, batch, r, q[0], k),
            lambda: zc.kv_rotate(cache, batch, r, q, k, w[:16], w), lambda: zc.kv_rotate(cache, batch, r, q, k, w.bfloat16(), w.bfloat16()),
            lambda: zc.kv_rotate(cache, batch, r, q, k, w.half(), w), lambda: zc.kv_rotate(cache, batch, r, q, k, w.cpu(), w),
            lambda: zc.kv_rotate(cache, batch, r, q, k, w, w, eps=0.0), lambda: zc.kv_rotate(cache, batch, r, q, k, w, w, eps=float("nan")),
            lambda: zc.kv_rotate(cache, batch, r, q, k, torch.ones(64, device=DEV)[::2], w),
            lambda: zc.kv_rotate(cache, batch, zc.KVRotation(_frequencies(48)), q, k),
            lambda: zc.kv_rotate(cache, batch, zc.KVRotation(_frequencies(32), device="cpu"), q, k),
            lambda: zc.kv_rotate_into(cache, batch, r, q, k, q[:, :2], k), lambda: zc.kv_rotate_into(cache, batch, r, q, k, q.float(), k.float()),
            lambda: zc.kv_rotate_into(cache, batch, r, q, k, q, torch.as_strided(k, (3, 2, 32), (32, 96, 1))),
            lambda: zc.kv_rotate(cache, batch, r, torch.zeros(3, 4, 33, device=DEV).half()[:, :, :32], k)]):
        with pytest.raises(zc.ZcError) as e:
            call()
        assert e.value.status == zc.EINVAL, i
    empty = zc.KVBatch(batch.block_table, torch.zeros(3, dtype=torch.int32, device=DEV), batch.lens, 0, 0)
    assert zc.kv_rotate(cache, empty, r, q[:0], k[:0])[0].shape == (0, 4, 32)
    out = zc.kv_rotate(cache, batch, r, q.requires_grad_(), k.requires_grad_())
    assert not out[0].requires_grad and not out[1].requires_grad
    cache.check()
