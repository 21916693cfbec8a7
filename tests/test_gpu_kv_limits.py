"""The 8-bit key/value cache on the GPU at the edges of what its calls take: layouts, counts, streams and states that
the ordinary tests do not reach."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import entropy_coding_gb300 as zc  # noqa: E402
from entropy_coding_gb300 import kv  # noqa: E402

from kv_reference import attend, to_codes  # noqa: E402

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


FALLING = [  # cu, lens: every pair but one or a few may be a sequence's
    ([0, 100, 110, 3, 200], [100, 210, 50, 197]),
    ([0, 100, 101, 102, 103, 5, 6, 7, 8], [300, 301, 302, 303, 100, 150, 151, 152]),
    ([0, 40, 90, 20, 25, 30, 35, 10, 15, 200], [200] * 9),
    ([60, 10, 70, 20, 80, 30, 90], [100] * 6),
]


@pytest.mark.parametrize("cu,lens", FALLING)
def test_counts_that_fall_are_reported_and_nothing_else_is_touched(cu, lens):
    """Blocks and scales that belong to no sequence keep their bytes, numbers around the outputs theirs."""
    n, width, total = len(lens), 20, 200
    g = torch.Generator(device=DEV).manual_seed(1)
    cache = _cache(n * width + 40, 2, 64, 16)
    table = torch.arange(20, 20 + n * width, dtype=torch.int32, device=DEV).view(n, width)
    batch = zc.KVBatch(table, _i32(cu), _i32(lens), total, total)
    before = [t.view(torch.uint8).clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    x = torch.randn(total, 2, 64, generator=g, device=DEV).half()
    q = torch.randn(total, 8, 64, generator=g, device=DEV).half()

    def attend():
        out = torch.full((total + 200, 8, 64), 3.0, dtype=torch.float16, device=DEV)
        lse = torch.full((total + 200, 8), 3.0, device=DEV)
        zc.kv_attend_into(cache, batch, q, out[100:-100], lse[100:-100])
        assert all((t[:100] == 3.0).all() and (t[-100:] == 3.0).all() for t in (out, lse))

    def read():
        k = torch.full((2, total + 200, 2, 64), 3.0, dtype=torch.float16, device=DEV)
        zc.kv_read_into(cache, batch, k[0, 100:-100], k[1, 100:-100])
        assert (k[:, :100] == 3.0).all() and (k[:, -100:] == 3.0).all()

    def write():
        zc.kv_write(cache, batch, x, x)
        for was, t in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)):
            now = t.view(torch.uint8)
            assert torch.equal(was[:20], now[:20]) and torch.equal(was[20 + n * width:], now[20 + n * width:])

    for call in (attend, read, write):
        call()
        with pytest.raises(zc.ZcError) as e:
            cache.check()
        assert e.value.status == zc.EFORMAT, call.__name__


def test_a_batch_whose_tokens_begin_inside_the_tensors():
    """cu that does not begin at 0: the rows before it are nobody's, and are left alone."""
    g = torch.Generator(device=DEV).manual_seed(2)
    lens, news, past = [1000, 37, 64], [3, 37, 1], 200
    table = torch.arange(3 * 63, dtype=torch.int32, device=DEV).view(3, 63)
    total = past + sum(news)
    x = torch.randn(total, 2, 64, generator=g, device=DEV).half()
    q = torch.randn(total, 4, 64, generator=g, device=DEV).half()
    caches = [_cache(3 * 63, 2, 64, 16) for _ in range(2)]
    got = []
    for c, off in zip(caches, (0, past)):
        cu = [off, off + 3, off + 40, off + 41]
        b = zc.KVBatch(table, _i32(cu), _i32(lens), off + sum(news), max(max(news), (off + sum(news) + 2) // 3))
        rows = slice(past - off, None)
        zc.kv_write(c, b, x[rows], x[rows])
        k = torch.full((2, off + 41, 2, 64), 3.0, dtype=torch.float16, device=DEV)
        zc.kv_read_into(c, b, k[0], k[1])
        out = torch.full((off + 41, 4, 64), 3.0, dtype=torch.float16, device=DEV)
        zc.kv_attend_into(c, b, q[rows], out)
        c.check()
        assert (k[:, :off] == 3.0).all() and (out[:off] == 3.0).all()
        got.append((k[:, off:], out[off:]))
    assert torch.equal(caches[0].k.view(torch.uint8), caches[1].k.view(torch.uint8)) and torch.equal(caches[0].k_scale, caches[1].k_scale)
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("seqs,new,dim,at", [(1, 1, 128, 0), (600, 1, 128, 0), (600, 1, 64, 40000), (1, 40, 128, 0), (160, 40, 128, 0),
                                             (160, 40, 64, 70000)])
@pytest.mark.parametrize("keys,share", [(8192, 0.99), (131072, 0.99), (131072, 0.999)])
def test_one_key_takes_nearly_all_of_the_weight_and_has_no_value(keys, share, seqs, new, dim, at, dtype):
    """The other keys' weights are the output then, each of them down to 2^-27 of the largest. Their numbers differ at
    random, as their roundings to half do: the output errs by no more than one such rounding, 2^-11 of what its values
    sum to in magnitude, and twice that is allowed, with the scores' own errors (2^-17 of their products' magnitudes)
    and the output's rounding to its type. Nothing in this grows with the keys. (The same tokens for many sequences: few of
    them share the key that takes the weight out with a short piece of the others.)"""
    rng = np.random.default_rng(keys + new + dim)
    block, heads, at = 64, 4, min(at, keys // 2)
    k, v = rng.standard_normal((keys, dim)) * dim ** -0.5, np.abs(rng.standard_normal((keys, dim)))
    k[:, -1], k[at], v[at] = 0.0, 0.0, 0.0
    k[at, -1] = 1.0
    q = rng.standard_normal((new, heads, dim))
    q[:, :, -1] = np.log(share / (1 - share) * keys * np.exp(0.5))
    kc, vc = (to_codes(x).reshape(keys // block, 1, block, dim) for x in (k, v))
    ones = np.ones((keys // block, 1), np.float32)
    table = rng.permutation(keys // block).astype(np.int32).reshape(1, -1)
    pool = [np.empty_like(c) for c in (kc, vc)]
    for p, c in zip(pool, (kc, vc)):
        p[table[0]] = c
    cache = zc.KVCache(*(torch.from_numpy(p).to(DEV) for p in pool), torch.from_numpy(ones).to(DEV), torch.from_numpy(ones).to(DEV))
    batch = zc.KVBatch(torch.from_numpy(table).to(DEV).repeat(seqs, 1), _i32(range(0, seqs * new + 1, new)), _i32([keys] * seqs),
                       seqs * new, new)
    qt = torch.from_numpy(q).to(DEV).to(dtype)
    out, lse = zc.kv_attend(cache, batch, qt.repeat(seqs, 1, 1), scale=1.0)
    cache.check()
    want, z, mass, size, _, _ = attend(qt.double().cpu().numpy(), pool[0], ones, pool[1], ones, table, [0, new], [keys], 1.0, True, 0)
    tol = mass * (2.0 ** -10 + 2.0 ** -16 * size)[..., None]
    low, high = (torch.from_numpy(want + d).to(dtype).double().numpy() for d in (-tol, tol))
    got = out.double().cpu().numpy().reshape(seqs, *want.shape)
    assert ((got >= low) & (got <= high)).all(), np.abs(got / want - 1).max()
    assert np.abs(lse.double().cpu().numpy().reshape(seqs, *z.shape) - z).max() < 2.0 ** -17 * size.max() + 2.0 ** -20 * np.abs(z).max()


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("exponent", [-118, 119])
def test_value_scales_near_the_ends_of_floats_range(exponent, new):
    """Outputs of 2^-118 and of 2^119 are bfloat16 numbers; 2^(mw - m) alone need not be a float. Weights are rounded to 11
    bits and the output to 8: 2^-8 of the values' magnitudes is allowed."""
    rng = np.random.default_rng(3)
    keys, dim, block = 512, 64, 16
    kc, vc = (to_codes(x).reshape(keys // block, 1, block, dim) for x in (rng.standard_normal((keys, dim)) * 0.5, np.abs(rng.standard_normal((keys, dim)))))
    ks, vs = np.ones((keys // block, 1), np.float32), np.full((keys // block, 1), 2.0 ** exponent, np.float32)
    table = np.arange(keys // block, dtype=np.int32).reshape(1, -1)
    cache = zc.KVCache(*(torch.from_numpy(np.array(a)).to(DEV) for a in (kc, vc, ks, vs)))
    batch = zc.KVBatch(torch.from_numpy(table).to(DEV), _i32([0, new]), _i32([keys]), new, new)
    q = torch.from_numpy(rng.standard_normal((new, 4, dim))).to(DEV).bfloat16()
    out, _ = zc.kv_attend(cache, batch, q, scale=1.0)
    cache.check()
    want, _, mass, _, _, _ = attend(q.double().cpu().numpy(), kc, ks, vc, vs, table, [0, new], [keys], 1.0, True, 0)
    assert (np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * mass).all()


MS = 2_000_000  # clocks: a millisecond and more


def _wrong(cache):
    """A batch that names a block which the pool does not have."""
    return zc.KVBatch(_i32([[cache.n_blocks]]), _i32([0, 1]), _i32([1]), 1, 1)


def test_check_waits_for_calls_on_other_streams():
    cache = _cache(4, 2, 64, 16)
    bad, side = _wrong(cache), torch.cuda.Stream()
    x = torch.zeros(1, 2, 64, device=DEV).half()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        with torch.cuda.stream(side):
            torch.cuda._sleep(100 * MS)
        zc.kv_write(cache, bad, x, x, stream=side)
        with pytest.raises(zc.ZcError) as e:
            cache.check()
        assert e.value.status == zc.EFORMAT
        cache.check()  # and has forgotten it


def _decoding(seqs=64, keys=4000, block=32):
    """A cache, and a maker of batches of one token for each sequence, whose items are cut and joined (by the counters of
    the workspace); queries, and what attention gives."""
    per = keys // block
    cache = _cache(per * 2, 2, 64, block)
    table = torch.stack([torch.randperm(per * 2, device=DEV)[:per].to(torch.int32) for _ in range(seqs)])
    cu, lens = torch.arange(seqs + 1, dtype=torch.int32, device=DEV), _i32([keys] * seqs)

    def batch():
        return zc.KVBatch(table, cu, lens, seqs, 1)

    q = torch.randn(seqs, 8, 64, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV).half()
    want, _ = zc.kv_attend(cache, batch(), q)
    cache.check()
    return cache, batch, q, want


def _leave_garbage(size):
    """Freed memory of this size, on the current stream, holds numbers that are not 0."""
    t = torch.full((size,), 0x55, dtype=torch.uint8, device=DEV)
    address = t.data_ptr()
    del t
    return address


def _size(cache, batch, heads):
    return max(16, zc.lib().zc_kv_attend_workspace_size(cache._ref, batch._ref, heads))


def test_one_batch_on_two_streams():
    """Its first stream is far behind: what that is to zero is not what the other one counts in."""
    cache, make, q, want = _decoding()
    batch, side = make(), torch.cuda.Stream()
    torch.cuda.synchronize()
    _leave_garbage(_size(cache, batch, 8))
    torch.cuda.synchronize()
    torch.cuda._sleep(100 * MS)
    first, _ = zc.kv_attend(cache, batch, q)
    other, _ = zc.kv_attend(cache, batch, q, stream=side)
    cache.check()
    assert torch.equal(first, want) and torch.equal(other, want)


def test_a_batch_that_is_dropped_while_another_stream_works_for_it():
    cache, make, q, want = _decoding()
    batch, side = make(), torch.cuda.Stream()
    assert torch.equal(zc.kv_attend(cache, batch, q)[0], want)
    size = _size(cache, batch, 8)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100 * MS)
    other, _ = zc.kv_attend(cache, batch, q, stream=side)
    del batch
    _leave_garbage(size)
    cache.check()
    assert torch.equal(other, want)


def test_an_error_before_the_status_is_zero_is_not_lost():
    """The stream on which the cache was made is far behind."""
    tensors, side = _cache(4, 2, 64, 16), torch.cuda.Stream()
    bad, x = _wrong(tensors), torch.zeros(1, 2, 64, device=DEV).half()
    zc.kv_write(tensors, bad, x, x, stream=side)  # (a kernel's first launch waits for the device)
    torch.cuda.synchronize()
    torch.cuda._sleep(100 * MS)
    cache = zc.KVCache(tensors.k, tensors.v, tensors.k_scale, tensors.v_scale)
    zc.kv_write(cache, bad, x, x, stream=side)
    with pytest.raises(zc.ZcError) as e:
        cache.check()
    assert e.value.status == zc.EFORMAT


def _give_up(cache, batch, q):
    """A call whose waits run out, and workspaces as CTAs that gave up at the worst moment leave them."""
    zc.lib().zc_kv_set_test_hooks(kv.HOOK_COPY_STALL)
    try:
        zc.kv_attend(cache, batch, q)
        torch.cuda.synchronize()
    finally:
        zc.lib().zc_kv_set_test_hooks(0)
    for ws in batch._ws.values():
        ws[2].fill_(1)
    with pytest.raises(zc.ZcError) as e:
        cache.check()
    assert e.value.status == zc.ETIMEOUT


def test_a_batch_is_used_again_after_a_call_that_gave_up():
    cache, make, q, want = _decoding()
    batch, other, side = make(), make(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        for b in (batch, other):
            assert torch.equal(zc.kv_attend(cache, b, q)[0], want)
        out, _ = zc.kv_attend(cache, batch, q, stream=side)
        cache.check()
        assert torch.equal(out, want)
        _give_up(cache, batch, q)


def test_a_captured_call_after_one_that_gave_up():
    cache, make, q, want = _decoding()
    batch, out = make(), torch.empty_like(want)
    zc.kv_attend_into(cache, batch, q, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        zc.kv_attend_into(cache, batch, q, out)
    _give_up(cache, batch, q)
    batch.reset()
    for _ in range(2):
        out.zero_()
        graph.replay()
        cache.check()
        assert torch.equal(out, want)


def test_a_first_call_in_a_capture_and_one_outside_it_before_the_replay():
    """The captured call's counters are zeroed when the graph runs: another call on the stream must not take them for zero
    before that (the graphs' memory held other numbers), and the graph keeps its memory when the batch is gone."""
    cache, make, q, want = _decoding()
    batch, side, pool = make(), torch.cuda.Stream(), torch.cuda.graph_pool_handle()
    size, out = _size(cache, batch, 8), torch.empty_like(want)
    garbage, graph = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(garbage, pool=pool, stream=side):
        _leave_garbage(size)
    garbage.replay()
    with torch.cuda.graph(graph, pool=pool, stream=side):
        zc.kv_attend_into(cache, batch, q, out)
    other, _ = zc.kv_attend(cache, batch, q, stream=side)
    cache.check()
    assert torch.equal(other, want)
    del batch
    _leave_garbage(size)
    for _ in range(2):
        out.zero_()
        graph.replay()
        cache.check()
        assert torch.equal(out, want)


@pytest.mark.parametrize("new", [1, 40])
def test_only_the_counters_of_a_workspace_are_zeroed(new):
    """The rest held other numbers, NaN as floats, before the batch's first call."""
    cache = _cache(200, 2, 64, 32)
    table = torch.randperm(200, device=DEV)[:190].to(torch.int32).view(2, 95)
    q = torch.randn(2 * new, 8, 64, device=DEV).half()
    outs = []
    for fill in (0x00, 0xFF):
        batch = zc.KVBatch(table, _i32([0, new, 2 * new]), _i32([3000, 2500]), 2 * new, new)
        t = torch.full((_size(cache, batch, 8),), fill, dtype=torch.uint8, device=DEV)
        address = t.data_ptr()
        del t
        outs.append(zc.kv_attend(cache, batch, q))
        assert batch.workspace(cache, 8)[0] == address  # (the allocator hands the freed memory on)
        del batch
    cache.check()
    assert not outs[0][0].isnan().any() and all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("new", [1, 40])
def test_windows_of_any_size(new):
    """From the sequence's length on, a window hides nothing, up to the largest that the C entry takes."""
    cache = _cache(10, 2, 64, 16)
    batch = zc.KVBatch(_i32([list(range(10))]), _i32([0, new]), _i32([150]), new, new)
    q = torch.randn(new, 8, 64, device=DEV).half()
    want, lse = zc.kv_attend(cache, batch, q)
    rows = kv._Rows(q.data_ptr(), 8 * 64, 64)
    address, size, _ = batch.workspace(cache, 8)
    for window in (150, 2 ** 20, 2 ** 30 - 1, 2 ** 30, 2 ** 31 - 1, 2 ** 31, 2 ** 32 - 1):
        out = torch.zeros_like(want)
        st = zc.lib().zc_kv_attend(cache._ref, batch._ref, zc.FP16, 8, ctypes.byref(rows),
                                   ctypes.byref(kv._Rows(out.data_ptr(), 8 * 64, 64)), None, 64 ** -0.5, 1, window, address, size,
                                   cache._status, torch.cuda.current_stream().cuda_stream)
        cache.check()
        assert st == zc.OK and torch.equal(out, want), window


def _against_reference(dtype, hkv, group, dim, block, lens, news, window=0):
    """Attention of a ragged batch against its definition. A weight is rounded to 11 bits, scores err by 2^-17 of their
    products' magnitudes, and the output is rounded to its type."""
    rng = np.random.default_rng(len(lens))
    per = [max(1, -(-n // block)) for n in lens]
    ids, table, at = rng.permutation(sum(per)), np.zeros((len(lens), max(per)), np.int32), 0
    for s, p in enumerate(per):
        table[s, :p] = ids[at: at + p]
        at += p
    kc, vc = (to_codes(rng.standard_normal((sum(per), hkv, block, dim)) * m) for m in (dim ** -0.5, 1.0))
    ks, vs = np.ones((sum(per), hkv), np.float32), np.exp2(rng.integers(-3, 4, (sum(per), hkv))).astype(np.float32)
    cache = zc.KVCache(*(torch.from_numpy(np.array(a)).to(DEV) for a in (kc, vc, ks, vs)))
    cu = np.concatenate([[0], np.cumsum(news)])
    batch = zc.KVBatch(torch.from_numpy(table).to(DEV), _i32(cu.tolist()), _i32(lens), int(cu[-1]), max(news))
    q = torch.from_numpy(rng.standard_normal((int(cu[-1]), hkv * group, dim))).to(DEV).to(dtype)
    out, lse = zc.kv_attend(cache, batch, q, scale=1.0, window=window)
    cache.check()
    want, z, mass, size, _, _ = attend(q.double().cpu().numpy(), kc, ks, vc, vs, table, cu, lens, 1.0, True, window)
    tol = mass * (2.0 ** -10 + 2.0 ** -16 * size)[..., None]
    low, high = (torch.from_numpy(want + d).to(dtype).double().numpy() for d in (-tol, tol))
    got = out.double().cpu().numpy()
    assert ((got >= low) & (got <= high)).all()
    seen = np.isfinite(z)
    got = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(got), ~seen) and (np.abs(got - z)[seen] < (2.0 ** -16 * size + 2.0 ** -19)[seen]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("seqs", [129, 256, 400])
def test_single_tokens_of_more_sequences_than_a_cta_has_threads(seqs, dtype):
    rng = np.random.default_rng(seqs)
    lens = rng.integers(1, 300, seqs).tolist()
    news = [0 if i % 17 == 5 else 1 for i in range(seqs)]
    _against_reference(dtype, 1, 4, 64, 16, lens, news)


@pytest.mark.parametrize("dim,window", [(64, 0), (128, 30)])
def test_prompts_of_more_slots_than_a_cta_has_threads(dim, window):
    """600 sequences of 17 to 40 tokens of 8 heads: more slots of 256 rows than 512."""
    rng = np.random.default_rng(dim)
    news = rng.integers(17, 41, 600).tolist()
    news[7] = news[599] = 0
    lens = [n + int(k) for n, k in zip(news, rng.integers(0, 30, 600))]
    _against_reference(torch.bfloat16, 1, 8, dim, 16, lens, news, window)


@pytest.mark.parametrize("at", [0, 130, 259])
def test_a_prompt_among_more_single_tokens_than_a_cta_has_threads(at):
    """Both kernels, each on its own sequences."""
    rng = np.random.default_rng(at)
    lens, news = rng.integers(1, 200, 260).tolist(), [1] * 260
    lens[at], news[at] = 700, 300
    _against_reference(torch.float16, 1, 4, 64, 32, lens, news)


@pytest.mark.parametrize("new", [1, 40])
def test_a_block_louder_by_more_than_a_float_holds(new):
    """The last block's value scale is 2^130 times the others', its keys' weights 2^-140 of theirs: 2^-10 of the output.
    (The same tokens for many sequences, so that whole sequences are one piece of work.)"""
    keys, dim, block, seqs = 256, 64, 16, 600
    rng = np.random.default_rng(4)
    k, v = np.zeros((keys, dim)), np.abs(rng.standard_normal((keys, dim)))
    k[-block:, -1] = -1.0
    kc, vc = (to_codes(x).reshape(keys // block, 1, block, dim) for x in (k, v))
    ks, vs = np.ones((keys // block, 1), np.float32), np.full((keys // block, 1), 2.0 ** -100, np.float32)
    vs[-1] = 2.0 ** 30
    table = np.arange(keys // block, dtype=np.int32).reshape(1, -1)
    cache = zc.KVCache(*(torch.from_numpy(np.array(a)).to(DEV) for a in (kc, vc, ks, vs)))
    batch = zc.KVBatch(torch.from_numpy(table).to(DEV).repeat(seqs, 1), _i32(range(0, seqs * new + 1, new)), _i32([keys] * seqs),
                       seqs * new, new)
    q = torch.zeros(new, 4, dim, device=DEV).bfloat16()
    q[..., -1] = 97.0  # 2^-140
    out, lse = zc.kv_attend(cache, batch, q.repeat(seqs, 1, 1), scale=1.0, causal=False)
    cache.check()
    want, z, mass, _, _, _ = attend(q.double().cpu().numpy(), kc, ks, vc, vs, table, [0, new], [keys], 1.0, False, 0)
    assert (np.abs(out.double().cpu().numpy().reshape(seqs, *want.shape) - want) <= 2.0 ** -7 * mass).all()
    assert np.abs(lse.double().cpu().numpy().reshape(seqs, *z.shape) - z).max() < 1e-5


def test_a_stream_in_every_form():
    """Current, as a torch stream, as a handle, the default one for a cache that was made on another, an external one."""
    cache, make, q, want = _decoding(seqs=20)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        there = zc.KVCache(cache.k, cache.v, cache.k_scale, cache.v_scale)
        outs = [zc.kv_attend(there, make(), q)[0]]
    batch = make()
    for stream in (None, side, side.cuda_stream, 0, torch.cuda.default_stream(), torch.cuda.ExternalStream(side.cuda_stream)):
        torch.cuda.synchronize()
        outs.append(zc.kv_attend(there, batch, q, stream=stream)[0])
        k, v = zc.kv_read(there, batch, dtype=torch.float16, stream=stream)
        zc.kv_write(there, batch, k, v, stream=stream)  # what is there already
    there.check()
    assert len(batch._ws) == 2 and all(torch.equal(o, want) for o in outs)
