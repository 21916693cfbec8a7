"""The 8-bit key/value cache on the GPU against its definitions in 64 bits.

Writing and reading back are exact: the codes, scales and numbers equal the
definition's. Attention's tolerance, for a row over n keys with scores whose
products sum to at most S in magnitude:

* a score is a float32 sum of head_dim products in at most 16 chained steps of
  the tensor cores, each within 2^-22 of what it adds up: 2^-18 S, and as much
  again for the scaling and the exponential's 2^-22 relative error;
* a weight is rounded to half (2^-11 relative, or 2^-25 of the largest
  contribution's unit), and at most n of them are added up in float32;
* the output is rounded once to its type: it lies between the roundings of
  the definition's value less and plus the above.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import entropy_coding_gb300 as zc  # noqa: E402
from entropy_coding_gb300 import kv  # noqa: E402

from kv_reference import VALUES, attend, rows_of, to_codes, write  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _table(lens, block, rng, spare=3):
    per = [max(1, -(-int(n) // block)) for n in lens]
    ids = rng.permutation(sum(per) + spare)
    t, at = np.zeros((len(lens), max(per)), np.int32), 0
    for s, p in enumerate(per):
        t[s, :p] = ids[at: at + p]
        at += p
    return t, len(ids)


def _batch(table, news, lens):
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    b = zc.KVBatch(torch.from_numpy(table).to(DEV), torch.from_numpy(cu).to(DEV),
                   torch.tensor(lens, dtype=torch.int32, device=DEV), int(cu[-1]), int(max(news)))
    return b, cu


def _pool(n_blocks, hkv, block, dim, rng, nan=False, spread=3):
    """Random codes (every code that is not NaN, or every code) and power-of-two scales."""
    c = rng.integers(0, 256, (n_blocks, hkv, block, dim), dtype=np.uint8)
    if not nan:
        c[(c & 0x7F) == 0x7F] = 0x40
    s = np.exp2(rng.integers(-9 - spread, -8 + spread, (n_blocks, hkv))).astype(np.float32)
    return c, s


def _cache(kc, ks, vc, vs):
    return zc.KVCache(*(torch.from_numpy(np.array(a)).to(DEV) for a in (kc, vc, ks, vs)))


def _strided(shape, dtype, kind):
    """A tensor of this shape that is contiguous, or a view of a fused projection, or head-major."""
    T, H, D = shape
    if kind == "fused":
        return torch.empty(T, 3 * H * D + 16, dtype=dtype, device=DEV)[:, 16 + H * D: 16 + 2 * H * D].view(T, H, D) \
            if H * D % 16 == 0 else torch.empty(shape, dtype=dtype, device=DEV)
    if kind == "heads":
        return torch.empty(H, T, D, dtype=dtype, device=DEV).transpose(0, 1)
    return torch.empty(shape, dtype=dtype, device=DEV)


WRITES = [  # dtype, block, kv heads, dim, lens, new tokens, strides
    ("bf16", 64, 8, 128, [1, 64, 65, 200], [1, 1, 1, 1], "plain"),
    ("bf16", 16, 2, 128, [500, 37, 16], [500, 21, 16], "fused"),
    ("fp16", 32, 3, 64, [100, 31, 33, 400], [0, 31, 2, 399], "heads"),
    ("fp32", 128, 1, 80, [129, 127, 300], [129, 1, 173], "fused"),
    ("fp32", 48, 5, 16, [47, 48, 49, 95], [3, 2, 2, 95], "heads"),
    ("fp16", 256, 2, 112, [700], [443], "plain"),
    ("bf16", 16, 1, 32, [33] * 300, [1] * 150 + [17] * 150, "plain"),
]


@pytest.mark.parametrize("dtype,block,hkv,dim,lens,news,strides", WRITES)
def test_write_gives_the_definitions_codes_and_scales(dtype, block, hkv, dim, lens, news, strides):
    rng = np.random.default_rng(7)
    table, n_blocks = _table(lens, block, rng)
    kc, ks = _pool(n_blocks, hkv, block, dim, rng)
    vc, vs = _pool(n_blocks, hkv, block, dim, rng, spread=8)
    batch, cu = _batch(table, news, lens)
    cache = _cache(kc, ks, vc, vs)
    T = int(cu[-1])
    xs = []
    for mag in (1.0, 30.0):
        x = rng.standard_normal((T, hkv, dim)) * mag * np.exp2(rng.integers(-6, 6, (T, 1, 1)))
        x[rng.random((T, hkv, dim)) < 0.05] = 0.0
        t = _strided((T, hkv, dim), DT[dtype], strides)
        t.copy_(torch.from_numpy(x))
        xs.append(t)
    for _ in range(2):  # writing the same tokens again changes nothing
        zc.kv_write(cache, batch, *xs)
    cache.check()
    write(kc, ks, xs[0].double().cpu().numpy(), table, cu, lens)
    write(vc, vs, xs[1].double().cpu().numpy(), table, cu, lens)
    for got, want in ((cache.k, kc), (cache.v, vc)):
        assert np.array_equal(VALUES[got.cpu().numpy()], VALUES[want])
    assert np.array_equal(cache.k_scale.cpu().numpy(), ks) and np.array_equal(cache.v_scale.cpu().numpy(), vs)


def test_write_of_zeros_extremes_and_non_finite_numbers():
    big, tiny = 3.3e38, 1e-45
    rows = [[0.0] * 16, [448.0] + [0.0] * 15, [449.0] + [-1.0] * 15, [big, -big] + [1.0] * 14, [tiny, -tiny] + [0.0] * 14,
            [float("inf"), float("-inf"), 1.0] + [0.5] * 13, [float("nan"), 2.0] + [0.25] * 14, [float("nan")] * 16,
            [448.0 * 2.0 ** -126] * 16, [2.0 ** -140] * 16, [-0.0] * 16]
    n = len(rows)
    x = torch.tensor(rows, dtype=torch.float32, device=DEV).view(n, 1, 16)
    table = np.arange(n, dtype=np.int32).reshape(n, 1)
    batch, cu = _batch(table, [1] * n, [1] * n)
    cache = zc.KVCache.empty(n, 1, 16, block_tokens=16)
    zc.kv_write(cache, batch, x, x)
    cache.check()
    kc, ks = np.zeros((n, 1, 16, 16), np.uint8), np.ones((n, 1), np.float32)
    write(kc, ks, x.double().cpu().numpy(), table, cu, [1] * n)
    assert np.array_equal(cache.k_scale.cpu().numpy(), ks)
    got = cache.k.view(torch.uint8).cpu().numpy()
    assert np.array_equal(VALUES[got[:, :, 0]], VALUES[kc[:, :, 0]], equal_nan=True)


def test_rows_written_one_by_one_move_to_the_scale_of_the_largest():
    rng = np.random.default_rng(3)
    n, block = 40, 32
    mags = np.exp2(rng.integers(-12, 13, n))
    x = torch.from_numpy(rng.standard_normal((n, 1, 64)) * mags[:, None, None]).to(DEV).float()
    cache = zc.KVCache.empty(2, 1, 64, block_tokens=block)
    table = np.array([[1, 0]], np.int32)
    kc, ks = np.zeros((2, 1, block, 64), np.uint8), np.ones((2, 1), np.float32)
    for i in range(n):
        batch, cu = _batch(table, [1], [i + 1])
        zc.kv_write(cache, batch, x[i: i + 1], x[i: i + 1])
        write(kc, ks, x[i: i + 1].double().cpu().numpy(), table, cu, [i + 1])
    cache.check()
    assert np.array_equal(cache.k_scale.cpu().numpy(), ks)
    assert np.array_equal(VALUES[cache.k.view(torch.uint8).cpu().numpy()], VALUES[kc])


def test_write_takes_scales_that_are_no_powers_of_two():
    rng = np.random.default_rng(4)
    kc, _ = _pool(2, 2, 16, 32, rng)
    ks = np.array([[0.3, 3.0], [1e-3, 7.5]], np.float32)
    table = np.array([[1, 0]], np.int32)
    batch, cu = _batch(table, [3], [12])
    cache = _cache(kc, ks, kc, ks)
    x = torch.randn(3, 2, 32, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    zc.kv_write(cache, batch, x, x)
    cache.check()
    write(kc, ks, x.double().cpu().numpy(), table, cu, [12])
    assert np.array_equal(cache.v_scale.cpu().numpy(), ks)
    assert np.array_equal(VALUES[cache.v.cpu().numpy()], VALUES[kc])


@pytest.mark.parametrize("dtype,block,hkv,dim,lens,news,strides", WRITES)
def test_read_gives_the_numbers_that_the_codes_stand_for(dtype, block, hkv, dim, lens, news, strides):
    rng = np.random.default_rng(8)
    table, n_blocks = _table(lens, block, rng)
    kc, ks = _pool(n_blocks, hkv, block, dim, rng, nan=True)
    vc, vs = _pool(n_blocks, hkv, block, dim, rng, spread=12)
    vs[0, 0], vs[-1, -1] = 2.0 ** 100, 0.7
    batch, cu = _batch(table, news, lens)
    cache = _cache(kc, ks, vc, vs)
    T = int(cu[-1])
    k, v = (_strided((T, hkv, dim), DT[dtype], strides) for _ in range(2))
    zc.kv_read_into(cache, batch, k, v)
    cache.check()
    for got, c, s in ((k, kc, ks), (v, vc, vs)):
        want = np.concatenate([rows_of(c, s, table[i], n)[:, n - m:].transpose(1, 0, 2)
                               for i, (n, m) in enumerate(zip(lens, news))])
        want = torch.from_numpy(want).float().to(DT[dtype])  # a code times a float32 scale is rounded to float32, then to the type
        assert torch.equal(got.cpu().nan_to_num(7.0), want.nan_to_num(7.0)) and torch.equal(got.cpu().isnan(), want.isnan())
    k2, v2 = zc.kv_read(cache, batch, dtype=DT[dtype])
    assert torch.equal(k2.nan_to_num(7.0), k.nan_to_num(7.0)) and torch.equal(v2, v)


def _attend_case(dtype, block, hkv, group, dim, lens, news, causal, window, scale=None, seed=11, strides="plain",
                 spread=1, edit=None, q_mag=1.0):
    rng = np.random.default_rng(seed)
    table, n_blocks = _table(lens, block, rng)
    kc, ks = _pool(n_blocks, hkv, block, dim, rng)
    vc, vs = _pool(n_blocks, hkv, block, dim, rng, spread=spread)
    ks *= 1.0 / 16  # scores of a few units
    batch, cu = _batch(table, news, lens)
    T, H = int(cu[-1]), hkv * group
    q = _strided((T, H, dim), DT[dtype], strides)
    q.copy_(torch.from_numpy(rng.standard_normal((T, H, dim)) * q_mag))
    if edit:
        edit(kc, ks, vc, vs, table, q)
    cache = _cache(kc, ks, vc, vs)
    out = _strided((T, H, dim), DT[dtype], strides)
    out.fill_(123.0)
    lse = torch.full((T, H), 5.0, device=DEV)
    zc.kv_attend_into(cache, batch, q, out, lse, scale, causal, window)
    cache.check()
    sc = dim ** -0.5 if scale is None else scale
    want = attend(q.double().cpu().numpy(), kc, ks, vc, vs, table, cu, lens, sc, causal, window)
    _compare(out, lse, want, dtype)
    return cache, batch, q, out, lse


def _compare(out, lse, want, dtype):
    o, z, mass, size, count, unit = want
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(o)) and np.array_equal(np.isnan(got_lse), np.isnan(z))
    assert np.array_equal(np.isneginf(got_lse), np.isneginf(z))
    score = 2.0 ** -17 * size + 2.0 ** -21
    rel = 2.0 ** -11 + 2 * score + count * 2.0 ** -23
    tol = mass * rel[..., None] + (count * unit * 448 * 2.0 ** -25)[..., None]
    fine = np.isfinite(o)
    low, high = (torch.from_numpy(o + d).to(DT[dtype]).double().numpy() for d in (-tol, tol))
    bad = fine & ((got < low) | (got > high))
    assert not bad.any(), (got[bad][:8], low[bad][:8], high[bad][:8])
    fine = np.isfinite(z)
    tol = (score + count * 2.0 ** -23)[fine] + 2.0 ** -21 * np.abs(z[fine])
    assert (np.abs(got_lse[fine] - z[fine]) <= tol).all(), (np.abs(got_lse[fine] - z[fine]) / tol).max()
    none = np.isneginf(z)
    assert (got[none] == 0).all()


ATTENDS = [  # dtype, block, kv heads, group, dim, lens, new, causal, window
    ("bf16", 64, 2, 4, 128, [1, 2, 63, 64, 65, 1000], [1] * 6, True, 0),          # single tokens
    ("fp16", 16, 1, 1, 64, [1, 15, 16, 17, 700], [1] * 5, True, 0),               # one head
    ("bf16", 32, 2, 8, 128, [400, 37, 2000], [1, 1, 1], True, 64),                # a window inside
    ("fp16", 16, 2, 7, 112, [300, 50], [1, 1], False, 0),
    ("bf16", 48, 3, 5, 80, [200, 33, 100], [4, 2, 7], True, 0),                   # drafted tokens
    ("fp16", 64, 2, 8, 128, [500, 900, 8], [8, 3, 8], True, 100),
    ("bf16", 16, 1, 3, 16, [77], [77], True, 0),                                  # whole prompts
    ("bf16", 128, 2, 4, 128, [300], [300], True, 0),
    ("fp16", 32, 1, 4, 64, [513, 129], [513, 129], False, 0),
    ("bf16", 64, 2, 1, 96, [390, 260], [390, 260], True, 50),
    ("fp16", 16, 1, 2, 32, [640, 300], [100, 260], False, 40),
    ("bf16", 256, 1, 16, 128, [600, 270], [64, 1], True, 0),                      # one key/value head for all
    ("fp16", 64, 2, 4, 128, [900, 1, 70, 640, 33], [1, 1, 70, 300, 2], True, 0),  # decoding and prompts
    ("bf16", 32, 2, 4, 128, [300, 20, 500, 64, 700, 33, 90, 10, 1000, 200], [1, 1, 1, 1, 300, 1, 2, 1, 0, 3], True, 0),  # one prompt among decoding
    ("fp16", 32, 1, 71, 64, [300, 50], [1, 2], True, 0),                          # an odd number of heads for one
    ("bf16", 16, 2, 2, 64, [200, 0, 10, 5, 0], [0, 3, 10, 9, 1], True, 0),        # no tokens, no keys, fewer keys than tokens
]


@pytest.mark.parametrize("strides", ["plain", "fused", "heads"])
@pytest.mark.parametrize("dtype,block,hkv,group,dim,lens,news,causal,window", ATTENDS)
def test_attend_matches_its_definition(dtype, block, hkv, group, dim, lens, news, causal, window, strides):
    _attend_case(dtype, block, hkv, group, dim, lens, news, causal, window, strides=strides)


@pytest.mark.parametrize("dim", [64, 128])
def test_items_of_one_row_tile_among_items_of_two(dim):
    """More items than the GPU has multiprocessors, over many key tiles whose block scales differ: the row threads of the
    second tile have nothing to do in some items and must not take the scales of others."""
    lens = [1700, 1300, 2100, 1500, 1900, 1200]
    news = [30, 150, 20, 140, 25, 160]
    _attend_case("fp16", 32, 40, 1, dim, lens, news, True, 0, spread=6)


SHAPES = [([700], [1], 0), ([333, 40], [3, 2], 50), ([300], [260], 0), ([600], [300], 100)]  # lens, new, window


@pytest.mark.parametrize("lens,news,window", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_value_scales_of_any_spread_keep_the_output_precise(dtype, lens, news, window):
    """Blocks of values whose scales differ by up to 2^40, the loud ones hardly attended to."""
    def edit(kc, ks, vc, vs, table, q):
        vs[table[0][0], :] = 2.0 ** 9
        vs[table[0][1], :] = 2.0 ** -30
        kc[table[0][0]] = 0  # score 0
        if len(table[0]) > 3:
            vs[table[0][3], :] = 2.0 ** -126
            vc[table[0][3]] = 0
    _attend_case(dtype, 16, 1, 4, 128, lens, news, True, window, spread=4, edit=edit, scale=1.0)


@pytest.mark.parametrize("lens,news,window", SHAPES)
def test_nothing_that_a_row_does_not_see_reaches_it(lens, news, window):
    """NaN codes, NaN scales' worth of them, in keys and values: past the sequences' ends, beyond the causal limit and
    outside the window; rows that see them are NaN, the others are not."""
    def edit(kc, ks, vc, vs, table, q):
        for s, n in enumerate(lens):
            last = table[s][(n - 1) // 16]
            kc[last][:, (n - 1) % 16 + 1:], vc[last][:, (n - 1) % 16 + 1:] = 0x7F, 0xFF
            used = set(table[s][: -(-n // 16)].tolist())
        spare = [b for b in range(len(kc)) if b not in {int(x) for r, n in zip(table, lens) for x in r[: -(-n // 16)]}]
        kc[spare], vc[spare] = 0x7F, 0x7F
        assert used
        n = lens[0]
        # a value's single column, and a key, near the end: rows before them do not see them
        vc[table[0][(n - 2) // 16]][:, (n - 2) % 16, 5] = 0x7F
        if news[0] > 20:
            kc[table[0][(n - 9) // 16]][:, (n - 9) % 16, 3] = 0xFF
            vc[table[0][(n - 200) // 16]][:, (n - 200) % 16, 17] = 0x7F
    _attend_case("bf16", 16, 2, 4, 64, lens, news, True, window, edit=edit)


@pytest.mark.parametrize("lens,news,window", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_queries_of_any_magnitude(dtype, lens, news, window):
    """Scores of hundreds (one key takes all), queries near the type's least and largest numbers, infinities, NaN."""
    def edit(kc, ks, vc, vs, table, q):
        q[0] *= 300.0
        if len(q) > 2:
            q[1] *= 2.0 ** -20 if dtype == "fp16" else 2.0 ** -100
            q[2, 0, 0] = float("inf")
            q[2, 1, 1] = float("nan")
        if dtype == "bf16" and len(q) > 4:
            q[3] = 0.0
            q[3, 0, :2] = torch.tensor([2.0 ** 20, 2.0 ** -20], device=DEV)
    with np.errstate(all="ignore"):
        _attend_case(dtype, 32, 1, 2, 128, lens, news, True, window, edit=edit)


def test_scale_is_the_callers():
    _attend_case("bf16", 64, 1, 4, 128, [300], [1], True, 0, scale=0.01)
    _attend_case("fp16", 64, 1, 4, 128, [300], [200], True, 0, scale=-0.2)
    _attend_case("fp16", 64, 1, 4, 128, [300], [200], True, 0, scale=0.0)


def test_blocks_past_four_gigabytes_and_slices_of_a_pool():
    """Blocks of one layer of a pool of several, with byte offsets above 2^32."""
    rng = np.random.default_rng(2)
    hkv, block, dim, layers, n = 2, 64, 128, 40, 7000
    pool = torch.empty(2, n, layers, hkv, block, dim, dtype=torch.uint8, device=DEV)
    scales = torch.empty(2, n, layers, hkv, dtype=torch.float32, device=DEV)
    assert pool[0].numel() > 1 << 32
    cache = zc.KVCache(pool[0, :, 3], pool[1, :, 3], scales[0, :, 3], scales[1, :, 3])
    table = np.array([[6999, 1, 6990, 4, 6500]], np.int32)
    lens, news = [300], [300]
    batch, cu = _batch(table, news, lens)
    x = torch.from_numpy(rng.standard_normal((300, hkv, dim))).to(DEV).bfloat16()
    zc.kv_write(cache, batch, x, x)
    k, v = zc.kv_read(cache, batch)
    used = torch.tensor(table[0].tolist(), device=DEV)
    small = zc.KVCache(cache.k[used], cache.v[used], cache.k_scale[used], cache.v_scale[used])
    b2, _ = _batch(np.arange(5, dtype=np.int32).reshape(1, 5), news, lens)
    k2, v2 = zc.kv_read(small, b2)
    q = torch.from_numpy(rng.standard_normal((300, 4, dim))).to(DEV).bfloat16()
    o1, l1 = zc.kv_attend(cache, batch, q)
    o2, l2 = zc.kv_attend(small, b2, q)
    cache.check()
    assert torch.equal(k, k2) and torch.equal(v, v2) and torch.equal(o1, o2) and torch.equal(l1, l2)
    assert (k.float() - x.float()).abs().max() < 0.3


def test_calls_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(5)
    lens, news, hkv, dim = [150, 60], [1, 1], 2, 64
    table, n = _table([l + 40 for l in lens], 16, rng)
    caches = [zc.KVCache.empty(n, hkv, dim, block_tokens=16) for _ in range(3)]
    fill, _ = _batch(table, lens, lens)
    x0 = torch.randn(210, hkv, dim, device=DEV).half()
    for c in caches:
        zc.kv_write(c, fill, x0, x0)
    batches = [_batch(table, news, lens)[0] for _ in caches]
    xs = [torch.randn(2, hkv, dim, device=DEV).half() for _ in range(10)]
    qs = [torch.randn(2, 4, dim, device=DEV).half() for _ in range(10)]
    x, q, out = xs[0].clone(), qs[0].clone(), torch.empty_like(qs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step(c, b, x, q, out, stream=None):
        zc.kv_write(c, b, x, x, stream=stream)
        zc.kv_attend_into(c, b, q, out, stream=stream)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step(caches[2], batches[2], x, q, out)
    torch.cuda.synchronize()
    for c, b in zip(caches[:2], batches):  # the same tokens in all caches
        zc.kv_write(c, b, x, x)
    with torch.cuda.graph(graph):
        step(caches[2], batches[2], x, q, out)
    for i in range(10):
        for b in batches:
            b.lens.add_(1)
        side.wait_stream(torch.cuda.current_stream())
        plain = torch.empty_like(out)
        step(caches[0], batches[0], xs[i], qs[i], plain)
        zc.kv_write(caches[1], batches[1], xs[i], xs[i], stream=side)
        other, _ = zc.kv_attend(caches[1], batches[1], qs[i], stream=side)
        x.copy_(xs[i])
        q.copy_(qs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(plain, out) and torch.equal(plain, other)
    for c in caches:
        c.check()


def test_the_same_call_gives_the_same_bits():
    cache, batch, q, out, lse = _attend_case("bf16", 64, 2, 4, 128, [3000, 100, 900], [1, 1, 1], True, 0)
    for _ in range(20):
        o2, l2 = zc.kv_attend(cache, batch, q)
        assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_device_errors_are_reported_and_nothing_else_is_touched():
    """Entries that the kernels check: blocks outside the pool, lengths beyond the table, counts that fall or are too large."""
    cache = zc.KVCache.empty(4, 1, 32, block_tokens=16)
    x = torch.randn(6, 1, 32, device=DEV).half()
    q = torch.randn(6, 2, 32, device=DEV).half()

    def batch(table, cu, lens, total=6, most=3):
        return zc.KVBatch(*(torch.tensor(t, dtype=torch.int32, device=DEV) for t in (table, cu, lens)), total, most)

    good = batch([[0], [1]], [0, 3, 6], [3, 16])
    for bad, status in ((batch([[4], [1]], [0, 3, 6], [3, 16]), zc.EFORMAT),
                        (batch([[-1], [1]], [0, 3, 6], [3, 16]), zc.EFORMAT),
                        (batch([[0], [1]], [0, 3, 6], [17, 16]), zc.ECAPACITY),
                        (batch([[0], [1]], [0, -1, 6], [3, 16], 6, 6), zc.EFORMAT),
                        (batch([[0], [1]], [0, 1, 6], [3, 16]), zc.EFORMAT),
                        (batch([[0], [1]], [0, 3, 9], [3, 16]), zc.EFORMAT),
                        (batch([[0], [1]], [0, 3, 6], [-2, 16]), zc.EFORMAT)):
        for call in (lambda: zc.kv_write(cache, bad, x, x), lambda: zc.kv_read(cache, bad), lambda: zc.kv_attend(cache, bad, q)):
            call()
            with pytest.raises(zc.ZcError) as e:
                cache.check()
            assert e.value.status & status
    short = batch([[0], [1]], [0, 3, 6], [2, 16])  # three new tokens of a sequence of two
    for call in (lambda: zc.kv_write(cache, short, x, x), lambda: zc.kv_read(cache, short)):
        call()
        with pytest.raises(zc.ZcError) as e:
            cache.check()
        assert e.value.status == zc.EFORMAT
    zc.kv_write(cache, good, x, x)
    cache.check()
    assert not cache.k.view(torch.uint8)[2:].any()


@pytest.mark.parametrize("lens,news", [([900, 300], [1, 1]), ([900, 300], [300, 10])])
def test_a_wait_that_runs_out_is_reported(lens, news):
    """With the test hook the copies of keys and values are never asked for: the kernels give up, return and report it,
    and a call after that, with a workspace of its own, is right."""
    cache, batch, q, out, lse = _attend_case("bf16", 64, 2, 4, 128, lens, news, True, 0)
    again = zc.KVBatch(batch.block_table, batch.cu_tokens, batch.lens, batch.total_tokens, batch.max_tokens)
    zc.lib().zc_kv_set_test_hooks(kv.HOOK_COPY_STALL)
    try:
        zc.kv_attend(cache, again, q)
        with pytest.raises(zc.ZcError) as e:
            cache.check()
    finally:
        zc.lib().zc_kv_set_test_hooks(0)
    assert e.value.status == zc.ETIMEOUT
    o2, l2 = zc.kv_attend(cache, batch, q)
    cache.check()
    assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_arguments_that_the_host_refuses():
    cache = zc.KVCache.empty(4, 2, 32, block_tokens=16)
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    batch = zc.KVBatch(t([[0], [1]]), t([0, 3, 6]), t([3, 16]), 6, 3)
    x = torch.zeros(6, 2, 32, device=DEV).half()
    refused = [
        lambda: zc.kv_write(cache, batch, x[:5], x),
        lambda: zc.kv_write(cache, batch, x, x.float()),
        lambda: zc.kv_write(cache, batch, x.double(), x.double()),
        lambda: zc.kv_write(cache, batch, x.cpu(), x.cpu()),
        lambda: zc.kv_write(cache, batch, x.transpose(1, 2).contiguous().transpose(1, 2), x),
        lambda: zc.kv_write(cache, batch, torch.zeros(6 * 64 + 1, device=DEV).half()[1:].view(6, 2, 32), x),
        lambda: zc.kv_write(cache, batch, torch.zeros(6, 2, 33, device=DEV).half()[:, :, :32], x),
        lambda: zc.kv_attend(cache, batch, torch.zeros(6, 3, 32, device=DEV).half()),
        lambda: zc.kv_attend(cache, batch, torch.zeros(6, 4, 32, device=DEV)),
        lambda: zc.kv_attend(cache, batch, x, scale=float("nan")),
        lambda: zc.kv_attend(cache, batch, x, window=-1),
        lambda: zc.kv_attend(cache, batch, x[0]),
        lambda: zc.kv_read(cache, batch, dtype=torch.float64),
        lambda: zc.kv_attend_into(cache, batch, x, torch.empty_like(x), torch.zeros(6, device=DEV)),
        lambda: zc.KVBatch(t([[0], [1]]), t([0, 3, 6]), t([3, 16]), 7, 3),
        lambda: zc.KVBatch(t([[0], [1]]), t([0, 3, 6]), t([3, 16]), 2, 3),
        lambda: zc.KVBatch(t([[0], [1]]), t([0, 6]), t([3, 16]), 6, 3),
        lambda: zc.KVBatch(t([[0], [1]]).long(), t([0, 3, 6]), t([3, 16]), 6, 3),
        lambda: zc.KVCache(cache.k, cache.v[:3], cache.k_scale, cache.v_scale),
        lambda: zc.KVCache(cache.k, cache.v, cache.k_scale.half(), cache.v_scale),
        lambda: zc.KVCache(cache.k.view(torch.uint8).transpose(1, 2), cache.v.view(torch.uint8).transpose(1, 2), cache.k_scale, cache.v_scale),
        lambda: zc.kv_write(zc.KVCache.empty(2, 1, 24, block_tokens=16), batch, x[:, :1, :24], x[:, :1, :24]),
        lambda: zc.kv_write(zc.KVCache.empty(2, 2, 32, block_tokens=20), batch, x, x),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(zc.ZcError) as e:
            call()
        assert e.value.status == zc.EINVAL, i
    empty = zc.KVBatch(t([[0], [1]]), t([0, 0, 0]), t([3, 16]), 0, 0)
    zc.kv_write(cache, empty, x[:0], x[:0])
    assert zc.kv_read(cache, empty)[0].shape == (0, 2, 32) and zc.kv_attend(cache, empty, x[:0])[0].shape == (0, 2, 32)
    cache.check()


@pytest.mark.parametrize("args", [[], ["--heads", "10", "--kv-heads", "2", "--dim", "80", "--steps", "3"]])
def test_the_example_of_a_layer_in_service(args):
    """Writing, attention, reading back, and a sequence parked without loss in host memory and restored: the outputs of
    a run in which it never left."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_cache.py")
    spec = importlib.util.spec_from_file_location("serve_cache", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.main(args)
    assert r["same"] and r["ratio"] < 1.0 and r["error"] < 2 ** -6


def test_reference_codes_are_torchs():
    """The oracle's table and rounding against torch's own E4M3 conversion."""
    b = torch.arange(256, dtype=torch.uint8)
    v = b.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, VALUES, equal_nan=True)
    x = torch.randn(20000, dtype=torch.float64, generator=torch.Generator().manual_seed(0)).float() * 40
    x = torch.cat([x, x / 4096, torch.tensor([0.0, -0.0, 448.0, 464.0, 2.0 ** -10, 2.0 ** -9 * 1.5])]).clamp(-448, 448)
    assert np.array_equal(VALUES[to_codes(x.double().numpy())], x.to(torch.float8_e4m3fn).double().numpy())
