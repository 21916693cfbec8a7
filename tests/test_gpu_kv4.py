"""The 4-bit key/value cache on the GPU against its definitions in 64 bits.

Writing and reading back are exact. Attention's tolerance is the 8-bit cache's (test_gpu_kv.py) but for the weights' unit,
which is the largest weight: for a row over n keys with scores whose products sum to at most S in magnitude,

* a score is a float32 sum of head_dim products in at most 16 chained steps of the tensor cores, each within 2^-22 of what it
  adds up: 2^-18 S, and as much again for the scaling and the exponential's 2^-22 relative error;
* a weight is rounded to half (2^-11 relative, or 2^-34 of the row's largest), and at most n of them are added up in float32;
* the output is rounded once to its type: it lies between the roundings of the definition's value less and plus the above.
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

from kv4_reference import attend, numbers, rows_of, write  # noqa: E402

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


def _pool(n_blocks, hkv, block, dim, rng, low=72, high=96):
    """Random codes and scales (2^-6 to 2^-3)."""
    return (rng.integers(0, 256, (n_blocks, hkv, block, -(-dim // 32) * 16), dtype=np.uint8),
            rng.integers(low, high, (n_blocks, hkv, block, dim // 16)).astype(np.uint8))


def _cache(kc, ks, vc, vs):
    return zc.KV4Cache(*(torch.from_numpy(np.array(a)).to(DEV) for a in (kc, vc, ks, vs)))


def _strided(shape, dtype, kind):
    """A tensor of this shape that is contiguous, or a view of a fused projection, or head-major."""
    T, H, D = shape
    if kind == "fused":
        return torch.empty(T, 3 * H * D + 16, dtype=dtype, device=DEV)[:, 16 + H * D: 16 + 2 * H * D].view(T, H, D)
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
    ("fp32", 16, 2, 96, [70, 5], [70, 5], "plain"),
]


@pytest.mark.parametrize("dtype,block,hkv,dim,lens,news,strides", WRITES)
def test_write_gives_the_definitions_codes_and_scales(dtype, block, hkv, dim, lens, news, strides):
    """And touches nothing else: the pool's other rows and the bytes behind a row's last column are compared too."""
    rng = np.random.default_rng(7)
    table, n_blocks = _table(lens, block, rng)
    kc, ks = _pool(n_blocks, hkv, block, dim, rng)
    vc, vs = _pool(n_blocks, hkv, block, dim, rng)
    batch, cu = _batch(table, news, lens)
    cache = _cache(kc, ks, vc, vs)
    T = int(cu[-1])
    xs = []
    for mag in (1.0, 30.0):
        x = rng.standard_normal((T, hkv, dim)) * mag * np.exp2(rng.integers(-8, 8, (T, 1, 1)))
        x[rng.random((T, hkv, dim)) < 0.05] = 0.0
        # halves of few digits, so that there are ties
        few = rng.random((T, hkv, dim)) < 0.5
        x[few] = np.round(x[few] * 4) / 4
        t = _strided((T, hkv, dim), DT[dtype], strides)
        t.copy_(torch.from_numpy(x))
        xs.append(t)
    for _ in range(2):  # writing the same tokens again changes nothing
        zc.kv_write(cache, batch, *xs)
    cache.check()
    for (c, s), x, got_c, got_s in (((kc, ks), xs[0], cache.k, cache.k_scale), ((vc, vs), xs[1], cache.v, cache.v_scale)):
        write(c, s, x.double().cpu().numpy(), table, cu, lens)
        assert np.array_equal(got_s.cpu().numpy(), s)
        assert np.array_equal(got_c.cpu().numpy(), c)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_write_of_every_border_and_of_extremes(dtype):
    """Numbers on the borders of two codes and of two scales and their neighbours in the type, under every scale; zeros,
    infinities, NaN, the type's ends."""
    t = DT[dtype]
    rows = []
    scale = (torch.arange(0xE3, dtype=torch.int16) << 7).view(torch.float16).double()
    info = torch.finfo(t)
    for b in range(1, 0xE3):
        s = float(scale[b])
        mid = [m * s for m in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)]
        base = torch.tensor([6.0 * s] + mid + [-m for m in mid] + [0.0], dtype=torch.float64)
        if base.abs().max() > info.max:
            continue
        up = (6.0 * (scale[min(b + 1, 0xE2)] + scale[b]) / 2).item()  # the border of two scales
        for x in (base, base * (1 + info.eps), base * (1 - info.eps / 2), torch.cat([torch.tensor([up], dtype=torch.float64), base[1:]])):
            rows.append(x)
    big, tiny = float(info.max), float(info.tiny)
    for x in ([0.0] * 16, [-0.0] * 16, [big, -big] + [1.0] * 14, [tiny, -tiny] + [0.0] * 14, [float("inf"), float("-inf"), 1.0] + [0.5] * 13,
              [float("inf")] + [0.0] * 15, [float("nan"), 2.0] + [0.25] * 14, [float("nan")] * 16, [2.0 ** -20] * 16, [12288.0 * 5] * 16):
        rows.append(torch.tensor(x, dtype=torch.float64))
    n = len(rows)
    x = torch.stack(rows).to(t).to(DEV).view(n, 1, 16)
    table = np.arange(-(-n // 16), dtype=np.int32)[None]
    batch, cu = _batch(table, [n], [n])
    cache = zc.KV4Cache.empty(table.size, 1, 16, block_tokens=16)
    zc.kv_write(cache, batch, x, -x)
    cache.check()
    for got_c, got_s, y in ((cache.k, cache.k_scale, x), (cache.v, cache.v_scale, -x)):
        c, s = np.zeros((table.size, 1, 16, 16), np.uint8), np.zeros((table.size, 1, 16, 1), np.uint8)
        write(c, s, y.double().cpu().numpy(), table, cu, [n])
        assert np.array_equal(got_s.cpu().numpy(), s) and np.array_equal(got_c.cpu().numpy(), c)


@pytest.mark.parametrize("dtype,block,hkv,dim,lens,news,strides", WRITES)
def test_read_gives_the_numbers_that_the_codes_stand_for(dtype, block, hkv, dim, lens, news, strides):
    rng = np.random.default_rng(8)
    table, n_blocks = _table(lens, block, rng)
    kc, ks = _pool(n_blocks, hkv, block, dim, rng, 0, 0xE3)
    vc, vs = _pool(n_blocks, hkv, block, dim, rng, 0, 0xE3)
    ks[rng.random(ks.shape) < 0.1] = 0xFF
    batch, cu = _batch(table, news, lens)
    cache = _cache(kc, ks, vc, vs)
    T = int(cu[-1])
    k, v = (_strided((T, hkv, dim), DT[dtype], strides) for _ in range(2))
    zc.kv_read_into(cache, batch, k, v)
    cache.check()
    for got, c, s in ((k, kc, ks), (v, vc, vs)):
        want = np.concatenate([rows_of(c, s, table[i], n)[:, n - m:].transpose(1, 0, 2) for i, (n, m) in enumerate(zip(lens, news))])
        assert np.array_equal(got.double().cpu().numpy(), want, equal_nan=True)
    k2, v2 = zc.kv_read(cache, batch, dtype=DT[dtype])
    assert torch.equal(k2.nan_to_num(7.0), k.nan_to_num(7.0)) and torch.equal(v2, v)


def test_rows_that_are_written_again_are_the_same_as_written_once():
    """What a read gives back is written with the same codes and scales: the cache's numbers are its own."""
    rng = np.random.default_rng(9)
    table, n_blocks = _table([200], 32, rng)
    batch, _ = _batch(table, [200], [200])
    a, b = (zc.KV4Cache.empty(n_blocks, 2, 128, 32) for _ in range(2))
    x = torch.randn(200, 2, 128, device=DEV)
    zc.kv_write(a, batch, x, x * 100)
    k, v = zc.kv_read(a, batch)
    zc.kv_write(b, batch, k, v)
    k2, v2 = zc.kv_read(b, batch, dtype=torch.float32)
    assert torch.equal(k.float(), k2) and torch.equal(v.float(), v2)
    assert ((k.float() - x).abs() <= x.abs().view(200, 2, 8, 16).amax(-1).repeat_interleave(16, -1) * 0.19).all()  # half the step of 4 to 6, of 6 less 1/16


def _attend_case(dtype, block, hkv, group, dim, lens, news, causal, window, scale=None, seed=11, strides="plain", edit=None):
    rng = np.random.default_rng(seed)
    table, n_blocks = _table(lens, block, rng)
    kc, ks = _pool(n_blocks, hkv, block, dim, rng, 80, 104)
    vc, vs = _pool(n_blocks, hkv, block, dim, rng)
    batch, cu = _batch(table, news, lens)
    T, H = int(cu[-1]), hkv * group
    q = _strided((T, H, dim), DT[dtype], strides)
    q.copy_(torch.from_numpy(rng.standard_normal((T, H, dim))))
    if edit:
        edit(kc, ks, vc, vs, table, q)
    cache = _cache(kc, ks, vc, vs)
    out = _strided((T, H, dim), DT[dtype], strides)
    out.fill_(123.0)
    lse = torch.full((T, H), 5.0, device=DEV)
    zc.kv_attend_into(cache, batch, q, out, lse, scale, causal, window)
    cache.check()
    sc = dim ** -0.5 if scale is None else scale
    _compare(out, lse, attend(q.double().cpu().numpy(), kc, ks, vc, vs, table, cu, lens, sc, causal, window), dtype)
    return cache, batch, q, out, lse


def _compare(out, lse, want, dtype):
    o, z, mass, size, count, unit = want
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(o)) and np.array_equal(np.isnan(got_lse), np.isnan(z))
    assert np.array_equal(np.isneginf(got_lse), np.isneginf(z))
    score = 2.0 ** -17 * size + 2.0 ** -21
    rel = 2.0 ** -11 + 2 * score + count * 2.0 ** -23
    tol = mass * rel[..., None] + (count * unit * 2.0 ** -34)[..., None]
    fine = np.isfinite(o)
    low, high = (torch.from_numpy(o + d).to(DT[dtype]).double().numpy() for d in (-tol, tol))
    bad = fine & ((got < low) | (got > high))
    assert not bad.any(), (got[bad][:8], low[bad][:8], high[bad][:8])
    fine = np.isfinite(z)
    tol = (score + count * 2.0 ** -23)[fine] + 2.0 ** -21 * np.abs(z[fine])
    assert (np.abs(got_lse[fine] - z[fine]) <= tol).all(), (np.abs(got_lse[fine] - z[fine]) / tol).max()
    assert (got[np.isneginf(z)] == 0).all()


ATTENDS = [  # dtype, block, kv heads, group, dim, lens, new, causal, window
    ("bf16", 64, 2, 4, 128, [1, 2, 31, 32, 33, 63, 64, 65, 1000], [1] * 9, True, 0),  # single tokens
    ("fp16", 16, 1, 1, 64, [1, 15, 16, 17, 33, 700], [1] * 6, True, 0),           # one head
    ("bf16", 32, 2, 8, 128, [400, 37, 2000], [1, 1, 1], True, 64),                # a window inside
    ("fp16", 16, 2, 7, 112, [300, 50], [1, 1], False, 0),
    ("bf16", 48, 3, 5, 80, [200, 33, 100], [4, 2, 7], True, 0),                   # drafted tokens
    ("fp16", 64, 2, 8, 128, [500, 900, 8], [8, 3, 8], True, 100),
    ("fp16", 80, 1, 2, 48, [500, 90], [3, 1], True, 33),
    ("bf16", 16, 1, 3, 16, [77], [77], True, 0),                                  # whole prompts
    ("bf16", 128, 2, 4, 128, [300], [300], True, 0),
    ("fp16", 32, 1, 4, 64, [513, 129], [513, 129], False, 0),
    ("bf16", 64, 2, 1, 96, [390, 260], [390, 260], True, 50),
    ("fp16", 16, 1, 2, 32, [640, 300], [100, 260], False, 40),
    ("bf16", 256, 1, 16, 128, [600, 270], [64, 1], True, 0),                      # one key/value head for all
    ("fp16", 112, 2, 3, 80, [330, 225], [200, 30], True, 0),
    ("fp16", 64, 2, 4, 128, [900, 1, 70, 640, 33], [1, 1, 70, 300, 2], True, 0),  # decoding and prompts
    ("bf16", 32, 2, 4, 128, [300, 20, 500, 64, 700, 33, 90, 10, 1000, 200], [1, 1, 1, 1, 300, 1, 2, 1, 0, 3], True, 0),  # one prompt among decoding
    ("fp16", 32, 1, 71, 64, [300, 50], [1, 2], True, 0),                          # an odd number of heads for one
    ("bf16", 16, 2, 2, 64, [200, 0, 10, 5, 0], [0, 3, 10, 9, 1], True, 0),        # no tokens, no keys, fewer keys than tokens
    ("fp16", 16, 1, 1, 128, [200, 0, 10, 5, 3], [0, 3, 10, 9, 1], True, 7),
]


@pytest.mark.parametrize("strides", ["plain", "fused", "heads"])
@pytest.mark.parametrize("dtype,block,hkv,group,dim,lens,news,causal,window", ATTENDS)
def test_attend_matches_its_definition(dtype, block, hkv, group, dim, lens, news, causal, window, strides):
    _attend_case(dtype, block, hkv, group, dim, lens, news, causal, window, strides=strides)


@pytest.mark.parametrize("dim", [64, 128])
def test_items_of_one_row_tile_among_items_of_two(dim):
    lens, news = [1700, 1300, 2100, 1500, 1900, 1200], [30, 150, 20, 140, 25, 160]
    _attend_case("fp16", 32, 20, 1, dim, lens, news, True, 0)


SHAPES = [([700], [1], 0), ([333, 40], [3, 2], 50), ([300], [260], 0), ([600], [300], 100)]  # lens, new, window


@pytest.mark.parametrize("lens,news,window", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_scales_of_any_spread(dtype, lens, news, window):
    """Groups of values whose scales lie at both ends of what a byte holds, and keys with scales of zero and the least."""
    def edit(kc, ks, vc, vs, table, q):
        vs[table[0][0]] = 1
        vs[table[0][1], :, ::2, 0] = 150
        ks[table[0][0]] = 0
        ks[table[0][1], :, :, 1] = 1
    _attend_case(dtype, 16, 1, 4, 128, lens, news, True, window, edit=edit, scale=0.2)


@pytest.mark.parametrize("dim", [64, 80, 128])
@pytest.mark.parametrize("lens,news,window", SHAPES)
def test_nothing_that_a_row_does_not_see_reaches_it(lens, news, window, dim):
    """Scales of NaN, and bytes that no scale has, in keys and values: past the sequences' ends, beyond the causal limit and
    outside the window; rows that see NaN are NaN in its columns, the others are not."""
    rng = np.random.default_rng(1)

    def edit(kc, ks, vc, vs, table, q):
        for s, n in enumerate(lens):
            last = table[s][(n - 1) // 16]
            for x in (ks, vs):
                x[last][:, (n - 1) % 16 + 1:] = rng.integers(0xE3, 0x100, x[last][:, (n - 1) % 16 + 1:].shape)
        spare = [b for b in range(len(kc)) if b not in {int(x) for r, n in zip(table, lens) for x in r[: -(-n // 16)]}]
        ks[spare], vs[spare] = 0xFF, 0xF9
        n = lens[0]
        # a value's single group, and a key's, near the end: rows before them do not see them
        vs[table[0][(n - 2) // 16]][:, (n - 2) % 16, 2] = 0xFF
        if news[0] > 20:
            ks[table[0][(n - 9) // 16]][:, (n - 9) % 16, 1] = 0xFF
            vs[table[0][(n - 200) // 16]][:, (n - 200) % 16, dim // 16 - 1] = 0xFF
    _attend_case("bf16", 16, 2, 4, dim, lens, news, True, window, edit=edit)


@pytest.mark.parametrize("lens,news", [([700], [1]), ([300], [260])])
def test_values_of_nan_in_the_midst_of_keys_that_all_rows_see(lens, news):
    def edit(kc, ks, vc, vs, table, q):
        vs[table[0][1]][:, 3, 1] = 0xFF
    _attend_case("fp16", 16, 1, 4, 64, lens, news, False, 0, edit=edit)


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
            # (an infinite query times a code of 0 is NaN, times others an infinity: the definition says which)
    with np.errstate(all="ignore"):
        _attend_case(dtype, 32, 1, 2, 128, lens, news, True, window, edit=edit)


@pytest.mark.parametrize("new", [1, 40])
def test_one_key_takes_nearly_all_of_the_weight_and_has_no_value(new):
    """The others' weights, 2^-24 of the largest together with a value of their own, are the output."""
    keys, dim = 8192, 64
    def edit(kc, ks, vc, vs, table, q):
        kc[:], ks[:], vc[:], vs[:] = 0, 120, 0x22, 120  # keys 0, values 1
        ks[table[0][0]] = 120
        kc[table[0][0], :, 5] = 0x22                    # key 5 is all ones
        vc[table[0][0], :, 5] = 0
        q.fill_(1.0)
    z = float(np.log(8191 * 99.0)) / dim                # the key has 0.99 of the weight
    _attend_case("fp16", 32, 1, 4, dim, [keys], [new], False, 0, edit=edit, scale=z)


@pytest.mark.parametrize("scale", [0.01, -0.2, 0.0, -0.0])
@pytest.mark.parametrize("dtype,new", [("bf16", 1), ("fp16", 3), ("bf16", 30), ("fp16", 200)])
def test_scale_is_the_callers(dtype, new, scale):
    _attend_case(dtype, 64, 1, 4, 128, [300], [new], True, 0, scale=scale)


@pytest.mark.parametrize("group,news", [(4, [20, 31, 5]), (8, [3, 16, 9]), (1, [100, 17, 128])])
@pytest.mark.parametrize("dim,window", [(64, 0), (128, 0), (80, 700), (128, 130)])
def test_rows_of_one_tile_over_one_to_many_key_tiles(dim, window, group, news):
    """Items of one row tile over one, two, three and many key tiles, and pieces that begin and end inside items."""
    for lens in ([128, 129, 256], [257, 300, 384], [385, 513, 1100], [3000, 2600, 150]):
        _attend_case("fp16", 32, 3, group, dim, [max(a, b) for a, b in zip(lens, news)], news, True, window)
        _attend_case("bf16", 16, 1, group, dim, [max(a, b) for a, b in zip(lens, news)], news, False, window)


def test_blocks_past_four_gigabytes_and_slices_of_a_pool():
    """Blocks of one layer of a pool of several, with byte offsets above 2^32 for codes and for scales."""
    rng = np.random.default_rng(2)
    hkv, block, dim, layers, n = 2, 64, 128, 40, 14000
    pool = torch.empty(2, n, layers, hkv, block, dim // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(2, n, layers * 8, hkv, block, dim // 16, dtype=torch.uint8, device=DEV)
    assert pool[0].numel() > 1 << 32 and scales[0].numel() > 1 << 32
    cache = zc.KV4Cache(pool[0, :, 3], pool[1, :, 3], scales[0, :, 3], scales[1, :, 3])
    table = np.array([[13999, 1, 13990, 4, 13500]], np.int32)
    lens, news = [300], [300]
    batch, cu = _batch(table, news, lens)
    x = torch.from_numpy(rng.standard_normal((300, hkv, dim))).to(DEV).bfloat16()
    zc.kv_write(cache, batch, x, x)
    k, v = zc.kv_read(cache, batch)
    used = torch.tensor(table[0].tolist(), device=DEV)
    small = zc.KV4Cache(cache.k[used], cache.v[used], cache.k_scale[used], cache.v_scale[used])
    b2, _ = _batch(np.arange(5, dtype=np.int32).reshape(1, 5), news, lens)
    k2, v2 = zc.kv_read(small, b2)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    for m in (300, 2):
        q = torch.from_numpy(rng.standard_normal((m, 4, dim))).to(DEV).bfloat16()
        (o1, l1), (o2, l2) = (zc.kv_attend(c, _batch(t, [m], lens)[0], q) for c, t in ((cache, table), (small, np.arange(5, dtype=np.int32)[None])))
        assert torch.equal(o1, o2) and torch.equal(l1, l2)
    cache.check()
    small.check()


def test_the_same_call_gives_the_same_bits():
    for lens, news in (([3000, 100, 900], [1, 1, 1]), ([900, 500], [300, 17])):
        cache, batch, q, out, lse = _attend_case("bf16", 64, 2, 4, 128, lens, news, True, 0)
        for _ in range(20):
            o2, l2 = zc.kv_attend(cache, batch, q)
            assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_device_errors_are_reported_and_nothing_else_is_touched():
    """Entries that the kernels check: blocks outside the pool, lengths beyond the table, counts that fall or are too large."""
    cache = zc.KV4Cache.empty(4, 1, 32, block_tokens=16)
    x = torch.randn(6, 1, 32, device=DEV).half()
    q = torch.randn(6, 2, 32, device=DEV).half()

    def batch(table, cu, lens, total=6, most=3):
        return zc.KVBatch(*(torch.tensor(t, dtype=torch.int32, device=DEV) for t in (table, cu, lens)), total, most)

    good = batch([[0], [1]], [0, 3, 6], [3, 16])
    calls = (lambda b: zc.kv_write(cache, b, x, x), lambda b: zc.kv_read(cache, b), lambda b: zc.kv_attend(cache, b, q))
    for bad, status in ((batch([[4], [1]], [0, 3, 6], [3, 16]), zc.EFORMAT),
                        (batch([[-1], [1]], [0, 3, 6], [3, 16]), zc.EFORMAT),
                        (batch([[0], [1]], [0, 3, 6], [17, 16]), zc.ECAPACITY),
                        (batch([[0], [1]], [0, -1, 6], [3, 16], 6, 6), zc.EFORMAT),
                        (batch([[0], [1]], [0, 1, 6], [3, 16]), zc.EFORMAT),
                        (batch([[0], [1]], [0, 3, 9], [3, 16]), zc.EFORMAT),
                        (batch([[0], [1]], [0, 3, 6], [-2, 16]), zc.EFORMAT)):
        for call in calls:
            call(bad)
            with pytest.raises(zc.ZcError) as e:
                cache.check()
            assert e.value.status & status
    short = batch([[0], [1]], [0, 3, 6], [2, 16])  # three new tokens of a sequence of two
    for call in calls[:2]:
        call(short)
        with pytest.raises(zc.ZcError) as e:
            cache.check()
        assert e.value.status == zc.EFORMAT
    zc.kv_write(cache, good, x, x)
    cache.check()
    assert not cache.k[2:].any() and not cache.k_scale[2:].any()


def test_rows_of_tokens_that_belong_to_no_sequence_stay_as_they_were():
    cache = zc.KV4Cache.empty(4, 1, 32, block_tokens=16)
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    batch = zc.KVBatch(t([[0], [1]]), t([1, 2, 4]), t([3, 16]), 7, 4)
    x = torch.randn(7, 1, 32, device=DEV).half()
    zc.kv_write(cache, batch, x, x)
    k, v, o = (torch.full_like(x, 9.0) for _ in range(3))
    zc.kv_read_into(cache, batch, k, v)
    zc.kv_attend_into(cache, batch, x, o)
    cache.check()
    for y in (k, v, o):
        assert (y[[0, 4, 5, 6]] == 9.0).all() and not (y[1:4] == 9.0).any()


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
    for b in (batch, again):
        o2, l2 = zc.kv_attend(cache, b, q)
        cache.check()
        assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_arguments_that_the_host_refuses():
    cache = zc.KV4Cache.empty(4, 2, 32, block_tokens=16)
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    batch = zc.KVBatch(t([[0], [1]]), t([0, 3, 6]), t([3, 16]), 6, 3)
    x = torch.zeros(6, 2, 32, device=DEV).half()
    pool = torch.zeros(4 * 512 + 64, dtype=torch.uint8, device=DEV)
    for i, call in enumerate([
            lambda: zc.kv_write(cache, batch, x[:5], x), lambda: zc.kv_write(cache, batch, x, x.float()),
            lambda: zc.kv_write(cache, batch, x.double(), x.double()), lambda: zc.kv_write(cache, batch, x.cpu(), x.cpu()),
            lambda: zc.kv_write(cache, batch, torch.zeros(6 * 64 + 1, device=DEV).half()[1:].view(6, 2, 32), x),
            lambda: zc.kv_attend(cache, batch, torch.zeros(6, 3, 32, device=DEV).half()),
            lambda: zc.kv_attend(cache, batch, torch.zeros(6, 4, 32, device=DEV)),
            lambda: zc.kv_attend(cache, batch, x, scale=float("nan")), lambda: zc.kv_attend(cache, batch, x, window=-1),
            lambda: zc.kv_read(cache, batch, dtype=torch.float64),
            lambda: zc.KV4Cache(cache.k, cache.v[:3], cache.k_scale, cache.v_scale),
            lambda: zc.KV4Cache(cache.k, cache.v, cache.k_scale, cache.v_scale.cpu()),
            lambda: zc.kv_write(zc.KV4Cache.empty(2, 2, 32, block_tokens=20), batch, x, x),
            # codes that begin beside a multiple of 16 bytes, blocks whose distance is none
            lambda: zc.kv_write(zc.KV4Cache(*[pool[8:2056].view(4, 2, 16, 16)] * 2, cache.k_scale, cache.v_scale), batch, x, x),
            lambda: zc.kv_write(zc.KV4Cache(*[pool.as_strided((4, 2, 16, 16), (520, 256, 16, 1))] * 2, cache.k_scale, cache.v_scale), batch, x, x)]):
        with pytest.raises(zc.ZcError) as e:
            call()
        assert e.value.status == zc.EINVAL, i
    empty = zc.KVBatch(t([[0], [1]]), t([0, 0, 0]), t([3, 16]), 0, 0)
    zc.kv_write(cache, empty, x[:0], x[:0])
    assert zc.kv_read(cache, empty)[0].shape == (0, 2, 32) and zc.kv_attend(cache, empty, x[:0])[0].shape == (0, 2, 32)
    cache.check()


@pytest.mark.parametrize("kind", [zc.KVCache, zc.KV4Cache])
@pytest.mark.parametrize("dim", [128, 80])
def test_a_layer_in_service(kind, dim):
    """Rotation, writing, attention and reading back, prompts and then tokens, eagerly, on another stream and as a graph that
    is replayed with new lengths: the same bits, and attention over what the cache holds."""
    g = torch.Generator(device=DEV).manual_seed(0)
    hkv, heads, block, lens, steps = 2, 8, 16, [150, 60], 6
    rng = np.random.default_rng(5)
    table, n = _table([l + steps for l in lens], block, rng)
    rotation = zc.KVRotation([10000.0 ** (-2 * i / dim) for i in range(dim // 2)])
    w = 1.0 + 0.1 * torch.randn(dim, generator=g, device=DEV)
    caches = [kind.empty(n, hkv, dim, block) for _ in range(3)]
    prompts, _ = _batch(table, lens, lens)
    batches = [_batch(table, [1, 1], lens)[0] for _ in caches]

    def tokens(T):
        return torch.randn(T, heads + 2 * hkv, dim, generator=g, device=DEV).bfloat16()

    def step(cache, batch, x, stream=None):
        q, k = zc.kv_rotate(cache, batch, rotation, x[:, :heads], x[:, heads: heads + hkv], w, w, stream=stream)
        zc.kv_write(cache, batch, k, x[:, heads + hkv:], stream=stream)
        return q, zc.kv_attend(cache, batch, q, stream=stream)

    x = tokens(sum(lens))
    first = [step(c, prompts, x) for c in caches]
    assert all(torch.equal(a[1][0], first[0][1][0]) for a in first)
    side, graph, x = torch.cuda.Stream(), torch.cuda.CUDAGraph(), tokens(2)
    for b in batches:
        b.lens.add_(1)
    side.wait_stream(torch.cuda.current_stream())
    for c, b in zip(caches, batches):
        step(c, b, x)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        _, captured = step(caches[2], batches[2], x)
    for _ in range(steps - 1):
        for b in batches:
            b.lens.add_(1)
        x.copy_(tokens(2))
        side.wait_stream(torch.cuda.current_stream())
        q, plain = step(caches[0], batches[0], x)
        _, other = step(caches[1], batches[1], x, stream=side)
        graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(plain[i], captured[i]) and torch.equal(plain[i], other[i])
    for c in caches:
        c.check()
    # the last step against float64 over the numbers that the cache holds
    now = [n + steps for n in lens]
    whole, _ = _batch(table, now, now)
    k, v = (t.double().split(now) for t in zc.kv_read(caches[0], whole, dtype=torch.float32))
    for s in range(2):
        z = torch.einsum("hgd,jhd->hgj", q[s].double().view(hkv, heads // hkv, dim), k[s]) * dim ** -0.5
        want = torch.einsum("hgj,jhd->hgd", z.softmax(-1), v[s]).reshape(heads, dim)
        assert torch.allclose(plain[0][s].double(), want, rtol=2 ** -8, atol=2 ** -9)
        assert torch.allclose(plain[1][s].double(), torch.logsumexp(z, -1).reshape(heads), rtol=0, atol=1e-4)


def test_both_caches_with_one_batch():
    """A batch keeps a workspace for each kind of cache."""
    rng = np.random.default_rng(6)
    table, n = _table([300, 40], 16, rng)
    batch, _ = _batch(table, [1, 1], [300, 40])
    fill, _ = _batch(table, [300, 40], [300, 40])
    x, q = torch.randn(340, 2, 64, device=DEV).half(), torch.randn(2, 8, 64, device=DEV).half()
    outs = []
    for _ in range(2):
        for kind in (zc.KVCache, zc.KV4Cache):
            c = kind.empty(n, 2, 64, 16)
            zc.kv_write(c, fill, x, x)
            outs.append(zc.kv_attend(c, batch, q)[0])
            c.check()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3]) and not torch.equal(outs[0], outs[1])
    assert (outs[0] - outs[1]).abs().max() < 0.5


@pytest.mark.parametrize("new", [1, 40])
def test_a_first_call_in_a_capture_among_other_kernels(new):
    """The graph zeroes the workspace itself; its calls follow kernels and copies of others, and one another."""
    rng = np.random.default_rng(7)
    lens = [300, 90]
    table, n = _table([l + 8 for l in lens], 32, rng)
    caches = [zc.KV4Cache.empty(n, 2, 64, 32) for _ in range(2)]
    fill, _ = _batch(table, lens, lens)
    x = torch.randn(390, 2, 64, device=DEV).bfloat16()
    for c in caches:
        zc.kv_write(c, fill, x, x)
    rotation = zc.KVRotation([0.5 ** i for i in range(32)])
    batches = [_batch(table, [new, new], lens)[0] for _ in caches]
    qs = torch.randn(2 * new, 8, 64, device=DEV).bfloat16()
    ks = torch.randn(2 * new, 2, 64, device=DEV).bfloat16()

    def step(c, b, q, k):
        b.lens.add_(1)
        q, k = zc.kv_rotate(c, b, rotation, q * 1.0, k + 0.0)
        zc.kv_write(c, b, k, k)
        out, lse = zc.kv_attend(c, b, q)
        return out * 2.0, lse, zc.kv_read(c, b)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = step(caches[1], batches[1], qs, ks)
    for _ in range(6):
        qs.copy_(torch.randn(2 * new, 8, 64, device=DEV))
        ks.copy_(torch.randn(2 * new, 2, 64, device=DEV))
        want = step(caches[0], batches[0], qs, ks)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((want[0], want[1], *want[2]), (captured[0], captured[1], *captured[2])):
            assert torch.equal(a, b)
    for c in caches:
        c.check()
    assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v_scale, caches[1].v_scale)


def test_calls_one_after_another_see_what_the_last_has_written():
    """Kernels that begin before the one in front of them has ended: each step reads what the last one wrote, many in a row."""
    rng = np.random.default_rng(8)
    table, n = _table([4000], 64, rng)
    cache = zc.KV4Cache.empty(n, 4, 128, 64)
    rotation = zc.KVRotation([1.0 / (i + 1) for i in range(64)])
    whole, _ = _batch(table, [4000], [4000])
    x = torch.randn(4000, 4, 128, device=DEV).half()
    results = []
    for _ in range(3):
        a = x
        for i in range(30):  # each pass through the cache and the rotation is the next one's input
            zc.kv_write(cache, whole, a, a)
            k, v = zc.kv_read(cache, whole, dtype=torch.float16)
            _, a = zc.kv_rotate(cache, whole, rotation, v, k)
        results.append(a)
    # the same with everything waited for
    a = x
    for i in range(30):
        zc.kv_write(cache, whole, a, a)
        torch.cuda.synchronize()
        k, v = zc.kv_read(cache, whole, dtype=torch.float16)
        torch.cuda.synchronize()
        _, a = zc.kv_rotate(cache, whole, rotation, v, k)
        torch.cuda.synchronize()
    cache.check()
    assert torch.isfinite(a).all() and all(torch.equal(a, r) for r in results)


@pytest.mark.parametrize("args", [["--bits", "4"], ["--bits", "4", "--rotate"], ["--rotate", "--heads", "10", "--kv-heads", "2", "--dim", "80", "--steps", "3"]])
def test_the_example_of_a_layer_in_service(args):
    """In 4 bits, and with norms and rotation: the outputs of a run in which the parked sequence never left."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_cache.py")
    spec = importlib.util.spec_from_file_location("serve_cache", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.main(args)
    assert r["same"] and r["ratio"] < 1.05 and r["error"] < 2 ** -6


@pytest.mark.parametrize("seqs", [1500, 5000])
def test_tokens_of_thousands_of_sequences(seqs):
    """More sequences than a CTA looks at one after another, some without new tokens: writing, reading and rotation."""
    rng = np.random.default_rng(10)
    news = rng.integers(0, 3, seqs)
    lens = news + rng.integers(0, 20, seqs)
    table = rng.permutation(seqs * 2).reshape(seqs, 2).astype(np.int32)
    kc, ks = _pool(seqs * 2, 1, 16, 32, rng)
    vc, vs = _pool(seqs * 2, 1, 16, 32, rng)
    batch, cu = _batch(table, news, lens)
    cache = _cache(kc, ks, vc, vs)
    T = int(cu[-1])
    x = torch.from_numpy(rng.standard_normal((T, 1, 32))).to(DEV).bfloat16()
    zc.kv_write(cache, batch, x, -x)
    cache.check()
    for c, s, y, got_c, got_s in ((kc, ks, x, cache.k, cache.k_scale), (vc, vs, -x, cache.v, cache.v_scale)):
        write(c, s, y.double().cpu().numpy(), table, cu, lens)
        assert np.array_equal(got_s.cpu().numpy(), s) and np.array_equal(got_c.cpu().numpy(), c)
    k, _ = zc.kv_read(cache, batch, dtype=torch.float32)
    want = np.concatenate([rows_of(kc, ks, table[i], n)[:, n - m:].transpose(1, 0, 2) for i, (n, m) in enumerate(zip(lens, news))])
    assert np.array_equal(k.double().cpu().numpy(), want)
    q, _ = zc.kv_rotate(cache, batch, zc.KVRotation([0.3 ** i for i in range(16)]), x.float(), x.float())
    cache.check()
    p = torch.tensor([n - m + i for n, m in zip(lens, news) for i in range(m)], device=DEV, dtype=torch.float64)
    t = p[:, None, None] * torch.tensor([0.3 ** i for i in range(16)], device=DEV, dtype=torch.float64)
    a, b = x.double().split(16, -1)
    want = torch.cat([a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()], -1)
    assert torch.allclose(q.double(), want, rtol=0, atol=2 ** -18)
