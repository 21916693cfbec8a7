"""Attention over scores whose own last place is many units wide, in both caches and for few and many rows.

A score of 10^9 has a float32 neighbour 64 away. What the softmax sees are differences of scores: of keys that are alike they
are 0 whatever the scores' size, and a key whose product is the largest by a last place or more has all of the weight. So:

* keys that are alike get one weight: the output is the values' mean, to what the 8- and 4-bit tests allow besides the
  scores' own error (2^-11 for a weight, 2^-23 for each addition, and the 8-bit cache's 2^-25 of the loudest block);
* a key that is above the others by more than a last place is the output, exactly (a value has no more than 6 bits);
* the same of the keys that a row sees, under a causal limit and a window;
* of any keys the output is a mean with some weights: between the least and the largest of a column's values, less and plus
  2^-10 of the largest magnitude for weights that are rounded to half and sums of them that are not (2^-11, and 2^-23 for
  each of 3000 keys), and one rounding to the type. The log sum is within the products' error, 2^-17 of the largest sum of
  magnitudes.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import entropy_coding_gb300 as zc  # noqa: E402

import kv4_reference  # noqa: E402
import kv_reference  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
BLOCK, HKV, GROUP = 16, 2, 4
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}

# (type, magnitude of a query's elements, the caller's scale)
SIZES = [("bf16", 1e7, None), ("bf16", 1e8, None), ("bf16", -1e9, None), ("bf16", 1e30, None), ("fp16", 1.0, 1e9), ("fp16", 6e4, -2.0),
         ("bf16", -3.0, 1e18), ("bf16", 5000.0, 0.125)]
SHAPES = [([3000], [1]), ([700, 90], [3, 1]), ([700], [260]), ([130], [130])]  # lens, new


class _Eight:
    ref, one, more = kv_reference, 0x38, 0x3C  # codes of 1 and of 1.5

    @staticmethod
    def pool(blocks, dim, rng, spread):
        codes = rng.integers(0, 256, (blocks, HKV, BLOCK, dim)).astype(np.uint8)
        codes[codes & 0x7F == 0x7F] = 0x18
        scales = np.exp2(rng.integers(-spread, spread + 1, (blocks, HKV))).astype(np.float32)
        return codes, scales

    @staticmethod
    def cache(kc, ks, vc, vs):
        k, v = (torch.from_numpy(c).to(DEV).view(torch.float8_e4m3fn) for c in (kc, vc))
        return zc.KVCache(k, v, torch.from_numpy(ks).to(DEV), torch.from_numpy(vs).to(DEV))

    @classmethod
    def alike(cls, kc, ks):
        kc[:], ks[:] = cls.one, 1.0

    @classmethod
    def above(cls, kc, ks, block, row):
        kc[block, :, row, 3] = cls.more


class _Four:
    ref = kv4_reference

    @staticmethod
    def pool(blocks, dim, rng, spread):
        codes = rng.integers(0, 256, (blocks, HKV, BLOCK, -(-dim // 32) * 16)).astype(np.uint8)
        return codes, rng.integers(max(1, 120 - 8 * spread), min(0xE2, 120 + 8 * spread) + 1, (blocks, HKV, BLOCK, dim // 16)).astype(np.uint8)

    @staticmethod
    def cache(kc, ks, vc, vs):
        return zc.KV4Cache(*(torch.from_numpy(x).to(DEV) for x in (kc, vc, ks, vs)))

    @staticmethod
    def alike(kc, ks):
        kc[:], ks[:] = 0x22, 120

    @staticmethod
    def above(kc, ks, block, row):
        kc[block, :, row, 1] = 0x32


CACHES = [pytest.param(_Eight, id="8"), pytest.param(_Four, id="4")]


def _case(kind, dim, lens, news, dtype, seed, spread):
    rng = np.random.default_rng(seed)
    width = max(-(-n // BLOCK) for n in lens)
    table = rng.permutation(len(lens) * width).astype(np.int32).reshape(len(lens), width)
    (kc, ks), (vc, vs) = (kind.pool(table.size, dim, rng, s) for s in (2, spread))
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    batch = zc.KVBatch(torch.from_numpy(table).to(DEV), torch.from_numpy(cu).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                       int(cu[-1]), max(news))
    q = torch.from_numpy(rng.standard_normal((int(cu[-1]), HKV * GROUP, dim))).to(DEV).to(DT[dtype])
    return rng, table, (kc, ks, vc, vs), cu, batch, q


def _attend(kind, pool, batch, q, scale):
    cache = kind.cache(*pool)
    out, lse = zc.kv_attend(cache, batch, q, scale=scale, causal=False)
    cache.check()
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def _rows(kind, pool, table, lens, news):
    """(row of the call, head, keys, values [keys, dim] of the row's head) of single rows, and of every 13th of many."""
    kc, ks, vc, vs = pool
    row = 0
    for s, n in enumerate(lens):
        k, v = kind.ref.rows_of(kc, ks, table[s], n), kind.ref.rows_of(vc, vs, table[s], n)
        for i in range(0, news[s], 13 if news[s] > 16 else 1):
            for h in range(HKV * GROUP):
                yield row + i, h, k[h // GROUP], v[h // GROUP]
        row += news[s]


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,news", SHAPES)
@pytest.mark.parametrize("dtype,size,scale", SIZES)
def test_keys_that_are_alike_get_one_weight(kind, dim, lens, news, dtype, size, scale):
    _, table, pool, _, batch, q = _case(kind, dim, lens, news, dtype, 1, 3)
    kind.alike(*pool[:2])
    q.fill_(size)
    out, lse = _attend(kind, pool, batch, q, scale)
    score = float(q.flatten()[0]) * dim * (dim ** -0.5 if scale is None else scale)
    for row, h, k, v in _rows(kind, pool, table, lens, news):
        want, mass = v.mean(0), np.abs(v).mean(0)
        tol = mass * (2.0 ** -11 + len(v) * 2.0 ** -23) + (np.abs(v).max() * 2.0 ** -25 if kind is _Eight else 0.0)
        tol += HALF_STEP[dtype] * (np.abs(want) + tol) + (2.0 ** -25 if dtype == "fp16" else 0.0)
        assert (np.abs(out[row, h] - want) <= tol).all(), (row, h, out[row, h][:4], want[:4])
        z = score + np.log(len(v))
        assert abs(lse[row, h] - z) <= 2.0 ** -17 * abs(score) + 2.0 ** -20 * abs(z), (row, h, lse[row, h], z)


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,news", SHAPES)
@pytest.mark.parametrize("at", [0, 89])
@pytest.mark.parametrize("dtype,size,scale", [s for s in SIZES if s[1] * (s[2] or 1) > 0])
def test_a_key_that_is_above_the_others_is_the_output(kind, dim, lens, news, at, dtype, size, scale):
    _, table, pool, _, batch, q = _case(kind, dim, lens, news, dtype, 2, 3)
    kind.alike(*pool[:2])
    for s in range(len(lens)):
        kind.above(pool[0], pool[1], table[s][at // BLOCK], at % BLOCK)
    q.fill_(size)
    out, _ = _attend(kind, pool, batch, q, scale)
    for row, h, k, v in _rows(kind, pool, table, lens, news):
        assert np.array_equal(out[row, h], v[at]), (row, h, out[row, h][:4], v[at][:4])


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("dim", [64, 112])
@pytest.mark.parametrize("lens,news", SHAPES)
@pytest.mark.parametrize("dtype,size,scale", SIZES)
@pytest.mark.parametrize("spread", [0, 7])
def test_an_output_is_a_mean_of_the_values(kind, dim, lens, news, dtype, size, scale, spread):
    """Random queries and keys; half of the rows with one element far above the others', so that keys differ by few last
    places. Value scales of one size and of many."""
    rng, table, pool, _, batch, q = _case(kind, dim, lens, news, dtype, 3, spread)
    x = q.double() * abs(size)
    x[:, 1::2] = torch.from_numpy(rng.integers(-4, 5, x[:, 1::2].shape)).to(DEV) * (abs(size) * 2.0 ** -20)
    x[:, 1::2, 0] = abs(size)
    q.copy_(x.clamp(-torch.finfo(q.dtype).max, torch.finfo(q.dtype).max))
    out, lse = _attend(kind, pool, batch, q, scale)
    sc = dim ** -0.5 if scale is None else scale
    q64 = q.double().cpu().numpy()
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    for row, h, k, v in _rows(kind, pool, table, lens, news):
        most = np.abs(v).max(0)
        tol = 2.0 ** -10 * most + (2.0 ** -24 if dtype == "fp16" else 0.0)
        low, high = (torch.from_numpy(b).to(DT[dtype]).double().numpy() for b in (v.min(0) - tol, v.max(0) + tol))
        assert ((out[row, h] >= low) & (out[row, h] <= high)).all(), (row, h)
        z = k @ q64[row, h] * sc
        want = z.max() + np.log(np.exp(z - z.max()).sum())
        tol = 2.0 ** -17 * (np.abs(k) @ np.abs(q64[row, h])).max() * abs(sc) + 2.0 ** -20 * abs(want) + 2.0 ** -20
        assert abs(lse[row, h] - want) <= tol, (row, h, lse[row, h], want)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,news", SHAPES)
@pytest.mark.parametrize("size,scale", [(1e7, None), (-1e9, None), (1e30, None), (3.0, 1e18)])
def test_value_scales_far_apart_under_large_scores(dim, lens, news, size, scale):
    """8 bits: blocks of values whose scales lie 2^-90 to 2^90 apart, under keys that are alike: the loudest are the mean, to
    one rounding and what is left of the others."""
    rng, table, pool, _, batch, q = _case(_Eight, dim, lens, news, "bf16", 4, 3)
    kc, ks, vc, vs = pool
    _Eight.alike(kc, ks)
    vs *= np.exp2(rng.choice([-90.0, -20.0, 0.0, 90.0], vs.shape)).astype(np.float32)
    q.fill_(size)
    out, _ = _attend(_Eight, pool, batch, q, scale)
    for row, h, k, v in _rows(_Eight, pool, table, lens, news):
        want, mass = v.mean(0), np.abs(v).mean(0)
        tol = mass * (2.0 ** -11 + len(v) * 2.0 ** -23) + np.abs(v).max() * 2.0 ** -25
        tol += HALF_STEP["bf16"] * (np.abs(want) + tol)
        assert (np.abs(out[row, h] - want) <= tol).all(), (row, h, out[row, h][:4], want[:4])


MASKS = [([3000], [1], True, 500), ([700, 90], [3, 1], True, 60), ([700], [260], True, 0), ([700], [260], True, 100), ([130, 300], [130, 150], True, 17),
         ([500], [200], False, 130)]  # lens, new, causal, window


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,news,causal,window", MASKS)
@pytest.mark.parametrize("dtype,size,scale", [s for s in SIZES if s[1] * (s[2] or 1) > 0])
def test_keys_that_a_row_does_not_see(kind, dim, lens, news, causal, window, dtype, size, scale):
    """Keys of four loudnesses, far apart as scores: a row's output is the mean of the values at the loudest keys that it sees.
    Past a sequence's end there is NaN."""
    rng, table, pool, _, batch, q = _case(kind, dim, lens, news, dtype, 5, 3)
    kc, ks, vc, vs = pool
    kind.alike(kc, ks)
    loud = rng.choice(4, p=[0.7, 0.2, 0.08, 0.02], size=kc.shape[:3])
    if kind is _Eight:
        kc[..., 3] = np.array([0x38, 0x3C, 0x40, 0x44], np.uint8)[loud]
    else:
        kc[..., 1] = np.array([0x22, 0x32, 0x42, 0x52], np.uint8)[loud]
    for s, n in enumerate(lens):
        if n % BLOCK:
            for codes, scales in ((kc, ks), (vc, vs)):
                (codes if kind is _Eight else scales)[table[s][n // BLOCK], :, n % BLOCK:] = 0x7F if kind is _Eight else 0xFF
    q.fill_(size)
    cache = kind.cache(*pool)
    out, _ = zc.kv_attend(cache, batch, q, scale=scale, causal=causal, window=window)
    cache.check()
    out, row = out.double().cpu().numpy(), 0
    for s, n in enumerate(lens):
        v = kind.ref.rows_of(vc, vs, table[s], n)
        at = loud[table[s]].transpose(1, 0, 2).reshape(HKV, -1)[:, :n]
        for i in range(0, news[s], 13 if news[s] > 16 else 1):
            p = n - news[s] + i
            lo, hi = (max(0, p - window + 1) if window else 0), (p + 1 if causal else n)
            for h in range(HKV * GROUP):
                seen = at[h // GROUP, lo:hi]
                values = v[h // GROUP, lo:hi][seen == seen.max()]
                want, mass = values.mean(0), np.abs(values).mean(0)
                tol = mass * (2.0 ** -11 + len(values) * 2.0 ** -23) + (np.abs(v).max() * 2.0 ** -25 if kind is _Eight else 0.0)
                tol += HALF_STEP[dtype] * (np.abs(want) + tol) + (2.0 ** -25 if dtype == "fp16" else 0.0)
                assert (np.abs(out[row + i, h] - want) <= tol).all(), (s, i, h, out[row + i, h][:4], want[:4])
        row += news[s]
