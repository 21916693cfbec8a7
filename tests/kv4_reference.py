"""The 4-bit cache operators and the rotation from their definitions, in 64
bits on the CPU. Shares no code with the package."""
from __future__ import annotations

import math

import numpy as np

CODES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MOST = 0xE2  # the largest scale byte that is written


def scale_of(byte: np.ndarray) -> np.ndarray:
    """5 exponent bits (bias 15) and 3 fraction bits; 0xFF is NaN (0xE3 to 0xFE stand for nothing)."""
    byte = np.asarray(byte).astype(np.int64)
    e, m = byte >> 3, byte & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 18.0), m * 2.0 ** -17)
    return np.where(byte > MOST, math.nan, v)


SCALES = scale_of(np.arange(MOST + 1))  # 0 .. 10240, rising


def nearest(a: np.ndarray, of: np.ndarray) -> np.ndarray:
    """Index of the nearest of the rising numbers `of`; ties go to the even index."""
    hi = np.searchsorted(of, a).clip(1, len(of) - 1)
    up, down = of[hi] - a, a - of[hi - 1]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def quantise(x: np.ndarray):
    """Codes (0 to 15) and scale bytes of x [..., dim] float64."""
    g = x.reshape(*x.shape[:-1], -1, 16)
    finite = np.where(np.isfinite(g), np.abs(g), 0.0)
    # the nearest scale to a / 6 is that whose sixfold is nearest to a: no quotient is rounded
    byte = nearest(finite.max(-1), 6.0 * SCALES).clip(1, MOST)
    a = np.minimum(np.where(np.isnan(g), 0.0, np.abs(g)), 1e300) / SCALES[byte][..., None]
    code = nearest(np.minimum(a, 6.0), CODES) | np.where(np.signbit(g), 8, 0)
    nan = np.isnan(g).any(-1)
    code[nan] = 0
    return code.reshape(x.shape), np.where(nan, 0xFF, byte)


def pack(code: np.ndarray) -> np.ndarray:
    return (code[..., 0::2] | code[..., 1::2] << 4).astype(np.uint8)


def numbers(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Numbers of rows of packed codes [..., row] and scale bytes [..., dim / 16]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])[..., : scales.shape[-1] * 16]
    v = np.where(c >= 8, -CODES[c & 7], CODES[c & 7])
    return v * np.repeat(scale_of(scales), 16, -1)


def places(table, cu, lens, block):
    """(row of the call, block, row of the block) of every token."""
    for s in range(len(lens)):
        n = int(cu[s + 1] - cu[s])
        for i in range(n):
            p = int(lens[s]) - n + i
            yield int(cu[s]) + i, int(table[s][p // block]), p % block


def write(codes, scales, x, table, cu, lens):
    """codes [blocks, heads, tokens, row] and scales, changed in place; x [tokens, heads, dim] float64."""
    code, byte = quantise(x)
    for t, b, r in places(table, cu, lens, codes.shape[2]):
        codes[b, :, r, : x.shape[-1] // 2] = pack(code[t])
        scales[b, :, r] = byte[t]


def rows_of(codes, scales, table_row, total):
    """[heads, total, dim] numbers of a sequence's first `total` positions."""
    at = [int(i) for i in table_row[: -(-total // codes.shape[2])]]
    x = numbers(codes[at], scales[at])
    return x.transpose(1, 0, 2, 3).reshape(codes.shape[1], len(at) * codes.shape[2], x.shape[-1])[:, :total]


def attend(q, kc, ks, vc, vs, table, cu, lens, scale, causal, window):
    """out, lse and, for the tolerances, for each row: sum p |v| (per column), the largest sum of |q k| scale, the
    number of keys, and the largest p times the largest |v|."""
    T, H, D = q.shape
    hkv = kc.shape[1]
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    mass, size, count, unit = np.zeros((T, H, D)), np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    for s in range(len(lens)):
        n, total = int(cu[s + 1] - cu[s]), int(lens[s])
        if not n or not total:
            continue
        k, v = rows_of(kc, ks, table[s], total), rows_of(vc, vs, table[s], total)
        for i in range(n):
            p = total - n + i
            lo, hi = (max(0, p - window + 1) if window else 0), (p + 1 if causal else total)
            if hi <= lo:
                continue
            for h in range(H):
                kh, r = h // (H // hkv), cu[s] + i
                with np.errstate(invalid="ignore", over="ignore"):
                    z = k[kh, lo:hi] @ q[r, h] * scale
                    m = z.max()
                    if m == -np.inf:
                        continue
                    w = np.exp(z - m)
                    out[r, h] = w @ v[kh, lo:hi] / w.sum()
                    lse[r, h] = m + math.log(w.sum()) if w.sum() == w.sum() else math.nan
                    mass[r, h] = w @ np.abs(v[kh, lo:hi]) / w.sum()
                    size[r, h] = (np.abs(k[kh, lo:hi]) @ np.abs(q[r, h])).max() * abs(scale)
                    count[r, h] = hi - lo
                    unit[r, h] = w.max() / w.sum() * np.nan_to_num(np.abs(v[kh, lo:hi])).max()
    return out, lse, mass, size, count, unit


def rotate(x, positions, frequencies, interleaved, weight, eps):
    """x [tokens, heads, dim] float64 rows, normed and turned."""
    y = x.copy()
    with np.errstate(invalid="ignore", over="ignore"):
        if weight is not None:
            y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
        half = len(frequencies)
        if half:
            t = np.exp(1j * np.array([[math.remainder(float(p) * f, 2 * math.pi) for f in frequencies] for p in positions]))[:, None]
            a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
            ya, yb = y[..., a].copy(), y[..., b].copy()
            y[..., a], y[..., b] = ya * t.real - yb * t.imag, yb * t.real + ya * t.imag
    return y
