"""The 8-bit cache operators from their definitions, in 64 bits on the CPU,
one sequence, block and head at a time. Shares no code with the package."""
from __future__ import annotations

import math

import numpy as np


def code_values() -> np.ndarray:
    """The 256 E4M3 values: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F and 0xFF are NaN, no infinities."""
    v = np.empty(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9
        v[c] = math.nan if c & 0x7F == 0x7F else -x if c & 0x80 else x
    return v


VALUES = code_values()
_POS = VALUES[:127]  # 0 .. 448, rising


def to_codes(x: np.ndarray) -> np.ndarray:
    """Nearest E4M3 codes (ties to the even code), saturating; NaN stays NaN (as 0x7F)."""
    a = np.minimum(np.abs(x), 448.0)
    nan = np.isnan(x)
    a = np.where(nan, 0.0, a)
    hi = np.searchsorted(_POS, a).clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _POS[hi] - a, a - _POS[lo]
    c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    c = np.where(np.signbit(x) & ~nan, c | 0x80, c)
    return np.where(nan, 0x7F, c).astype(np.uint8)


def need_scale(a: float) -> float:
    e = -126
    if a > 0:
        e = max(-126, math.frexp(a / 448.0)[1] - 1)
        while 448.0 * 2.0 ** e < a:
            e += 1
    return 2.0 ** e


def ceil_pow2(s: float) -> float:
    e = math.frexp(s)[1] - 1
    return max(2.0 ** (e if 2.0 ** e == s else e + 1), 2.0 ** -126)


def write(codes, scales, x, table, cu, lens):
    """codes [blocks, heads, tokens, dim] uint8 and scales, changed in place; x [tokens, heads, dim] float64."""
    B = codes.shape[2]
    for s in range(len(lens)):
        n = int(cu[s + 1] - cu[s])
        start = int(lens[s]) - n
        for b in range(start // B, -(-int(lens[s]) // B) if n else 0):
            lo, hi = max(start, b * B), min(int(lens[s]), (b + 1) * B)
            at, n0 = int(table[s][b]), lo - b * B
            for h in range(codes.shape[1]):
                rows = x[cu[s] + lo - start: cu[s] + hi - start, h]
                fin = np.abs(rows[np.isfinite(rows)])
                now = need_scale(float(fin.max()) if fin.size else 0.0)
                if n0:
                    old = float(scales[at, h])
                    now = max(now, ceil_pow2(old))
                    if now != old:
                        codes[at, h, :n0] = to_codes(VALUES[codes[at, h, :n0]] * (old / now))
                scales[at, h] = now
                codes[at, h, n0: n0 + hi - lo] = to_codes(rows / now)


def rows_of(codes, scales, table_row, total):
    """[heads, total, dim] numbers of a sequence's first `total` positions."""
    B = codes.shape[2]
    at = [int(i) for i in table_row[: -(-total // B)]]
    x = VALUES[codes[at]] * scales[at].astype(np.float64)[:, :, None, None]
    return x.transpose(1, 0, 2, 3).reshape(codes.shape[1], -1, codes.shape[3])[:, :total]


def attend(q, kc, ks, vc, vs, table, cu, lens, scale, causal, window):
    """out, lse and, for the tolerances, for each row: sum p |v| (per column), the largest sum of |q k| scale, the
    number of keys, and the largest p_j * (value scale)_j."""
    T, H, D = q.shape
    hkv, B = kc.shape[1], kc.shape[2]
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    mass, size, count, unit = np.zeros((T, H, D)), np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    for s in range(len(lens)):
        n, total = int(cu[s + 1] - cu[s]), int(lens[s])
        if not n or not total:
            continue
        k, v = rows_of(kc, ks, table[s], total), rows_of(vc, vs, table[s], total)
        at = [int(i) for i in table[s][: -(-total // B)]]
        by = np.repeat(vs[at].astype(np.float64), B, axis=0)[:total]
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
                    unit[r, h] = (w * by[lo:hi, kh]).max() / w.sum()
    return out, lse, mass, size, count, unit
