"""Sines and cosines of the rotation, alone: pairs (1, 0) in float32 become (cos t, sin t).

t is the position times the frequency. Its fraction of a turn is right to half a unit of 2^-64 for each position; what is left
of it beside the nearest quarter of a turn is rounded once to float32, 2^-24 of itself, and a sine or cosine of that is
sincospif's, within two units (2^-22). So a sine is right relative to itself, however small the angle."""
from __future__ import annotations

import math
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import entropy_coding_gb300 as zc  # noqa: E402

DEV = torch.device("cuda:0")
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def _cos_sin(frequency: float, position: int):
    """To more than 16 digits of each, from an exact product and a quotient of 70 digits."""
    with localcontext() as c:
        c.prec = 70
        turns = Decimal(position) * Decimal(frequency) / (2 * PI)
        quarter = int((turns * 4).to_integral_value())
        rest = float((turns - Decimal(quarter) / 4) * 2 * PI)
    cs, sn = math.cos(rest), math.sin(rest)
    return [(cs, sn), (-sn, cs), (-cs, -sn), (sn, -cs)][quarter % 4]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("base", [1e2, 5e5, 1e7, 1e12])
def test_sines_and_cosines_are_right_relative_to_themselves(base, interleaved):
    positions = [0, 1, 2, 7, 100, 4095, 131071, 9999991, (1 << 30) - 2]
    frequencies = [base ** (-i / 64) * (1 if i % 5 else -1) for i in range(64)]
    n = len(positions)
    batch = zc.KVBatch(torch.zeros(n, 1, dtype=torch.int32, device=DEV), torch.arange(n + 1, dtype=torch.int32, device=DEV),
                       torch.tensor([p + 1 for p in positions], dtype=torch.int32, device=DEV), n, 1)
    cache = zc.KVCache.empty(1, 1, 128, 16)
    x = torch.zeros(n, 1, 128, device=DEV)
    a, b = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, 64), slice(64, 128))
    x[..., a] = 1.0
    got, _ = zc.kv_rotate(cache, batch, zc.KVRotation(frequencies, interleaved), x, x)
    cache.check()
    got = got[:, 0].double().cpu().numpy()
    want = np.array([[_cos_sin(f, p) for f in frequencies] for p in positions])
    for which, of in ((0, a), (1, b)):
        w = want[..., which]
        tol = np.abs(w) * (2.0 ** -24 + 2.0 ** -22) + np.array(positions)[:, None] * 2.0 ** -65 * 2 * math.pi
        bad = np.abs(got[:, of] - w) > tol
        assert not bad.any(), (which, [(positions[i], frequencies[j], got[i, of][j], w[i, j]) for i, j in np.argwhere(bad)[:4]])
