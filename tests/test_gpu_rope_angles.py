"""Angles of far positions: near a whole turn, where the sine is small, an
error of the angle shows undiluted."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from indexer_top_sparse_c4_b200 import build, qsa
    build.build()
    return qsa


def _rest(p, f):
    """p * f less the nearest whole turns."""
    a = Decimal(int(p)) * Decimal(float(f))
    return float(a - (a / (2 * PI)).to_integral_value() * 2 * PI)


def _near_whole_turns(f, lo, hi, n):
    """The n positions of [lo, hi) whose angles are nearest to whole turns."""
    p = np.arange(lo, hi, dtype=np.int64)
    a = p.astype(np.longdouble) * np.longdouble(f)
    t = a / (2 * np.arccos(np.longdouble(-1)))
    return p[np.argsort(np.abs(t - np.rint(t)))[:n]]


@pytest.mark.parametrize("lo, hi", [(1, 1 << 20), ((1 << 30) - (1 << 19), (1 << 30) + (1 << 19)),
                                    ((1 << 31) - (1 << 20), (1 << 31) - 1)])
@pytest.mark.parametrize("adjacent", [False, True])
def test_small_sines_of_far_positions(q, lo, hi, adjacent):
    """Every pair is (1, 0), so that the kernel returns the cosine and the sine
    themselves.  With r the angle's rest (|r| <= pi): the fraction of a turn is
    rounded to FP32, 2^-24 of r, which moves the sine by |r cos r| 2^-24 and
    the cosine by |r sin r| 2^-24; sincospi is within 2 units, 2^-22 of its
    value.  What the product, 1 / (2 pi) and the sum add in 64 bits and their
    remainders is below 2^-50 of a radian."""
    getcontext().prec = 60
    half, n = 8, 12
    freqs = np.float32([1.0, 0.74989420, 0.31622776, 0.1, 0.98765433, 0.05623413, 0.5, 0.7071068])
    pos = np.concatenate([_near_whole_turns(f, lo, hi, n) for f in freqs] + [[hi - 1, lo]])
    T, D = len(pos), 64
    x = torch.zeros((T, 1, D), device="cuda")
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if adjacent else (slice(0, half), slice(half, 2 * half))
    x[..., a] = 1
    kc, vc = (torch.zeros((-(-T // 64), 64, 1, D), device="cuda") for _ in range(2))
    out = torch.zeros_like(x)
    q.qsa_rope_write(x, x, x, torch.tensor(pos, dtype=torch.int32, device="cuda"), torch.tensor(freqs).cuda(),
                     torch.arange(T, dtype=torch.int32, device="cuda"), out, kc, vc, adjacent_pairs=adjacent)
    got = out[:, 0].double().cpu().numpy()
    for t in range(T):
        for i in range(half):
            r = _rest(pos[t], freqs[i])
            c, s = math.cos(r), math.sin(r)
            for y, want, slope in ((got[t, a][i], c, s), (got[t, b][i], s, c)):
                tol = abs(r * slope) * 2.0 ** -24 + abs(want) * 2.0 ** -22 + 2.0 ** -50
                assert abs(y - want) <= tol, f"position {pos[t]}, frequency {freqs[i]}: {y} for {want}, rest {r}"
