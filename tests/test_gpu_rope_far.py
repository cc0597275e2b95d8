"""Angles of far positions against whole-number arithmetic: the bound that include/pa.h gives."""
import math

import pytest
import torch

from test_gpu_rope import DEV, pa  # noqa: F401 (pa: the fixture)

pytestmark = pytest.mark.gpu

BITS = 320


def _arctan_inverse(x):
    """arctan(1 / x) 2^BITS (its series, in whole numbers)."""
    total, term, k = 0, (1 << BITS) // x, 0
    while term:
        total += (-1) ** k * (term // (2 * k + 1))
        term //= x * x
        k += 1
    return total


def _turn(position, freq, pi):
    """position * freq / (2 pi) without its whole turns, in 64 bits."""
    num, den = float(freq).as_integer_ratio()
    one = 2 * pi * den
    return (position * num * (1 << BITS)) % one / one


@pytest.mark.parametrize("far", [20, 37, 45, 52, 60])
def test_angles_of_far_positions(pa, far):  # noqa: F811
    pi = 4 * (4 * _arctan_inverse(5) - _arctan_inverse(239))
    n, half = 24, 16
    gen = torch.Generator().manual_seed(far)
    pos = (1 << far) - torch.randint(0, 1 << min(far, 40), (n,), generator=gen)
    pos[::3] *= -1
    inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    inv[1], inv[2], inv[3] = 3.7, -0.83, 41.25
    x = torch.zeros((n, 1, 2 * half))
    x[..., :half] = 1.0  # the rotation of (1, 0): its cosine and sine
    out = torch.empty((n, 1, 2 * half), device=DEV)
    kc, vc = (torch.zeros((3, 8, 1, 2 * half), device=DEV) for _ in range(2))
    dx = x.to(DEV)
    pa.pa_rope_write_kv(out, dx, dx, dx, pos.to(DEV), inv.to(DEV), torch.arange(n, device=DEV), kc, vc)
    got = out.cpu().double()[:, 0]
    for t in range(n):
        for i in range(half):
            f, p = float(inv[i]), int(pos[t])
            turn = _turn(p, f, pi)
            # the bound, the angle's rounding to fp32, and sincospif's and the products'
            tol = 2 * math.pi * (abs(p) * max(1.0, abs(f)) * 2.0 ** -63 + 2.0 ** -26) + 4 * 2.0 ** -24
            assert abs(got[t, i] - math.cos(2 * math.pi * turn)) <= tol, (p, f)
            assert abs(got[t, half + i] - math.sin(2 * math.pi * turn)) <= tol, (p, f)
