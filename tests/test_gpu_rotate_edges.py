"""lmc_rotate and lmc_append_rotated at the ends of their ranges: the largest
frequencies at the farthest positions, fp8 scales and factors whose product
leaves binary32; against plain arithmetic in 64 bits and fractions."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import linear_reference as R
import state_cache_paging_gb300 as lmc

pytestmark = pytest.mark.gpu
DEV = "cuda"
TWO_PI = Fraction(62831853071795864769252867665590057683943387987502, 10 ** 49)


@pytest.mark.parametrize("pairs", [False, True])
def test_the_largest_frequencies_at_the_farthest_positions(pairs):
    """Angles of up to 2^55 rad. A reduced angle is off by 2^-31 turns and its binary32
    form by pi 2^-25; sine, products and sums as in R.turned (2^-21 in all)."""
    rows, half = 66, 16
    g = torch.Generator().manual_seed(5)
    angles = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows,), generator=g).int()
    angles[:4] = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, -1])
    freqs = torch.tensor([2.0 ** 24 - 1, 2.0 ** 23, 2.0 ** 23 + 1, -1.6e7, 8388607.5, 5e6, -1234567.0, 1e5, 12345.67, -4097.3,
                          1000.1, 63.0, 6.2831855, 1.0, 0.999, 2.0 ** -40])
    x = torch.randn(rows, 2, 2 * half, generator=g).half()
    out = torch.empty(rows, 2, 2 * half, dtype=torch.float16, device=DEV)
    lmc.lmc_rotate(x.cuda(), angles.cuda(), out, freqs.cuda(), pairs=pairs)
    t = torch.tensor([[float(int(a) * Fraction(float(f)) / TWO_PI % 1) for f in freqs] for a in angles],
                     dtype=torch.float64)[:, None] * (2 * np.pi)
    u, w = (x[..., 0::2], x[..., 1::2]) if pairs else (x[..., :half], x[..., half:])
    u, w, got = u.double(), w.double(), out.cpu().double()
    got_u, got_w = (got[..., 0::2], got[..., 1::2]) if pairs else (got[..., :half], got[..., half:])
    for y, want in ((got_u, u * torch.cos(t) - w * torch.sin(t)), (got_w, u * torch.sin(t) + w * torch.cos(t))):
        tol = (u.abs() + w.abs()) * 2.0 ** -21
        err = (y - want).abs()
        assert bool((err <= tol + (want.abs() + tol) * R.HALF_STEP["f16"] + 2.0 ** -25).all()), float((err - tol).max())
