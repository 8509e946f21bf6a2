"""lmc_rotate and lmc_append_rotated at the ends of their ranges: the largest
frequencies at the farthest positions, fp8 scales and factors whose product
leaves binary32; against plain arithmetic in 64 bits and fractions."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import linear_reference as R
import state_cache_paging_gb300 as lmc
import token_reference as T

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


@pytest.mark.parametrize("shape,E", [((1, 576, 512, 512, 64, True), 576), ((4, 64, 64, 0, 64, False), 320),
                                     ((3, 10, 10, 2, 6, True), 50)])
@pytest.mark.parametrize("mscale,scale,size", [(1e30, 1e-20, 1.0), (-1e37, 0.01, 1.0), (1.0, 1e-25, 1e-15)])
def test_fp8_scales_beside_large_factors(shape, E, mscale, scale, size):
    """mscale / scale, or the norm's factor over it, is past binary32: zeros stay zeros,
    and what is past the codes is the largest one."""
    heads, dim, norm, first, rot, pairs = shape
    rows, N = 40, 20
    M = T.Model(lmc, E, "e4m3", N, blocks=4)
    x = torch.randn(rows, E, generator=torch.Generator().manual_seed(2)) * size
    x[:, ::3] = 0
    x[5] = 0
    x = x.bfloat16()
    freqs = (10000.0 ** -(torch.arange(rot // 2) * 2.0 / rot)).float()
    pool, status = M.pool.cuda(), torch.zeros(1, dtype=torch.int32, device=DEV)
    table = torch.tensor([[3, 1]], dtype=torch.int32)
    lmc.lmc_append_rotated(M.layout, M.layers[0], pool, table.cuda(), torch.zeros(rows, dtype=torch.int32, device=DEV),
                           torch.arange(rows, dtype=torch.int32, device=DEV), x.cuda(), status, freqs.cuda(), num_heads=heads,
                           head_dim=dim, rot_first=first, pairs=pairs, mscale=mscale, norm_dim=norm, eps=1e-30 if size < 1 else 1e-6,
                           scale=scale)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    width = heads * dim
    want, _ = R.turned(x[:, :width].reshape(rows, heads, dim), norm, None, 1e-30 if size < 1 else 1e-6, torch.arange(rows), freqs,
                       first, pairs, mscale)
    want = torch.cat([want.reshape(rows, width), x[:, width:].double()], 1) / scale
    p = torch.arange(rows)
    got = M.pages(0, pool.cpu())[table[0, p // N].long(), p % N].contiguous().view(torch.float8_e4m3fn).double()
    assert bool((got[want == 0] == 0).all())
    far = want.abs() > 500
    assert bool((got[far] == 448 * want[far].sign()).all()) and int(far.sum()) > rows * heads * rot // 4
