"""lmc_rotate and lmc_append_rotated of long heads by eight lanes each, many and few, and
fp8 scales without an inverse, against plain 64-bit arithmetic."""
import numpy as np
import pytest
import torch

import linear_reference as R
import state_cache_paging_gb300 as lmc
import token_reference as T
from test_gpu_rotate import check, draw, rotation

pytestmark = pytest.mark.gpu

# (heads, dim, norm_dim, rot_first, rot_dim, pairs): 33 to 72 pieces of eight values a head
LONG = [(1, 576, 512, 512, 64, True), (1, 576, 512, 512, 64, False), (1, 576, 576, 0, 576, True), (1, 576, 0, 64, 128, False),
        (2, 288, 264, 8, 96, False), (32, 264, 264, 200, 64, True), (33, 272, 16, 0, 16, False), (1, 512, 512, 0, 0, False),
        (1, 568, 40, 24, 160, False)]


@pytest.mark.parametrize("shape", LONG)
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_rotate_many_long_heads(shape, act):
    heads, dim, norm, first, rot, pairs = shape
    rows = 19500 // heads + 3
    x = draw(rows, heads, dim, act)
    angles, freqs, weight = rotation(shape, rows)
    for in_place in (False, True):
        big = torch.full((rows, heads, dim + 8), 7.0, dtype=x.dtype, device="cuda")
        xg = x.cuda() if not in_place else big[:, :, :dim]
        xg.copy_(x)
        out = big[:, :, :dim]
        lmc.lmc_rotate(xg, angles.cuda(), out, None if freqs is None else freqs.cuda(), rot_first=first, pairs=pairs,
                       norm_dim=norm, norm_weight=None if weight is None else weight.cuda())
        check(out.cpu(), x, shape, angles, freqs, weight, act)
        assert bool((big[:, :, dim:] == 7.0).all())


def entries(shape, E, kind, act, scale, rows, N=100):
    """Appends `rows` rows, some of them padding, in a random order; checks every byte."""
    heads, dim, norm, first, rot, pairs = shape
    rng = np.random.default_rng(3)
    cols = -(-rows // N) + 1
    M = T.Model(lmc, E, kind, N, layers=2, blocks=cols + 2, state=0)
    table = torch.from_numpy(rng.permutation(cols + 2)[:cols].astype(np.int32))[None]
    pos = rng.permutation(cols * N)[:rows].astype(np.int32)
    req = np.where(rng.random(rows) < 0.05, -1, 0).astype(np.int32)
    req, pos = torch.from_numpy(req), torch.from_numpy(pos)
    x = torch.randn(rows, E, generator=torch.Generator().manual_seed(1)).to(R.TYPES[act])
    _, freqs, weight = rotation(shape, rows)
    pool, status = M.pool.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    lmc.lmc_append_rotated(M.layout, M.layers[1], pool, table.cuda(), req.cuda(), pos.cuda(), x.cuda(), status, freqs.cuda(),
                           num_heads=heads, head_dim=dim, rot_first=first, pairs=pairs, norm_dim=norm,
                           norm_weight=weight.cuda(), scale=scale)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    width = heads * dim
    want, lost = R.turned(x[:, :width].reshape(rows, heads, dim), norm, weight, 1e-6, pos, freqs, first, pairs, 1.0)
    want = torch.cat([want.reshape(rows, width), x[:, width:].double()], 1)
    lost = torch.cat([lost.reshape(rows, width), torch.zeros(rows, E - width, dtype=torch.float64)], 1)
    got = pool.cpu()
    at = req >= 0
    block, token = table[0, (pos[at] // N).long()].long(), (pos[at] % N).long()
    y = M.pages(1, got)[block, token].contiguous().view(T.TYPES[kind]).double() * scale
    half, tiny = T.HALF_STEP[kind], {"bf16": 2.0 ** -133, "f16": 2.0 ** -25, "e4m3": 2.0 ** -10 * scale}[kind]
    want, lost = want[at], lost[at]
    if kind == "e4m3":
        want = want.clamp(-448 * scale, 448 * scale)  # (satfinite)
    assert bool(((y - want).abs() <= lost + (want.abs() + lost) * half + tiny).all())
    expect = M.pool.clone()
    M.pages(1, expect)[block, token] = M.pages(1, got)[block, token]
    assert torch.equal(expect, got)  # nothing else was written


@pytest.mark.parametrize("kind,act", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("shape", [LONG[0], LONG[1], LONG[4], LONG[8]])
def test_append_many_long_heads(shape, kind, act):
    heads, dim = shape[:2]
    entries(shape, heads * dim, kind, act, 0.05 if kind == "e4m3" else 1.0, 19500 // heads + 7)


@pytest.mark.parametrize("scale", [float(np.uint32(0x3fffffff).view(np.float32)), 2.0 ** -102, 2.0 ** 101])
@pytest.mark.parametrize("shape,E,rows", [(LONG[0], 576, 50), (LONG[0], 576, 19600), ((4, 64, 64, 0, 64, False), 512, 50),
                                          ((3, 10, 10, 2, 6, True), 50, 50)])
def test_fp8_scales_without_an_inverse(shape, E, rows, scale):
    """Codes of quotients where 1 / scale would not do."""
    entries(shape, E, "e4m3", "bf16", scale, rows)
