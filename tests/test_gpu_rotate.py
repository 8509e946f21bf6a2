"""lmc_rotate and lmc_append_rotated on the GPU against plain 64-bit arithmetic."""
import numpy as np
import pytest
import torch

import linear_reference as R
import state_cache_paging_gb300 as lmc
import token_reference as T

pytestmark = pytest.mark.gpu

# (heads, dim, norm_dim, rot_first, rot_dim, pairs)
SHAPES = [
    (4, 192, 0, 128, 64, True), (8, 128, 128, 0, 128, False), (1, 576, 512, 512, 64, True), (5, 64, 64, 0, 32, False),
    (3, 80, 40, 16, 64, True), (2, 80, 80, 24, 48, False),  # eights, but not all of them pairs of eights
    (7, 33, 20, 3, 10, False), (2, 50, 50, 1, 48, True), (1, 2, 2, 0, 2, True),   # nothing on eights
    (2, 1024, 1024, 0, 1024, False), (1, 4096, 4096, 2048, 2048, True), (3, 3000, 17, 5, 2, False),  # long heads
    (2, 64, 64, 0, 0, False), (6, 16, 0, 0, 16, False), (65, 8, 8, 0, 8, True), (300, 16, 8, 8, 8, True)]


def draw(rows, heads, dim, act, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, heads, dim, generator=g).to(R.TYPES[act])


def rotation(shape, rows, seed=1, far=True):
    heads, dim, norm, first, rot, pairs = shape
    g = torch.Generator().manual_seed(seed)
    angles = torch.randint(0, 200000 if far else 100, (rows,), generator=g).int()
    freqs = (10000.0 ** -(torch.arange(rot // 2) * 2.0 / max(rot, 1))).float() if rot else None
    weight = (1 + 0.2 * torch.randn(norm, generator=g)) if norm else None
    return angles, freqs, weight


def check(got, x, shape, angles, freqs, weight, act, eps=1e-6, mscale=1.0, scale=None):
    heads, dim, norm, first, rot, pairs = shape
    want, lost = R.turned(x, norm, weight, eps, angles, freqs, first, pairs, mscale)
    tiny = 2.0 ** -25 if act == "f16" else 2.0 ** -133
    tol = lost + (want.abs() + lost) * R.HALF_STEP[act] + tiny
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("rows", [1, 37])
def test_rotate(shape, act, rows):
    heads, dim, norm, first, rot, pairs = shape
    x = draw(rows, heads, dim, act)
    angles, freqs, weight = rotation(shape, rows)
    dev = [None if t is None else t.cuda() for t in (angles, freqs, weight)]
    for in_place in (False, True):
        xg = x.cuda()
        out = xg if in_place else torch.full_like(xg, float("nan"))
        lmc.lmc_rotate(xg, dev[0], out, dev[1], rot_first=first, pairs=pairs, norm_dim=norm, norm_weight=dev[2])
        check(out.cpu(), x, shape, angles, freqs, weight, act)
        if not in_place:
            assert torch.equal(xg.cpu(), x)


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[1], SHAPES[6]])
@pytest.mark.parametrize("order", ["wide", "head-major", "odd"])
def test_rotate_strides(shape, order):
    heads, dim, norm, first, rot, pairs = shape
    rows = 19
    x = draw(rows, heads, dim, "bf16")
    angles, freqs, weight = rotation(shape, rows)

    def place():
        if order == "wide":
            big = torch.full((rows, heads, dim + 24), 7.0, dtype=torch.bfloat16, device="cuda")
            return big, big[:, :, 8:8 + dim]
        if order == "odd":
            big = torch.full((rows * heads * (dim + 3) + 1,), 7.0, dtype=torch.bfloat16, device="cuda")
            return big, torch.as_strided(big, (rows, heads, dim), (heads * (dim + 3), dim + 3, 1), 1)
        big = torch.full((heads, rows, dim), 7.0, dtype=torch.bfloat16, device="cuda")
        return big, big.transpose(0, 1)
    for in_place in (False, True):
        big, view = place()
        view.copy_(x)
        kept, out = (big, view) if in_place else place()
        before = kept.clone()
        lmc.lmc_rotate(view, angles.cuda(), out, freqs.cuda(), rot_first=first, pairs=pairs, norm_dim=norm,
                       norm_weight=None if weight is None else weight.cuda())
        check(out.cpu(), x, shape, angles, freqs, weight, "bf16")
        out.fill_(0)
        probe = before.clone()
        torch.as_strided(probe, out.shape, out.stride(), out.storage_offset()).fill_(0)
        assert torch.equal(kept, probe)  # nothing beside the heads was written


def test_rotate_far_and_negative_positions_and_odd_frequencies():
    rows, half = 64, 16
    shape = (2, 32, 0, 0, 32, False)
    x = draw(rows, 2, 32, "f16")
    g = torch.Generator().manual_seed(3)
    angles = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows,), generator=g).int()
    angles[:4] = torch.tensor([0, -1, 2 ** 31 - 1, -2 ** 31])
    freqs = torch.tensor([1.0, -1.0, 0.0, 3.14159, 6.2831855, 100.5, 1e-3, -1e-7, 1e-20, 2.0 ** -130, 0.7071, 5e3, 1e-5,
                          0.1, 2.5, 12345.67])
    out = torch.empty(rows, 2, 32, dtype=torch.float16, device="cuda")
    lmc.lmc_rotate(x.cuda(), angles.cuda(), out, freqs.cuda())
    # The reference's own angle: whole numbers of 2^-100 turns
    from fractions import Fraction
    two_pi_digits = 62831853071795864769252867665590057683943387987502
    turns = [[(int(a) * Fraction(float(f)) * Fraction(10 ** 49, two_pi_digits)) % 1 for f in freqs] for a in angles]
    t = torch.tensor([[float(y) for y in z] for z in turns], dtype=torch.float64)[:, None] * (2 * np.pi)
    a, b = x[..., :half].double(), x[..., half:].double()
    want = torch.cat([a * torch.cos(t) - b * torch.sin(t), a * torch.sin(t) + b * torch.cos(t)], -1)
    both = torch.cat([a.abs() + b.abs()] * 2, -1)
    # as R.turned; a step's own rounding (2^-61 of a frequency of at most 2^11 turns, times 2^31
    # positions) adds 2 pi 2^-19
    far = 2 * np.pi * 2.0 ** -30 * torch.clamp(freqs.abs().double() / 6.28, min=1.0)
    tol = both * (2.0 ** -21 + torch.cat([far, far])) + want.abs() * 2.0 ** -11 + 2.0 ** -25
    err = (out.cpu().double() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


def test_rotate_scales_and_eps():
    shape = (2, 64, 64, 0, 64, False)
    x = draw(9, 2, 64, "bf16") * 1e-3
    x[3] = 0
    angles, freqs, weight = rotation(shape, 9)
    out = torch.empty(9, 2, 64, dtype=torch.bfloat16, device="cuda")
    lmc.lmc_rotate(x.cuda(), angles.cuda(), out, freqs.cuda(), norm_dim=64, norm_weight=weight.cuda(), eps=1e-4, mscale=1.3)
    check(out.cpu(), x, shape, angles, freqs, weight, "bf16", eps=1e-4, mscale=1.3)
    assert bool((out[3] == 0).all())
    lmc.lmc_rotate(x.cuda(), None, out, None, norm_dim=64, norm_weight=None, eps=1e-4)
    check(out.cpu(), x, (2, 64, 64, 0, 0, False), angles, None, None, "bf16", eps=1e-4)


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("E,shape,wide", [
    (576, (1, 576, 512, 512, 64, True), 576), (576, (1, 576, 512, 512, 64, False), 600), (128, (2, 32, 16, 8, 16, False), 131),
    (1024, (8, 64, 64, 0, 64, False), 1024), (112, (2, 48, 48, 0, 16, True), 120), (50, (3, 10, 10, 2, 6, True), 50),
    (1040, (4, 64, 0, 0, 64, False), 1040), (2000, (1, 1200, 1200, 0, 96, True), 2000), (16, (1, 8, 0, 0, 8, True), 16)])
@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_append_rotated(E, shape, wide, act, cache):
    heads, dim, norm, first, rot, pairs = shape
    kind = act if cache == "same" else "e4m3"
    N, had, new = 20, [0, 7, 19, 40], [31, 1, 22, 0]
    rng = np.random.default_rng(2)
    blocks = 12
    M = T.Model(lmc, E, kind, N, layers=2, blocks=blocks, state=0)
    table = T.tables([h + n for h, n in zip(had, new)], N, blocks, rng)
    rows = sum(new) + 2
    req = np.concatenate([np.repeat(np.arange(4), new), [-1, -1]]).astype(np.int32)
    pos = np.concatenate([np.concatenate([np.arange(n) + h for h, n in zip(had, new)]), [0, 5]]).astype(np.int32)
    order = rng.permutation(rows)
    req, pos = torch.from_numpy(req[order]), torch.from_numpy(pos[order])
    g = torch.Generator().manual_seed(1)
    x = torch.randn(rows, wide, generator=g).to(R.TYPES[act])[:, :E]
    _, freqs, weight = rotation(shape, rows)
    scale = 0.05 if kind == "e4m3" else 1.0
    for angles in (None, (pos + 1000).int()):
        pool, status = M.pool.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
        xg = torch.empty(rows, wide, dtype=x.dtype, device="cuda")[:, :E]
        xg.copy_(x)
        lmc.lmc_append_rotated(M.layout, M.layers[1], pool, table.cuda(), req.cuda(), pos.cuda(), xg, status, freqs.cuda(),
                               num_heads=heads, head_dim=dim, rot_first=first, pairs=pairs, norm_dim=norm,
                               norm_weight=None if weight is None else weight.cuda(), scale=scale,
                               angles=None if angles is None else angles.cuda())
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        width = heads * dim
        want, lost = R.turned(x[:, :width].reshape(rows, heads, dim), norm, weight, 1e-6, pos if angles is None else angles,
                              freqs, first, pairs, 1.0)
        want = torch.cat([want.reshape(rows, width), x[:, width:].double()], 1)
        lost = torch.cat([lost.reshape(rows, width), torch.zeros(rows, E - width, dtype=torch.float64)], 1)
        got = pool.cpu()
        pages, expect = M.pages(1, got), M.pool.clone()
        for i in range(rows):
            if int(req[i]) < 0:
                continue
            b, t = int(table[int(req[i]), int(pos[i]) // N]), int(pos[i]) % N
            y = pages[b, t].contiguous().view(T.TYPES[kind]).double() * scale
            half, tiny = T.HALF_STEP[kind], {"bf16": 2.0 ** -133, "f16": 2.0 ** -25, "e4m3": 2.0 ** -10 * scale}[kind]
            assert bool(((y - want[i]).abs() <= lost[i] + (want[i].abs() + lost[i]) * half + tiny).all()), i
            M.pages(1, expect)[b, t] = pages[b, t]
        assert torch.equal(expect, got)  # nothing else was written


def test_append_rotated_without_norm_and_rotation_is_append():
    """No norm, no rotation: lmc_append's bytes, in each type."""
    for kind, act in (("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")):
        M = T.Model(lmc, 576, kind, 20, blocks=4)
        x = (torch.randn(45, 576) * 8).to(R.TYPES[act]).cuda()
        table = torch.tensor([[2, 0, 3]], dtype=torch.int32).cuda()
        req, pos = torch.zeros(45, dtype=torch.int32).cuda(), torch.arange(45, dtype=torch.int32).cuda()
        pools, status = [], torch.zeros(1, dtype=torch.int32, device="cuda")
        scale = 0.3 if kind == "e4m3" else 1.0
        for f in (lmc.lmc_append, lambda *a, **kw: lmc.lmc_append_rotated(*a, None, **kw)):
            pool = M.pool.cuda()
            f(M.layout, M.layers[0], pool, table, req, pos, x, status, scale=scale)
            pools.append(pool.cpu())
        assert int(status.item()) == 0 and torch.equal(*pools)


def test_append_rotated_bad_rows():
    M = T.Model(lmc, 64, "bf16", 8, blocks=4)
    table = torch.tensor([[0, -1], [9, 1]], dtype=torch.int32).cuda()
    req = torch.tensor([0, 0, 1, 1, 2, -2, 1, 0], dtype=torch.int32).cuda()
    pos = torch.tensor([3, 9, 0, 8, 0, 0, 16, -1], dtype=torch.int32).cuda()
    x = torch.ones(8, 64, dtype=torch.bfloat16).cuda()
    pool, status = M.pool.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    lmc.lmc_append_rotated(M.layout, 0, pool, table, req, pos, x, status, torch.ones(8).cuda())
    torch.cuda.synchronize()
    assert int(status.item()) == lmc.LMC_ST_BAD_JOB | lmc.LMC_ST_NO_BLOCK | lmc.LMC_ST_BLOCK_OOR
    written = (M.pages(0, pool.cpu()) != 0xFF).any(-1).nonzero().tolist()
    assert written == [[0, 3], [1, 0]]


def test_rotate_repeats_streams_and_graphs():
    shape = (8, 128, 128, 0, 128, False)
    x = draw(300, 8, 128, "bf16").cuda()
    angles, freqs, weight = (t.cuda() for t in rotation(shape, 300))
    call = lambda out, stream=None: lmc.lmc_rotate(x, angles, out, freqs, norm_dim=128, norm_weight=weight,  # noqa: E731
                                                   stream=stream)
    outs = [torch.zeros_like(x) for _ in range(3)]
    call(outs[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(outs[1], s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(outs[2])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
