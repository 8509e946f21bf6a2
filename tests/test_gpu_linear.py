"""lmc_linear_step and lmc_linear_scan on the GPU against plain 64-bit
arithmetic, token by token."""
import numpy as np
import pytest
import torch

import linear_reference as R
import state_cache_paging_gb300 as lmc

pytestmark = pytest.mark.gpu


def inputs(rows, H, Hk, dk, dv, act, decay, seed, fused=False):
    g = torch.Generator().manual_seed(seed)
    t = R.TYPES[act]
    if fused:  # slices of one product's rows
        width = 2 * Hk * dk + H * dv + 8
        x = torch.randn(rows, width, generator=g).to(t)
        q, k = x[:, :Hk * dk].view(rows, Hk, dk), x[:, Hk * dk:2 * Hk * dk].view(rows, Hk, dk)
        v = x[:, 2 * Hk * dk:2 * Hk * dk + H * dv].view(rows, H, dv)
        k.mul_(dk ** -0.5)
    else:
        q, v = torch.randn(rows, Hk, dk, generator=g).to(t), torch.randn(rows, H, dv, generator=g).to(t)
        k = (torch.randn(rows, Hk, dk, generator=g) * dk ** -0.5).to(t)
        x = None
    if decay == "head":
        d = torch.log(1 - 2.0 ** -torch.linspace(2, 10, H)).expand(rows, H)
    elif decay == "none":
        d = torch.zeros(1, 1).expand(rows, H)
    elif decay == "resets":  # some tokens forget everything, by any number that says so
        d = -torch.exp(2 * torch.randn(rows, H, generator=g) - 4)
        u = torch.rand(rows, H, generator=g)
        d = torch.where(u < 0.03, torch.tensor(-float("inf")), torch.where(u < 0.05, torch.tensor(-5000.0), d))
        d = torch.where((u > 0.05) & (u < 0.08), torch.tensor(-90.0), d)
    else:
        d = -torch.exp(2 * torch.randn(rows, H, generator=g) - 4)
    return q, k, v, d, x


def on_gpu(t, x=None, base=None):
    """To the device with the strides it has."""
    if base is not None:
        return torch.as_strided(base.cuda() if not base.is_cuda else base, t.shape, t.stride(), t.storage_offset())
    if 0 in t.stride():
        return t[:1, :1].cuda().expand(t.shape) if t.stride() == (0, 0) else t[:1].cuda().expand(t.shape)
    return t.cuda()


def run(had, new, H=2, Hk=None, dk=64, dv=64, N=48, act="bf16", decay="token", packed=False, held=None, fused=False,
        op="scan", pad=0, seed=1, scale=None, stream=None):
    Hk = Hk or H
    rng = np.random.default_rng(seed)
    blocks = sum(-(-(max(h, 0) + t) // N) for h, t in zip(had, new)) + 3
    P = R.States(lmc, H, dk, dv, N, blocks, packed=packed)
    table = R.tables(had, new, N, blocks, rng, held)
    g = torch.Generator().manual_seed(seed + 5)
    pages = P.pages()
    for r, h in enumerate(had):
        if h > 0:
            pages[int(table[r, (h - 1) // N])] = torch.randn(H, dk, dv, generator=g)
    rows = sum(new) + pad
    q, k, v, d, x = inputs(rows, H, Hk, dk, dv, act, decay, seed, fused)
    scale = dk ** -0.5 if scale is None else scale
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    pool, out = P.pool.cuda(), torch.full((rows, H, dv), float("nan"), dtype=R.TYPES[act], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lengths = torch.tensor(had, dtype=torch.int32, device="cuda")
    xg = None if x is None else x.cuda()
    args = [on_gpu(q, base=xg), on_gpu(k, base=xg), on_gpu(v, base=xg), on_gpu(d)]
    if op == "scan":
        ws = torch.full((lmc.lmc_linear_scan_workspace(P.layout, P.layer, len(had), rows, H),), 0xFF, dtype=torch.uint8,
                        device="cuda")
        lmc.lmc_linear_scan(P.layout, P.layer, pool, table.cuda(), torch.from_numpy(start).cuda(), lengths, *args, out, ws,
                            status, scale=scale)
    else:
        lmc.lmc_linear_step(P.layout, P.layer, pool, table.cuda(), lengths, *args, out, status, scale=scale)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    check(P, pool.cpu(), out.cpu(), had, new, table, start, q, k, v, d, scale, act)
    return out


def check(P, pool, out, had, new, table, start, q, k, v, d, scale, act):
    want_pool = P.pool.clone()
    got, want = P.pages(pool), P.pages(want_pool)
    half, N = R.HALF_STEP[act], P.N
    touched = torch.zeros(out.shape[0], dtype=torch.bool)
    written = []
    for r, (h, t) in enumerate(zip(had, new)):
        if h < 0 or t == 0:
            continue
        s, e = int(start[r]), int(start[r]) + t
        touched[s:e] = True
        S0 = P.pages()[int(table[r, (h - 1) // N])].double() if h > 0 else torch.zeros(P.H, P.dk, P.dv, dtype=torch.float64)
        ends = [n - h for n in range(h + 1, h + t + 1) if n % N == 0 or n == h + t]
        o, mag, kept = R.linear(S0, q[s:e], k[s:e], v[s:e], d[s:e], scale, ends)
        err = (out[s:e].double() - o).abs()
        # The result and the weights inside a chunk are rounded to the type, and the
        # rest is binary32: sums of up to t + 128 terms, decays of 2^-20.
        tol = half * o.abs() + mag * (half + (t + 256) * 2.0 ** -23 + 2.0 ** -14) + (2.0 ** -24 if act == "f16" else 0)
        assert bool((err <= tol).all()), (r, float((err - tol).max()), float(err.max()))
        # As many independent roundings of half a step: their 2-norm stays below one
        assert float(err.norm()) <= half * float(o.norm()) + 1e-30, (r, float(err.norm() / o.norm()))
        for n, (S, A) in kept.items():
            b = int(table[r, (h + n - 1) // N])
            if b < 0:
                continue
            written.append(b)
            es = (got[b].double() - S).abs()
            assert bool((es <= A * ((t + 256) * 2.0 ** -23 + 2.0 ** -18) + 1e-37).all()), (r, n, float(es.max()))
            assert float(es.norm()) <= 2.0 ** -18 * float(S.norm()) + 1e-37, (r, n, float(es.norm() / S.norm()))
            want[b] = got[b]
    assert len(set(written)) == len(written)
    # what is not written stays: other rows, pages, the conv part, the other layers
    assert bool(torch.isnan(out[~touched].float()).all())
    assert torch.equal(want_pool, pool)


DIMS = [(64, 64), (128, 128), (128, 40), (24, 128), (96, 96), (8, 8), (72, 104)]


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("dims", DIMS)
def test_step(dims, act):
    run([0, 5, 47, 48, 49, -1, 96], [1] * 7, H=4, Hk=2, dk=dims[0], dv=dims[1], op="step", act=act)


@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 1), (6, 3), (8, 8)])
def test_step_heads_and_strides(H, Hk):
    run([7, 100, 0], [1] * 3, H=H, Hk=Hk, dk=64, dv=128, op="step", fused=True, packed=True, decay="head")


def test_step_decays():
    run([9] * 40, [1] * 40, H=4, op="step", decay="resets")


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("dims", DIMS)
def test_scan_dims(dims, act):
    run([0, 30, 48], [130, 70, 1], H=2, Hk=1, dk=dims[0], dv=dims[1], act=act)


@pytest.mark.parametrize("N", [16, 48, 64, 65, 100, 200, 1000])
@pytest.mark.parametrize("decay", ["token", "head", "none", "resets"])
def test_scan_blocks_and_decays(N, decay):
    run([0, 3, N, 2 * N - 1, -1, 17, 64], [1, 200, 63, 66, 20, 0, 129], N=N, decay=decay, pad=5)


def test_scan_ragged_many():
    rng = np.random.default_rng(4)
    run(rng.integers(0, 90, 37).tolist(), rng.integers(0, 150, 37).tolist(), H=3, Hk=3, dk=128, dv=128, N=100)


@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_scan_one_long_request(act):
    run([100], [2500], H=2, dk=128, dv=128, N=144, act=act, held=lambda r, b: b % 2 == 1)


def test_scan_long_beside_short():
    run([0, 10, 3], [1700, 3, 40], H=1, dk=128, dv=64, N=300, held=lambda r, b: False)


def test_scan_strided_inputs():
    run([0, 50], [90, 75], H=4, Hk=2, dk=64, dv=128, N=60, fused=True, packed=True)


def test_scan_equals_step_by_step():
    """A prompt, then tokens one at a time, and the prompt with those tokens at once."""
    H, d, N, T, m = 2, 64, 48, 100, 20
    q, k, v, dec, _ = inputs(T + m, H, H, d, d, "f16", "token", 3)
    P = R.States(lmc, H, d, d, N, 8)
    table = torch.arange(3, dtype=torch.int32)[None].cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    outs, pools = [], []
    for first in (T, T + m):
        pool, out = P.pool.cuda(), torch.zeros(T + m, H, d, dtype=torch.float16, device="cuda")
        ws = torch.empty(lmc.lmc_linear_scan_workspace(P.layout, P.layer, 1, T + m, H), dtype=torch.uint8, device="cuda")
        a = [x.cuda() for x in (q, k, v, dec)]
        lmc.lmc_linear_scan(P.layout, P.layer, pool, table, ints([0, first]), ints([0]), *a, out, ws, status, scale=0.1)
        for t in range(first, T + m):
            lmc.lmc_linear_step(P.layout, P.layer, pool, table, ints([t]), *[x[t:t + 1] for x in a], out[t:t + 1], status,
                                scale=0.1)
        torch.cuda.synchronize()
        outs.append(out.float().cpu())
        pools.append(P.pages(pool.cpu())[:3].clone())
    assert int(status.item()) == 0
    # each is within the type's half step (2^-11) of the exact one twice over, in the 2-norm
    assert float((outs[0] - outs[1]).norm()) <= 2 * 2.0 ** -11 * float(outs[0].norm())
    assert float((pools[0] - pools[1]).norm()) <= 2.0 ** -17 * float(pools[0].norm())


@pytest.mark.parametrize("op", ["step", "scan"])
def test_bad_requests_are_left_out(op):
    H, d, N, blocks = 2, 64, 32, 6
    P = R.States(lmc, H, d, d, N, blocks)
    P.pages()[:] = 0.25
    had = [-2, 40, 40, 40, 64, 96, 31, 5]
    # positions: (read, written) block 1 of row 1 missing, of row 2 outside, of row 3 fine, row 4's new one
    # missing, row 5 past the table, row 6: fine in block 0, row 7's outside
    table = [[0, 0, 0], [0, -1, 0], [0, 99, 0], [0, 1, 0], [0, 2, -1], [0, 0, 0], [3, 0, 0], [-7, 0, 0]]
    rows = len(had)
    q, k, v, dec, _ = inputs(rows, H, H, d, d, "bf16", "token", 1)
    pool, out = P.pool.cuda(), torch.full((rows, H, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    a = [x.cuda() for x in (q, k, v, dec)]
    if op == "step":
        lmc.lmc_linear_step(P.layout, P.layer, pool, ints(table), ints(had), *a, out, status)
    else:
        ws = torch.empty(lmc.lmc_linear_scan_workspace(P.layout, P.layer, rows, rows, H), dtype=torch.uint8, device="cuda")
        lmc.lmc_linear_scan(P.layout, P.layer, pool, ints(table), ints(list(range(rows + 1))), ints(had), *a, out, ws, status)
    torch.cuda.synchronize()
    assert int(status.item()) == lmc.LMC_ST_BAD_JOB | lmc.LMC_ST_NO_SNAPSHOT | lmc.LMC_ST_BLOCK_OOR
    fine = [3, 6]
    assert [bool(torch.isfinite(out[r].float()).all()) for r in range(rows)] == [r in fine for r in range(rows)]
    changed = (P.pages(pool.cpu()) != 0.25).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [1, 3]


def test_scan_bad_starts():
    H, d, N = 1, 64, 32
    P = R.States(lmc, H, d, d, N, 8)
    q, k, v, dec, _ = inputs(10, H, H, d, d, "bf16", "token", 1)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for starts, fine in (([0, 4, 11], range(0, 4)), ([0, 6, 4], range(0, 6)), ([-1, 3, 5], range(3, 5))):
        pool, out = P.pool.cuda(), torch.full((10, H, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = torch.empty(lmc.lmc_linear_scan_workspace(P.layout, P.layer, 2, 10, H), dtype=torch.uint8, device="cuda")
        lmc.lmc_linear_scan(P.layout, P.layer, pool, ints([[0], [1]]), ints(starts), ints([0, 0]),
                            *[x.cuda() for x in (q, k, v, dec)], out, ws, status)
        torch.cuda.synchronize()
        assert int(status.item()) == lmc.LMC_ST_BAD_JOB
        ok = torch.isfinite(out.float()).flatten(1).all(1).tolist()
        assert ok == [i in fine for i in range(10)]


def test_scan_leaves_a_bad_snapshot_out():
    """An entry outside the pool in between raises its bit; all else is done."""
    H, d, N = 1, 64, 32
    P = R.States(lmc, H, d, d, N, 8)
    q, k, v, dec, _ = inputs(96, H, H, d, d, "bf16", "token", 1)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pool, out = P.pool.cuda(), torch.full((96, H, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(lmc.lmc_linear_scan_workspace(P.layout, P.layer, 1, 96, H), dtype=torch.uint8, device="cuda")
    lmc.lmc_linear_scan(P.layout, P.layer, pool, ints([[2, 50, 4]]), ints([0, 96]), ints([0]),
                        *[x.cuda() for x in (q, k, v, dec)], out, ws, status, scale=0.1)
    torch.cuda.synchronize()
    assert int(status.item()) == lmc.LMC_ST_BLOCK_OOR
    got = P.pages(pool.cpu())
    assert [bool(torch.isfinite(got[b]).all()) for b in range(8)] == [b in (2, 4) for b in range(8)]
    assert bool(torch.isfinite(out.float()).all())


def test_rows_of_other_requests_do_not_leak():
    """NaN and infinities in one request's rows stay with it."""
    H, d, N = 2, 64, 48
    new = [37, 70, 41]
    q, k, v, dec, _ = inputs(sum(new), H, H, d, d, "bf16", "token", 2)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    got = []
    for bad in (False, True):
        if bad:
            for x, y in ((q, float("nan")), (k, float("inf")), (v, float("nan"))):
                x[37:107] = y
            dec[37:107] = float("nan")
        P = R.States(lmc, H, d, d, N, 8)
        pool, out = P.pool.cuda(), torch.zeros(sum(new), H, d, dtype=torch.bfloat16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = torch.empty(lmc.lmc_linear_scan_workspace(P.layout, P.layer, 3, sum(new), H), dtype=torch.uint8, device="cuda")
        lmc.lmc_linear_scan(P.layout, P.layer, pool, ints([[0, -1, -1], [1, 2, 3], [4, 5, 6]]), ints([0, 37, 107, 148]),
                            ints([0, 0, 0]), *[x.cuda() for x in (q, k, v, dec)], out, ws, status, scale=0.1)
        torch.cuda.synchronize()
        got.append((out.cpu(), P.pages(pool.cpu()).clone()))
    for i in (slice(0, 37), slice(107, 148)):
        assert torch.equal(got[0][0][i], got[1][0][i])
    assert bool(torch.isnan(got[1][0][37:107].float()).all())
    assert torch.equal(got[0][1][[0, 4]], got[1][1][[0, 4]])


@pytest.mark.parametrize("op", ["step", "scan"])
def test_repeats_streams_and_graphs_give_the_same_bits(op):
    H, d, N, Rq = 4, 128, 100, 5
    had = [0, 50, 100, 150, 199]
    new = [1] * Rq if op == "step" else [90, 1, 250, 64, 0]
    rows = sum(new)
    q, k, v, dec, _ = inputs(rows, H, H, d, d, "bf16", "token", 7)
    P = R.States(lmc, H, d, d, N, 24)
    for b in range(24):
        P.pages()[b] = torch.randn(H, d, d, generator=torch.Generator().manual_seed(b))
    table = R.tables(had, new, N, 24, np.random.default_rng(0)).cuda()
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    starts, lengths = ints(np.concatenate([[0], np.cumsum(new)]).tolist()), ints(had)
    a = [x.cuda() for x in (q, k, v, dec)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fresh = P.pool.cuda()
    need = lmc.lmc_linear_scan_workspace(P.layout, P.layer, Rq, rows, H) if op == "scan" else 0

    def call(pool, out, ws, stream=None):
        if op == "step":
            lmc.lmc_linear_step(P.layout, P.layer, pool, table, lengths, *a, out, status, stream=stream)
        else:
            lmc.lmc_linear_scan(P.layout, P.layer, pool, table, starts, lengths, *a, out, ws, status, stream=stream)

    def state():
        return fresh.clone(), torch.zeros(rows, H, d, dtype=torch.bfloat16, device="cuda"), \
            torch.empty(need, dtype=torch.uint8, device="cuda")
    first = state()
    call(*first)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    both = [state(), state()]
    torch.cuda.synchronize()
    for _ in range(3):
        for (pool, out, ws), s in zip(both, sides):
            with torch.cuda.stream(s):
                pool.copy_(fresh)
            call(pool, out, ws, stream=s)
    torch.cuda.synchronize()
    graphed = state()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        graphed[0].copy_(fresh)
        call(*graphed)
        graphed[0].copy_(fresh)
        call(*graphed)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for x in (*both, graphed):
        assert torch.equal(x[0], first[0]) and torch.equal(x[1], first[1])
    assert int(status.item()) == 0
