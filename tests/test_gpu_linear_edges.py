"""lmc_linear_scan and lmc_linear_step where a call is easily wrong: starts that
decrease, tables that name a page twice, long slow decays, f16's range; against
plain 64-bit arithmetic."""
import numpy as np
import pytest
import torch

import linear_reference as R
import state_cache_paging_gb300 as lmc
import test_gpu_linear as G
from test_gpu_linear_uses import flag, ints, workspace

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _decreasing(case, n, most):
    if case == 0:
        return np.array([0, n, n // 2, n])
    if case == 1:
        return np.array([n - 1000, n, 0, n - 1000])
    rng = np.random.default_rng(case)
    starts = np.sort(rng.integers(0, n + 1, most + 1))
    swap = rng.permutation(most + 1)[:2 + 3 * (case % 3)]
    starts[swap] = starts[np.roll(swap, 1)]
    return starts


@pytest.mark.parametrize("case", range(6))
def test_a_request_is_done_from_its_own_tokens_or_left_out(case):
    """Starts that decrease: nothing comes from a workspace that nobody wrote. Each
    request is made whole or not touched, and those too short to be cut are made."""
    H, d, N, n = 1, 64, 1 << 13, 6000
    starts = _decreasing(case, n, 6)
    Rq = len(starts) - 1
    assert (np.diff(starts) < 0).any()
    q, k, v, dec, _ = G.inputs(n, H, H, d, d, "bf16", "token", 1)
    P = R.States(lmc, H, d, d, N, Rq + 2)
    pool, out, status = P.pool.cuda(), torch.full((n, H, d), float("nan"), dtype=torch.bfloat16, device=DEV), flag()
    ws = workspace(P, Rq, n)[0].fill_(0xFF)
    lmc.lmc_linear_scan(P.layout, P.layer, pool, ints([[r] for r in range(Rq)]), ints(starts.tolist()), ints([0] * Rq),
                        *[x.cuda() for x in (q, k, v, dec)], out, ws, status, scale=0.1)
    torch.cuda.synchronize()
    assert int(status.item()) == lmc.LMC_ST_BAD_JOB
    got, out, half = P.pages(pool.cpu()), out.cpu(), R.HALF_STEP["bf16"]
    makers = [[] for _ in range(n)]
    for r in range(Rq):
        s, e = int(starts[r]), int(starts[r + 1])
        if bool(torch.isnan(got[r]).all()):
            assert e <= s or e - s >= 1024, r  # (segments are of 512 tokens)
            continue
        assert e > s
        o, _, kept = R.linear(torch.zeros(H, d, d, dtype=torch.float64), q[s:e], k[s:e], v[s:e], dec[s:e], 0.1, (e - s,))
        assert float((got[r].double() - kept[e - s][0]).norm()) <= 2.0 ** -18 * float(kept[e - s][0].norm()), r
        for i in range(s, e):
            makers[i].append(o[i - s])
    # (rows of several requests hold the result of one of them)
    for i, o in enumerate(makers):
        x = out[i].double()
        if not o:
            assert bool(torch.isnan(x).all()), i
        else:  # as many as 64 independent roundings of a weight and a result: below twice the half step of the norm
            assert min(float((x - y).norm() / y.norm()) for y in o) <= 4 * half, i


@pytest.mark.parametrize("n,N,H", [(6000, 144, 1), (5900, 64, 1), (6000, 16, 1), (4000, 100, 2), (8000, 200, 1), (900, 64, 2)])
def test_one_page_at_every_position(n, N, H):
    """Requests that keep one state each: the page is read and ends with the state after
    the last token, whatever positions and segments lie between."""
    d, had, new = 64, [70, 0, N], [n, 33, 0]
    blocks = max(-(-(h + t) // N) for h, t in zip(had, new))
    P = R.States(lmc, H, d, d, N, 4)
    P.pages()[2] = torch.randn(H, d, d, generator=torch.Generator().manual_seed(2))
    table = torch.tensor([[2], [0], [1]], dtype=torch.int32).expand(3, blocks).contiguous()
    rows = sum(new)
    q, k, v, dec, _ = G.inputs(rows, H, H, d, d, "bf16", "token", 14)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    a = [x.cuda() for x in (q, k, v, dec)]
    kept = [R.linear(P.pages()[2].double(), q[:n], k[:n], v[:n], dec[:n], 0.1, (n,))[2][n][0],
            R.linear(torch.zeros(H, d, d, dtype=torch.float64), q[n:], k[n:], v[n:], dec[n:], 0.1, (33,))[2][33][0]]
    for _ in range(20):
        pool, out, status = P.pool.cuda(), torch.zeros(rows, H, d, dtype=torch.bfloat16, device=DEV), flag()
        lmc.lmc_linear_scan(P.layout, P.layer, pool, table.cuda(), ints(start.tolist()), ints(had), *a, out,
                            workspace(P, 3, rows)[0], status, scale=0.1)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        got = P.pages(pool.cpu())
        for b, S in ((2, kept[0]), (0, kept[1])):
            assert float((got[b].double() - S).norm()) <= 2.0 ** -18 * float(S.norm()), b
        assert bool(torch.isnan(got[[1, 3]]).all())


# ---- digits of the states ------------------------------------------------------------

def _by_weights(k, v, g, n):
    """The states after n tokens of one decay g per head: sums of k v^T times exp(g
    (tokens since)), in 64 bits. k [T, dk] of all heads, v [T, H, dv]."""
    since = torch.arange(n - 1, -1, -1, dtype=torch.float64, device=v.device)
    return torch.stack([(k[:n].double() * torch.exp(float(g[h]) * since)[:, None]).t() @ v[:n, h].double()
                        for h in range(v.shape[1])])


def _off(got, want):
    """Per head: the difference's 2-norm over the state's."""
    return (got.double().cpu() - want.cpu()).flatten(1).norm(dim=1) / want.cpu().flatten(1).norm(dim=1)


def test_a_cut_request_of_slow_decays():
    """Three segments of 5400 tiles each, a decay for all tokens of a head: what
    joins them keeps the digits of the 5400 decays' product.

    A state is rounded once a tile, by at most 2^-24 of itself and independently,
    so n tiles that all count move it by less than sqrt(n) 2^-24 in the 2-norm, with
    rounding's mean square (0.4 of the most) room for a tile's own sums. (One
    binary32 sum of a segment's decays would be off by 5e-5 for some of these heads,
    a quarter of it in the state at 786432 tokens.)"""
    H, d, n, N = 50, 8, 1 << 20, 1 << 18
    rec = H * d * d * 4
    L = lmc.lmc_layout_build([{"kind": "KDA", "conv_bytes": 16, "rec_bytes": rec}], N, False, 4 * (rec + 16))
    g = torch.Generator(device=DEV).manual_seed(6)
    q, k = ((1 + torch.randn(n, 1, d, generator=g, device=DEV)).bfloat16() for _ in range(2))
    v = torch.randn(n, H, d, generator=g, device=DEV, dtype=torch.bfloat16) + 1
    decay = -torch.logspace(-6, -5.2, H)
    decay[0] = -2.4030030090216314e-06
    pool, out, status = torch.zeros(L.pool_bytes, dtype=torch.uint8, device=DEV), torch.empty_like(v), flag()
    ws = torch.empty(lmc.lmc_linear_scan_workspace(L, 0, 1, n, H), dtype=torch.uint8, device=DEV)
    lmc.lmc_linear_scan(L, 0, pool, ints([[0, 1, 2, 3]]), ints([0, n]), ints([0]), q, k, v, decay.cuda()[None].expand(n, H),
                        out, ws, status, scale=1e-6)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for b in range(4):
        at = L.base[0] + b * L.stride[0] + 16
        S = pool[at:at + rec].view(torch.float32).view(H, d, d)
        off = _off(S, _by_weights(k[:, 0], v, decay, (b + 1) * N))
        assert float(off.max()) <= ((b + 1) * N / 64) ** 0.5 * 2.0 ** -24, (b, int(off.argmax()), float(off.max()))


@pytest.mark.parametrize("op", ["scan", "step"])
def test_states_of_slow_decays(op):
    """Thousands of decays near 1, the same for all tokens of a head, as prompts and
    as steps. One rounding of the state a tile or step, as above; a decay rounded to
    binary32 would make it sum to 2^-25 a time, the same way every time."""
    H, d = 152, 8
    n = 25600 if op == "scan" else 4096
    N, rec = n, H * d * d * 4
    L = lmc.lmc_layout_build([{"kind": "KDA", "conv_bytes": 16, "rec_bytes": rec}], N, False, 2 * (rec + 16))
    g = torch.Generator(device=DEV).manual_seed(7)
    q, k = ((1 + torch.randn(n, 1, d, generator=g, device=DEV)).bfloat16() for _ in range(2))
    v = torch.randn(n, H, d, generator=g, device=DEV, dtype=torch.bfloat16) + 1
    decay = -2.0 ** torch.linspace(-15, -13, H) if op == "scan" else -2.0 ** torch.linspace(-13, -11, H)
    far = decay.cuda()[None].expand(n, H)
    pool, out, status = torch.zeros(L.pool_bytes, dtype=torch.uint8, device=DEV), torch.empty_like(v), flag()
    if op == "scan":
        ws = torch.empty(lmc.lmc_linear_scan_workspace(L, 0, 1, n, H), dtype=torch.uint8, device=DEV)
        lmc.lmc_linear_scan(L, 0, pool, ints([[1]]), ints([0, n]), ints([0]), q, k, v, far, out, ws, status, scale=1e-4)
    else:
        lengths, table = torch.arange(n, dtype=torch.int32, device=DEV), ints([[1]])
        for t in range(n):
            s = slice(t, t + 1)
            lmc.lmc_linear_step(L, 0, pool, table, lengths[s], q[s], k[s], v[s], far[s], out[s], status, scale=1e-4)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    at = L.base[0] + L.stride[0] + 16
    S = pool[at:at + rec].view(torch.float32).view(H, d, d)
    off = _off(S, _by_weights(k[:, 0], v, decay, n))
    assert float(off.max()) <= (n / 64 if op == "scan" else n) ** 0.5 * 2.0 ** -24, (int(off.argmax()), float(off.max()))


@pytest.mark.parametrize("op", ["scan", "step"])
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("decay", ["token", "head", "resets"])
@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (24, 40)])
def test_states_keep_binary32s_digits(dims, decay, act, op):
    """One to three tiles behind a state, and a step.

    A step's product, decay and sums are off by a few 2^-24, not alike: below 2^-21 of
    the state in the 2-norm. A tile's products of 16 tokens are added up part by part,
    the large part's last, and the tensor cores cut each of those four sums off below
    binary32's last place, by up to 2^-23 of it, half of that on average, all of them
    the same way: 2^-22; decays and the parts' own steps add less than half of that.
    (Three bf16 parts of a value times its decay would be off by 2^-18.7; the large
    part's sums first, by 2^-21.)"""
    H, N = 3, 200
    had, new = ([0, 30, 7, 190], [64, 170, 1, 10]) if op == "scan" else ([0, 30, 7, 190], [1, 1, 1, 1])
    P = R.States(lmc, H, *dims, N, 6)
    table = R.tables(had, new, N, 6, np.random.default_rng(0))
    g = torch.Generator().manual_seed(3)
    for r, h in enumerate(had):
        if h:
            P.pages()[int(table[r, (h - 1) // N])] = torch.randn(H, *dims, generator=g)
    rows = sum(new)
    q, k, v, dec, _ = G.inputs(rows, H, H, *dims, act, decay, 4)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    pool, out, status = P.pool.cuda(), torch.zeros(rows, H, dims[1], dtype=R.TYPES[act], device=DEV), flag()
    a = [x.cuda() for x in (q, k, v)] + [dec.contiguous().cuda()]
    if op == "scan":
        lmc.lmc_linear_scan(P.layout, P.layer, pool, table.cuda(), ints(start.tolist()), ints(had), *a, out,
                            workspace(P, len(new), rows)[0], status, scale=0.1)
    else:
        lmc.lmc_linear_step(P.layout, P.layer, pool, table.cuda(), ints(had), *a, out, status, scale=0.1)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    got = P.pages(pool.cpu())
    for r, (h, t) in enumerate(zip(had, new)):
        s = slice(int(start[r]), int(start[r]) + t)
        S0 = P.pages()[int(table[r, (h - 1) // N])].double() if h else torch.zeros(H, *dims, dtype=torch.float64)
        _, _, kept = R.linear(S0, q[s], k[s], v[s], dec[s], 0.1, (t,))
        off = _off(got[int(table[r, (h + t - 1) // N])], kept[t][0])
        assert float(off.max()) <= (1.5 * 2.0 ** -22 if op == "scan" else 2.0 ** -21), (r, off.tolist())


# ---- f16 -----------------------------------------------------------------------------

@pytest.mark.parametrize("n", [20, 64, 200])
@pytest.mark.parametrize("forgotten", [-float("inf"), -60.0])
def test_f16_weights_beside_a_forgotten_tokens(n, forgotten):
    """A first token whose product with every query is 2^32 times the others', and is
    forgotten by the second: the others' weights keep f16's digits. As many independent
    roundings of half a step: their 2-norm stays below one."""
    H, d, N = 2, 64, 256
    q, k, v, dec, _ = G.inputs(n, H, H, d, d, "f16", "token", 12)
    q, k = q * 16, (k.float() * 2.0 ** -16).half()  # (k: randn / 8)
    k[0] = (torch.randn(H, d, generator=torch.Generator().manual_seed(1)) * 2.0 ** 13).half()
    v[0] = (v[0].float() * 2.0 ** -22).half()
    dec[1] = forgotten
    P = R.States(lmc, H, d, d, N, 2)
    pool, out, status = P.pool.cuda(), torch.full((n, H, d), float("nan"), dtype=torch.float16, device=DEV), flag()
    lmc.lmc_linear_scan(P.layout, P.layer, pool, ints([[1]]), ints([0, n]), ints([0]), *[x.cuda() for x in (q, k, v, dec)],
                        out, workspace(P, 1, n)[0], status, scale=2.0 ** 12)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    o, _, _ = R.linear(torch.zeros(H, d, d, dtype=torch.float64), q, k, v, dec, 2.0 ** 12)
    assert 1e-2 < float(o[1:].abs().mean()) and float(o.abs().max()) < 65504
    assert float((out.cpu().double() - o)[1:].norm()) <= R.HALF_STEP["f16"] * float(o[1:].norm())


@pytest.mark.parametrize("n", [1, 20, 37, 64])
def test_f16_rows_of_other_requests_do_not_leak(n):
    """NaN, infinities and the largest values in the next request's rows, which lie in the
    same tile's boxes, change no bit of a request's results and states."""
    H, d, N, new = 2, 64, 48, [n, 70, 41]
    rows = sum(new)
    q, k, v, dec, _ = G.inputs(rows, H, H, d, d, "f16", "resets", 2)
    start, got = np.concatenate([[0], np.cumsum(new)]).astype(np.int32), []
    for bad in (None, 65504.0, float("inf"), float("nan")):
        if bad is not None:
            for x in (q, k, v):
                x[n:n + 70] = bad
            dec[n:n + 70] = -1e30 if bad == 65504.0 else bad
        P = R.States(lmc, H, d, d, N, 8)
        pool, out, status = P.pool.cuda(), torch.zeros(rows, H, d, dtype=torch.float16, device=DEV), flag()
        lmc.lmc_linear_scan(P.layout, P.layer, pool, ints([[0, 7, -1], [1, 2, 3], [4, 5, 6]]), ints(start.tolist()),
                            ints([0, 0, 0]), *[x.cuda() for x in (q, k, v, dec)], out, workspace(P, 3, rows)[0], status, scale=0.1)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        got.append((out.cpu(), P.pages(pool.cpu()).clone()))
    for out, pages in got[1:]:
        for s in (slice(0, n), slice(n + 70, rows)):
            assert torch.equal(got[0][0][s], out[s])
        assert torch.equal(got[0][1][[0, 4]], pages[[0, 4]])
