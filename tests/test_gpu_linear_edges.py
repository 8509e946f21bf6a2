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
