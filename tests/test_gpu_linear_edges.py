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
