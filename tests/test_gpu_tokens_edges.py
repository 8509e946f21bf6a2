"""Token operators on the GPU where they are easily got wrong: host threads
side by side and the ends of the types' ranges."""
import threading

import numpy as np
import pytest
import torch

import token_reference as T

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture()
def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _int32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).to(DEV)


def test_select_from_four_threads(lmc):
    """Four host threads, each on its own stream, select from rows of very
    different lengths at once: every call is accepted and gives what it gives
    alone."""
    jobs = []
    for k, tokens in enumerate((131_072, 100, 40_000, 600_001)):
        x = torch.rand((1, 1, tokens), device=DEV, generator=torch.Generator(DEV).manual_seed(k))
        jobs.append((x, _int32([tokens]), tokens // 3))

    def call(job, stream=None):
        x, lengths, budget = job
        kept = torch.full((1, 1, budget), -7, dtype=torch.int32, device=DEV)
        kl, status = _int32([-7]), _int32([0])
        lmc.lmc_select_tokens(x, lengths, budget, 5, kept, None, kl, status, stream=stream)
        return kept, kl, status

    want = [call(j)[0] for j in jobs]
    torch.cuda.synchronize()
    failures, start = [], threading.Barrier(len(jobs))

    def work(k):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                start.wait()
                got = [call(jobs[k]) for _ in range(300)]
                stream.synchronize()
                for kept, kl, status in got:
                    assert torch.equal(kept, want[k]) and int(kl) == jobs[k][2] and int(status) == 0
        except Exception as e:  # noqa: BLE001 (a thread's failure is the test's)
            failures.append((k, repr(e)))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures


def _call(lmc, M, table, lengths, q, V, status, softmax_scale, scale=1.0, weights=None):
    R, H, _ = q.shape
    out = torch.full((R, H, V), 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full((R, H), 7.0, device=DEV)
    most = max(lengths)
    ws = torch.empty(lmc.lmc_attend_workspace(M.layout, M.layers[0], R, H, V, most, weights is not None),
                     dtype=torch.uint8, device=DEV)
    lmc.lmc_attend(M.layout, M.layers[0], M.pool.to(DEV), table.to(DEV), _int32(lengths), q, V, softmax_scale, out, ws,
                   status, max_length=most, scale=scale, lse=lse, weights=weights)
    assert status.item() == 0
    return out.cpu().double(), lse.cpu().double()


@pytest.mark.parametrize("act,exponent", [
    ("bf16", 126), ("bf16", 120), ("bf16", 116), ("bf16", 113), ("bf16", 0), ("bf16", -86), ("bf16", -100),
    ("bf16", -120), ("bf16", -126), ("f16", 14), ("f16", 0), ("f16", -14)])
def test_attend_fp8_queries_over_the_whole_range(lmc, status, act, exponent):
    """Queries of every size that the type has, with a softmax_scale that brings
    the logits back near one: over an fp8 cache, whose queries are held as f16
    times a power of two. Heads of one call lie far apart, too."""
    rng = np.random.default_rng(exponent + 200)
    N, E, V, H, n = 64, 64, 32, 6, 150
    M = T.Model(lmc, E, "e4m3", N, blocks=3)
    table = T.tables([n], N, 3, rng)
    M.write(0, table, 0, 0, torch.from_numpy(rng.standard_normal((n, E))))
    # at most 1.75 times 2^exponent: finite in every case
    q = torch.from_numpy(np.clip(rng.standard_normal((1, H, E)), -1.75, 1.75)) * 2.0 ** exponent
    q[:, 4] *= 2.0 ** -20 if act == "bf16" and exponent > 0 else 1.0
    q[:, 5] = 0.0
    q = q.to(T.TYPES[act])
    # |x| is about 8 here; softmax_scale stays a normal number
    softmax_scale = 2.0 ** max(-exponent, -126)
    out, lse = _call(lmc, M, table, [n], q.to(DEV), V, status, softmax_scale)
    o, l, _, d_o, d_l, _ = T.attend(M.read(0, table, 0, list(range(n))), q[0].double(), V, softmax_scale, 1.0, "e4m3",
                                    act)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert ((out[0] - o).abs() <= d_o).all(), float((out[0] - o).abs().max())
    assert ((lse[0] - l).abs() <= d_l).all(), float((lse[0] - l).abs().max())
