"""Token operators on the GPU where they are easily got wrong: host threads
side by side."""
import threading

import numpy as np
import pytest
import torch

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
