"""Token operators on the GPU where they are easily got wrong: host threads
side by side, the ends of the types' ranges, values that are not finite, the
calls from C, and the largest sizes."""
import math
import os
import shutil
import subprocess
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


@pytest.mark.parametrize("n", [100, 5000])
@pytest.mark.parametrize("cache", ["bf16", "f16"])
def test_attend_infinite_keys(lmc, status, cache, n):
    """One key with an infinity among its last values: a head that it gives a
    logit of -inf goes on without that token, one that it gives +inf has no
    softmax (NaN). n = 5000: the request is shared by several CTAs."""
    rng = np.random.default_rng(n)
    N, E, V, H = 64, 64, 32, 4
    blocks = -(-n // N)
    M = T.Model(lmc, E, cache, N, blocks=blocks)
    table = T.tables([n], N, blocks, rng)
    e = torch.from_numpy(rng.standard_normal((n, E)))
    e[n // 2, 40] = math.inf
    M.write(0, table, 0, 0, e)
    q = torch.from_numpy(rng.standard_normal((1, H, E)))
    q[0, :, 40] = torch.tensor([1.0, -1.0, -2.0, 0.5])
    q = q.to(T.TYPES[cache])
    out, lse = _call(lmc, M, table, [n], q.to(DEV), V, status, 0.125)
    at = [t for t in range(n) if t != n // 2]
    o, l, _, d_o, d_l, _ = T.attend(M.read(0, table, 0, at), q[0].double(), V, 0.125, 1.0, cache, cache)
    for h in (1, 2):
        assert ((out[0, h] - o[h]).abs() <= d_o[h]).all() and abs(lse[0, h] - l[h]) <= d_l[h]
    for h in (0, 3):
        assert torch.isnan(out[0, h]).all() and torch.isnan(lse[0, h])
    # with weights, the heads that have a softmax alone; then one that has none
    weights = torch.zeros((1, n), device=DEV)
    _call(lmc, M, table, [n], q[:, 1:3].contiguous().to(DEV), V, status, 0.125, weights=weights)
    assert weights[0, n // 2] == 0 and abs(float(weights.double().sum()) - 2) < 1e-4
    _call(lmc, M, table, [n], q[:, :3].contiguous().to(DEV), V, status, 0.125, weights=weights)
    assert torch.isnan(weights).all()


@pytest.mark.parametrize("n", [100, 5000])
@pytest.mark.parametrize("cache,act", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")])
def test_attend_heads_whose_logits_are_all_minus_infinity(lmc, status, cache, act, n):
    """Such a head is as one without tokens: zeros, lse of -inf, nothing added
    to the weights, whatever other finite values its query holds (an fp8 cache
    holds the query as f16: what f16 cannot hold must not become an infinity
    of its own, which would make NaN beside the other)."""
    rng = np.random.default_rng(n)
    N, E, V, H = 64, 64, 32, 3
    blocks = -(-n // N)
    M = T.Model(lmc, E, cache, N, blocks=blocks)
    table = T.tables([n], N, blocks, rng)
    e = torch.from_numpy(rng.standard_normal((n, E)))
    e[:, 40], e[:, 41] = 1.0, 1.0
    M.write(0, table, 0, 0, e)
    q = torch.from_numpy(rng.standard_normal((1, H, E)))
    q[0, 0, 40], q[0, 0, 41] = -math.inf, 6e4 if act == "f16" else 1e30
    q[0, 1, 40] = -math.inf
    q = q.to(T.TYPES[act])
    before = torch.from_numpy(rng.random((1, n))).float()
    weights = before.to(DEV)
    out, lse = _call(lmc, M, table, [n], q.to(DEV), V, status, 0.125, weights=weights)
    assert (out[0, :2] == 0).all() and (lse[0, :2] == -math.inf).all()
    o, l, w, d_o, d_l, d_w = T.attend(M.read(0, table, 0, list(range(n))), q[0, 2:].double(), V, 0.125, 1.0, cache, act)
    assert ((out[0, 2:] - o).abs() <= d_o).all() and abs(lse[0, 2] - l[0]) <= d_l[0]
    added = weights[0].cpu().double() - before[0].double()
    # (the sum with what was there before is rounded once: at most half a step of 2)
    assert ((added - w).abs() <= d_w + 2.0 ** -23).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_attend_nan_just_before_a_window(lmc, status, cache):
    """Tokens before the window, in the window's first tile too, do not show."""
    rng = np.random.default_rng(2)
    N, E, V, H, n, window = 64, 64, 32, 4, 300, 70
    M = T.Model(lmc, E, cache, N, window=window, blocks=5)
    table = T.tables([n], N, 5, rng)
    e = torch.from_numpy(rng.standard_normal((n, E)))
    e[:n - window] = math.nan
    M.write(0, table, 0, 0, e)
    q = torch.from_numpy(rng.standard_normal((1, H, E))).to(torch.bfloat16)
    out, lse = _call(lmc, M, table, [n], q.to(DEV), V, status, 0.125)
    o, l, _, d_o, d_l, _ = T.attend(M.read(0, table, 0, list(range(n - window, n))), q[0].double(), V, 0.125, 1.0,
                                    cache, "bf16")
    assert ((out[0] - o).abs() <= d_o).all() and ((lse[0] - l).abs() <= d_l).all()


def test_token_operators_from_c(lmc, tmp_path):
    """A C11 program (tests/c_abi_tokens_client.c) makes the four calls through
    the C ABI alone; its results against the 64-bit forms."""
    here = os.path.dirname(os.path.abspath(__file__))
    root = os.path.dirname(here)
    cuda = next((d for d in (os.environ.get("CUDA_HOME"), "/usr/local/cuda")
                 if d and os.path.exists(os.path.join(d, "include", "cuda_runtime.h"))), None)
    if shutil.which("gcc") is None or cuda is None:
        pytest.skip("gcc or the CUDA toolkit headers not available")
    exe, libdir = tmp_path / "tokens_client", os.path.join(root, "state_cache_paging_gb300")
    subprocess.run(["gcc", "-std=c11", "-pedantic", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(root, "include"),
                    "-I", os.path.join(cuda, "include"), os.path.join(here, "c_abi_tokens_client.c"), "-o", str(exe),
                    f"-L{libdir}", "-llmc", f"-L{os.path.join(cuda, 'lib64')}", "-lcudart", "-lm",
                    f"-Wl,-rpath,{libdir}", f"-Wl,-rpath,{os.path.join(cuda, 'lib64')}"],
                   check=True, capture_output=True, text=True)
    N, E, V, H, n, budget, recent = 64, 192, 128, 5, 500, 96, 32
    rng = np.random.default_rng(6)
    rows = torch.from_numpy(rng.standard_normal((n, E))).bfloat16()
    q = torch.from_numpy(rng.standard_normal((H, E))).bfloat16()
    (tmp_path / "case.txt").write_text(f"{N} {E} {V} {H} {n} {budget} {recent}\n")
    rows.view(torch.int16).numpy().tofile(tmp_path / "rows.bin")
    q.view(torch.int16).numpy().tofile(tmp_path / "q.bin")
    r = subprocess.run([str(exe), str(tmp_path)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stdout + r.stderr

    def read(name, dtype):
        return torch.from_numpy(np.fromfile(tmp_path / name, dtype=dtype))

    assert (tmp_path / "status.out").read_text().split() == ["0", str(budget)]
    scale = float(np.float32(1.0) / np.sqrt(np.float32(E)))
    o, l, w, d_o, d_l, d_w = T.attend(rows.double(), q.double(), V, scale, 1.0, "bf16", "bf16")
    out = read("out.out", np.int16).view(torch.bfloat16).view(H, V).double()
    assert ((out - o).abs() <= d_o).all()
    assert ((read("lse.out", np.float32).double() - l).abs() <= d_l).all()
    weights = read("weights.out", np.float32)
    assert ((weights.double() - w).abs() <= d_w).all()
    want = T.select(weights.tolist(), n, budget, recent)  # by the weights as the kernel accumulated them
    assert read("kept.out", np.int32).tolist() == want
    assert torch.equal(read("scores.out", np.float32), weights[want])
    moved = read("moved.out", np.int16).view(torch.bfloat16).view(budget, E)
    assert torch.equal(moved.view(torch.int16), rows[want].view(torch.int16))


# Sixteen values a token, all below 6: logits are below 16. In units of log 2 the
# sum of products (8 of absolute value) is off by 8 * 1.45 * 2^-22 at most, the two
# roundings behind it by 16 * 1.45 * 2^-24 each, the exponential by 2^-20: together
# 2^-17, and the same again in lse.
OFF = 2.0 ** -16
# p and the result in f16: half a step each
OUT_OFF = 6 * (2.0 ** -10 + OFF) + 2.0 ** -24


def _plain(entries, q, V, softmax_scale):
    """[R, T, E] and [R, H, E] in 64 bits, none of a request's tokens left out."""
    x = torch.einsum("rhe,rte->rht", q, entries) * softmax_scale
    return torch.softmax(x, -1) @ entries[:, :, :V], torch.logsumexp(x, -1), torch.softmax(x, -1).sum(1)


def test_attend_of_the_most_requests(lmc, status):
    """65535 requests of up to three tokens over shared blocks, one of them of
    a thousand: walked, shared out and joined."""
    g = torch.Generator().manual_seed(1)
    N, E, V, R, long = 16, 16, 8, 65535, 1000
    blocks = 64
    L = lmc.lmc_layout_build([{"kind": "MLA", "token_bytes": 2 * E}], N, False, blocks * N * E * 2)
    entries = torch.randn((blocks, N, E), generator=g).half()
    pool = entries.to(DEV).view(torch.uint8).flatten()
    lengths = torch.randint(0, 4, (R,), generator=g).int()
    at = 40_000
    lengths[at] = long
    table = torch.randint(0, blocks, (R, 1), generator=g).int().repeat(1, 63)
    table[at] = torch.randperm(blocks, generator=g)[:63].int()
    q = torch.randn((R, 1, E), generator=g).half()
    out, lse = torch.full((R, 1, V), 7.0, dtype=torch.half, device=DEV), torch.full((R, 1), 7.0, device=DEV)
    weights = torch.zeros((R, long), device=DEV)
    ws = torch.empty(lmc.lmc_attend_workspace(L, 0, R, 1, V, long, True), dtype=torch.uint8, device=DEV)
    lmc.lmc_attend(L, 0, pool, table.to(DEV), lengths.to(DEV), q.to(DEV), V, 0.25, out, ws, status, max_length=long,
                   lse=lse, weights=weights)
    assert status.item() == 0
    out, lse, weights = out.cpu().double(), lse.cpu().double(), weights.cpu().double()
    for n in (0, 1, 2, 3, long):
        at_n = torch.nonzero(lengths == n).flatten()
        if n == 0:
            assert (out[at_n] == 0).all() and (lse[at_n] == -math.inf).all() and (weights[at_n] == 0).all()
            continue
        e = entries[table[at_n, :-(-n // N)].long()].reshape(len(at_n), -1, E)[:, :n].double()
        o, l, w = _plain(e, q[at_n].double(), V, 0.25)
        assert float((out[at_n] - o).abs().max()) <= OUT_OFF
        assert float((lse[at_n] - l).abs().max()) <= OFF
        assert float((weights[at_n, :n] - w).abs().max()) <= OFF and (weights[at_n, n:] == 0).all()


@pytest.mark.parametrize("H", [9999, 65535])
def test_attend_of_more_heads_than_the_device_has_groups_for(lmc, status, H):
    g = torch.Generator().manual_seed(H)
    N, E, V, n = 64, 16, 8, 200
    L = lmc.lmc_layout_build([{"kind": "MLA", "token_bytes": 2 * E}], N, False, 4 * N * E * 2)
    entries = torch.randn((4 * N, E), generator=g).half()
    q = torch.randn((2, H, E), generator=g).half()
    out, lse = torch.full((2, H, V), 7.0, dtype=torch.half, device=DEV), torch.full((2, H), 7.0, device=DEV)
    ws = torch.empty(lmc.lmc_attend_workspace(L, 0, 2, H, V, 4 * N, True), dtype=torch.uint8, device=DEV)
    lengths = [n, 70]
    for most in (n, 4 * N):
        weights = torch.zeros((2, most), device=DEV)
        lmc.lmc_attend(L, 0, entries.to(DEV).view(torch.uint8).flatten(), _int32([[0, 1, 2, 3]] * 2), _int32(lengths),
                       q.to(DEV), V, 0.25, out, ws, status, max_length=most, lse=lse, weights=weights)
        assert status.item() == 0
        for r, k in enumerate(lengths):
            o, l, w = _plain(entries[None, :k].double(), q[r:r + 1].double(), V, 0.25)
            assert float((out[r].cpu().double() - o[0]).abs().max()) <= OUT_OFF
            assert float((lse[r].cpu().double() - l[0]).abs().max()) <= OFF
            # H terms, each off by OFF of itself at most, added in binary32
            got = weights[r].cpu().double()
            assert float(((got[:k] - w[0]).abs() / w[0]).max()) <= OFF + H * 2.0 ** -24 and (got[k:] == 0).all()


def test_attend_weights_in_turns_behind_a_window(lmc, status):
    """400 requests that could have 26 blocks' tokens each, one more than their
    share of the grid; windows that begin on odd tokens."""
    rng = np.random.default_rng(13)
    N, E, V, H, R, window = 64, 16, 8, 2, 400, 6400
    lengths = [6401, 6500, 6400, 12_801] + [int(x) for x in rng.integers(0, 70, R - 4)]
    blocks = sum(-(-n // N) for n in lengths)
    M = T.Model(lmc, E, "f16", N, window=window, blocks=blocks)
    raw = torch.from_numpy(rng.standard_normal((blocks, N, E))).half()
    M.pages(0).copy_(raw.view(torch.uint8))
    table = T.tables(lengths, N, blocks, rng)
    q = torch.from_numpy(rng.standard_normal((R, H, E))).half()
    before = torch.from_numpy(rng.random((R, max(lengths)))).float()
    weights = before.to(DEV)
    _call(lmc, M, table, lengths, q.to(DEV), V, status, 0.25, weights=weights)
    got = weights.cpu()
    for r, n in enumerate(lengths):
        lo = max(0, n - window)
        assert torch.equal(got[r, :lo], before[r, :lo]) and torch.equal(got[r, n:], before[r, n:])
        if n:
            _, _, w, _, _, d_w = T.attend(M.read(0, table, r, list(range(lo, n))), q[r].double(), V, 0.25, 1.0, "f16", "f16")
            want = before[r, lo:n].double() + w
            assert ((got[r, lo:n].double() - want).abs() <= d_w + want * 2.0 ** -23).all(), r


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
def test_attend_of_three_hundred_million_tokens(lmc, status, cache):
    """One request whose entries take more than 2^32 bytes: a value that is 1 in
    the tokens of every fourth page, the others' 0, and a last token that all
    of one head's weight falls on."""
    N, V, H, n = 1000, 8, 2, 300_000_007
    E = 16
    elem = 2 if cache == "f16" else 1
    blocks = -(-n // N)
    L = lmc.lmc_layout_build([{"kind": "MLA", "token_bytes": E * elem}], N, False, blocks * N * E * elem)
    pool = torch.zeros(L.pool_bytes, dtype=torch.uint8, device=DEV)
    one = torch.ones((1,), device=DEV).to(T.TYPES[cache])
    # the table is the blocks in reverse: page k of the request lies in block blocks - 1 - k
    table = torch.arange(blocks - 1, -1, -1, dtype=torch.int32, device=DEV)[None]
    raw = pool.view(torch.int16 if elem == 2 else torch.uint8).view(blocks, N, E)
    raw[torch.arange(blocks - 1, -1, -4, device=DEV), :, 0] = one.view(raw.dtype)
    last = raw[blocks - 1 - (n - 1) // N, (n - 1) % N]
    last[0], last[1], last[15] = 0, one.view(raw.dtype), (one.float() * 64).to(T.TYPES[cache]).view(raw.dtype)
    q = torch.zeros((1, H, E), dtype=torch.half, device=DEV)
    q[0, 1, 15] = 1.0
    out, lse = torch.empty((1, H, V), dtype=torch.half, device=DEV), torch.empty((1, H), device=DEV)
    ws = torch.empty(lmc.lmc_attend_workspace(L, 0, 1, H, V, n), dtype=torch.uint8, device=DEV)
    lmc.lmc_attend(L, 0, pool, table, _int32([n]), q, V, 1.0, out, ws, status, max_length=n, lse=lse)
    assert status.item() == 0
    ones = ((blocks + 3) // 4 - (1 if (blocks - 1) % 4 == 0 else 0)) * N
    ones += (n - (blocks - 1) * N - 1) if (blocks - 1) % 4 == 0 else 0
    got = out[0].cpu().double()
    # sums of whole numbers that one thread holds stay below 2^24; parts are joined in binary32; the result is f16
    assert abs(float(got[0, 0]) - ones / n) <= ones / n * (2.0 ** -11 + 2.0 ** -16)
    assert (got[0, 2:] == 0).all() and float(got[0, 1]) <= 2.0 ** -24
    assert abs(float(lse[0, 0]) - math.log(n)) <= 2.0 ** -16
    # the others' n - 1 weigh e^-64 each
    assert float(got[1, 1]) == 1.0 and (got[1, [0, 2, 3, 4, 5, 6, 7]] == 0).all()
    assert abs(float(lse[0, 1]) - 64.0) <= 2.0 ** -16
