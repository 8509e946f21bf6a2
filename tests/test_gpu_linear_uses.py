"""Linear attention, rotations and the calls beside them as they are used:
together, from C, in graphs and on several streams, over other layouts of the
same tensors, at the ends of the ranges."""
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import linear_reference as R
import state_cache_paging_gb300 as lmc
import test_gpu_linear as G
import token_reference as T

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def flag():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def workspace(P, requests, rows, guard=0):
    n = lmc.lmc_linear_scan_workspace(P.layout, P.layer, requests, rows, P.H)
    return torch.full((n + 2 * guard,), 0xA5, dtype=torch.uint8, device=DEV), n


# ---- together -------------------------------------------------------------------

@pytest.fixture(scope="module")
def hybrid():
    import example_hybrid
    torch.manual_seed(11)
    return example_hybrid.run(DEV)


def test_hybrid_linear_layer(hybrid):
    """Scan, steps and the scan from the restored snapshot, four of 32 heads."""
    x = hybrid
    assert x["status"] == 0
    h = slice(0, 32, 10)
    q, k, v, d = (x[n].cpu()[:, h] for n in ("q", "k", "v", "decay"))
    n = q.shape[0]
    o, mag, kept = R.linear(torch.zeros(4, 128, 128, dtype=torch.float64), q, k, v, d, 128 ** -0.5, (x["N"], n))
    half = R.HALF_STEP["bf16"]
    for got, want, m in ((x["o"].cpu()[:, h], o, mag), (x["o2"].cpu()[:, h], o[x["N"]:], mag[x["N"]:])):
        err = (got.double() - want).abs()
        # the result's rounding and those of the weights inside a tile; sums and decays in binary32
        assert bool((err <= half * want.abs() + m * (half + (n + 256) * 2.0 ** -23 + 2.0 ** -14)).all())
        assert float(err.norm()) <= half * float(want.norm())
    # the states after the prompt's first block (stored, loaded) and after all tokens, in both pools
    L, g = x["layout"], x["layout"].kv_group[0]
    for pool, tables in ((x["pool"], x["tables"]), (x["fresh"], x["others"])):
        for n, position in ((x["N"], 0), (n, 1)):
            at = L.base[0] + int(tables[g][0, position]) * L.stride[0] + 12288 * 3 * 2
            S = pool[at:at + 32 * 128 * 128 * 4].view(torch.float32).view(32, 128, 128)[h].cpu().double()
            assert float((S - kept[n][0]).norm()) <= 2.0 ** -18 * float(kept[n][0].norm())


def test_hybrid_attention_layer(hybrid):
    """Entries against the 64-bit norm and rotation; attention over the entries as they lie."""
    x, half = hybrid, R.HALF_STEP["bf16"]
    L, n = x["layout"], x["entries"].shape[0]
    want, lost = R.turned(x["entries"].cpu()[:, None], 512, x["norm"].cpu(), 1e-6, torch.arange(n), x["freqs"].cpu(), 512,
                          True, 1.0)
    for pool, tables, outs in ((x["pool"], x["tables"], x["a"]), (x["fresh"], x["others"], x["a2"])):
        rows = []
        for position, m in ((0, x["N"]), (1, n - x["N"])):
            at = L.base[3] + int(tables[L.kv_group[3]][0, position]) * L.stride[3]
            rows.append(pool[at:at + m * 1152].view(torch.bfloat16).view(m, 576).cpu())
        rows = torch.cat(rows)
        err = (rows.double() - want[:, 0]).abs()
        assert bool((err <= half * want[:, 0].abs() + (1 + half) * lost[:, 0]).all())
        first = n - outs.shape[0]
        for i in range(outs.shape[0]):
            m = first + i + 1
            o, _, _, d_o, _, _ = T.attend(rows[:m].double(), x["aq"][m - 1].cpu().double(), 512, 192 ** -0.5, 1.0, "bf16",
                                          "bf16")
            assert bool(((outs[i].cpu().double() - o).abs() <= d_o).all())


def test_a_captured_decode_step_of_both_layers():
    """Rotation in place, append, attention and a state's step in one graph,
    replayed with new inputs in the same memory: the bits of the eager calls."""
    H, N, steps = 4, 64, 5
    layers = [{"kind": "KDA", "conv_bytes": 48, "rec_bytes": H * 64 * 64 * 4}, {"kind": "MLA", "token_bytes": 1152}]
    L = lmc.lmc_layout_build(layers, N, False, 16 * N * 1152)
    assert L.num_blocks == 16
    g = torch.Generator(device=DEV).manual_seed(1)
    draw = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()  # noqa: E731
    had = [0, 61, 130]
    # (a block's pages of both layers are the same memory)
    table, latents = ints([[6, -1, -1], [0, 1, -1], [-1, 2, 3]]), ints([[8, -1, -1], [9, 10, -1], [11, 12, 13]])
    freqs = 10000.0 ** (-torch.arange(32, device=DEV) / 32)
    fresh = draw(L.pool_bytes // 2).view(torch.uint8)  # (two bf16 numbers are a binary32 number near the second)
    new = [(draw(3, H, 576), draw(3, 576), draw(3, H, 64), draw(3, H, 64), draw(3, H, 64),
            -torch.rand(3, H, generator=g, device=DEV)) for _ in range(steps)]
    held = [torch.empty_like(t) for t in new[0]]
    lengths, after, positions = ints(had), ints([n + 1 for n in had]), ints(had)
    ws = torch.empty(lmc.lmc_attend_workspace(L, 1, 3, H, 512, 192), dtype=torch.uint8, device=DEV)
    status, requests = flag(), ints([0, 1, 2])
    out, o = torch.empty(3, H, 512, dtype=torch.bfloat16, device=DEV), torch.empty(3, H, 64, dtype=torch.bfloat16, device=DEV)

    def step(pool):
        aq, e, q, k, v, d = held
        lmc.lmc_rotate(aq, positions, aq, freqs, rot_first=512)
        lmc.lmc_append_rotated(L, 1, pool, latents, requests, positions, e, status, freqs, rot_first=512, norm_dim=512)
        lmc.lmc_attend(L, 1, pool, latents, after, aq, 512, 0.07, out, ws, status, max_length=192)
        lmc.lmc_linear_step(L, 0, pool, table, lengths, q, k, v, d, o, status, scale=0.125)

    def all_steps(call, pool):
        got = []
        for x in (lengths, after, positions):
            x.copy_(ints(had) + (x is after))
        for x in new:
            for to, t in zip(held, x):
                to.copy_(t)
            call()
            got += [out.clone(), o.clone()]
            for c in (lengths, after, positions):
                c.add_(1)
        return got + [pool.clone()]

    pool = fresh.clone()
    eager = all_steps(lambda: step(pool), pool)
    pool2 = fresh.clone()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        step(pool2)
    torch.cuda.synchronize()
    pool2.copy_(fresh)
    again = all_steps(graph.replay, pool2)
    assert int(status.item()) == 0
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(eager, again))


def test_linear_calls_from_c(tmp_path):
    """A C11 program (tests/c_abi_linear_client.c): a prompt, then a token, and a
    rotation in place, through the C ABI alone."""
    here = os.path.dirname(os.path.abspath(__file__))
    root = os.path.dirname(here)
    cuda = next((d for d in (os.environ.get("CUDA_HOME"), "/usr/local/cuda")
                 if d and os.path.exists(os.path.join(d, "include", "cuda_runtime.h"))), None)
    if shutil.which("gcc") is None or cuda is None:
        pytest.skip("gcc or the CUDA toolkit headers not available")
    exe, libdir = tmp_path / "linear_client", os.path.join(root, "state_cache_paging_gb300")
    subprocess.run(["gcc", "-std=c11", "-pedantic", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(root, "include"),
                    "-I", os.path.join(cuda, "include"), os.path.join(here, "c_abi_linear_client.c"), "-o", str(exe),
                    f"-L{libdir}", "-llmc", f"-L{os.path.join(cuda, 'lib64')}", "-lcudart",
                    f"-Wl,-rpath,{libdir}", f"-Wl,-rpath,{os.path.join(cuda, 'lib64')}"],
                   check=True, capture_output=True, text=True)
    N, H, d, n = 48, 3, 64, 101
    q, k, v, dec, _ = G.inputs(n, H, H, d, d, "bf16", "token", 8)
    (tmp_path / "case.txt").write_text(f"{N} {H} {d} {n}\n")
    for name, t in (("q", q), ("k", k), ("v", v)):
        t.contiguous().view(torch.int16).numpy().tofile(tmp_path / f"{name}.bin")
    dec.contiguous().numpy().tofile(tmp_path / "decay.bin")
    freqs = (10000.0 ** (-torch.arange(d // 2) / (d // 2))).float()
    freqs.numpy().tofile(tmp_path / "frequencies.bin")
    r = subprocess.run([str(exe), str(tmp_path)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stdout + r.stderr

    def read(name):
        return torch.from_numpy(np.fromfile(tmp_path / name, dtype=np.int16)).view(torch.bfloat16).view(n, H, d).double()

    assert (tmp_path / "status.out").read_text().split() == ["0"]
    half = R.HALF_STEP["bf16"]
    o, mag, _ = R.linear(torch.zeros(H, d, d, dtype=torch.float64), q, k, v, dec, float(np.float32(0.125)))
    err = (read("out.out") - o).abs()
    assert bool((err <= half * o.abs() + mag * (half + (n + 256) * 2.0 ** -23 + 2.0 ** -14)).all())
    want, lost = R.turned(q, 0, None, 1e-6, torch.arange(n), freqs, 0, False, 1.0)
    assert bool(((read("turned.out") - want).abs() <= half * want.abs() + (1 + half) * lost).all())


# ---- other layouts of the same tensors: the same bits ------------------------------

def _like(t, order, pad, offset):
    """t's values in memory of another order, with `pad` elements behind each row,
    `offset` elements from an aligned address."""
    rows, heads, dim = t.shape
    if order == "heads":  # heads of rows
        x = torch.full((heads * (rows * (dim + pad)) + offset + 64,), 7.0, dtype=t.dtype, device=DEV)
        y = torch.as_strided(x, t.shape, (dim + pad, rows * (dim + pad), 1), offset)
    else:
        x = torch.full((rows * (heads * dim + pad) + offset + 64,), 7.0, dtype=t.dtype, device=DEV)
        y = torch.as_strided(x, t.shape, (heads * dim + pad, dim, 1), offset)
    y.copy_(t)
    return y


@pytest.mark.parametrize("op", ["scan", "step"])
@pytest.mark.parametrize("order,pad,offset", [("heads", 0, 0), ("heads", 8, 16), ("rows", 8, 0), ("rows", 1, 0),
                                              ("heads", 3, 1), ("rows", 0, 1)])
@pytest.mark.parametrize("dv", [64, 104])
def test_layouts_of_inputs_and_results(order, pad, offset, dv, op):
    H, Hk, dk, N = 6, 3, 72, 80
    had, new = ([30, 0, 79], [1, 1, 1]) if op == "step" else ([30, 0, 80], [130, 64, 3])
    rows = sum(new)
    q, k, v, dec, _ = G.inputs(rows, H, Hk, dk, dv, "bf16", "token", 5)
    P = R.States(lmc, H, dk, dv, N, 12)
    P.pages()[:] = torch.randn(12, H, dk, dv, generator=torch.Generator().manual_seed(3))
    table = R.tables(had, new, N, 12, np.random.default_rng(2)).cuda()
    starts, lengths = ints(np.concatenate([[0], np.cumsum(new)]).tolist()), ints(had)
    got = []
    for other in (False, True):
        a, out = [x.cuda() for x in (q, k, v)], torch.zeros(rows, H, dv, dtype=torch.bfloat16, device=DEV)
        d = dec.cuda()
        if other:
            even = offset % 8 == 0 and pad % 8 == 0  # inputs are 16-byte aligned, results are not
            if even:
                a = [_like(x, order, pad, offset) for x in a]
            out = _like(out, order, pad, offset)
            d = d.t().contiguous().t()
        pool, status = P.pool.cuda(), flag()
        if op == "scan":
            lmc.lmc_linear_scan(P.layout, P.layer, pool, table, starts, lengths, *a, d, out, workspace(P, 3, rows)[0],
                                status, scale=0.1)
        else:
            lmc.lmc_linear_step(P.layout, P.layer, pool, table, lengths, *a, d, out, status, scale=0.1)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        got.append((out.contiguous().view(torch.int16).cpu(), pool.cpu()))
        if other:  # what lies between the rows stays
            base = torch.as_strided(out, (out.untyped_storage().nbytes() // 2,), (1,), 0).clone()
            torch.as_strided(base, out.shape, out.stride(), offset).fill_(7.0)
            assert bool((base == 7.0).all())
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


# ---- the ends of the ranges ---------------------------------------------------------

@pytest.mark.parametrize("had,new,pad", [([0], [1], 0), ([64], [1], 0), ([5], [0], 3), ([0, 0, 3], [0, 0, 0], 4),
                                         ([-1, -1], [2, 1], 0), ([0, 7, 0, 128], [0, 1, 64, 0], 0), ([63], [65], 0)])
def test_small_scans(had, new, pad):
    G.run(had, new, N=64, pad=pad)


@pytest.mark.parametrize("op", ["scan", "step"])
def test_the_most_heads(op):
    """65535 states of 8 x 8 in a page; two requests."""
    G.run([0, 3], [1, 1] if op == "step" else [3, 1], H=65535, Hk=1, dk=8, dv=8, N=16, op=op)


@pytest.mark.parametrize("op", ["scan", "step"])
def test_the_most_requests(op):
    """2^20 requests' first tokens: the state is k v^T, the result scale (q . k) v."""
    n, d = 1 << 20, 8
    layers = [{"kind": "KDA", "conv_bytes": 16, "rec_bytes": d * d * 4}]
    L = lmc.lmc_layout_build(layers, 16, False, n * (16 + d * d * 4))
    assert L.num_blocks == n
    g = torch.Generator(device=DEV).manual_seed(2)
    q, k, v = (torch.randn(n, 1, d, generator=g, device=DEV).bfloat16() for _ in range(3))
    pool = torch.full((L.pool_bytes,), 0xFF, dtype=torch.uint8, device=DEV)
    table = torch.randperm(n, generator=g, device=DEV).int()[:, None]
    out, status = torch.empty_like(v), flag()
    lengths, decay = torch.zeros(n, dtype=torch.int32, device=DEV), torch.zeros(1, 1, device=DEV).expand(n, 1)
    if op == "scan":
        ws = torch.empty(lmc.lmc_linear_scan_workspace(L, 0, n, n, 1), dtype=torch.uint8, device=DEV)
        lmc.lmc_linear_scan(L, 0, pool, table, torch.arange(n + 1, dtype=torch.int32, device=DEV), lengths, q, k, v, decay,
                            out, ws, status)
    else:
        lmc.lmc_linear_step(L, 0, pool, table, lengths, q, k, v, decay, out, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    S = torch.as_strided(pool.view(torch.float32), (n, d, d), (L.stride[0] // 4, d, 1), (L.base[0] + 16) // 4)
    # a product of two bf16 numbers is a binary32 number
    assert torch.equal(S[table[:, 0].long()], k[:, 0, :, None].float() * v[:, 0, None, :].float())
    qk = q.double() * k.double()
    want, mag = qk.sum(2, keepdim=True) * v.double(), qk.abs().sum(2, keepdim=True) * v.double().abs()
    half = R.HALF_STEP["bf16"]
    # a rounded result of a weight that is rounded (scan), 8 terms in binary32
    assert bool(((out.double() - want).abs() <= half * (2 + half) * want.abs() + 16 * 2.0 ** -24 * mag).all())


def test_scan_of_rows_past_32_bits():
    """140000 tokens of 128 heads: v and out have 2.3 billion values. A token near
    the end forgets what came before, so the last ones follow from few."""
    n, H, d, tail = 140_000, 128, 128, 100
    layers = [{"kind": "KDA", "conv_bytes": 0, "rec_bytes": H * d * d * 4}]
    L = lmc.lmc_layout_build(layers, 1 << 18, False, 2 * H * d * d * 4)
    g = torch.Generator(device=DEV).manual_seed(3)
    v = torch.randn(n, H, d, generator=g, device=DEV, dtype=torch.bfloat16)
    q, k = torch.randn(n, 1, d, generator=g, device=DEV).bfloat16(), (torch.randn(n, 1, d, generator=g, device=DEV) / 16).bfloat16()
    decay = torch.full((n, 1), -0.01, device=DEV)
    decay[n - tail] = -float("inf")
    out, status = torch.full_like(v, float("nan")), flag()
    pool = torch.zeros(L.pool_bytes, dtype=torch.uint8, device=DEV)
    ws = torch.empty(lmc.lmc_linear_scan_workspace(L, 0, 1, n, H), dtype=torch.uint8, device=DEV)
    lmc.lmc_linear_scan(L, 0, pool, ints([[1]]), ints([0, n]), ints([0]), q, k, v, decay.expand(n, H), out, ws, status,
                        scale=0.125)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    heads = [0, 77, 127]
    o, mag, kept = R.linear(torch.zeros(3, d, d, dtype=torch.float64), q[-tail:].cpu(), k[-tail:].cpu(),
                            v[-tail:, heads].cpu(), decay[-tail:].expand(tail, 3).cpu(), 0.125, (tail,))
    half = R.HALF_STEP["bf16"]
    err = (out[-tail:, heads].cpu().double() - o).abs()
    assert bool((err <= half * o.abs() + mag * (half + (tail + 256) * 2.0 ** -23 + 2.0 ** -14)).all())
    S = pool[L.base[0] + L.stride[0]:].view(torch.float32).view(-1)[:H * d * d].view(H, d, d)[heads].cpu().double()
    assert float((S - kept[tail][0]).norm()) <= 2.0 ** -18 * float(kept[tail][0].norm())
    assert not bool(torch.isnan(out).any())


def test_pages_past_32_bits():
    """Blocks whose states lie more than 2^32 floats into a pool of 20 GB."""
    H, d, N = 32, 128, 16
    rec = H * d * d * 4
    L = lmc.lmc_layout_build([{"kind": "KDA", "conv_bytes": 32, "rec_bytes": rec}], N, False, 9600 * (rec + 32))
    assert L.num_blocks == 9600
    pool = torch.empty(L.pool_bytes, dtype=torch.uint8, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    q, k, v = (torch.randn(2, H, d, generator=g, device=DEV).half() for _ in range(3))
    out, status, decay = torch.empty_like(v), flag(), torch.full((2, H), -0.5, device=DEV)
    ws = torch.empty(lmc.lmc_linear_scan_workspace(L, 0, 1, 1, H), dtype=torch.uint8, device=DEV)
    table = ints([[9599, 8300]])
    lmc.lmc_linear_scan(L, 0, pool, table, ints([0, 1]), ints([0]), q[:1], k[:1], v[:1], decay[:1], out[:1], ws, status,
                        scale=0.01)
    page = lambda b: pool[L.base[0] + b * L.stride[0] + 32:][:rec].view(torch.float32).view(H, d, d)  # noqa: E731
    first = page(9599).clone()
    lmc.lmc_linear_step(L, 0, pool, table, ints([16]), q[1:], k[1:], v[1:], decay[1:], out[1:], status, scale=0.01)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    want = k[0, :, :, None].double() * v[0, :, None, :].double()
    assert float((first.double() - want).norm()) <= 2.0 ** -18 * float(want.norm())
    assert torch.equal(page(9599), first)
    want = first.double() * float(np.exp(-0.5)) + k[1, :, :, None].double() * v[1, :, None, :].double()
    # a decay and two products in binary32: three steps of each term at most
    bound = first.double().abs() + (k[1, :, :, None].double() * v[1, :, None, :].double()).abs()
    assert bool(((page(8300).double() - want).abs() <= bound * 2.0 ** -22).all())


@pytest.mark.parametrize("what", ["v", "k", "q"])
@pytest.mark.parametrize("op", ["scan", "step"])
def test_f16_of_all_its_range(what, op):
    """Values of 2^-14 to 2^14 beside each other: neither the weights nor the
    state may leave f16's range on their way to the products."""
    H, d, N = 2, 64, 100
    had, new = ([40, 0], [150, 64]) if op == "scan" else ([40, 0], [1, 1])
    rows = sum(new)
    q, k, v, dec, _ = G.inputs(rows, H, H, d, d, "f16", "resets", 9)
    g = torch.Generator().manual_seed(10)
    grown = lambda t, most: (t * 2.0 ** (most * (2 * torch.rand(rows, H, 1, generator=g) - 1)).half())  # noqa: E731
    if what == "v":
        v = grown(v, 14).clamp(-60000, 60000)
    elif what == "k":
        k = grown(k, 12)
    else:
        q = grown(q, 12)
    scale = {"v": 2.0 ** -6, "k": 2.0 ** -4, "q": 2.0 ** -4}[what]  # (results below 65504)
    P = R.States(lmc, H, d, d, N, 8)
    table = R.tables(had, new, N, 8, np.random.default_rng(0))
    P.pages()[int(table[0, 0])] = torch.randn(H, d, d, generator=g)
    pool, out, status = P.pool.cuda(), torch.full((rows, H, d), float("nan"), dtype=torch.float16, device=DEV), flag()
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    a = [x.cuda() for x in (q, k, v, dec)]
    if op == "scan":
        lmc.lmc_linear_scan(P.layout, P.layer, pool, table.cuda(), ints(start.tolist()), ints(had), *a, out,
                            workspace(P, 2, rows)[0], status, scale=scale)
    else:
        lmc.lmc_linear_step(P.layout, P.layer, pool, table.cuda(), ints(had), *a, out, status, scale=scale)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    G.check(P, pool.cpu(), out.cpu(), had, new, table, start, q, k, v, dec, scale, "f16")


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("N,new", [(64, [1, 2, 5, 16, 17, 31, 32]), (20, [90, 21]), (96, [200, 96, 100])])
def test_short_tiles_hold_their_weights_twice_as_long(N, new, act):
    """Tiles of at most 32 tokens, alone and between whole ones: the first ones of
    fresh requests are off by no more than the result's own rounding."""
    H, d = 2, 64
    P = R.States(lmc, H, d, d, N, 32)
    table = R.tables([0] * len(new), new, N, 32, np.random.default_rng(0))
    rows = sum(new)
    q, k, v, dec, _ = G.inputs(rows, H, H, d, d, act, "token", 21)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    pool, out, status = P.pool.cuda(), torch.full((rows, H, d), float("nan"), dtype=R.TYPES[act], device=DEV), flag()
    lmc.lmc_linear_scan(P.layout, P.layer, pool, table.cuda(), ints(start.tolist()), ints([0] * len(new)),
                        *[x.cuda() for x in (q, k, v, dec)], out, workspace(P, len(new), rows)[0], status, scale=0.1)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    out, half = out.cpu(), R.HALF_STEP[act]
    G.check(P, pool.cpu(), out, [0] * len(new), new, table, start, q, k, v, dec, 0.1, act)
    for r, n in enumerate(new):
        n = min(n, N) if min(n, N) <= 32 else 0  # the request's first tile
        s = slice(int(start[r]), int(start[r]) + n)
        o, mag, _ = R.linear(torch.zeros(H, d, d, dtype=torch.float64), q[s], k[s], v[s], dec[s], 0.1)
        # a weight in two parts is off by half a step squared (2^-16 in bf16); sums and decays in binary32
        most = half * o.abs() * (1 + 2.0 ** -10) + mag * (2.0 ** -14) + (2.0 ** -24 if act == "f16" else 0)
        assert bool(((out[s].double() - o).abs() <= most).all()), (r, n)


# ---- several calls at once, bad starts, pages that are shared -------------------------

@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_cut_requests_on_two_streams(act):
    """Long requests (three passes over a workspace) on two streams at a time."""
    H, d, N, new = 2, 128, 1000, [4100, 3, 2000]
    rows = sum(new)
    q, k, v, dec, _ = G.inputs(rows, H, H, d, d, act, "token", 7)
    P = R.States(lmc, H, d, d, N, 12)
    table = R.tables([0] * 3, new, N, 12, np.random.default_rng(0)).cuda()
    starts, lengths = ints([0, 4100, 4103, 6103]), ints([0] * 3)
    a = [x.cuda() for x in (q, k, v, dec)]

    def state():
        return P.pool.cuda(), torch.zeros(rows, H, d, dtype=R.TYPES[act], device=DEV), workspace(P, 3, rows)[0], flag()
    sets = [state() for _ in range(3)]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    for i, (pool, out, ws, status) in enumerate(sets):
        for _ in range(2):  # the second call finds the first one's workspace
            lmc.lmc_linear_scan(P.layout, P.layer, pool, table, starts, lengths, *a, out, ws, status, scale=0.1,
                                stream=sides[i] if i < 2 else None)
    torch.cuda.synchronize()
    for pool, out, _, status in sets:
        assert int(status.item()) == 0
        assert torch.equal(out.view(torch.int16), sets[0][1].view(torch.int16)) and torch.equal(pool, sets[0][0])
    G.check(P, sets[0][0].cpu(), sets[0][1].cpu(), [0] * 3, new, table.cpu(), starts.cpu().numpy(), q, k, v, dec, 0.1, act)


@pytest.mark.parametrize("seed", range(4))
def test_starts_that_decrease(seed):
    """Whatever starts hold, BAD_JOB is raised and nothing outside the rows, the
    pages of the table and the workspace is written."""
    H, d, N, n, most = 1, 64, 1 << 12, 6000, 40
    rng = np.random.default_rng(seed)
    starts = np.sort(rng.integers(0, n + 1, most + 1))
    swap = rng.permutation(most + 1)[:2 + 12 * (seed % 3)]
    starts[swap] = starts[np.roll(swap, 1)]
    if seed == 3:
        starts = rng.integers(-5000, 3 * n, most + 1)
    assert (np.diff(starts) < 0).any()
    q, k, v, dec, _ = G.inputs(n, H, H, d, d, "bf16", "token", 1)
    P = R.States(lmc, H, d, d, N, most + 4)
    pool, out, status = P.pool.cuda(), torch.full((n + 256, H, d), 3.0, dtype=torch.bfloat16, device=DEV), flag()
    ws, size = workspace(P, most, n, guard=4096)
    lmc.lmc_linear_scan(P.layout, P.layer, pool, ints([[2 + r] for r in range(most)]), ints(starts.tolist()), ints([0] * most),
                        *[x.cuda() for x in (q, k, v, dec)], out[128:128 + n], ws[4096:4096 + size], status)
    torch.cuda.synchronize()
    assert int(status.item()) == lmc.LMC_ST_BAD_JOB
    assert bool((out[:128] == 3.0).all()) and bool((out[128 + n:] == 3.0).all())
    assert bool((ws[:4096] == 0xA5).all()) and bool((ws[4096 + size:] == 0xA5).all())
    got, want = pool.cpu(), P.pool.clone()
    P.pages(want)[2:2 + most] = P.pages(got)[2:2 + most]
    assert torch.equal(want, got)


@pytest.mark.parametrize("op", ["scan", "step"])
def test_a_shared_prefix(op):
    """Two requests go on from one page at a block's end, each to a page of its own."""
    H, d, N = 2, 64, 32
    P = R.States(lmc, H, d, d, N, 6)
    P.pages()[0] = torch.randn(H, d, d, generator=torch.Generator().manual_seed(1))
    table = torch.tensor([[0, 1], [0, 2]], dtype=torch.int32)
    new = [1, 1] if op == "step" else [20, 32]
    q, k, v, dec, _ = G.inputs(sum(new), H, H, d, d, "bf16", "token", 1)
    pool, out, status = P.pool.cuda(), torch.full((sum(new), H, d), float("nan"), dtype=torch.bfloat16, device=DEV), flag()
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    a = [x.cuda() for x in (q, k, v, dec)]
    if op == "scan":
        lmc.lmc_linear_scan(P.layout, P.layer, pool, table.cuda(), ints(start.tolist()), ints([N, N]), *a, out,
                            workspace(P, 2, sum(new))[0], status, scale=0.1)
    else:
        lmc.lmc_linear_step(P.layout, P.layer, pool, table.cuda(), ints([N, N]), *a, out, status, scale=0.1)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    G.check(P, pool.cpu(), out.cpu(), [N, N], new, table, start, q, k, v, dec, 0.1, "bf16")


@pytest.mark.parametrize("op", ["scan", "step"])
def test_the_binding_refuses(op):
    """Tensors of other memory, types and shapes, before anything is enqueued."""
    H, d, N = 2, 64, 32
    P = R.States(lmc, H, d, d, N, 4)
    x, status = torch.randn(1, H, d, device=DEV).bfloat16(), flag()
    args = dict(q=x, k=x, v=x, decay=torch.zeros(1, H, device=DEV), out=torch.zeros_like(x))
    pool = P.pool.cuda()

    def call(lengths=ints([0]), table=ints([[0]]), starts=ints([0, 1]), ws=None, **kw):
        a = {**args, **kw}
        a = [a[n] for n in ("q", "k", "v", "decay", "out")]
        if op == "scan":
            lmc.lmc_linear_scan(P.layout, P.layer, pool, table, starts, lengths, *a, workspace(P, 1, 1)[0] if ws is None else ws,
                                status)
        else:
            lmc.lmc_linear_step(P.layout, P.layer, pool, table, lengths, *a, status)
    call()
    bad = [dict(q=x.cpu().pin_memory()), dict(out=torch.zeros(1, H, d).bfloat16().pin_memory()), dict(q=x.half()),
           dict(v=x[:, :, :32]), dict(k=x[:, :1]), dict(q=x[0]), dict(decay=args["decay"].double()),
           dict(decay=args["decay"][:, :1]), dict(decay=torch.zeros(1, H)), dict(lengths=torch.zeros(1, dtype=torch.int64, device=DEV)),
           dict(lengths=ints([0, 0])), dict(table=ints([0])), dict(out=x), dict(q=x.expand(2, H, d))]
    if op == "scan":
        bad += [dict(starts=ints([0])), dict(ws=torch.zeros(16, dtype=torch.uint8, device=DEV))]
    for kw in bad:
        with pytest.raises(lmc.LmcError):
            call(**kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0


@pytest.mark.parametrize("N", [1, 7, 33])
def test_small_blocks(N):
    """Tiles of a token or a few, each with its snapshot."""
    G.run([0, 5, 12], [40, 1, 9], N=N, act="f16")


def test_a_captured_scan_of_other_lengths():
    """A padded batch: one graph, replayed with other starts, lengths and tables in
    the same memory (requests that are skipped, empty, and cut into segments)."""
    H, d, N, rows, R_ = 2, 64, 1024, 5000, 4
    P = R.States(lmc, H, d, d, N, 14)
    P.pages()[:] = torch.randn(14, H, d, d, generator=torch.Generator().manual_seed(5))
    q, k, v, dec, _ = G.inputs(rows, H, H, d, d, "bf16", "token", 31)
    a = [x.cuda() for x in (q, k, v, dec)]
    pool, out, status = P.pool.cuda(), torch.zeros(rows, H, d, dtype=torch.bfloat16, device=DEV), flag()
    table, starts, lengths = ints([[-1] * 5] * R_), ints([0] * (R_ + 1)), ints([-1] * R_)
    ws = workspace(P, R_, rows)[0]
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        lmc.lmc_linear_scan(P.layout, P.layer, pool, table, starts, lengths, *a, out, ws, status, scale=0.1)
    for had, new in (([0, 3, 1024, 0], [4096, 1, 500, 403]), ([-1, 0, 2047, 9], [7, 0, 1, 300]), ([0] * 4, [0, 0, 0, 5000]),
                     ([-1] * 4, [0] * 4)):
        t = torch.full((R_, 5), -1, dtype=torch.int32)
        made = R.tables(had, new, N, 14, np.random.default_rng(1))
        t[:, :made.shape[1]] = made
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        pool.copy_(P.pool)
        out.fill_(float("nan"))
        table.copy_(t)
        starts.copy_(torch.from_numpy(start))
        lengths.copy_(torch.tensor(had, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        G.check(P, pool.cpu(), out.cpu(), had, new, t, start, q, k, v, dec, 0.1, "bf16")
