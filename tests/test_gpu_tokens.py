"""Token operators on the GPU against their plain 64-bit forms: appending
entries, attention of one new token over the pages, selecting the tokens a
request keeps, moving them, and the four together."""
import math

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


# ----------------------------------------------------------------------------
# Append
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("E,cache,act,N,packed,scale,pad", [
    (576, "bf16", "bf16", 944, False, 1.0, 0),
    (576, "f16", "f16", 64, True, 1.0, 8),
    (576, "e4m3", "bf16", 768, False, 0.05, 0),
    (112, "e4m3", "f16", 16, True, 0.0625, 16),
    (112, "e4m3", "bf16", 7, False, 0.3, 3),      # rows not 16-byte aligned
    (33, "bf16", "bf16", 5, True, 1.0, 1),        # odd entries: two-byte boundaries
    (35, "e4m3", "f16", 5, True, 0.7, 0),
    (6, "f16", "f16", 3, False, 1.0, 0),          # 12-byte entries
])
def test_append_writes_exactly_the_named_rows(lmc, status, E, cache, act, N, packed, scale, pad):
    rng = np.random.default_rng(E + N)
    M = T.Model(lmc, E, cache, N, packed, layers=2, state=N * E, blocks=12)
    lengths = [1, N, 2 * N + 1]
    table = T.tables(lengths, N, 12, rng)
    req = np.concatenate([np.full(n, r) for r, n in enumerate(lengths)] + [[-1]]).astype(np.int32)
    pos = np.concatenate([np.arange(n) for n in lengths] + [[12345]]).astype(np.int32)
    order = rng.permutation(len(req))
    req, pos = req[order], pos[order]
    x = (torch.from_numpy(rng.standard_normal((len(req), E + pad))) * 3).to(T.TYPES[act])
    x[0, :3] = torch.tensor([1e4, -1e4, 0.0]).to(x.dtype)       # past e4m3's range
    x[1, 0] = math.nan
    want = M.pool.clone()
    pages = M.pages(1, want)
    for i in range(len(req)):
        if req[i] < 0:
            continue
        v = x[i, :E]
        if cache == "e4m3":
            # IEEE binary32 quotient, saturated, rounded half to even
            v = (v.float() / torch.tensor(scale, dtype=torch.float32)).clamp(-448, 448).to(torch.float8_e4m3fn)
        pages[int(table[req[i], pos[i] // N]), pos[i] % N] = v.contiguous().view(torch.uint8)
    pool = M.pool.to(DEV)
    lmc.lmc_append(M.layout, M.layers[1], pool, table.to(DEV), _int32(req), _int32(pos), x.to(DEV)[:, :E], status,
                   scale=scale)
    got = pool.cpu()
    assert status.item() == 0
    # NaN codes differ in sign between converters: compare such bytes as NaN
    diff = torch.nonzero(got != want).flatten()
    if cache == "e4m3":
        assert all((int(got[i]) & 0x7F) == 0x7F and (int(want[i]) & 0x7F) == 0x7F for i in diff)
    else:
        assert diff.numel() == 0


@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_append_codes_of_every_value(lmc, status, act):
    """All 65536 patterns of the rows' type under scales that are powers of
    two, odd, near the ends of binary32 and with every significand bit set:
    the code of the IEEE quotient each time."""
    patterns = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(T.TYPES[act]).view(128, 512).to(DEV)
    L = lmc.lmc_layout_build([{"kind": "MLA", "token_bytes": 512}], 128, False, 128 * 512)
    req, pos = _int32(np.zeros(128)), _int32(np.arange(128))
    all_ones = float(np.uint32(0x3FFFFFFF).view(np.float32))
    for scale in (1.0, 0.05, 0.0625, 3.0, 1 / 3, 448.0, 2.0 ** -90, 1.7e-31, 2.0 ** -126, 1e-42, 2.0 ** 99, 3e38,
                  all_ones, all_ones * 2.0 ** -5, 0.0123):
        pool = torch.full((L.pool_bytes,), 0x55, dtype=torch.uint8, device=DEV)
        lmc.lmc_append(L, 0, pool, _int32([[0]]), req, pos, patterns, status, scale=scale)
        s = torch.tensor(scale, dtype=torch.float32, device=DEV)
        want = (patterns.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        got = pool.view(128, 512)
        nan = torch.isnan(patterns.float())
        assert torch.equal(got[~nan], want[~nan]), scale
        assert ((got[nan] & 0x7F) == 0x7F).all()
    assert status.item() == 0


def test_append_skips_bad_rows_with_status(lmc, status):
    M = T.Model(lmc, 32, "bf16", 4, layers=1, blocks=3)
    table = _int32([[0, -1], [99, 1]])
    x = torch.ones((1, 32), dtype=torch.bfloat16, device=DEV)
    pool = M.pool.to(DEV)
    for req, pos, bit in [(0, 4, lmc.LMC_ST_NO_BLOCK), (1, 0, lmc.LMC_ST_BLOCK_OOR), (2, 0, lmc.LMC_ST_BAD_JOB),
                          (-2, 0, lmc.LMC_ST_BAD_JOB), (0, 8, lmc.LMC_ST_BAD_JOB), (0, -1, lmc.LMC_ST_BAD_JOB)]:
        status.zero_()
        lmc.lmc_append(M.layout, 0, pool, table, _int32([req]), _int32([pos]), x, status)
        assert status.item() == bit, (req, pos)
    assert torch.equal(pool.cpu(), M.pool)
    lmc.lmc_append(M.layout, 0, pool, table, _int32([]), _int32([]), x[:0], status)  # no rows


# ----------------------------------------------------------------------------
# Attention
# ----------------------------------------------------------------------------

def _attend(lmc, M, i, table, lengths, q, V, status, scale=1.0, softmax_scale=None, weights=None, pool=None,
            max_length=None, **kw):
    R, H, E = q.shape
    max_length = max_length or max(1, max(lengths))
    softmax_scale = softmax_scale or 1.0 / math.sqrt(E)
    out = kw.pop("out", None)
    if out is None:
        out = torch.full((R, H, V), 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full((R, H), 7.0, device=DEV)
    n = lmc.lmc_attend_workspace(M.layout, M.layers[i], R, H, V, max_length, weights is not None)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    lmc.lmc_attend(M.layout, M.layers[i], M.pool.to(DEV) if pool is None else pool, table.to(DEV), _int32(lengths), q,
                   V, softmax_scale, out, ws, status, max_length=max_length, scale=scale, lse=lse, weights=weights,
                   **kw)
    return out, lse, softmax_scale


def _check_attend(M, i, table, lengths, q, V, scale, softmax_scale, out, lse, act, weights=None, before=None,
                  skip=()):
    """Each request against the 64-bit form; positions in skip[r] are missing."""
    for r, n in enumerate(lengths):
        lo = max(0, n - M.window) if M.window else 0
        at = [t for t in range(lo, n) if not (skip and t in skip[r])]
        e = M.read(i, table, r, at) if at else torch.zeros((0, M.E), dtype=torch.float64)
        o, l, w, d_o, d_l, d_w = T.attend(e, q[r].cpu().double(), V, softmax_scale, scale, M.cache, act)
        got = out[r].cpu().double()
        assert torch.isfinite(got).all(), f"request {r}"
        assert ((got - o).abs() <= d_o).all(), (r, n, float((got - o).abs().max()), float(o.abs().max()))
        gl = lse[r].cpu().double()
        assert torch.equal(torch.isinf(gl), torch.isinf(l))
        if at:
            assert ((gl - l).abs() <= d_l).all(), (r, n, float((gl - l).abs().max()))
        if weights is not None:
            want = before[r].double()
            slack = want.abs() * 2.0 ** -23
            if at:
                want[at] += w
                slack[at] += d_w
            assert ((weights[r].cpu().double() - want).abs() <= slack).all(), (r, n)
            outside = [t for t in range(want.numel()) if t not in set(at)]
            assert torch.equal(weights[r].cpu()[outside], before[r][outside])


CASES = [
    # E, V, heads, cache, act, N, packed, window, lengths
    (576, 512, 4, "bf16", "bf16", 64, False, 0, [300, 517]),
    (576, 512, 32, "bf16", "bf16", 944, False, 0, [1, 943, 944, 945, 0, 2000]),
    (576, 512, 64, "bf16", "bf16", 768, True, 0, [1536, 63, 64, 65, 129]),
    (576, 512, 64, "e4m3", "bf16", 768, False, 0, [1537, 1, 0, 800]),
    (576, 512, 16, "e4m3", "f16", 100, True, 0, [99, 100, 101, 256]),
    (576, 512, 96, "bf16", "bf16", 64, False, 0, [130, 5]),
    (576, 512, 128, "f16", "f16", 64, True, 0, [64, 127, 128, 200]),
    (576, 512, 20, "f16", "f16", 16, False, 0, [1, 15, 16, 17, 100]),
    (576, 512, 32, "bf16", "bf16", 944, True, 700, [500, 699, 700, 701, 1900, 0]),
    (576, 512, 8, "e4m3", "bf16", 64, False, 1, [1, 64, 65, 0]),
    (320, 256, 40, "bf16", "bf16", 48, False, 0, [47, 48, 96, 200]),
    (192, 128, 1, "f16", "f16", 7, True, 0, [6, 7, 8, 50]),
    (112, 96, 12, "e4m3", "f16", 24, False, 33, [32, 33, 34, 100]),
    (80, 72, 5, "bf16", "bf16", 1, False, 0, [1, 2, 9, 0]),
    (16, 8, 3, "f16", "f16", 2, True, 0, [1, 2, 3, 30]),
    (64, 64, 64, "e4m3", "bf16", 1000, False, 0, [999, 64, 1]),
    (192, 128, 8, "bf16", "bf16", 75, True, 151, [150, 151, 400, 77]),   # whole tiles that begin on odd tokens
    (576, 512, 48, "e4m3", "f16", 8, False, 0, [7, 8, 9, 70]),           # eight pages in a tile
    (128, 128, 130, "bf16", "bf16", 40, True, 0, [40, 41, 300]),         # three groups of heads, one of them short
]


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("E,V,H,cache,act,N,packed,window,lengths", CASES)
def test_attend_matches_64_bits(lmc, status, E, V, H, cache, act, N, packed, window, lengths, weights):
    rng = np.random.default_rng(E * 7 + H)
    blocks = sum(-(-n // N) for n in lengths) + 2
    scale = 0.0625 if cache == "e4m3" else 1.0
    M = T.Model(lmc, E, cache, N, packed, layers=2, window=window, state=16 * N, blocks=blocks)
    table = T.tables(lengths, N, blocks, rng)
    for r, n in enumerate(lengths):
        # only the range is written: everything else in the pool stays NaN
        lo = max(0, n - window) if window else 0
        M.write(1, table, r, lo, torch.from_numpy(rng.standard_normal((n - lo, E))) / scale)
    q = torch.from_numpy(rng.standard_normal((len(lengths), H, E))).to(T.TYPES[act]).to(DEV)
    W = before = None
    if weights:
        before = torch.from_numpy(rng.random((len(lengths), max(lengths) + 3))).float()
        W = before.to(DEV)
    out, lse, ss = _attend(lmc, M, 1, table, lengths, q, V, status, scale, weights=W)
    assert status.item() == 0
    _check_attend(M, 1, table, lengths, q, V, scale, ss, out, lse, act, W, before)


@pytest.mark.parametrize("R,longest,N,window,H,cache,act", [
    (1, 128, 64, 0, 32, "bf16", "bf16"), (5, 190, 64, 0, 4, "f16", "f16"), (153, 64, 944, 0, 8, "e4m3", "bf16"),
    (300, 128, 16, 0, 20, "bf16", "bf16"), (40, 400, 944, 33, 96, "bf16", "bf16"), (310, 60, 20, 0, 3, "e4m3", "f16"),
    (700, 60, 64, 0, 2, "f16", "f16"), (90, 1, 64, 0, 130, "bf16", "bf16")])
def test_attend_of_short_caches(lmc, status, R, longest, N, window, H, cache, act):
    """Caches of a tile or a few, so that requests are not split; one length
    among them cannot be served. The same again sized for long caches."""
    E, V = 128, 96
    rng = np.random.default_rng(R)
    lengths = [int(n) for n in rng.integers(0, longest + 1, R)]
    lengths[-1] = longest
    blocks = sum(-(-n // N) for n in lengths) + 2
    scale = 0.0625 if cache == "e4m3" else 1.0
    M = T.Model(lmc, E, cache, N, False, layers=2, window=window, state=16 * N, blocks=blocks)
    table = T.tables(lengths, N, blocks, rng)
    for r, n in enumerate(lengths):
        lo = max(0, n - window) if window else 0
        M.write(1, table, r, lo, torch.from_numpy(rng.standard_normal((n - lo, E))) / scale)
    q = torch.from_numpy(rng.standard_normal((R, H, E))).to(T.TYPES[act]).to(DEV)
    bad = R // 2 if R > 2 else None
    given = [1 << 20 if r == bad else n for r, n in enumerate(lengths)]
    before = torch.from_numpy(rng.random((R, 4096))).float()
    for max_length in (longest, 4096):
        W = before.to(DEV)
        status.zero_()
        out, lse, ss = _attend(lmc, M, 1, table, given, q, V, status, scale, weights=W, max_length=max_length)
        assert status.item() == (0 if bad is None else lmc.LMC_ST_BAD_JOB)
        if bad is not None:
            assert (out[bad] == 7.0).all() and (lse[bad] == 7.0).all()
            assert torch.equal(W[bad].cpu(), before[bad])
        at = [r for r in range(R) if r != bad]
        sub = table[at]
        _check_attend(M, 1, sub, [lengths[r] for r in at], q[at], V, scale, ss, out[at], lse[at], act, W[at],
                      before[at])


@pytest.mark.parametrize("cache,act", [("bf16", "bf16"), ("e4m3", "bf16"), ("f16", "f16")])
def test_attend_split_over_a_long_cache_and_many_requests(lmc, status, cache, act):
    """One long request beside many short ones: the work is shared over the
    device, so single requests are split and joined; lengths in a wide batch
    are 0, 1 and odd."""
    rng = np.random.default_rng(11)
    N, E, V, H = 944, 576, 512, 32
    lengths = [40_001, 0, 1, 2500] + [int(n) for n in rng.integers(0, 130, 300)]
    blocks = sum(-(-n // N) for n in lengths) + 1
    scale = 0.0625 if cache == "e4m3" else 1.0
    M = T.Model(lmc, E, cache, N, layers=1, blocks=blocks)
    M.pool = torch.from_numpy(rng.integers(0, 256, M.pool.numel(), dtype=np.uint8))
    raw = torch.from_numpy(rng.standard_normal((blocks, N, E)).astype(np.float32)) / scale
    M.pages(0).copy_(raw.to(T.TYPES[cache]).view(torch.uint8))
    table = T.tables(lengths, N, blocks, rng)
    q = torch.from_numpy(rng.standard_normal((len(lengths), H, E))).to(T.TYPES[act]).to(DEV)
    before = torch.zeros((len(lengths), max(lengths)))
    W = before.to(DEV)
    out, lse, ss = _attend(lmc, M, 0, table, lengths, q, V, status, scale, weights=W)
    again = torch.zeros_like(W)
    out2, lse2, _ = _attend(lmc, M, 0, table, lengths, q, V, status, scale, weights=again)
    assert status.item() == 0
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and torch.equal(W, again)  # the same bits again
    few = [0, 1, 2, 3, 10, 100, 303]
    _check_attend(M, 0, table[few], [lengths[r] for r in few], q[few], V, scale, ss, out[few], lse[few], act, W[few],
                  before[few])
    total = W.double().sum(1).cpu()
    want = torch.tensor([H if n else 0 for n in lengths], dtype=torch.float64)
    assert (total - want).abs().max() <= H * 1e-4


@pytest.mark.parametrize("softmax_scale,shift", [(4.0, 0.0), (-0.5, 0.0), (1.0, 60.0), (1e-8, 0.0)])
def test_attend_peaked_growing_and_flat_logits(lmc, status, softmax_scale, shift):
    """Logits of some hundreds, a running maximum that grows with every token
    (and in steps no threshold hides), a scale below zero, a flat softmax."""
    rng = np.random.default_rng(3)
    N, E, V, H, n = 64, 64, 64, 16, 500
    M = T.Model(lmc, E, "bf16", N, blocks=9)
    table = T.tables([n], N, 9, rng)
    e = rng.standard_normal((n, E))
    e[:, 0] += shift * np.arange(n) / n
    M.write(0, table, 0, 0, torch.from_numpy(e))
    q = torch.from_numpy(rng.standard_normal((1, H, E)))
    q[:, :, 0] += 8.0 if shift else 0.0
    q = q.to(torch.bfloat16).to(DEV)
    out, lse, ss = _attend(lmc, M, 0, table, [n], q, V, status, softmax_scale=softmax_scale)
    assert status.item() == 0
    _check_attend(M, 0, table, [n], q, V, 1.0, ss, out, lse, "bf16")


def test_attend_one_large_weight_among_many_small(lmc, status):
    """A first token that outweighs each of the others by 2^24 and 2^30, all of
    them together by a factor of 2^9 and less: in f16 the small weights must
    not be lost (they are lifted), whatever the order."""
    rng = np.random.default_rng(4)
    N, E, V, H, n = 64, 64, 64, 16, 40_000
    blocks = -(-n // N)
    for where in (0, n // 2, n - 1):
        M = T.Model(lmc, E, "f16", N, blocks=blocks)
        table = T.tables([n], N, blocks, rng)
        e = rng.standard_normal((n, E)) * 0.01
        e[:, 0], e[:, 1] = 0.0, 1.0   # the second value is 1 for all but the large one
        e[where, 0], e[where, 1] = 16.0, 0.0
        pages = M.pages(0)
        flat = torch.from_numpy(e).to(torch.float16).view(torch.uint8)
        pad = torch.zeros((blocks * N, E * 2), dtype=torch.uint8)
        pad[:n] = flat
        pages[table[0].long()] = pad.view(blocks, N, E * 2)
        q = torch.zeros((1, H, E), dtype=torch.float16, device=DEV)
        q[:, :8, 0] = 24 * math.log(2) / 16
        q[:, 8:, 0] = 30 * math.log(2) / 16
        out, lse, ss = _attend(lmc, M, 0, table, [n], q, V, status, softmax_scale=1.0)
        assert status.item() == 0
        # the others' share of the weight, by their second value
        for h in (0, 8):
            bits = float(q[0, h, 0]) * 16 / math.log(2)  # as f16 holds q
            share = (n - 1) / (n - 1 + 2.0 ** bits)
            got = float(out[0, h, 1])
            # p of the small ones is 2^(7 - bits) where the large one comes first: f16's half step is 2^-25 there;
            # the output's is 2^-11 of it, or 2^-25 where it is not normal
            slack = share * (2.0 ** -25 / 2.0 ** (7 - bits) + 2.0 ** -10) + 2.0 ** -24
            assert abs(got - share) <= slack, (where, bits, got, share)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("N", [64, 16, 100])
def test_attend_missing_blocks_bad_lengths_and_status(lmc, status, N, cache):
    """A missing page's tokens are left out; a request all of whose pages are
    missing gives zeros; a bad length leaves its rows as they were."""
    rng = np.random.default_rng(5)
    E, V, H = 64, 64, 8
    lengths = [3 * N, 2 * N, 2 * N, N, N]
    blocks = 12
    M = T.Model(lmc, E, cache, N, blocks=blocks)
    table = T.tables(lengths, N, blocks, rng, cols=4)
    for r, n in enumerate(lengths):
        M.write(0, table, r, 0, torch.from_numpy(rng.standard_normal((n, E))))
    good = table.clone()
    table[0, 1] = -1
    table[1, :] = -1
    table[2, 0] = blocks
    given = [3 * N, 2 * N, 2 * N, -1, 3 * N + 1]  # -1, and above max_length
    q = torch.from_numpy(rng.standard_normal((5, H, E))).to(torch.bfloat16).to(DEV)
    before = torch.rand((5, 3 * N))
    W = before.to(DEV)
    out, lse, ss = _attend(lmc, M, 0, table, given, q, V, status, weights=W, max_length=3 * N)
    assert status.item() == lmc.LMC_ST_NO_BLOCK | lmc.LMC_ST_BLOCK_OOR | lmc.LMC_ST_BAD_JOB
    skip = [set(range(N, 2 * N)), set(range(2 * N)), set(range(N))]
    _check_attend(M, 0, good, lengths[:3], q[:3], V, 1.0, ss, out[:3], lse[:3], "bf16", W[:3], before[:3], skip)
    for r in (3, 4):
        assert (out[r] == 7).all() and (lse[r] == 7).all() and torch.equal(W[r].cpu(), before[r])
    # a length past the table's columns
    status.zero_()
    _attend(lmc, M, 0, table[:1], [4 * N + 1], q[:1], V, status, max_length=5 * N)
    assert status.item() == lmc.LMC_ST_BAD_JOB


def test_attend_strides_untouched_bytes_and_side_stream(lmc, status):
    """q, out and lse as slices of wider buffers (head-major too), a block
    table with a row stride; on another stream than the current one; bytes
    between the rows are left alone."""
    rng = np.random.default_rng(8)
    N, E, V, H, lengths = 64, 192, 128, 6, [100, 1, 0, 64]
    M = T.Model(lmc, E, "f16", N, packed=True, layers=2, blocks=8)
    table = T.tables(lengths, N, 8, rng)
    for r, n in enumerate(lengths):
        M.write(0, table, r, 0, torch.from_numpy(rng.standard_normal((n, E))))
    R = len(lengths)
    wide = torch.from_numpy(rng.standard_normal((H, R, E + 8))).to(torch.float16).to(DEV)
    q = wide[:, :, :E].transpose(0, 1)  # [R, H, E], head-major
    buf = torch.full((H, R, V + 3), 5.0, dtype=torch.float16, device=DEV)
    out = buf[:, :, :V].transpose(0, 1)
    tab = torch.full((R, table.shape[1] + 3), 77, dtype=torch.int32)
    tab[:, : table.shape[1]] = table
    tab = tab.to(DEV)[:, : table.shape[1]]
    pool = M.pool.to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse, ss = _attend(lmc, M, 0, tab, lengths, q, V, status, out=out, pool=pool, stream=side)
    side.synchronize()
    assert status.item() == 0
    _check_attend(M, 0, table, lengths, q, V, 1.0, ss, out, lse, "f16")
    assert (buf[:, :, V:] == 5).all()
    assert torch.equal(pool.cpu(), M.pool)


def test_attend_on_two_streams_beside_matrix_products(lmc, status):
    """Two batches at once on two streams, each with its own workspace, while
    a third stream multiplies matrices: the same bits as one after the other."""
    rng = np.random.default_rng(12)
    N, E, V, H = 64, 192, 128, 24
    jobs = []
    for cache, lengths in (("bf16", [3000, 17, 900]), ("e4m3", [2500, 64, 1, 0])):
        blocks = sum(-(-n // N) for n in lengths)
        M = T.Model(lmc, E, cache, N, blocks=blocks)
        raw = torch.from_numpy(rng.standard_normal((blocks, N, E)).astype(np.float32)).to(T.TYPES[cache])
        M.pages(0).copy_(raw.view(torch.uint8))
        table = T.tables(lengths, N, blocks, rng).to(DEV)
        q = torch.from_numpy(rng.standard_normal((len(lengths), H, E))).to(torch.bfloat16).to(DEV)
        n = lmc.lmc_attend_workspace(M.layout, 0, len(lengths), H, V, 3000, True)
        jobs.append((M, M.pool.to(DEV), table, _int32(lengths), q, torch.empty(n, dtype=torch.uint8, device=DEV)))

    def call(job, out, lse, weights, stream=None):
        M, pool, table, lengths, q, ws = job
        lmc.lmc_attend(M.layout, 0, pool, table, lengths, q, V, 0.1, out, ws, status, max_length=3000, lse=lse,
                       weights=weights, stream=stream)

    def buffers(job):
        R = job[4].shape[0]
        return (torch.empty((R, H, V), dtype=torch.bfloat16, device=DEV), torch.empty((R, H), device=DEV),
                torch.zeros((R, 3000), device=DEV))

    want = [buffers(j) for j in jobs]
    for j, w in zip(jobs, want):
        call(j, *w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    a = torch.randn((2048, 2048), device=DEV).bfloat16()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        with torch.cuda.stream(streams[2]):
            for _ in range(4):
                a @ a
        for j, s in zip(jobs, streams):
            g = buffers(j)
            s.wait_stream(torch.cuda.current_stream())
            call(j, *g, stream=s)
            got.append((j, g))
    torch.cuda.synchronize()
    assert status.item() == 0
    for j, g in got:
        for x, y in zip(g, want[0] if j is jobs[0] else want[1]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_attend_values_that_are_not_finite_reach_the_result(lmc, status):
    """An infinity or NaN in a token that is attended shows in the output, as
    in the plain softmax; one behind the length or before the window does not."""
    N, E, V, H = 64, 64, 64, 4
    rng = np.random.default_rng(9)
    M = T.Model(lmc, E, "bf16", N, blocks=4)
    table = T.tables([100], N, 4, rng)
    e = torch.from_numpy(rng.standard_normal((100, E)))
    e[50, 3] = math.nan
    M.write(0, table, 0, 0, e)
    q = torch.ones((1, H, E), dtype=torch.bfloat16, device=DEV)
    out, lse, _ = _attend(lmc, M, 0, table, [100], q, V, status)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    out, lse, ss = _attend(lmc, M, 0, table, [50], q, V, status)
    _check_attend(M, 0, table, [50], q, V, 1.0, ss, out, lse, "bf16")


def test_attend_blocks_past_four_gigabytes(lmc, status):
    """Block offsets that need more than 32 bits."""
    N, E, V, H = 64, 576, 512, 8
    blocks = (5 << 30) // (N * E * 2)
    L = lmc.lmc_layout_build([{"kind": "MLA", "token_bytes": E * 2}], N, False, blocks * N * E * 2)
    pool = torch.empty(L.pool_bytes, dtype=torch.uint8, device=DEV)
    small = T.Model(lmc, E, "bf16", N, blocks=4)
    rng = np.random.default_rng(10)
    small_table = T.tables([200], N, 4, rng)
    small.write(0, small_table, 0, 0, torch.from_numpy(rng.standard_normal((200, E))))
    table = small_table + (blocks - 4)
    pool[-small.pool.numel():] = small.pool.to(DEV)
    q = torch.from_numpy(rng.standard_normal((1, H, E))).to(torch.bfloat16).to(DEV)
    big = T.Model.__new__(T.Model)
    big.layout, big.layers = L, [0]
    out, lse, ss = _attend(lmc, big, 0, table, [200], q, V, status, pool=pool)
    assert status.item() == 0
    _check_attend(small, 0, small_table, [200], q, V, 1.0, ss, out, lse, "bf16")
    # the appended row and the moved rows land there too
    x = torch.ones((1, E), dtype=torch.bfloat16, device=DEV)
    lmc.lmc_append(L, 0, pool, table.to(DEV), _int32([0]), _int32([199]), x, status)
    kept = _int32([[[199, 5]]])
    lmc.lmc_move_tokens(L, 0, pool, table.to(DEV), _int32([[0]]), kept, _int32([2]), status)
    assert status.item() == 0
    got = pool[: 2 * E * 2].view(torch.bfloat16).view(2, E)
    assert (got[0] == 1).all()
    assert torch.equal(got[1].cpu().double(), small.read(0, small_table, 0, [5])[0])


# ----------------------------------------------------------------------------
# Select and move
# ----------------------------------------------------------------------------

def _select(lmc, scores, lengths, budget, recent, status, with_scores=True):
    S, R, _ = scores.shape
    kept = torch.full((S, R, budget), -7, dtype=torch.int32, device=DEV)
    ks = torch.full((S, R, budget), -7.0, device=DEV) if with_scores else None
    kl = torch.full((R,), -7, dtype=torch.int32, device=DEV)
    lmc.lmc_select_tokens(scores, _int32(lengths), budget, recent, kept, ks, kl, status)
    return kept.cpu(), None if ks is None else ks.cpu(), kl.cpu()


def _check_select(scores, lengths, budget, recent, kept, ks, kl):
    x = scores.cpu()
    for r, n in enumerate(lengths):
        assert int(kl[r]) == min(n, budget)
        for s in range(x.shape[0]):
            want = T.select(x[s, r].tolist(), n, budget, recent)
            assert kept[s, r].tolist() == want + [-7] * (budget - len(want)), (s, r, n)
            if ks is not None:
                a, b = ks[s, r, : len(want)], x[s, r][want]
                assert torch.equal(a.view(torch.int32), b.contiguous().view(torch.int32))  # the bits
                assert (ks[s, r, len(want):] == -7).all()


@pytest.mark.parametrize("tokens,budget,recent,lengths", [
    (600, 128, 32, [300, 517, 128, 129, 0, 1, 600]),
    (5000, 7, 7, [5000, 7, 8, 3]),          # only the last tokens
    (5000, 4999, 0, [5000, 4999, 2500]),    # all but one
    (5000, 1, 0, [5000, 1, 2]),
    (5000, 0, 0, [5000, 0]),                # an empty cache
    (40_000, 3000, 100, [40_000, 39_999, 3001, 16385]),
])
@pytest.mark.parametrize("kind", ["normal", "ties", "one_value"])
def test_select_matches_a_sort(lmc, status, tokens, budget, recent, lengths, kind):
    g = torch.Generator().manual_seed(tokens + budget)
    x = torch.randn((3, len(lengths), tokens + 5), generator=g)
    if kind == "ties":
        x = (x * 2).round() / 2
    elif kind == "one_value":
        x = torch.full_like(x, -0.25)
    wide = x.to(DEV)
    scores = wide[:, :, :tokens]  # a stride past the tokens
    kept, ks, kl = _select(lmc, scores, lengths, budget, recent, status)
    assert status.item() == 0
    _check_select(scores, lengths, budget, recent, kept, ks, kl)


def test_select_special_values_and_no_scores(lmc, status):
    x = torch.tensor([math.nan, -math.inf, 0.0, -0.0, math.inf, 1e-45, -1e-45, math.nan, 3.0, -math.inf]).repeat(1, 1, 1)
    for budget in range(0, 10):
        kept, ks, kl = _select(lmc, x.to(DEV), [10], budget, 0, status)
        _check_select(x, [10], budget, 0, kept, ks, kl)
    kept, ks, kl = _select(lmc, x.to(DEV), [10], 4, 1, status, with_scores=False)
    _check_select(x, [10], 4, 1, kept, ks, kl)
    assert status.item() == 0
    # bad lengths: nothing is written for that request
    kept, ks, kl = _select(lmc, x.to(DEV).expand(1, 3, 10), [-1, 11, 10], 2, 0, status)
    assert status.item() == lmc.LMC_ST_BAD_JOB
    assert (kept[0, :2] == -7).all() and kl.tolist() == [-7, -7, 2]


def test_select_rows_of_every_cluster_shape(lmc, status):
    """Lengths around the points where a row is shared by more CTAs, and one
    that no CTA's shared memory holds."""
    for tokens in (2048, 2049, 16384, 16385, 131_072, 131_073, 600_001):
        x = torch.rand((1, 2, tokens), device=DEV, generator=torch.Generator(DEV).manual_seed(tokens))
        x = (x * 50_000).floor() / 50_000
        lengths, budget, recent = [tokens, tokens - 1], tokens // 3, 17
        kept, ks, kl = _select(lmc, x, lengths, budget, recent, status)
        for r, n in enumerate(lengths):
            v, order = torch.sort(x[0, r, : n - recent], descending=True, stable=True)
            want = torch.cat([order[: budget - recent].sort().values, torch.arange(n - recent, n, device=DEV)])
            assert torch.equal(kept[0, r].long(), want.cpu())
            assert torch.equal(ks[0, r], x[0, r][want].cpu())
    assert status.item() == 0


@pytest.mark.parametrize("E,cache,N,packed,shared", [
    (576, "bf16", 64, False, False), (576, "e4m3", 100, True, False), (576, "bf16", 944, True, True),
    (33, "bf16", 5, True, False), (35, "e4m3", 4, False, False), (6, "f16", 3, True, True),
])
def test_move_copies_exactly_the_kept_entries(lmc, status, E, cache, N, packed, shared):
    rng = np.random.default_rng(E + N)
    lengths, keep = [3 * N + 1, N, 0, 2 * N], [2 * N, 1, 0, N - 1]
    n_src = sum(-(-n // N) for n in lengths)
    blocks = n_src + sum(-(-n // N) for n in keep) + 1
    M = T.Model(lmc, E, cache, N, packed, layers=3, state=8 * N, blocks=blocks)
    M.pool = torch.from_numpy(rng.integers(0, 256, M.pool.numel(), dtype=np.uint8))
    ids = rng.permutation(blocks)
    src = T.tables(lengths, N, n_src, rng)
    dst = T.tables(keep, N, blocks - n_src, rng)
    src = torch.where(src >= 0, torch.from_numpy(ids.astype(np.int32))[src.long()], src)
    dst = torch.where(dst >= 0, torch.from_numpy(ids.astype(np.int32))[n_src + dst.long()], dst)
    S, K = (1 if shared else 3), max(keep) + 2
    kept = torch.full((S, 4, K), -9, dtype=torch.int32)  # not looked at behind the kept
    want = M.pool.clone()
    for s in range(S):
        for r in range(4):
            kept[s, r, : keep[r]] = torch.from_numpy(np.sort(rng.permutation(lengths[r])[: keep[r]]).astype(np.int32))
    for i in range(3):
        a, b = M.pages(i), M.pages(i, want)
        for r in range(4):
            for j in range(keep[r]):
                t = int(kept[0 if shared else i, r, j])
                b[int(dst[r, j // N]), j % N] = a[int(src[r, t // N]), t % N]
    pool = M.pool.to(DEV)
    lmc.lmc_move_tokens(M.layout, M.group, pool, src.to(DEV), dst.to(DEV), kept.to(DEV), _int32(keep), status)
    assert status.item() == 0
    assert torch.equal(pool.cpu(), want)


def test_move_skips_bad_entries_with_status(lmc, status):
    M = T.Model(lmc, 32, "bf16", 4, blocks=6)
    src, dst = _int32([[0, -1], [1, 9]]), _int32([[2], [-1]])
    pool = M.pool.to(DEV)
    B = lmc
    for kept, lens, bit in [([[[4]], ], [1, 0], B.LMC_ST_NO_BLOCK), ([[[8]]], [1, 0], B.LMC_ST_BAD_JOB),
                            ([[[-1]]], [1, 0], B.LMC_ST_BAD_JOB), ([[[0]]], [2, 0], B.LMC_ST_BAD_JOB),
                            ([[[0]]], [-1, 0], B.LMC_ST_BAD_JOB), ([[[4]]], [0, 1], B.LMC_ST_BLOCK_OOR | B.LMC_ST_NO_BLOCK)]:
        status.zero_()
        k = _int32(kept).expand(1, 2, 1).contiguous()
        lmc.lmc_move_tokens(M.layout, 0, pool, src, dst, k, _int32(lens), status)
        assert status.item() == bit, (kept, lens)
    assert torch.equal(pool.cpu(), M.pool)


# ----------------------------------------------------------------------------
# Together
# ----------------------------------------------------------------------------

def _sequence(lmc, cache, act, status, seed, capture):
    """A small model's serving loop: a prefill is appended, steps append one
    token per request and attend with accumulated weights, then the cache is
    cut to a budget and attended again. Returns everything it computed."""
    rng = np.random.default_rng(seed)
    N, E, V, H, n_layers, R = 64, 192, 128, 16, 2, 3
    scale = 0.05 if cache == "e4m3" else 1.0
    prompt, steps, budget, recent = np.array([100, 1, 190]), 3, 80, 16
    M = T.Model(lmc, E, cache, N, packed=True, layers=n_layers, state=4096, blocks=24)
    L = M.layout
    full = prompt + steps
    cols = int(-(-full.max() // N))
    ids = rng.permutation(24).astype(np.int32)
    table, fresh = _int32(ids[:R * cols].reshape(R, cols)), _int32(ids[R * cols:R * cols + 2 * R].reshape(R, 2))
    pool = M.pool.to(DEV)
    most = int(full.max())
    weights = torch.zeros((n_layers, R, most), device=DEV)
    ws = torch.empty(lmc.lmc_attend_workspace(L, M.layers[0], R, H, V, most, True), dtype=torch.uint8, device=DEV)
    kept = torch.full((n_layers, R, budget), -1, dtype=torch.int32, device=DEV)
    kept_scores = torch.zeros((n_layers, R, budget), device=DEV)
    kept_lengths = torch.zeros(R, dtype=torch.int32, device=DEV)
    draw = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(T.TYPES[act]).to(DEV)  # noqa: E731
    rows = int(prompt.sum())
    req = _int32(np.repeat(np.arange(R), prompt))
    pos = _int32(np.concatenate([np.arange(n) for n in prompt]))
    first = [draw(rows, E) for _ in range(n_layers)]
    tokens = [[draw(R, E) for _ in range(n_layers)] for _ in range(steps)]
    queries = [[draw(R, H, E) for _ in range(n_layers)] for _ in range(steps + 1)]
    outs = [[torch.empty((R, H, V), dtype=T.TYPES[act], device=DEV) for _ in range(n_layers)] for _ in range(steps + 1)]
    every = _int32(np.arange(R))
    lens = [_int32(prompt + k + 1) for k in range(steps)]
    at = [_int32(prompt + k) for k in range(steps)]

    def work():
        weights.zero_()
        for i, l in enumerate(M.layers):
            lmc.lmc_append(L, l, pool, table, req, pos, first[i], status, scale=scale)
        for k in range(steps):
            for i, l in enumerate(M.layers):
                lmc.lmc_append(L, l, pool, table, every, at[k], tokens[k][i], status, scale=scale)
                lmc.lmc_attend(L, l, pool, table, lens[k], queries[k][i], V, 0.1, outs[k][i], ws, status,
                               max_length=most, scale=scale, weights=weights[i])
        lmc.lmc_select_tokens(weights, lens[-1], budget, recent, kept, kept_scores, kept_lengths, status)
        lmc.lmc_move_tokens(L, M.group, pool, table, fresh, kept, kept_lengths, status)
        for i, l in enumerate(M.layers):
            lmc.lmc_attend(L, l, pool, fresh, kept_lengths, queries[steps][i], V, 0.1, outs[steps][i], ws, status,
                           max_length=most, scale=scale)

    if capture:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            work()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            work()
        for o in outs:
            for x in o:
                x.zero_()
        graph.replay()
        graph.replay()
    else:
        work()
    torch.cuda.synchronize()
    assert status.item() == 0
    return dict(M=M, scale=scale, prompt=prompt, steps=steps, budget=budget, recent=recent, first=first,
                tokens=tokens, queries=queries, outs=outs, weights=weights, kept=kept, kept_lengths=kept_lengths,
                kept_scores=kept_scores, V=V, R=R, pool=pool)


@pytest.mark.parametrize("cache,act", [("bf16", "bf16"), ("e4m3", "bf16"), ("e4m3", "f16")])
def test_serving_loop_of_all_four(lmc, status, cache, act):
    s = _sequence(lmc, cache, act, status, 21, capture=False)
    n_layers = len(s["first"])
    offsets = np.concatenate([[0], np.cumsum(s["prompt"])])
    for r in range(s["R"]):
        for i in range(n_layers):
            rows = [s["first"][i][offsets[r]:offsets[r + 1]]] + [s["tokens"][k][i][r:r + 1] for k in range(s["steps"])]
            x = torch.cat(rows).cpu()
            if cache == "e4m3":
                x = (x.float() / torch.tensor(s["scale"])).clamp(-448, 448).to(torch.float8_e4m3fn)
            e = x.double()
            total, slack = torch.zeros(len(e), dtype=torch.float64), torch.zeros(len(e), dtype=torch.float64)
            for k in range(s["steps"]):
                n = int(s["prompt"][r]) + k + 1
                o, _, w, d_o, _, d_w = T.attend(e[:n], s["queries"][k][i][r].cpu().double(), s["V"], 0.1, s["scale"],
                                                cache, act)
                assert ((s["outs"][k][i][r].cpu().double() - o).abs() <= d_o).all()
                total[:n] += w
                slack[:n] += d_w + 2.0 ** -23 * total[:n]
            got = s["weights"][i, r, : len(e)].cpu()
            assert ((got.double() - total).abs() <= slack).all()
            # the selection follows the weights as the kernels accumulated them
            want = T.select(got.tolist(), len(e), s["budget"], s["recent"])
            assert s["kept"][i, r, : len(want)].tolist() == want
            assert int(s["kept_lengths"][r]) == len(want)
            o, _, _, d_o, _, _ = T.attend(e[want], s["queries"][s["steps"]][i][r].cpu().double(), s["V"], 0.1,
                                          s["scale"], cache, act)
            assert ((s["outs"][s["steps"]][i][r].cpu().double() - o).abs() <= d_o).all()


def test_serving_loop_captured_and_replayed(lmc, status):
    a = _sequence(lmc, "bf16", "bf16", status, 22, capture=False)
    b = _sequence(lmc, "bf16", "bf16", status, 22, capture=True)
    for k in ("weights", "kept", "kept_lengths", "kept_scores"):
        assert torch.equal(a[k], b[k]), k
    for x, y in zip(a["outs"], b["outs"]):
        for u, v in zip(x, y):
            assert torch.equal(u, v)


def test_decode_example_runs():
    """The decode example (tests/example_decode.py, also printed in the README)
    runs as written. Each step adds one unit of weight per head; the last 64
    of 1203 tokens are kept."""
    import example_decode
    got = example_decode.run(DEV)
    assert got["status"] == 0 and got["finite"] and got["kept_length"] == 256
    assert all(abs(w - 3 * 32) <= 3 * 32 * 1e-4 for w in got["weight"])
    assert got["kept"][192:] == list(range(1203 - 64, 1203)) and got["kept"] == sorted(set(got["kept"]))
