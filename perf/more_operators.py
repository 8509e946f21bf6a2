"""What is measured of the operators by which a hybrid model's layers fill the
paged pool: linear attention with a decay for each head over the state pages
(prompts, and one new token per request), entries normalised and rotated on
their way into a paged attention layer, and norms and rotations of queries.

Sizes are those of the library's own workloads: Kimi-Linear (N = 944, 32 state
heads of 128 x 128, a 576-value latent entry of which 64 are rotated), Kimi K3
(N = 768, fp8 entries, 64 state heads, eight of them per GPU where the state is
sharded, 131072 tokens), the mixed step's 256 requests and the tiny four-layer
workload (N = 64, four heads of 64 x 64, requests of 300 and 517 tokens).

`run` with `own` false is the plain form: elementary torch operations in 32
bits (sums of log decays and angles in 64). With `own` true it makes the calls
a user of the library makes.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
CHUNK = 64  # tokens of the plain form's products


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------

def _case(op, **kw):
    c = {"op": op, "packed": False, "N": 944, "act": "bf16", "R": 32, "lo": 8192, "hi": 8192, "fresh": False}
    if op in ("step", "scan"):
        c.update(H=32, Hk=32, dk=128, dv=128, conv=73728, decay="token", snapshots="block")
    else:
        c.update(heads=1, dim=576, norm=512, rot_first=512, rot=64, pairs=True)
    if op == "append":
        c.update(E=576, cache="bf16", scale=1.0, wide=576, state=2170880)
    if op == "rotate":
        c.update(in_place=False)
    c.update(kw)
    return c


_TINY = dict(N=64, R=2, lo=300, hi=517)
_TINY_STATE = dict(H=4, Hk=4, dk=64, dv=64, conv=4608, **_TINY)


def listed():
    return [
        # the rotated part of 256 requests' queries in a decode step, where they lie (latency)
        _case("rotate", name="rotate_decode_256", R=256, lo=1, hi=1, heads=32, dim=192, norm=0, rot_first=128, rot=64,
              in_place=True),
        # queries of a prefill with a norm for each head, halves rotated against one another
        _case("rotate", name="rotate_norm_32x1024", lo=1024, hi=1024, heads=32, dim=128, norm=128, rot_first=0, rot=128,
              pairs=False),
        # the new token's latent of 256 requests: its norm, the rotation of its last 64 values
        _case("append", name="append_decode_256", R=256, lo=1, hi=1),
        # a prefill of 131072 tokens written as fp8 entries
        _case("append", name="append_k3_prefill", N=768, R=4, lo=32768, hi=32768, cache="e4m3", scale=0.0625, state=542720),
        # eight key heads with norms and rotation and eight value heads of 64 as one entry, ragged
        # prompts, rows that are part of a wider product
        _case("append", name="append_kv_ragged_64", packed=True, R=64, lo=1024, hi=32768, E=1024, wide=1536, act="f16",
              cache="f16", heads=8, dim=64, norm=64, rot_first=0, rot=64, pairs=False),
        # one token of the smallest model's state layer (latency)
        _case("step", name="step_tiny", **_TINY_STATE),
        # one state layer of a decode step of the mixed step's 256 requests
        _case("step", name="step_kimi_256", packed=True, R=256, lo=1024, hi=32768),
        # one state layer of K3 with all its heads, four long contexts
        _case("step", name="step_k3_4", N=768, R=4, lo=131072, hi=131072, H=64, Hk=64, conv=147456, act="f16"),
        # the smallest model's two prompts
        _case("scan", name="scan_tiny", fresh=True, **_TINY_STATE),
        # one state layer of Kimi-Linear's prefill of 32 prompts of 8192 tokens
        _case("scan", name="scan_kimi_32x8192", fresh=True),
        # one long prompt on one of eight GPUs of K3, a snapshot at every second block
        _case("scan", name="scan_k3_131072", N=768, R=1, lo=131072, hi=131072, H=8, Hk=8, conv=18432, fresh=True,
              snapshots="second"),
        # ragged prompts that follow cached prefixes, one decay per head for all tokens
        _case("scan", name="scan_ragged_64", packed=True, R=64, lo=1024, hi=32768, act="f16", decay="head"),
    ]


def _between(rng, lo, hi):
    """A whole number, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "step", "append", "rotate"])
    c = {"op": op}
    c["N"] = rng.choice([64, 100, 768, 944, rng.randrange(48, 1000)])
    c["packed"] = rng.random() < 0.5
    c["act"] = rng.choice(["bf16", "bf16", "f16"])
    c["R"] = _between(rng, 1, 256)
    c["fresh"] = rng.random() < 0.5
    if op in ("step", "scan"):
        c["H"] = rng.choice([1, 4, 8, 16, 20, 32, 64])
        c["Hk"] = rng.choice([c["H"], c["H"], 1, c["H"] // 4 if c["H"] % 4 == 0 else 1])
        c["dk"], c["dv"] = rng.choice([(128, 128), (128, 128), (64, 64), (96, 96), (64, 128), (128, 40)])
        c["conv"] = rng.choice([0, 4608, 73728])
        c["decay"] = rng.choice(["token", "token", "head"])
        c["snapshots"] = rng.choice(["block", "second", "last"])
    else:
        c["heads"] = rng.choice([1, 1, 4, 8, 20, 32]) if op == "append" else rng.choice([1, 8, 20, 32, 64])
        c["dim"] = 576 if c["heads"] == 1 and op == "append" else rng.choice([64, 128, 192, 80])
        c["rot"] = rng.choice([64, c["dim"] // 4 * 2, 32])
        c["rot_first"] = rng.choice([0, c["dim"] - c["rot"]])
        c["norm"] = rng.choice([0, c["dim"], c["dim"] - c["rot"] if c["dim"] > c["rot"] else 0])
        c["pairs"] = rng.random() < 0.5
    if op == "append":
        c["E"] = c["heads"] * c["dim"] * (1 if c["heads"] == 1 else 2)
        c["wide"] = c["E"] + rng.choice([0, 64, 3])
        c["cache"] = rng.choice([c["act"], c["act"], "e4m3"])
        c["scale"] = rng.choice([0.03125, 0.0625, 0.05]) if c["cache"] == "e4m3" else 1.0
        c["state"] = rng.choice([0, 542720])
    if op == "rotate":
        c["in_place"] = rng.random() < 0.5
    # tokens of a call: at most the largest listed case's
    per = c["H"] * 8 if op == "scan" else c["heads"] * c["dim"] // 16 if op == "rotate" else c.get("E", 16) // 16
    most = 1 if op == "step" else max(1, min(131072, (1 << 25) // per // c["R"]))
    c["hi"] = _between(rng, 1, most)
    if op == "step":
        c["hi"] = _between(rng, 1, 131072)
    c["lo"] = rng.choice([0, c["hi"], c["hi"] // 2]) if op != "step" else rng.choice([0, c["hi"]])
    return c


# ----------------------------------------------------------------------------
# What a program has in hand
# ----------------------------------------------------------------------------

def _lengths(c, seed=0):
    """The requests' lengths: the case gives them, the seed their order (so
    that the pool's size, and with it an output's shape, is the case's)."""
    g = np.random.default_rng(c["R"] + c["hi"])
    if c["lo"] == c["hi"]:
        x = np.full(c["R"], c["hi"])
    elif (c["lo"], c["hi"]) == (300, 517):
        x = np.array([300, 517])
    elif c["lo"] == 1024:
        x = np.clip(np.floor(np.exp(g.normal(math.log(4096.0), 1.0, c["R"]))), c["lo"], c["hi"])
    else:
        x = g.integers(c["lo"], c["hi"] + 1, c["R"])
        x[0] = c["hi"]
    return np.random.default_rng(seed).permutation(x.astype(np.int64))


def _before(c, lengths):
    """Tokens that a request holds before the call."""
    if c["op"] == "step":
        return lengths
    return np.zeros_like(lengths) if c["fresh"] else lengths * 7919 % (3 * c["N"])


def _blocks(total, N):
    return -(-total // N)


def _state_blocks(c, had, new):
    """Which block positions of each request hold a state, [R, cols]: the one
    before the call's tokens, the last one, and snapshots between."""
    N = c["N"]
    cols = max(1, int(_blocks(had + new, N).max()))
    at = np.arange(cols)[None, :]
    first, last = _blocks(had, N)[:, None] - 1, _blocks(had + new, N)[:, None] - 1
    step = {"block": 1, "second": 2, "last": cols + 1}[c["snapshots"]]
    return (at == first) | (at == last) | ((at > first) & (at < last) & (at % step == step - 1))


def _randn(gen, shape, act):
    return torch.randn(shape, generator=gen, device=DEV, dtype=DTYPES[act])


def _plan(c, had, new, table):
    """The plain form's chunks: runs of up to CHUNK tokens of one block of one
    request, in order, with the page (or -1) that the state after them is
    written to, and each request's chunks in turn."""
    N, rows, chunks, turns = c["N"], 0, [], []
    for r in range(len(new)):
        p, end, mine = int(had[r]), int(had[r] + new[r]), []
        while p < end:
            stop = min(end, (p // N + 1) * N, p + CHUNK)
            keep = stop == end or stop % N == 0
            mine.append(len(chunks))
            chunks.append((rows + p - int(had[r]), stop - p, r, int(table[r, (stop - 1) // N]) if keep else -1))
            p = stop
        rows += int(new[r])
        turns.append(mine)
    a = np.array(chunks or [(0, 0, 0, -1)], dtype=np.int64)
    seq = np.full((max((len(t) for t in turns), default=0), len(new)), len(a), dtype=np.int64)
    for r, t in enumerate(turns):
        seq[: len(t), r] = t
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
    return {"first": up(a[:, 0]), "count": up(a[:, 1]), "page": up(a[:, 3]), "turns": up(seq)}


def _prepare_state(c, s, seed):
    gen, g = s["gen"], np.random.default_rng(seed + 77)
    had = _before(c, s["host_lengths"])
    new = np.ones_like(had) if c["op"] == "step" else s["host_lengths"]
    N, R, H, Hk, dk, dv = c["N"], c["R"], c["H"], c["Hk"], c["dk"], c["dv"]
    held = _state_blocks(c, had, new)
    blocks = int(held.sum()) + 2
    table = np.full(held.shape, -1, dtype=np.int32)
    table[held] = g.permutation(blocks)[: int(held.sum())]
    # one state layer, beside an attention layer of small entries
    rec = H * dk * dv * 4
    page = c["conv"] + rec
    stride = max(page, N * 16)
    s["pool"] = torch.zeros(blocks * stride, dtype=torch.uint8, device=DEV)
    s["pages"] = torch.as_strided(s["pool"].view(torch.float32), (blocks, H, dk, dv), (stride // 4, dk * dv, dv, 1),
                                  c["conv"] // 4)
    s["pages"].normal_(0.0, 0.3, generator=gen)
    s["table"] = torch.from_numpy(table).to(DEV)
    s["had"] = torch.from_numpy(had.astype(np.int32)).to(DEV)
    rows = int(new.sum())
    s["starts"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).to(DEV)
    s["q"] = _randn(gen, (rows, Hk, dk), c["act"])
    s["k"] = _randn(gen, (rows, Hk, dk), c["act"]).mul_(dk ** -0.5)
    s["v"] = _randn(gen, (rows, H, dv), c["act"])
    if c["decay"] == "head":
        # one decay per head: 1 - 2^-5 ... 1 - 2^-11
        x = 1.0 - 2.0 ** -torch.linspace(5.0, 11.0, H, device=DEV, dtype=torch.float64)
        s["decay"] = torch.log(x).float().expand(rows, H)
    else:
        # gates of a token: most forget little, some nearly all
        x = torch.randn((rows, H), generator=gen, device=DEV)
        s["decay"] = -torch.exp(2.0 * x - 4.0)
    s["scale"] = dk ** -0.5
    s["out"] = torch.zeros((rows, H, dv), dtype=DTYPES[c["act"]], device=DEV)
    if c["op"] == "scan":
        s["plan"] = _plan(c, had, new, table)
    else:
        at = np.arange(R)
        s["from"] = torch.from_numpy(np.where(had > 0, table[at, np.maximum(had - 1, 0) // N], -1)).to(DEV).long()
        s["to"] = torch.from_numpy(table[at, had // N]).to(DEV).long()
    if own:
        import state_cache_paging_gb300 as lmc

        spec = [{"kind": "KDA", "conv_bytes": c["conv"], "rec_bytes": rec}, {"kind": "MLA", "token_bytes": 16}]
        s["layout"] = lmc.lmc_layout_build(spec, N, c["packed"], blocks * stride)
        assert s["layout"].num_blocks == blocks
        if c["op"] == "scan":
            n = lmc.lmc_linear_scan_workspace(s["layout"], 0, R, rows, H)
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)


def _prepare_rotation(c, s, seed):
    gen, g = s["gen"], np.random.default_rng(seed + 77)
    new, R, N = s["host_lengths"], c["R"], c["N"]
    had, rows = _before(c, new), int(new.sum())
    pos = np.arange(rows) - np.repeat(np.cumsum(new) - new, new) + np.repeat(had, new)
    s["positions"] = torch.from_numpy(pos.astype(np.int32)).to(DEV)
    # angles of contexts far into a long conversation
    s["angles"] = s["positions"] + 100000
    s["frequencies"] = (10000.0 ** -(torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64) * 2 / c["rot"])).float()
    s["weight"] = 1.0 + 0.1 * torch.randn(c["norm"], generator=gen, device=DEV) if c["norm"] else None
    s["eps"] = 1e-6
    if c["op"] == "rotate":
        s["x"] = _randn(gen, (rows, c["heads"], c["dim"]), c["act"])
        s["out"] = s["x"] if c["in_place"] else torch.zeros_like(s["x"])
        return
    s["entries"] = _randn(gen, (rows, c["wide"]), c["act"])[:, : c["E"]]
    s["requests"] = torch.from_numpy(np.repeat(np.arange(R), new).astype(np.int32)).to(DEV)
    per = _blocks(had + new, N)
    blocks = int(per.sum()) + 3
    table = np.full((R, max(1, int(per.max()))), -1, dtype=np.int32)
    table[np.arange(table.shape[1])[None, :] < per[:, None]] = g.permutation(blocks)[: int(per.sum())]
    s["table"] = torch.from_numpy(table).to(DEV)
    tb = c["E"] * (1 if c["cache"] == "e4m3" else 2)
    stride = max(N * tb, c["state"])
    s["pool"] = torch.zeros(blocks * stride, dtype=torch.uint8, device=DEV)
    s["view"] = torch.as_strided(s["pool"], (blocks, N, tb), (stride, tb, 1))
    if own:
        import state_cache_paging_gb300 as lmc

        spec = [{"kind": "KDA", "conv_bytes": 0, "rec_bytes": c["state"]}] if c["state"] else []
        s["layer"] = len(spec)
        s["layout"] = lmc.lmc_layout_build(spec + [{"kind": "MLA", "token_bytes": tb}], N, c["packed"], blocks * stride)
        assert s["layout"].num_blocks == blocks


def prepare(case, seed):
    c = _case(**case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"case": c, "gen": gen, "host_lengths": _lengths(c, seed),
         "status": torch.zeros(1, dtype=torch.int32, device=DEV)}
    (_prepare_state if c["op"] in ("step", "scan") else _prepare_rotation)(c, s, seed)
    return s


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------

def _heads(x, H):
    """Values of key heads, 32 bits, for each of the H state heads."""
    return x.float().repeat_interleave(H // x.shape[-2], dim=-2)


def _step(s):
    c = s["case"]
    S = s["pages"][s["from"].clamp(min=0)] * (s["from"] >= 0)[:, None, None, None]
    k, q = _heads(s["k"], c["H"]), _heads(s["q"], c["H"])
    S = S * torch.exp(s["decay"])[:, :, None, None] + k[..., None] * s["v"].float()[:, :, None, :]
    s["out"].copy_((q[..., None] * S).sum(-2) * s["scale"])
    s["pages"][s["to"]] = S
    return {"out": s["out"], "state": s["pages"]}


def _scan(s):
    c, p = s["case"], s["plan"]
    H = c["H"]
    at = torch.arange(CHUNK, device=DEV)
    valid = at < p["count"][:, None]
    row = torch.where(valid, p["first"][:, None] + at, torch.zeros_like(p["first"])[:, None])
    if s["q"].shape[0] == 0:
        return {"out": s["out"], "state": s["pages"]}
    take = lambda x: torch.where(valid[:, :, None, None], x[row], torch.zeros((), dtype=x.dtype, device=DEV))  # noqa: E731
    q = _heads(take(s["q"]), H).permute(0, 2, 1, 3)
    k = _heads(take(s["k"]), H).permute(0, 2, 1, 3)
    v = take(s["v"]).float().permute(0, 2, 1, 3)
    G = torch.where(valid[:, :, None], s["decay"][row].double(), 0.0).cumsum(1).permute(0, 2, 1)  # [chunks, H, CHUNK]
    U = (k * torch.exp(G[:, :, -1:] - G).float()[..., None]).transpose(2, 3) @ v
    U = torch.cat([U, torch.zeros_like(U[:1])])  # the last one: no chunk
    decay = torch.cat([torch.exp(G[:, :, -1]).float(), torch.ones((1, H), device=DEV)])
    before = torch.empty_like(U)
    had = s["had"].long()
    first = s["table"].long().gather(1, ((had - 1).clamp(min=0) // c["N"])[:, None])[:, 0]
    S = s["pages"][first.clamp(min=0)] * (had > 0)[:, None, None, None]
    for now in p["turns"]:
        before[now] = S
        S = S * decay[now][:, :, None, None] + U[now]
        U[now] = S
        U[-1] = 0.0
    inside = torch.tril(torch.exp(G[..., :, None] - G[..., None, :]).nan_to_num(posinf=0.0).float())
    o = (q @ before[:-1]) * torch.exp(G).float()[..., None] + ((q @ k.transpose(2, 3)) * inside) @ v
    s["out"][row[valid]] = (o * s["scale"]).permute(0, 2, 1, 3)[valid].to(s["out"].dtype)
    kept = torch.nonzero(p["page"] >= 0)[:, 0]
    s["pages"][p["page"][kept]] = U[kept]
    return {"out": s["out"], "state": s["pages"]}


def _turned(c, s, x):
    """Heads [rows, heads, dim] in 32 bits, normalised and rotated."""
    x = x.float()
    if c["norm"]:
        n = x[..., : c["norm"]]
        n = n * torch.rsqrt((n * n).mean(-1, keepdim=True) + s["eps"]) * s["weight"]
        x = torch.cat([n, x[..., c["norm"]:]], dim=-1)
    f, rot = c["rot_first"], c["rot"]
    angle = s["angles"].double()[:, None, None] * s["frequencies"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    y = x[..., f: f + rot]
    a, b = (y[..., 0::2], y[..., 1::2]) if c["pairs"] else (y[..., : rot // 2], y[..., rot // 2:])
    a, b = a * cos - b * sin, a * sin + b * cos
    y = torch.stack([a, b], dim=-1).flatten(-2) if c["pairs"] else torch.cat([a, b], dim=-1)
    return torch.cat([x[..., :f], y, x[..., f + rot:]], dim=-1)


def _append(s):
    c, req, pos = s["case"], s["requests"].long(), s["positions"].long()
    width = c["heads"] * c["dim"]
    x = s["entries"]
    y = _turned(c, s, x[:, :width].unflatten(1, (c["heads"], c["dim"]))).flatten(1)
    y = torch.cat([y, x[:, width:].float()], dim=1)
    if c["cache"] == "e4m3":
        y = (y / c["scale"]).clamp(-448.0, 448.0)
    y = y.to(DTYPES[c["cache"]])
    block = s["table"].long()[req, pos // c["N"]]
    s["view"][block, pos % c["N"]] = y.view(torch.uint8)
    return _typed(s)


def _typed(s):
    return s["view"].view(DTYPES[s["case"]["cache"]])


def run(s):
    c = s["case"]
    if not own:
        if c["op"] == "rotate":
            return s["out"].copy_(_turned(c, s, s["x"]))
        return {"append": _append, "step": _step, "scan": _scan}[c["op"]](s)
    import state_cache_paging_gb300 as lmc

    if c["op"] == "rotate":
        lmc.lmc_rotate(s["x"], s["angles"], s["out"], s["frequencies"], rot_first=c["rot_first"], pairs=c["pairs"],
                       norm_dim=c["norm"], norm_weight=s["weight"], eps=s["eps"])
        return s["out"]
    if c["op"] == "append":
        lmc.lmc_append_rotated(s["layout"], s["layer"], s["pool"], s["table"], s["requests"], s["positions"], s["entries"],
                               s["status"], s["frequencies"], num_heads=c["heads"], head_dim=c["dim"],
                               rot_first=c["rot_first"], pairs=c["pairs"], norm_dim=c["norm"], norm_weight=s["weight"],
                               eps=s["eps"], angles=s["angles"], scale=c["scale"])
        return _typed(s)
    if c["op"] == "step":
        lmc.lmc_linear_step(s["layout"], 0, s["pool"], s["table"], s["had"], s["q"], s["k"], s["v"], s["decay"], s["out"],
                            s["status"], scale=s["scale"])
    else:
        lmc.lmc_linear_scan(s["layout"], 0, s["pool"], s["table"], s["starts"], s["had"], s["q"], s["k"], s["v"],
                            s["decay"], s["out"], s["workspace"], s["status"], scale=s["scale"])
    return {"out": s["out"], "state": s["pages"]}


# ----------------------------------------------------------------------------
# What a pass cannot do without, and its values in 64 bits
# ----------------------------------------------------------------------------

def work(case):
    c = _case(**case)
    lengths = _lengths(c)
    had, rows = _before(c, lengths), int(lengths.sum())
    if c["op"] == "rotate":
        i, j = c["rot_first"], c["rot_first"] + c["rot"]
        touched = c["dim"]
        if c["in_place"]:  # what is neither normalised nor rotated stays where it is
            touched = max(0, c["norm"] - (max(0, min(j, c["norm"]) - i))) + c["rot"] if i < c["norm"] else c["norm"] + c["rot"]
        return {"bytes": rows * (4 * c["heads"] * touched + 4), "flops": rows * c["heads"] * (3 * c["rot"] + 4 * c["norm"])}
    if c["op"] == "append":
        tb = c["E"] * (1 if c["cache"] == "e4m3" else 2)
        return {"bytes": rows * (2 * c["E"] + tb + 12), "flops": rows * c["heads"] * (3 * c["rot"] + 4 * c["norm"])}
    new = np.ones_like(lengths) if c["op"] == "step" else lengths
    state = c["H"] * c["dk"] * c["dv"] * 4
    some = new > 0
    held = _state_blocks(c, had, new)
    at = np.arange(held.shape[1])[None, :]
    # pages read: the state before the call; pages written: every one from the first token's on
    read = int((some & (had > 0)).sum())
    written = int((held & (at >= (had // c["N"])[:, None]) & some[:, None]).sum())
    tokens = int(new.sum())
    decays = 4 * c["H"] if c["decay"] == "head" else 4 * c["H"] * tokens
    return {"bytes": tokens * 4 * (c["Hk"] * c["dk"] + c["H"] * c["dv"]) + decays + (read + written) * state,
            "flops": 4 * tokens * c["H"] * c["dk"] * c["dv"]}


def _exact_state(c, s):
    """Token by token, requests side by side, the longest first."""
    had = _before(c, s["host_lengths"])
    new = np.ones_like(had) if c["op"] == "step" else s["host_lengths"]
    start = np.cumsum(new) - new
    order = np.argsort(-new, kind="stable")
    table = s["table"].cpu().numpy()
    pages, H, N = s["pages"].double(), c["H"], c["N"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    S = torch.zeros((c["R"], H, c["dk"], c["dv"]), dtype=torch.float64, device=DEV)
    for i, r in enumerate(order):
        if had[r] > 0:
            S[i] = pages[int(table[r, (had[r] - 1) // N])]
    first = torch.from_numpy(start[order]).to(DEV)
    head = torch.arange(H, device=DEV) // (H // c["Hk"])
    k, q, v = s["k"].double()[:, head], s["q"].double()[:, head], s["v"].double()
    a = torch.exp(s["decay"].double())
    for t in range(int(new.max(initial=0))):
        n = int((new > t).sum())
        rows = first[:n] + t
        here = S[:n].view(n * H, c["dk"], c["dv"])
        here.mul_(a[rows].view(-1, 1, 1)).baddbmm_(k[rows].view(n * H, -1, 1), v[rows].view(n * H, 1, -1))
        out[rows] = torch.bmm(q[rows].view(n * H, 1, -1), here).view(n, H, c["dv"])
        done = had[order[:n]] + t + 1
        for i in np.nonzero((done % N == 0) | (new[order[:n]] == t + 1))[0]:
            page = int(table[order[i], (done[i] - 1) // N])
            if page >= 0:
                pages[page] = S[i]
    return {"out": out.mul_(s["scale"]), "state": pages}


def _exact_heads(c, s, x):
    """Complex numbers in 64 bits."""
    x = x.double().clone()
    if c["norm"]:
        power = x[..., : c["norm"]].square().sum(-1, keepdim=True) / c["norm"]
        x[..., : c["norm"]] *= s["weight"].double() / torch.sqrt(power + s["eps"])
    f, rot = c["rot_first"], c["rot"]
    i = torch.arange(rot // 2, device=DEV)
    a, b = (f + 2 * i, f + 2 * i + 1) if c["pairs"] else (f + i, f + rot // 2 + i)
    z = torch.complex(x[..., a], x[..., b])
    angle = s["angles"].double()[:, None, None] * s["frequencies"].double()
    z = z * torch.polar(torch.ones_like(angle), angle)
    x[..., a], x[..., b] = z.real, z.imag
    return x


def exact(case, seed):
    c = _case(**case)
    s = prepare(case, seed)
    if c["op"] in ("step", "scan"):
        return _exact_state(c, s)
    if c["op"] == "rotate":
        return _exact_heads(c, s, s["x"])
    if c["cache"] == "e4m3":
        return None  # a rounding to eight bits, not a number in 64
    got, pos, width = _typed(s).double(), s["positions"].long(), c["heads"] * c["dim"]
    x = s["entries"].double()
    heads = _exact_heads(c, s, x[:, :width].reshape(-1, c["heads"], c["dim"]))
    x = torch.cat([heads.reshape(-1, width), x[:, width:]], dim=1)
    got[s["table"].long()[s["requests"].long(), pos // c["N"]], pos % c["N"]] = x
    return got
