"""What is measured of the paged-cache operators: appending token entries to a
paged attention layer, attention of one new token over the paged cache,
selecting the tokens a request keeps by their accumulated attention weight,
and moving the kept tokens' entries into other blocks.

Sizes are those of the library's own workloads: Kimi-Linear (24 layers,
N = 944, a 576-value latent entry of which 512 are the value, 32 heads), Kimi
K3 (N = 768, fp8 entries, 64 heads, 131072 tokens, KDA state sharded over
eight GPUs), the mixed step's sliding window (4096) and the tiny four-layer
workload (N = 64, requests of 300 and 517 tokens).

`run` with `own` false is the plain form: elementary torch operations in 32
bits. With `own` true it makes the calls a user of the library makes.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------

def _case(op, **kw):
    c = {"op": op, "packed": False, "N": 944, "layers": 6, "state": 2170880, "E": 576, "V": 512, "cache": "bf16",
         "act": "bf16", "R": 32, "lo": 8192, "hi": 8192, "heads": 32, "window": 0, "weights": False, "scale": 1.0,
         "budget": 0, "recent": 0, "shared": False}
    c.update(kw)
    return c


_TINY = dict(N=64, layers=1, state=70144, R=2, lo=300, hi=517)
_K3 = dict(N=768, layers=24, state=542720, cache="e4m3", scale=0.0625, heads=64, R=4, lo=131072, hi=131072)


def listed():
    return [
        # one decode step of the smallest model: four heads, two short requests (latency)
        _case("attend", name="attend_tiny", heads=4, **_TINY),
        # one MLA layer of a decode step of Kimi-Linear, 32 requests of 8192 tokens
        _case("attend", name="attend_kimi_32x8192"),
        # the same layer in the packed layout, ragged lengths (median 4096, 1k to 32k), the attention
        # weights accumulated for a later eviction
        _case("attend", name="attend_ragged_weights", packed=True, R=64, lo=1024, hi=32768, weights=True),
        # one MLA layer of K3 over four long contexts, fp8 entries
        _case("attend", name="attend_k3_4x131072", **_K3),
        # a sliding-window layer of the mixed step, 256 ragged requests
        _case("attend", name="attend_window_256", packed=True, R=256, lo=1024, hi=32768, window=4096),
        # the new token's entry of 256 requests (a decode step)
        _case("append", name="append_decode_256", R=256, lo=1, hi=1),
        # a prefill of 131072 tokens written as fp8 entries
        _case("append", name="append_k3_prefill", **{**_K3, "lo": 32768, "hi": 32768}),
        # ragged prompts of 64 requests in the packed layout
        _case("append", name="append_ragged_64", packed=True, R=64, lo=1024, hi=32768),
        # the smallest eviction: two short requests
        _case("select", name="select_tiny", budget=128, recent=32, **_TINY),
        # every layer of K3 selects a quarter of four long contexts
        _case("select", name="select_k3_4x131072", budget=32768, recent=1024, **_K3),
        # six layers, 32 requests: 4096 of 8192 tokens are moved into fresh blocks
        _case("move", name="move_kimi_32x4096", budget=4096, recent=256),
        # 24 layers of K3: 32768 of 131072 tokens of each of four requests
        _case("move", name="move_k3_4x32768", budget=32768, recent=1024, **_K3),
    ]


def _between(rng, lo, hi):
    """A whole number, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "select", "move"])
    c = {"op": op}
    c["N"] = rng.choice([16, 64, 100, 768, 944, rng.randrange(48, 1000)])
    c["packed"] = rng.random() < 0.5
    c["layers"] = rng.randrange(1, 7)
    c["E"], c["V"] = rng.choice([(576, 512), (576, 512), (320, 256), (192, 128), (112, 96)])
    c["cache"] = rng.choice(["bf16", "bf16", "f16", "e4m3"])
    c["act"] = rng.choice(["bf16", "f16"]) if c["cache"] == "e4m3" else c["cache"]
    c["scale"] = rng.choice([0.03125, 0.0625, 0.05]) if c["cache"] == "e4m3" else 1.0
    c["R"] = _between(rng, 1, 256)
    c["hi"] = _between(rng, 1, min(131072, 262144 // c["R"]))
    c["lo"] = rng.choice([0, c["hi"], c["hi"] // 2])
    c["heads"] = rng.choice([1, 4, 8, 16, 20, 32, 64, 96])
    c["window"] = rng.choice([0, 0, _between(rng, 1, 8192)]) if op == "attend" else 0
    c["weights"] = op == "attend" and rng.random() < 0.4
    # the unified page also holds a state page of up to twice the attention page
    page = c["N"] * c["E"] * (1 if c["cache"] == "e4m3" else 2)
    c["state"] = rng.choice([0, page // 2 // 16 * 16, page * 2])
    c["budget"] = _between(rng, 1, max(1, c["hi"])) if op in ("select", "move") else 0
    c["recent"] = rng.randrange(0, c["budget"] + 1) if c["budget"] else 0
    c["shared"] = op in ("select", "move") and rng.random() < 0.3
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


def _token_bytes(c):
    return c["E"] * (1 if c["cache"] == "e4m3" else 2)


def _pool(c, blocks, gen, fill_layers):
    """A pool of `blocks` blocks: c["layers"] paged layers of one group, with
    three state layers beside each where c["state"] > 0. The paged layers
    `fill_layers` hold drawn entries. Returns the pool (bytes) and the layers
    as [layers, blocks, N, entry bytes]: a view of it."""
    tb, n = _token_bytes(c), c["layers"]
    page = c["N"] * tb
    if c["packed"]:
        stride = n * max(page, c["state"])
        base, per_layer = 0, page
        total = blocks * stride
    else:
        stride = max(page, c["state"])
        base, per_layer = 0, stride * blocks
        total = blocks * stride * n
    pool = torch.empty(total, dtype=torch.uint8, device=DEV)
    view = torch.as_strided(pool, (n, blocks, c["N"], tb), (per_layer, stride, tb, 1), base)
    for i in fill_layers:
        x = torch.randn((blocks, c["N"], c["E"]), generator=gen, device=DEV, dtype=torch.float16)
        if c["cache"] == "e4m3":
            x = (x / c["scale"]).to(DTYPES["e4m3"])
        else:
            x = x.to(DTYPES[c["cache"]])
        view[i].copy_(x.view(torch.uint8))
    return pool, view


def _tables(lengths, N, ids):
    """int32 [R, cols]: blocks of `ids` for every position, -1 behind the end."""
    per = -(-lengths // N)
    cols = max(1, int(per.max()))
    t = np.full((len(lengths), cols), -1, dtype=np.int32)
    at = np.arange(cols)[None, :] < per[:, None]
    t[at] = ids[: int(per.sum())]
    return torch.from_numpy(t).to(DEV)


def _blocks_of(lengths, N):
    return int((-(-lengths // N)).sum())


def _handle(c, blocks):
    """The layout handle a user's program keeps."""
    import state_cache_paging_gb300 as lmc

    page = c["N"] * _token_bytes(c)
    paged = {"kind": "SWA" if c["window"] else "MLA", "token_bytes": _token_bytes(c), "window": c["window"]}
    state = {"kind": "KDA", "conv_bytes": 0, "rec_bytes": c["state"]}
    layers = ([state] * 3 if c["state"] else []) + [paged]
    per_block = c["layers"] * max(page, c["state"])
    L = lmc.lmc_layout_build(layers * c["layers"], c["N"], c["packed"], blocks * per_block)
    assert L.num_blocks == blocks
    return L, len(layers) - 1  # the first paged layer


def prepare(case, seed):
    c = _case(**case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    g = np.random.default_rng(seed + 77)
    lengths = _lengths(c, seed)
    s = {"case": c, "lengths": torch.from_numpy(lengths.astype(np.int32)).to(DEV), "max": int(lengths.max()),
         "status": torch.zeros(1, dtype=torch.int32, device=DEV)}
    R, N, act = c["R"], c["N"], DTYPES[c["act"]]
    blocks = 0
    if c["op"] == "attend":
        blocks = max(1, _blocks_of(lengths, N)) + 3
        s["pool"], s["view"] = _pool(c, blocks, gen, [0])
        s["table"] = _tables(lengths, N, g.permutation(blocks).astype(np.int32))
        s["q"] = torch.randn((R, c["heads"], c["E"]), generator=gen, device=DEV).to(act)
        s["softmax_scale"] = 1.0 / math.sqrt(192.0)
        if c["weights"]:
            s["weights"] = torch.rand((R, max(1, s["max"])), generator=gen, device=DEV)
    elif c["op"] == "append":
        # every request holds up to 3 N tokens already; its new rows follow them
        had = lengths * 7919 % (3 * N)
        blocks = _blocks_of(had + lengths, N) + 3
        s["pool"], s["view"] = _pool(c, blocks, gen, [0])
        s["table"] = _tables(had + lengths, N, g.permutation(blocks).astype(np.int32))
        rows = int(lengths.sum())
        req = np.repeat(np.arange(R), lengths)
        pos = np.arange(rows) - np.repeat(np.cumsum(lengths) - lengths, lengths) + np.repeat(had, lengths)
        s["requests"] = torch.from_numpy(req.astype(np.int32)).to(DEV)
        s["positions"] = torch.from_numpy(pos.astype(np.int32)).to(DEV)
        s["entries"] = torch.randn((rows, c["E"]), generator=gen, device=DEV).to(act)
    else:
        sets = 1 if c["shared"] else c["layers"]
        s["kept_lengths"] = torch.zeros(R, dtype=torch.int32, device=DEV)
        if c["op"] == "select":
            # accumulated weights: many small, a few large, some equal
            x = torch.rand((sets, R, max(1, s["max"])), generator=gen, device=DEV)
            x = torch.exp(6.0 * x * x - 3.0)
            s["scores"] = torch.where(x < 0.0625, torch.full_like(x, 0.0625), x)
            s["kept"] = torch.full((sets, R, c["budget"]), -1, dtype=torch.int32, device=DEV)
            s["kept_scores"] = torch.zeros((sets, R, c["budget"]), device=DEV)
        else:
            keep = np.minimum(lengths, c["budget"])
            src, dst = _blocks_of(lengths, N), _blocks_of(keep, N)
            blocks = max(1, src + dst)
            s["pool"], s["view"] = _pool(c, blocks, gen, range(c["layers"]))
            s["src_table"] = _tables(lengths, N, g.permutation(src).astype(np.int32))
            s["dst_table"] = _tables(keep, N, (src + g.permutation(dst)).astype(np.int32))
            s["first_dst"] = src
            # the kept tokens of each set: a drawn choice, in order
            x = torch.rand((sets, R, max(1, s["max"])), generator=gen, device=DEV)
            at = torch.arange(x.shape[2], device=DEV)
            x = torch.where(at < s["lengths"][None, :, None], x, torch.full_like(x, 2.0))
            s["kept_lengths"] = torch.from_numpy(keep.astype(np.int32)).to(DEV)
            rank = torch.argsort(torch.argsort(x, dim=-1), dim=-1)
            chosen = rank < s["kept_lengths"][None, :, None]
            s["kept"] = torch.full((sets, R, c["budget"] + 1), -1, dtype=torch.int32, device=DEV)
            put = torch.where(chosen, torch.cumsum(chosen, -1) - 1, c["budget"])
            s["kept"].scatter_(2, put, at.int().expand_as(put).contiguous())
            s["kept"] = s["kept"][:, :, : c["budget"]].contiguous()
    if own:
        import state_cache_paging_gb300 as lmc

        if c["op"] != "select":
            s["layout"], s["layer"] = _handle(c, blocks)
        if c["op"] == "attend":
            s["out"] = torch.empty((R, c["heads"], c["V"]), dtype=act, device=DEV)
            s["lse"] = torch.empty((R, c["heads"]), device=DEV)
            n = lmc.lmc_attend_workspace(s["layout"], s["layer"], R, c["heads"], c["V"], s["max"], c["weights"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    return s


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------

def _typed(s):
    """The first paged layer as [blocks, N, E] values."""
    return s["view"][0].view(DTYPES[s["case"]["cache"]])


def _attend(s):
    c, lengths = s["case"], s["lengths"].long()
    N, T = c["N"], max(1, min(s["max"], c["window"] or s["max"]))
    first = (lengths - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(lengths)
    pos = first[:, None] + torch.arange(T, device=DEV)[None, :]
    valid = pos < lengths[:, None]
    pos = torch.where(valid, pos, torch.zeros_like(pos))
    block = s["table"].long().gather(1, pos // N).clamp(min=0)
    e = s["view"].view(torch.int64)[0][block, pos % N].view(DTYPES[c["cache"]]).float()
    if c["scale"] != 1.0:
        e.mul_(c["scale"])
    e.masked_fill_(~valid[:, :, None], 0.0)
    x = torch.bmm(s["q"].float(), e.transpose(1, 2)) * s["softmax_scale"]
    x.masked_fill_(~valid[:, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    out = torch.bmm(p, e[:, :, : c["V"]]).to(s["q"].dtype)
    if c["weights"]:
        s["weights"].scatter_add_(1, pos, p.sum(1) * valid)
        return {"out": out, "lse": lse, "weights": s["weights"]}
    return {"out": out, "lse": lse}


def _append(s):
    c, req, pos = s["case"], s["requests"].long(), s["positions"].long()
    block = s["table"].long()[req, pos // c["N"]]
    x = s["entries"]
    if c["cache"] == "e4m3":
        x = (x.float() / c["scale"]).clamp(-448.0, 448.0).to(DTYPES["e4m3"])
    s["view"].view(torch.int64)[0][block, pos % c["N"]] = x.view(torch.int64)
    return _typed(s)


def _select(s):
    c, L = s["case"], s["lengths"].long()[None, :, None]
    x = s["scores"]
    at = torch.arange(x.shape[2], device=DEV)[None, None, :]
    everything = L <= c["budget"]
    ranked = at < L - c["recent"]
    order = torch.argsort(torch.where(ranked, x, torch.full_like(x, -math.inf)), dim=-1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(2, order, at.expand_as(order))
    chosen = (at < L) & (everything | ~ranked | (rank < c["budget"] - c["recent"]))
    put = torch.where(chosen, torch.cumsum(chosen, -1) - 1, c["budget"])
    pad = torch.nn.functional.pad
    kept = pad(s["kept"], (0, 1)).scatter_(2, put, at.int().expand_as(put).contiguous())
    scores = pad(s["kept_scores"], (0, 1)).scatter_(2, put, x)
    return {"kept": kept[:, :, :-1], "scores": scores[:, :, :-1],
            "lengths": s["lengths"].clamp(max=c["budget"])}


def _move(s):
    c, N = s["case"], s["case"]["N"]
    n, R, K = c["layers"], c["R"], c["budget"]
    kept = s["kept"].long().expand(n, R, K)
    at = torch.arange(K, device=DEV)
    layer, req, j = torch.nonzero((at < s["kept_lengths"][:, None]).expand(n, R, K), as_tuple=True)
    pos = kept[layer, req, j]
    words = s["view"].view(torch.int64)
    words[layer, s["dst_table"].long()[req, j // N], j % N] = words[layer, s["src_table"].long()[req, pos // N], pos % N]
    return words[:, s["first_dst"]:]


def run(s):
    c = s["case"]
    if not own:
        return {"attend": _attend, "append": _append, "select": _select, "move": _move}[c["op"]](s)
    import state_cache_paging_gb300 as lmc

    if c["op"] == "attend":
        lmc.lmc_attend(s["layout"], s["layer"], s["pool"], s["table"], s["lengths"], s["q"], c["V"],
                       s["softmax_scale"], s["out"], s["workspace"], s["status"], max_length=s["max"],
                       scale=c["scale"], lse=s["lse"], weights=s.get("weights"))
        got = {"out": s["out"], "lse": s["lse"]}
        return {**got, "weights": s["weights"]} if c["weights"] else got
    if c["op"] == "append":
        lmc.lmc_append(s["layout"], s["layer"], s["pool"], s["table"], s["requests"], s["positions"], s["entries"],
                       s["status"], scale=c["scale"])
        return _typed(s)
    if c["op"] == "select":
        lmc.lmc_select_tokens(s["scores"], s["lengths"], c["budget"], c["recent"], s["kept"], s["kept_scores"],
                              s["kept_lengths"], s["status"])
        return {"kept": s["kept"], "scores": s["kept_scores"], "lengths": s["kept_lengths"]}
    lmc.lmc_move_tokens(s["layout"], s["layout"].kv_group[s["layer"]], s["pool"], s["src_table"], s["dst_table"],
                        s["kept"], s["kept_lengths"], s["status"])
    return s["view"].view(torch.int64)[:, s["first_dst"]:]


# ----------------------------------------------------------------------------
# What a pass cannot do without, and its values in 64 bits
# ----------------------------------------------------------------------------

def work(case):
    c = _case(**case)
    lengths = _lengths(c)
    tb = _token_bytes(c)
    tokens = int(np.minimum(lengths, c["window"]).sum() if c["window"] else lengths.sum())
    if c["op"] == "attend":
        vectors = c["R"] * c["heads"] * (2 * (c["E"] + c["V"]) + 4)
        return {"bytes": tokens * (tb + (8 if c["weights"] else 0)) + vectors + 4 * c["R"],
                "flops": 2 * tokens * c["heads"] * (c["E"] + c["V"])}
    if c["op"] == "append":
        return {"bytes": tokens * (2 * c["E"] + tb + 8), "flops": 0}
    sets = 1 if c["shared"] else c["layers"]
    keep = int(np.minimum(lengths, c["budget"]).sum())
    if c["op"] == "select":
        return {"bytes": 4 * sets * tokens + 8 * sets * keep + 8 * c["R"], "flops": 0}
    return {"bytes": 2 * c["layers"] * keep * tb + 4 * sets * keep, "flops": 0}


def exact(case, seed):
    c = _case(**case)
    s = prepare(case, seed)
    if c["op"] == "append":
        if c["cache"] == "e4m3":
            return None  # a rounding to eight bits, not a number in 64
        got = _typed(s).double()
        req, pos = s["requests"].long(), s["positions"].long()
        got[s["table"].long()[req, pos // c["N"]], pos % c["N"]] = s["entries"].double()
        return got
    if c["op"] != "attend":
        return None  # whole numbers, and values that are only moved
    entries = _typed(s)
    out = torch.zeros((c["R"], c["heads"], c["V"]), dtype=torch.float64, device=DEV)
    lse = torch.full((c["R"], c["heads"]), -math.inf, dtype=torch.float64, device=DEV)
    weights = s["weights"].double() if c["weights"] else None
    table, lengths = s["table"].cpu().numpy(), s["lengths"].cpu().numpy()
    for r in range(c["R"]):
        n = int(lengths[r])
        lo = max(0, n - c["window"]) if c["window"] else 0
        if n == 0:
            continue
        first, last = lo // c["N"], (n - 1) // c["N"] + 1
        ids = torch.from_numpy(table[r, first:last].astype(np.int64)).to(DEV)
        e = s["view"][0][ids].view(entries.dtype).reshape(-1, c["E"])
        e = e[lo - first * c["N"]: n - first * c["N"]].double() * c["scale"]
        x = (s["q"][r].double() @ e.T) * s["softmax_scale"]
        lse[r] = torch.logsumexp(x, dim=-1)
        w = torch.exp(x - lse[r][:, None])
        out[r] = w @ e[:, : c["V"]]
        if weights is not None:
            weights[r, lo:n] += w.sum(0)
    return {"out": out, "lse": lse, "weights": weights} if c["weights"] else {"out": out, "lse": lse}
