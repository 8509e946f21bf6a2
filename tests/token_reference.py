"""Plain 64-bit forms of the token operators, and the pools their tests use.

Everything here works on host tensors from the layout's descriptors; nothing
is shared with the library's kernels. `Model` is one group of paged layers
(with state layers beside them) over a pool whose every byte starts as a
pattern that reads as NaN in each entry type, so a read outside the entries
written shows.
"""
from __future__ import annotations

import math

import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
#: half a step relative to the value
HALF_STEP = {k: torch.finfo(t).eps / 2 for k, t in TYPES.items()}


class Model:
    def __init__(self, lmc, E, cache, N, packed=False, layers=1, window=0, state=0, blocks=8):
        self.E, self.cache, self.N, self.n = E, cache, N, layers
        tb = E * (1 if cache == "e4m3" else 2)
        paged = {"kind": "SWA" if window else "MLA", "token_bytes": tb, "window": window}
        spec = ([{"kind": "KDA", "rec_bytes": state}] * 3 if state else []) + [paged]
        per = max(N * tb, state) * layers
        self.layout = lmc.lmc_layout_build(spec * layers, N, packed, blocks * per)
        assert self.layout.num_blocks == blocks
        self.layers = [i for i, k in enumerate(self.layout.kinds) if k != "KDA"]
        self.group = self.layout.kv_group[self.layers[0]]
        self.window, self.tb, self.blocks = window, tb, blocks
        # 0xFF: NaN as bf16, f16 and e4m3
        self.pool = torch.full((self.layout.pool_bytes,), 0xFF, dtype=torch.uint8)

    def pages(self, i, pool=None):
        """Layer i (of the paged ones) as [blocks, N, entry bytes]: a view of the pool."""
        L, l = self.layout, self.layers[i]
        return torch.as_strided(self.pool if pool is None else pool, (self.blocks, self.N, self.tb),
                                (L.stride[l], self.tb, 1), L.base[l])

    def write(self, i, table, r, t0, values):
        """Values [tokens, E] become the entries t0.. of request r."""
        if values.shape[0] == 0:
            return
        raw = values.to(TYPES[self.cache]).contiguous().view(torch.uint8)
        pages = self.pages(i)
        for k in range(raw.shape[0]):
            b = int(table[r, (t0 + k) // self.N])
            pages[b, (t0 + k) % self.N] = raw[k]

    def read(self, i, table, r, positions):
        """Entries in 64 bits (as the cached type holds them)."""
        pages = self.pages(i)
        t = torch.as_tensor(positions, dtype=torch.long)
        raw = pages[table[r].long()[t // self.N], t % self.N].contiguous()
        return raw.view(TYPES[self.cache]).double()


def tables(lengths, N, blocks, rng, cols=None):
    per = [-(-int(n) // N) for n in lengths]
    ids = rng.permutation(blocks)
    t = np.full((len(lengths), cols or max(1, max(per, default=1))), -1, dtype=np.int32)
    k = 0
    for r, p in enumerate(per):
        t[r, :p] = ids[k:k + p]
        k += p
    return torch.from_numpy(t)


def attend(entries, q, value_dim, softmax_scale, scale, cache, act):
    """One request: entries [T, E] and q [H, E] in 64 bits. Returns out, lse,
    the token weights and for each the most that the kernel's roundings can
    move it (see below)."""
    H, E = q.shape
    if entries.shape[0] == 0:
        zero = torch.zeros((H, value_dim), dtype=torch.float64)
        return zero, torch.full((H,), -math.inf, dtype=torch.float64), torch.zeros(0, dtype=torch.float64), zero, 0.0, 0.0
    k = entries * scale
    x = (q @ k.T) * softmax_scale
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[:, None])
    v = k[:, :value_dim]
    out = p @ v
    # The products are exact in binary32 accumulators; a sum of E of them in
    # any order, truncated at each step, is off by at most E * 2^-23 of the
    # absolute sum. Scaling, the change to base two and the exponential add
    # 2^-20 relative. Where the cache is fp8 and q bf16, q is brought to f16
    # with a power of two: what lies 2^24 below the head's largest is lost.
    absolute = (q.abs() @ k.abs().T) * abs(softmax_scale)
    lost = (q.abs().amax(-1, keepdim=True) * 2.0 ** -24) * k.abs().sum(-1)[None] * abs(softmax_scale)
    dx = (absolute * E * 2.0 ** -23 + lost).amax(-1) + x.abs().amax(-1) * 2.0 ** -22
    dp = 2 * dx + 2.0 ** -20
    # p is rounded to the tensor cores' type (f16 for an fp8 cache) before the
    # second product, and the result to the output's; the T sums in binary32.
    half = HALF_STEP["f16" if cache == "e4m3" else cache]
    T = entries.shape[0]
    spread = p @ v.abs()
    d_out = spread * (half + dp[:, None] + T * 2.0 ** -23) + out.abs() * HALF_STEP[act]
    # values under the smallest normal are rounded to steps of fixed size
    tiny = 2.0 ** -24 if "f16" in (act, cache) or cache == "e4m3" else 0.0
    d_out = d_out + tiny * (1 + v.abs().amax())
    weights = p.sum(0)
    return (out, lse, weights, d_out, dx + T * 2.0 ** -23 + 2.0 ** -20 * (1 + lse.abs()),
            (p * (dp + T * 2.0 ** -23)[:, None]).sum(0) + H * 2.0 ** -23 * weights)


def select(scores, length, budget, recent):
    """One request: the kept positions, in increasing order."""
    if length <= budget:
        return list(range(length))
    n = length - recent
    x = [float(s) for s in scores[:n]]
    order = sorted(range(n), key=lambda t: (1 if x[t] != x[t] else 0, -x[t] if x[t] == x[t] else 0.0, t))
    return sorted(order[: budget - recent]) + list(range(n, length))
