"""Plain 64-bit forms of linear attention over state pages and of norms and
rotations, and the pools their tests use. Works on host tensors from the
layout's descriptors; nothing is shared with the library's kernels."""
from __future__ import annotations

import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
#: half a step relative to the value
HALF_STEP = {k: torch.finfo(t).eps / 2 for k, t in TYPES.items()}


class States:
    """State layers of a pool whose every byte starts as 0xFF (NaN in binary32)."""

    def __init__(self, lmc, H, dk, dv, N, blocks, conv=48, packed=False, layers=2):
        self.H, self.dk, self.dv, self.N, self.blocks = H, dk, dv, N, blocks
        rec = H * dk * dv * 4
        spec = [{"kind": "KDA", "conv_bytes": conv, "rec_bytes": rec}, {"kind": "MLA", "token_bytes": 16}] * layers
        per = max(conv + rec, N * 16) * layers
        self.layout = lmc.lmc_layout_build(spec, N, packed, blocks * per)
        assert self.layout.num_blocks == blocks
        self.layer = 2 * (layers - 1)  # the last state layer
        self.conv = conv
        self.pool = torch.full((self.layout.pool_bytes,), 0xFF, dtype=torch.uint8)

    def pages(self, pool=None):
        """[blocks, H, dk, dv] float32: a view of the pool."""
        L, l = self.layout, self.layer
        p = (self.pool if pool is None else pool).view(torch.float32)
        return torch.as_strided(p, (self.blocks, self.H, self.dk, self.dv),
                                (L.stride[l] // 4, self.dk * self.dv, self.dv, 1), (L.base[l] + self.conv) // 4)


def tables(had, new, N, blocks, rng, held=None):
    """int32 [R, cols]: a block of its own for every position; positions that
    `held` (r, position) says no to, before the last one, get -1."""
    per = [-(-(max(0, h) + t) // N) for h, t in zip(had, new)]
    t = np.full((len(had), max([1, *per])), -1, dtype=np.int32)
    ids = iter(rng.permutation(blocks))
    for r, p in enumerate(per):
        for b in range(p):
            if b == p - 1 or b == (had[r] - 1) // N or held is None or held(r, b):
                t[r, b] = next(ids)
    return torch.from_numpy(t)


def linear(S, q, k, v, decay, scale, ends=()):
    """One request, token by token: S [H, dk, dv] (64 bits), q, k [T, Hk, dk], v
    [T, H, dv], decay [T, H]. Returns out, the sums of the absolute terms that
    make out, the states after the tokens counted in `ends` (1 ..) and theirs."""
    T, H = v.shape[0], S.shape[0]
    head = torch.arange(H) // (H // q.shape[1])
    S, A = S.clone(), S.abs()
    out, mag, kept = torch.zeros(v.shape, dtype=torch.float64), torch.zeros(v.shape, dtype=torch.float64), {}
    for t in range(T):
        a = torch.exp(decay[t].double())[:, None, None]
        x = k[t, head].double()[:, :, None] * v[t].double()[:, None, :]
        S, A = S * a + x, A * a + x.abs()
        y = q[t, head].double()
        out[t] = scale * torch.einsum("hi,hij->hj", y, S)
        mag[t] = abs(scale) * torch.einsum("hi,hij->hj", y.abs(), A)
        if t + 1 in ends:
            kept[t + 1] = (S.clone(), A.clone())
    return out, mag, kept


def turned(x, norm_dim, weight, eps, angles, freqs, rot_first, pairs, mscale):
    """Heads [rows, heads, dim] in 64 bits, and a bound on what binary32 may
    lose of each value."""
    x = x.double().clone()
    # A sum of n squares in any order is off by at most n 2^-24 of itself; mean,
    # root, quotient and two products add less than 8 more steps.
    lost = torch.zeros_like(x)
    if norm_dim:
        n = x[..., :norm_dim]
        w = torch.ones(norm_dim, dtype=torch.float64) if weight is None else weight.double()
        x[..., :norm_dim] = n / torch.sqrt(n.square().mean(-1, keepdim=True) + eps) * w
        lost[..., :norm_dim] = x[..., :norm_dim].abs() * (norm_dim + 8) * 2.0 ** -24
    half = 0 if freqs is None else len(freqs)
    if half:
        i = torch.arange(half)
        a, b = (rot_first + 2 * i, rot_first + 2 * i + 1) if pairs else (rot_first + i, rot_first + half + i)
        t = angles.double()[:, None, None] * freqs.double()
        c, s = mscale * torch.cos(t), mscale * torch.sin(t)
        u, w = x[..., a], x[..., b]
        lu, lw = lost[..., a], lost[..., b]
        x[..., a], x[..., b] = u * c - w * s, u * s + w * c
        # The angle is off by pi 2^-25 (its fraction as binary32) and 2^-30, the
        # sine by two steps, three products and sums by half a step each: less
        # than 2^-21 of |u| + |w| times mscale.
        lost[..., a] = lost[..., b] = abs(mscale) * (lu + lw + (u.abs() + w.abs()) * 2.0 ** -21)
    return x, lost
