"""The decode example shown in the README, as a module the tests run.

A Kimi-Linear layout; two requests' prompts are appended to one MLA layer,
three decode steps append a token each and attend, the second request's cache
is cut to a budget by its accumulated attention weight and attended again.
run() returns the values a test checks.
"""


def run(device="cuda"):
    import torch

    import state_cache_paging_gb300 as lmc

    kda = {"kind": "KDA", "conv_bytes": 12288 * 3 * 2, "rec_bytes": 32 * 128 * 128 * 4}
    mla = {"kind": "MLA", "token_bytes": (512 + 64) * 2}
    L = lmc.lmc_layout_build([kda, kda, kda, mla] * 6, 944, packed=False, mem_bytes=16 * 6 * 2170880)
    layer, group, heads = 3, 3, 32                                    # the first MLA layer and its KV group
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=device)  # noqa: E731
    draw = lambda *s: torch.randn(*s, device=device).bfloat16()         # noqa: E731
    pool = torch.empty(L.pool_bytes, dtype=torch.uint8, device=device)
    status = torch.zeros(1, dtype=torch.int32, device=device)
    table = ints([[0, 1], [2, 3]])                                    # blocks of each request

    prompt, most = [500, 1200], 2 * 944
    lmc.lmc_append(L, layer, pool, table, ints([0] * 500 + [1] * 1200),
                   ints([*range(500), *range(1200)]), draw(1700, 576), status)
    ws = torch.empty(lmc.lmc_attend_workspace(L, layer, 2, heads, 512, most, weights=True), dtype=torch.uint8,
                     device=device)
    out = torch.empty(2, heads, 512, dtype=torch.bfloat16, device=device)
    lse = torch.empty(2, heads, device=device)
    weights = torch.zeros(2, most, device=device)
    for k in range(3):                                                # one new token per request and step
        lmc.lmc_append(L, layer, pool, table, ints([0, 1]), ints([n + k for n in prompt]), draw(2, 576), status)
        lmc.lmc_attend(L, layer, pool, table, ints([n + k + 1 for n in prompt]), draw(2, heads, 576), 512, 192 ** -0.5,
                       out, ws, status, max_length=most, lse=lse, weights=weights)

    # request 1 keeps its last 64 tokens and the 192 that weighed most, in a fresh block
    kept, kept_len = ints([[[-1] * 256]]), ints([0])
    lmc.lmc_select_tokens(weights[None, 1:], ints([1203]), 256, 64, kept, None, kept_len, status)
    lmc.lmc_move_tokens(L, group, pool, table[1:], ints([[4]]), kept, kept_len, status)
    lmc.lmc_attend(L, layer, pool, ints([[4]]), kept_len, draw(1, heads, 576), 512, 192 ** -0.5, out[1:], ws, status)
    torch.cuda.synchronize()
    return {"status": int(status.item()), "weight": weights.sum(1).tolist(), "kept": kept.flatten().tolist(),
            "kept_length": int(kept_len.item()), "finite": bool(torch.isfinite(out.float()).all())}
