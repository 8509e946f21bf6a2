"""The hybrid model example shown in the README, as a module the tests run.

Pages of Kimi-Linear's sizes, whose state layers decay by the head here (KDA's own
recurrence is another one); one request's prompt passes a linear-attention layer and
an attention layer, three decode steps follow, and its first chunk is stored,
loaded into a fresh pool and continued from there. run() returns the tensors a
test checks.
"""


def run(device="cuda"):
    import numpy as np
    import torch

    import state_cache_paging_gb300 as lmc

    kda = {"kind": "KDA", "conv_bytes": 12288 * 3 * 2, "rec_bytes": 32 * 128 * 128 * 4}
    mla = {"kind": "MLA", "token_bytes": (512 + 64) * 2}
    N, prompt, steps, heads = 944, 1200, 3, 32
    total = prompt + steps
    L = lmc.lmc_layout_build([kda, kda, kda, mla] * 6, N, packed=False, mem_bytes=16 * 6 * 2170880)
    state, latent = 0, 3                                              # a state layer, an MLA layer
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=device)  # noqa: E731
    draw = lambda *s: torch.randn(*s, device=device).bfloat16()         # noqa: E731
    pool = torch.zeros(L.pool_bytes, dtype=torch.uint8, device=device)
    status = torch.zeros(1, dtype=torch.int32, device=device)
    tables = [ints([[2 * g, 2 * g + 1]]) for g in range(L.num_kv_groups)]
    states, latents = tables[L.kv_group[state]], tables[L.kv_group[latent]]

    # the prompt: its states (the one at the block's end is a snapshot) and its entries
    q, k, v = draw(total, heads, 128), draw(total, heads, 128) * 128 ** -0.5, draw(total, heads, 128)
    decay = -0.2 * torch.rand(total, heads, device=device)
    o = torch.empty(total, heads, 128, dtype=torch.bfloat16, device=device)
    ws = torch.empty(lmc.lmc_linear_scan_workspace(L, state, 1, total, heads), dtype=torch.uint8, device=device)
    lmc.lmc_linear_scan(L, state, pool, states, ints([0, prompt]), ints([0]), q, k, v, decay, o, ws, status,
                        scale=128 ** -0.5)
    entries, norm = draw(total, 576), 1 + 0.1 * torch.randn(512, device=device)
    freqs = 10000.0 ** (-torch.arange(32, device=device) / 32)
    where = dict(frequencies=freqs, rot_first=512, pairs=True)         # the last 64 values turn
    lmc.lmc_append_rotated(L, latent, pool, latents, ints([0] * prompt), ints(range(prompt)), entries[:prompt], status,
                           norm_dim=512, norm_weight=norm, **where)

    # one token at a time
    aq, a = draw(total, heads, 576), torch.empty(total, heads, 512, dtype=torch.bfloat16, device=device)
    aws = torch.empty(lmc.lmc_attend_workspace(L, latent, 1, heads, 512, total), dtype=torch.uint8, device=device)
    lmc.lmc_rotate(aq, ints(range(total)), aq, **where)                # in place
    for t in range(prompt, total):
        one = slice(t, t + 1)
        lmc.lmc_linear_step(L, state, pool, states, ints([t]), q[one], k[one], v[one], decay[one], o[one], status,
                            scale=128 ** -0.5)
        lmc.lmc_append_rotated(L, latent, pool, latents, ints([0]), ints([t]), entries[one], status, norm_dim=512,
                               norm_weight=norm, **where)
        lmc.lmc_attend(L, latent, pool, latents, ints([t + 1]), aq[one], 512, 192 ** -0.5, a[one], aws, status,
                       max_length=total)

    # the first chunk goes out and comes back elsewhere; the rest is one prompt from there
    sizes = [L.object_bytes(N, g) for g in range(L.num_object_groups)]
    jobs = [lmc.jobs_to_device(np.array([(0, 0, sum(sizes[:g]))], dtype=lmc.JOB_DTYPE), device) for g in range(len(sizes))]
    arena = torch.empty(sum(sizes), dtype=torch.uint8, device=device)
    lmc.lmc_store(L, N, pool, tables, jobs, arena, status)
    fresh, others = torch.zeros_like(pool), [t + 8 for t in tables]
    lmc.lmc_load(L, N, fresh, others, jobs, arena, status)
    o2, a2 = torch.empty_like(o[N:]), torch.empty_like(a[:1])
    lmc.lmc_linear_scan(L, state, fresh, others[L.kv_group[state]], ints([0, total - N]), ints([N]), q[N:], k[N:], v[N:],
                        decay[N:], o2, ws, status, scale=128 ** -0.5)
    lmc.lmc_append_rotated(L, latent, fresh, others[L.kv_group[latent]], ints([0] * (total - N)), ints(range(N, total)),
                           entries[N:], status, norm_dim=512, norm_weight=norm, **where)
    lmc.lmc_attend(L, latent, fresh, others[L.kv_group[latent]], ints([total]), aq[-1:], 512, 192 ** -0.5, a2, aws, status,
                   max_length=total)
    torch.cuda.synchronize()
    return dict(status=int(status.item()), layout=L, pool=pool, fresh=fresh, tables=tables, others=others, q=q, k=k, v=v,
                decay=decay, o=o, o2=o2, entries=entries, norm=norm, freqs=freqs, aq=aq, a=a[prompt:], a2=a2, N=N,
                prompt=prompt)
