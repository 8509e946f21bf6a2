"""Argument checks of the token operators (no GPU): what is refused on the
host before anything is enqueued, through the C ABI with host pointers that
are never read."""
import ctypes

import numpy as np
import pytest

import workloads as W


@pytest.fixture()
def env(lmc):
    layers = [W.kda(768, 3, 4, 64), W.mla(1152), W.swa(64, 128)]
    L = lmc.lmc_layout_build(layers, 64, False, 1 << 24)
    buf = np.zeros(4096 + 256, dtype=np.uint8)
    base = (buf.ctypes.data + 255) // 256 * 256
    return L, base, buf


def _entries(lmc, base, **kw):
    a = dict(layer=1, dtype=lmc.LMC_E_BF16, entry_dim=576, num_requests=2, scale=1.0, cols=3, row=3, table=base)
    a.update(kw)
    return lmc.lmc_entries(a["layer"], a["dtype"], a["entry_dim"], a["num_requests"], a["scale"], 0,
                           lmc.lmc_block_table(a["table"], a["row"], a["cols"]))


BAD_ENTRIES = [dict(layer=0), dict(layer=-1), dict(layer=3), dict(dtype=9), dict(entry_dim=575), dict(entry_dim=0),
               dict(dtype=2), dict(scale=2.0), dict(scale=float("nan")), dict(num_requests=-1), dict(row=2),
               dict(cols=-1), dict(table=None)]


@pytest.mark.parametrize("kw", BAD_ENTRIES)
def test_bad_entries_are_refused_by_append_and_attend(lmc, env, kw):
    L, base, _ = env
    e = _entries(lmc, base, **kw)
    assert _append(lmc, L, base, e) == lmc.LMC_ERR_INVALID_ARG
    assert _attend(lmc, L, base, e) == lmc.LMC_ERR_INVALID_ARG


def _append(lmc, L, base, e, **kw):
    a = dict(pool=base, requests=base, positions=base, rows=base, dtype=lmc.LMC_E_BF16, stride=576, n=2, status=base)
    a.update(kw)
    return lmc._lib.lmc_append(L.handle, ctypes.byref(e), a["pool"], a["requests"], a["positions"], a["rows"],
                               a["dtype"], a["stride"], a["n"], a["status"], None)


@pytest.mark.parametrize("kw", [dict(pool=None), dict(requests=None), dict(positions=None), dict(rows=None),
                                dict(dtype=2), dict(dtype=1), dict(stride=575), dict(n=-1), dict(status=None)])
def test_append_refusals(lmc, env, kw):
    L, base, _ = env
    assert _append(lmc, L, base, _entries(lmc, base), **kw) == lmc.LMC_ERR_INVALID_ARG
    assert _append(lmc, L, base, _entries(lmc, base), status=base + 2) == lmc.LMC_ERR_ALIGN
    assert _append(lmc, L, base, _entries(lmc, base), rows=base + 1) == lmc.LMC_ERR_ALIGN
    assert _append(lmc, L, base, _entries(lmc, base), n=0) == lmc.LMC_OK


def _attend(lmc, L, base, e, **kw):
    a = dict(lengths=base, max_length=100, q=base, qr=576 * 4, qh=576, out=base, outr=512 * 4, outh=512, lse=None,
             lse_r=0, weights=None, w_r=0, dtype=lmc.LMC_E_BF16, heads=4, value=512, scale=0.1, pool=base, ws=base,
             ws_bytes=1 << 40, status=base)
    a.update(kw)
    t = lmc.lmc_attention(a["lengths"], a["max_length"], a["q"], a["qr"], a["qh"], a["out"], a["outr"], a["outh"],
                          a["lse"], a["lse_r"], a["weights"], a["w_r"], a["dtype"], a["heads"], a["value"], a["scale"])
    return lmc._lib.lmc_attend(L.handle, ctypes.byref(e), a["pool"], ctypes.byref(t), a["ws"], a["ws_bytes"],
                               a["status"], None)


@pytest.mark.parametrize("kw", [
    dict(lengths=None), dict(q=None), dict(out=None), dict(pool=None), dict(ws=None), dict(status=None),
    dict(max_length=0), dict(max_length=1 << 31), dict(qr=-8), dict(qr=577), dict(qh=575), dict(outr=-1),
    dict(outh=511), dict(outr=511), dict(dtype=2), dict(dtype=1), dict(heads=0), dict(value=0), dict(value=516),
    dict(value=500), dict(scale=float("inf")), dict(ws_bytes=0)])
def test_attend_refusals(lmc, env, kw):
    L, base, _ = env
    assert _attend(lmc, L, base, _entries(lmc, base), **kw) == lmc.LMC_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(pool=8), dict(q=8), dict(out=1), dict(ws=16), dict(status=2), dict(lengths=1),
                                dict(lse=2, lse_r=4), dict(weights=2, w_r=100)])
def test_attend_alignment(lmc, env, kw):
    L, base, _ = env
    kw = {k: base + v if k not in ("lse_r", "w_r") else v for k, v in kw.items()}
    assert _attend(lmc, L, base, _entries(lmc, base), **kw) == lmc.LMC_ERR_ALIGN


def test_attend_refuses_short_buffers_and_odd_entries(lmc, env):
    L, base, _ = env
    e = _entries(lmc, base)
    assert _attend(lmc, L, base, e, lse=base, lse_r=3) == lmc.LMC_ERR_INVALID_ARG
    assert _attend(lmc, L, base, e, weights=base, w_r=99) == lmc.LMC_ERR_INVALID_ARG
    assert _attend(lmc, L, base, _entries(lmc, base, num_requests=0)) == lmc.LMC_OK
    for dim in (24, 592):  # not a multiple of 16; past 576
        M = lmc.lmc_layout_build([W.mla(2 * dim)], 64, False, 1 << 24)
        e = _entries(lmc, base, layer=0, entry_dim=dim)
        assert _attend(lmc, M, base, e, qr=4096, qh=dim, value=16) == lmc.LMC_ERR_INVALID_ARG


def test_attend_workspace_sizes_and_refusals(lmc, env):
    L, _, _ = env
    a = lmc.lmc_attend_workspace(L, 1, 2, 4, 512, 100)
    assert lmc.lmc_attend_workspace(L, 1, 2, 4, 512, 100, True) >= a > 0
    assert lmc.lmc_attend_workspace(L, 1, 64, 64, 512, 1 << 20, True) > a
    for args in [(0, 2, 4, 512, 100), (7, 2, 4, 512, 100), (1, -1, 4, 512, 100), (1, 2, 0, 512, 100),
                 (1, 2, 4, 0, 100), (1, 2, 4, 520, 100), (1, 2, 4, 512, 0), (1, 2, 4, 512, 1 << 31)]:
        with pytest.raises(lmc.LmcError) as ei:
            lmc.lmc_attend_workspace(L, *args)
        assert ei.value.code == lmc.LMC_ERR_INVALID_ARG, args


def test_attend_workspace_takes_no_window_from_a_full_attention_layer(lmc):
    """Only SWA layers have one; the logits of all tokens are kept."""
    plain, odd = W.mla(1152), dict(W.mla(1152), window=16)
    need = [lmc.lmc_attend_workspace(lmc.lmc_layout_build([x], 64, False, 1 << 24), 0, 2, 4, 512, 1000, True)
            for x in (plain, odd)]
    assert need[0] == need[1]
    assert need[1] >= 2 * 4 * 1000 * 4


def _select(lmc, base, **kw):
    a = dict(scores=base, ss=100, rs=10, sets=2, n=2, lengths=base, most=10, budget=4, recent=1, kept=base, ks=base,
             kl=base, status=base)
    a.update(kw)
    return lmc._lib.lmc_select_tokens(a["scores"], a["ss"], a["rs"], a["sets"], a["n"], a["lengths"], a["most"],
                                      a["budget"], a["recent"], a["kept"], a["ks"], a["kl"], a["status"], None)


@pytest.mark.parametrize("kw", [dict(scores=None), dict(lengths=None), dict(kept=None), dict(kl=None),
                                dict(status=None), dict(sets=-1), dict(n=-1), dict(most=-1), dict(most=1 << 31),
                                dict(budget=-1), dict(recent=5), dict(recent=-1), dict(ss=-1), dict(rs=-1)])
def test_select_refusals(lmc, env, kw):
    _, base, _ = env
    assert _select(lmc, base, **kw) == lmc.LMC_ERR_INVALID_ARG
    assert _select(lmc, base, scores=base + 2) == lmc.LMC_ERR_ALIGN
    assert _select(lmc, base, n=0) == _select(lmc, base, sets=0) == lmc.LMC_OK


def _move(lmc, L, base, **kw):
    a = dict(group=1, pool=base, n=2, src=(base, 3, 3), dst=(base + 64, 3, 3), kept=base, sets=1, ss=0, rs=8,
             kl=base, most=8, status=base)
    a.update(kw)
    src, dst = (lmc.lmc_block_table(*t) if t else None for t in (a["src"], a["dst"]))
    return lmc._lib.lmc_move_tokens(L.handle, a["group"], a["pool"], a["n"], src and ctypes.byref(src),
                                    dst and ctypes.byref(dst), a["kept"], a["sets"], a["ss"], a["rs"], a["kl"],
                                    a["most"], a["status"], None)


@pytest.mark.parametrize("kw", [dict(group=-1), dict(group=0), dict(group=3), dict(pool=None), dict(n=-1),
                                dict(src=None), dict(dst=None), dict(kept=None), dict(kl=None), dict(status=None),
                                dict(sets=2), dict(sets=0), dict(ss=-1), dict(rs=7), dict(most=-1),
                                dict(src=(None, 3, 3)), dict(dst=(None, 3, 3))])
def test_move_refusals(lmc, env, kw):
    L, base, _ = env
    assert [L.kv_group_kind[g] for g in range(3)] == ["KDA", "MLA", "SWA"]
    assert _move(lmc, L, base, **kw) == lmc.LMC_ERR_INVALID_ARG


def test_move_refuses_one_table_as_both(lmc, env):
    L, base, _ = env
    assert _move(lmc, L, base, dst=(base, 3, 3)) == lmc.LMC_ERR_OVERLAP
    assert _move(lmc, L, base, kept=base + 2) == lmc.LMC_ERR_ALIGN
    assert _move(lmc, L, base, n=0) == _move(lmc, L, base, most=0) == lmc.LMC_OK


def test_binding_refuses_wrong_tensors(lmc, env):
    """The binding's own checks: host tensors, wrong types and shapes."""
    import torch
    L, _, _ = env
    host = torch.zeros(L.pool_bytes, dtype=torch.uint8)
    t = torch.zeros((2, 3), dtype=torch.int32)
    x = torch.zeros((2, 576), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (
        lambda: lmc.lmc_append(L, 1, host, t, i, i, x, i),
        lambda: lmc.lmc_append(L, 1, host, t, i, i, x.float(), i),
        lambda: lmc.lmc_append(L, 1, host, t, i, i, x[0], i),
        lambda: lmc.lmc_attend(L, 1, host, t, i, x[:, None], 512, 0.1, x[:, None, :512], host, i),
        lambda: lmc.lmc_attend(L, 1, host, t, i, x[:, None].float(), 512, 0.1, x[:, None, :512], host, i),
        lambda: lmc.lmc_select_tokens(torch.zeros((1, 2, 5)), i, 2, 1, t[None, :, :2], None, i, i),
        lambda: lmc.lmc_select_tokens(torch.zeros((2, 5)), i, 2, 1, t[None, :, :2], None, i, i),
        lambda: lmc.lmc_move_tokens(L, 1, host, t, t.clone(), t[None], i, i),
    ):
        with pytest.raises(lmc.LmcError) as ei:
            call()
        assert ei.value.code == lmc.LMC_ERR_INVALID_ARG


@pytest.fixture()
def as_if_on_device(lmc, monkeypatch):
    """Host tensors pass as ones of the current device; nothing is launched."""
    import torch
    monkeypatch.setattr(lmc, "_torch", torch)
    monkeypatch.setattr(lmc, "_home", lambda name, t: -1)
    monkeypatch.setattr(lmc, "_stream_ptr", lambda stream, *buffers: None)

    class Library:
        calls = 0

        def __getattr__(self, name):
            if name == "lmc_strerror":
                return lambda code: b"refused"

            def call(*args):
                Library.calls += 1
                return lmc.LMC_OK
            return call
    monkeypatch.setattr(lmc, "_lib", Library())
    return Library


def test_binding_refuses_rows_that_overlap(lmc, env, as_if_on_device):
    """An expanded tensor's rows lie 0 apart: taken as rows of their own they
    would be read past its memory."""
    import torch
    L, _, _ = env
    pool = torch.zeros(L.pool_bytes, dtype=torch.uint8)
    t = torch.zeros((2, 3), dtype=torch.int32)
    x = torch.zeros((2, 576), dtype=torch.bfloat16)
    q, out = torch.zeros((2, 4, 576), dtype=torch.bfloat16), torch.zeros((2, 4, 512), dtype=torch.bfloat16)
    f = torch.zeros((2, 200))
    i, kept = torch.zeros(2, dtype=torch.int32), torch.zeros((1, 2, 4), dtype=torch.int32)
    ws = torch.zeros(1024, dtype=torch.uint8)

    def append(table=t, rows=x, status=i):
        lmc.lmc_append(L, 1, pool, table, i, i, rows, status)

    def attend(table=t, workspace=ws, **kw):
        lmc.lmc_attend(L, 1, pool, table, i, q, 512, 0.1, out, workspace, i, max_length=190, **kw)

    def move(src=t, dst=t.clone(), kept=kept):
        lmc.lmc_move_tokens(L, 1, pool, src, dst, kept, i, i)

    one = [torch.Tensor.expand(y[:1], *y.shape) for y in (t, x, f)]
    for call in (lambda: append(table=one[0]), lambda: append(rows=one[1]),
                 lambda: append(status=torch.zeros(1, dtype=torch.uint8).expand(4)),
                 lambda: attend(table=one[0]), lambda: attend(lse=one[2]), lambda: attend(weights=one[2]),
                 lambda: attend(workspace=torch.zeros(1, dtype=torch.uint8).expand(1024)),
                 lambda: attend(weights=torch.zeros(2 * 150).as_strided((2, 200), (100, 1))),
                 lambda: move(src=one[0]), lambda: move(dst=one[0]), lambda: move(kept=kept[:, :1].expand(1, 2, 4))):
        before = as_if_on_device.calls
        with pytest.raises(lmc.LmcError) as ei:
            call()
        assert ei.value.code == lmc.LMC_ERR_INVALID_ARG
        assert as_if_on_device.calls == before
    for call in (append, attend, move):  # the same calls without one
        call()
    assert as_if_on_device.calls >= 3


def test_binding_refuses_tensors_of_another_device(lmc, monkeypatch):
    import torch
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)

    class On:
        def __init__(self, device):
            self.is_cuda, self.get_device = device >= 0, lambda: device

        def is_pinned(self):
            return True

    assert lmc._home("pool", On(0)) == lmc._home("pool", On(-1)) == 0
    lmc._away("q", On(-1), 0)
    for call in (lambda: lmc._home("pool", On(1)), lambda: lmc._away("q", On(1), 0),
                 lambda: lmc._ints("lengths", On(1), 0, 2)):
        with pytest.raises(lmc.LmcError) as ei:
            call()
        assert ei.value.code == lmc.LMC_ERR_INVALID_ARG
