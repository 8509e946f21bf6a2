"""Argument checks of lmc_linear_step, lmc_linear_scan, lmc_rotate and
lmc_append_rotated (no GPU): what is refused on the host before anything is
enqueued, through the C ABI with host pointers that are never read."""
import ctypes

import numpy as np
import pytest

import workloads as W

BIG = 1 << 40


@pytest.fixture()
def env(lmc):
    layers = [W.kda(768, 3, 4, 64), W.mla(1152), W.swa(64, 128), W.kda(4, 1, 4, 64)]
    L = lmc.lmc_layout_build(layers, 64, False, 1 << 24)
    buf = np.zeros(4096 + 256, dtype=np.uint8)
    return L, (buf.ctypes.data + 255) // 256 * 256, buf


def _linear(lmc, base, **kw):
    # (addresses are only compared: nothing lies there)
    a = dict(layer=0, dtype=lmc.LMC_E_BF16, R=2, H=4, K=2, dk=64, dv=64, scale=0.1, cols=3, row=3, table=base,
             lengths=base, q=base, k=base, v=base, out=base + BIG, decay=base, qr=128, qh=64, kr=128, kh=64, vr=256, vh=64,
             outr=256, outh=64, dr=4, dh=1)
    a.update(kw)
    return lmc.lmc_linear(a["layer"], a["dtype"], a["R"], a["H"], a["K"], a["dk"], a["dv"], a["scale"],
                          lmc.lmc_block_table(a["table"], a["row"], a["cols"]), a["lengths"], a["q"], a["k"], a["v"],
                          a["out"], a["decay"], a["qr"], a["qh"], a["kr"], a["kh"], a["vr"], a["vh"], a["outr"], a["outh"],
                          a["dr"], a["dh"])


def _step(lmc, L, base, pool=True, status=0, **kw):
    return lmc._lib.lmc_linear_step(L.handle, ctypes.byref(_linear(lmc, base, **kw)), base if pool is True else pool,
                                    None if status is None else base + status, None)


def _scan(lmc, L, base, pool=True, status=0, starts=0, n=2, ws=0, ws_bytes=1 << 40, **kw):
    return lmc._lib.lmc_linear_scan(L.handle, ctypes.byref(_linear(lmc, base, **kw)), None if starts is None else base + starts,
                                    n, base if pool is True else pool, None if ws is None else base + ws, ws_bytes,
                                    None if status is None else base + status, None)


BAD = [dict(layer=1), dict(layer=-1), dict(layer=4), dict(dtype=2), dict(dtype=9), dict(R=-1), dict(R=(1 << 20) + 1),
       dict(H=0), dict(H=3), dict(K=0), dict(K=3), dict(H=65536), dict(dk=0), dict(dk=60), dict(dk=128), dict(dv=136),
       dict(dv=32), dict(dk=-64), dict(scale=float("nan")), dict(scale=float("inf")), dict(cols=-1), dict(row=2),
       dict(table=None), dict(lengths=None), dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(decay=None),
       dict(qr=63), dict(qr=-128), dict(qh=60), dict(qh=68), dict(kr=129), dict(kh=0), dict(vr=8), dict(vh=-64), dict(vh=2),
       dict(outr=63), dict(outh=63), dict(outr=-256), dict(outr=100, outh=100), dict(dr=-1), dict(dh=-1), dict(pool=None),
       dict(status=None), dict(qr=1 << 40), dict(vh=1 << 61)]


@pytest.mark.parametrize("kw", BAD)
def test_linear_refusals(lmc, env, kw):
    L, base, _ = env
    assert _step(lmc, L, base, **kw) == lmc.LMC_ERR_INVALID_ARG
    assert _scan(lmc, L, base, **kw) == lmc.LMC_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(starts=None), dict(n=-1), dict(ws=None), dict(ws_bytes=0)])
def test_scan_refusals(lmc, env, kw):
    L, base, _ = env
    assert _scan(lmc, L, base, **kw) == lmc.LMC_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(q=8), dict(k=2), dict(v=8), dict(out=BIG + 1), dict(decay=2), dict(lengths=1)])
def test_linear_alignment(lmc, env, kw):
    L, base, _ = env
    kw = {k: base + v for k, v in kw.items()}
    assert _step(lmc, L, base, **kw) == lmc.LMC_ERR_ALIGN
    assert _scan(lmc, L, base, **kw) == lmc.LMC_ERR_ALIGN


def test_linear_alignment_of_the_call(lmc, env):
    L, base, _ = env
    assert _step(lmc, L, base, status=2) == lmc.LMC_ERR_ALIGN
    assert _step(lmc, L, base, pool=base + 8) == lmc.LMC_ERR_ALIGN
    assert _scan(lmc, L, base, starts=2) == lmc.LMC_ERR_ALIGN
    assert _scan(lmc, L, base, ws=16) == lmc.LMC_ERR_ALIGN
    assert _step(lmc, L, base, layer=3) == lmc.LMC_ERR_ALIGN  # conv_bytes of 8


def test_linear_overlaps(lmc, env):
    """out may touch none of the inputs, from the first element to the last."""
    L, base, _ = env
    ends = dict(q=2 * (128 + 64 + 64), k=2 * (128 + 64 + 64), v=2 * (256 + 192 + 64), decay=4 * (4 + 3 + 1))
    out_end = 2 * (256 + 192 + 64)
    for name, end in ends.items():
        for at in (0, end - 16, 16 - out_end):
            kw = {n: base + 2 * BIG for n in ends}
            kw[name] = base + BIG - (at // 16 * 16)
            assert _step(lmc, L, base, **kw) == lmc.LMC_ERR_OVERLAP, (name, at)
            assert _scan(lmc, L, base, **kw) == lmc.LMC_ERR_OVERLAP, (name, at)


def test_nothing_to_do(lmc, env):
    L, base, _ = env
    assert _step(lmc, L, base, R=0) == lmc.LMC_OK
    assert _scan(lmc, L, base, R=0) == lmc.LMC_OK
    assert _scan(lmc, L, base, n=0) == lmc.LMC_OK


def test_scan_workspace(lmc, env):
    L, _, _ = env
    assert lmc.lmc_linear_scan_workspace(L, 0, 2, 1000, 4) > 0
    for args in [(1, 2, 10, 4), (-1, 2, 10, 4), (4, 2, 10, 4), (0, -1, 10, 4), (0, (1 << 20) + 1, 10, 4), (0, 2, -1, 4),
                 (0, 2, 10, 0), (0, 2, 10, 65536)]:
        with pytest.raises(lmc.LmcError) as ei:
            lmc.lmc_linear_scan_workspace(L, *args)
        assert ei.value.code == lmc.LMC_ERR_INVALID_ARG, args


def _rotation(lmc, base, **kw):
    a = dict(heads=4, dim=128, norm=128, first=64, rot=64, mode=0, eps=1e-6, mscale=1.0, weight=base, freqs=base, pos=base)
    a.update(kw)
    return lmc.lmc_rotation(a["heads"], a["dim"], a["norm"], a["first"], a["rot"], a["mode"], a["eps"], a["mscale"],
                            a["weight"], a["freqs"], a["pos"])


def _rotate(lmc, base, x=0, out=BIG, dtype=0, xr=512, xh=128, outr=512, outh=128, n=3, **kw):
    return lmc._lib.lmc_rotate(ctypes.byref(_rotation(lmc, base, **kw)), dtype, None if x is None else base + x, xr, xh,
                               None if out is None else base + out, outr, outh, n, None)


def _append(lmc, L, base, entry=576, layer=1, dtype=0, rows=0, stride=576, n=2, status=0, pool=0, req=0, positions=0,
            scale=1.0, rows_dtype=0, **kw):
    at = lambda v: None if v is None else base + v  # noqa: E731
    kw = {**dict(heads=1, dim=576, norm=512, first=512, rot=64), **kw}
    e = lmc.lmc_entries(layer, dtype, entry, 2, scale, 0, lmc.lmc_block_table(base, 3, 3))
    return lmc._lib.lmc_append_rotated(L.handle, ctypes.byref(e), ctypes.byref(_rotation(lmc, base, **kw)), at(pool),
                                       at(req), at(positions), at(rows), rows_dtype, stride, n, at(status), None)


ROTATION = [dict(heads=0), dict(dim=0), dict(dim=4097), dict(norm=-1), dict(norm=577), dict(first=-1), dict(first=577),
            dict(rot=-2), dict(rot=63), dict(first=513), dict(mode=2), dict(eps=-1.0), dict(eps=float("nan")),
            dict(mscale=float("inf")), dict(freqs=None)]


@pytest.mark.parametrize("kw", ROTATION)
def test_rotation_refusals(lmc, env, kw):
    L, base, _ = env
    full = {**dict(heads=1, dim=576, norm=512, first=512, rot=64), **kw}
    assert _rotate(lmc, base, xr=8192, outr=8192, xh=4200, outh=4200, **full) == lmc.LMC_ERR_INVALID_ARG
    assert _append(lmc, L, base, **kw) == lmc.LMC_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(x=None), dict(out=None), dict(pos=None), dict(dtype=2), dict(n=-1), dict(xr=127),
                                dict(xr=300), dict(xh=127), dict(outr=511), dict(outh=100), dict(outr=-512),
                                dict(xr=200, xh=300), dict(xr=1 << 62)])
def test_rotate_refusals(lmc, env, kw):
    _, base, _ = env
    assert _rotate(lmc, base, **kw) == lmc.LMC_ERR_INVALID_ARG


def test_rotate_alignment_and_overlap(lmc, env):
    _, base, _ = env
    for kw in (dict(x=1), dict(out=BIG + 1), dict(weight=base + 2), dict(freqs=base + 1), dict(pos=base + 2)):
        assert _rotate(lmc, base, **kw) == lmc.LMC_ERR_ALIGN, kw
    end = 2 * (2 * 512 + 512)
    for out in (2, end - 2, 128):
        assert _rotate(lmc, base, out=out) == lmc.LMC_ERR_OVERLAP, out
        assert _rotate(lmc, base, x=out, out=0) == lmc.LMC_ERR_OVERLAP, out
    assert _rotate(lmc, base, out=0, outr=1024) == lmc.LMC_ERR_OVERLAP  # in place with other strides
    assert _rotate(lmc, base, n=0) == lmc.LMC_OK
    assert _rotate(lmc, base, out=0, norm=0, rot=0) == lmc.LMC_OK       # in place, nothing to do


@pytest.mark.parametrize("kw", [dict(layer=0), dict(layer=9), dict(entry=575), dict(dtype=2), dict(dtype=1), dict(scale=2.0),
                                dict(rows=None), dict(pool=None), dict(req=None), dict(positions=None), dict(status=None),
                                dict(stride=575), dict(n=-1), dict(rows_dtype=2), dict(heads=2), dict(heads=1 << 30)])
def test_append_rotated_refusals(lmc, env, kw):
    L, base, _ = env
    assert _append(lmc, L, base, **kw) == lmc.LMC_ERR_INVALID_ARG


def test_append_rotated_alignment(lmc, env):
    L, base, _ = env
    for kw in (dict(rows=1), dict(status=2), dict(req=1), dict(positions=2), dict(weight=base + 1)):
        assert _append(lmc, L, base, **kw) == lmc.LMC_ERR_ALIGN, kw
    assert _append(lmc, L, base, n=0) == lmc.LMC_OK
