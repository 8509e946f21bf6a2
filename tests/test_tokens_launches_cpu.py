"""What the token operators' host code launches, without a GPU: their own
translation units linked with a fake of the CUDA calls they make
(tests/fake_cuda.cpp), which writes launches down and can be made to fail."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import workloads as W

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "state_cache_paging_gb300", "csrc")
CUDA = next((d for d in (os.environ.get("CUDA_HOME"), "/usr/local/cuda")
             if d and os.path.exists(os.path.join(d, "include", "cuda_runtime.h"))), None)


@pytest.fixture(scope="module")
def fake_lib(lmc, tmp_path_factory):
    nvcc = os.environ.get("NVCC", "nvcc")
    if shutil.which(nvcc) is None or shutil.which("g++") is None or CUDA is None:
        pytest.skip("the CUDA compiler is not available")
    d = tmp_path_factory.mktemp("fake")
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    cmds = [[nvcc, "-O1", "-std=c++17", "-gencode", "arch=compute_103a,code=compute_103a", "-Xcompiler", "-fPIC", *inc,
             "-c", os.path.join(CSRC, f"{u}.cu"), "-o", str(d / f"{u}.o")] for u in ("tokens", "attend")]
    cmds += [["g++", "-O1", "-std=c++17", "-fPIC", *inc, "-I", os.path.join(CUDA, "include"), "-c", src, "-o",
              str(d / (os.path.basename(src)[:-4] + ".o"))]
             for src in (os.path.join(CSRC, "layout.cpp"), os.path.join(CSRC, "checks.cpp"),
                         os.path.join(HERE, "fake_cuda.cpp"))]
    procs = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for c in cmds]
    for c, p in zip(cmds, procs):
        out, _ = p.communicate()
        assert p.returncode == 0, f"{' '.join(c)}\n{out}"
    so = d / "libfake.so"
    # -Bsymbolic: the fake's calls, whatever CUDA runtime is loaded beside it
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", str(so), *map(str, sorted(d.glob("*.o")))], check=True,
                   capture_output=True, text=True)
    lib = ctypes.CDLL(str(so))
    lib.fake_launch.restype = ctypes.c_char_p
    for name in ("lmc_select_tokens", "lmc_attend", "lmc_attend_workspace", "lmc_append", "lmc_move_tokens"):
        getattr(lib, name).argtypes = getattr(lmc._lib, name).argtypes
    return lib


@pytest.fixture()
def fake(fake_lib):
    fake_lib.fake_reset()
    return fake_lib


@pytest.fixture()
def env(lmc):
    layers = [W.kda(768, 3, 4, 64), W.mla(1152), W.swa(64, 128), W.mla(576)]
    L = lmc.lmc_layout_build(layers, 64, False, 1 << 28)
    buf = np.zeros(8192, dtype=np.uint8)
    return L, (buf.ctypes.data + 255) // 256 * 256, buf


def launches(lib):
    out = []
    for i in range(lib.fake_launches()):
        x = (ctypes.c_longlong * 5)()
        name = lib.fake_launch(i, x).decode()
        out.append((name, tuple(x[:3]), x[3], x[4]))
    return out


def select(lib, base, sets=1, requests=1, most=100, budget=4, recent=1, **kw):
    # (addresses are only compared: nothing lies there)
    a = dict(kept=base, ks=base + (1 << 30), kl=base + (2 << 30), lengths=base + (3 << 30), status=base + (4 << 30),
             scores=base + (5 << 30))
    a.update(kw)
    return lib.lmc_select_tokens(a["scores"], most * requests, most, sets, requests, a["lengths"], most, budget, recent,
                                 a["kept"], a["ks"], a["kl"], a["status"], None)


def test_a_selection_between_anothers_preparation_and_launch(lmc, fake, env):
    """Two host threads select at once: a call of short rows that comes between
    another's preparation and its launch takes nothing from it (the shared
    memory a kernel may take belongs to the kernel, not to the call)."""
    _, base, _ = env
    inner = []
    for sizes in ((131_072, 100), (300_000, 2_000_000), (100, 131_072)):
        fake.fake_reset()
        hook = ctypes.CFUNCTYPE(None)(lambda: inner.append(select(fake, base, most=sizes[1])))
        fake.fake_before_launch(hook)
        assert select(fake, base, most=sizes[0]) == lmc.LMC_OK, sizes
        assert inner.pop() == lmc.LMC_OK
        assert len(launches(fake)) == 2


@pytest.mark.parametrize("which,at", [
    ("kl", "lengths"), ("kl", "lengths+4"), ("kept", "lengths"), ("ks", "lengths"), ("kept", "scores"),
    ("ks", "scores"), ("ks", "scores+1596"), ("kl", "scores+1596"), ("ks", "kept"), ("kl", "kept+60"), ("kl", "ks+60")])
def test_select_refuses_outputs_over_inputs_and_each_other(lmc, fake, env, which, at):
    """Cutting the lengths in place is the obvious call: other CTAs still read
    what one of them cuts. Two sets of two requests of 100 scores (400 floats)
    and a budget of 4 (16 elements kept)."""
    _, base, _ = env
    place = dict(scores=base, kept=base + 1600, ks=base + 1664, kl=base + 1728, lengths=base + 1736)

    def call(**kw):
        a = {**place, **kw}
        return fake.lmc_select_tokens(a["scores"], 200, 100, 2, 2, a["lengths"], 100, 4, 1, a["kept"], a["ks"], a["kl"],
                                      base + 2000, None)

    assert call() == call(ks=None) == lmc.LMC_OK  # side by side, to the byte
    n = len(launches(fake))
    name, _, off = at.partition("+")
    assert call(**{which: place[name] + int(off or 0)}) == lmc.LMC_ERR_OVERLAP
    assert len(launches(fake)) == n


def test_select_of_nothing_overlaps_nothing(lmc, fake, env):
    """Memory of no elements may lie anywhere; sizes past 64 bits are refused."""
    _, base, _ = env
    assert select(fake, base, budget=0, recent=0, kept=base + (5 << 30), ks=base + (3 << 30)) == lmc.LMC_OK
    assert select(fake, base, most=0, scores=base) == lmc.LMC_OK
    big = 1 << 62
    assert fake.lmc_select_tokens(base, big, 100, 9, 1, base, 100, 4, 1, base, None, base, base, None) == \
        lmc.LMC_ERR_OVERFLOW


@pytest.mark.parametrize("unit", ["tokens.cu", "attend.cu"])
def test_kernels_that_start_early_read_no_constant_memory(unit):
    """These kernels are launched while the one before them may still write
    what they read. The read-only path (__ldg, ld.global.nc, restrict) is for
    memory that does not change while the kernel is there."""
    import re
    with open(os.path.join(CSRC, unit)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert "follow(" in text
    assert not re.findall(r"__ldg|\.nc\b|__restrict__", text)


def attend(lmc, lib, L, base, requests=2, heads=4, max_length=190, weights=False, cols=3, layer=1, scale=0.1, dtype=0,
           entry_scale=1.0, ws=None, **kw):
    """One call over addresses that are only compared. Layer 1 holds 576 16-bit
    values, layer 3 as many fp8 codes."""
    far = base + (1 << 40)
    e = lmc.lmc_entries(layer, dtype, 576, requests, entry_scale, 0, lmc.lmc_block_table(far, cols, cols))
    a = lmc.lmc_attention(far, max_length, base, 576 * heads, 576, far, 512 * heads, 512, None, 0,
                          far if weights else None, max_length, lmc.LMC_E_BF16, heads, 512, scale)
    n = ctypes.c_int64()
    rc = lib.lmc_attend_workspace(L.handle, layer, requests, heads, 512, max_length, int(weights), ctypes.byref(n))
    assert rc == lmc.LMC_OK
    return lib.lmc_attend(L.handle, ctypes.byref(e), base, ctypes.byref(a), far, n.value, far, None)


def test_attend_does_not_answer_for_another_calls_error(lmc, fake, env):
    """An error that some earlier call left behind is neither reported (the
    caller would make the call again and add the weights twice) nor cleared."""
    L, base, _ = env
    for kw in (dict(), dict(weights=True), dict(max_length=128, cols=2)):
        fake.fake_reset()
        fake.fake_set_last_error(98)
        assert attend(lmc, fake, L, base, **kw) == lmc.LMC_OK
        assert fake.fake_last_error() == 98


@pytest.mark.parametrize("fails", [0, 1, 2])
def test_attend_reports_a_launch_that_fails(lmc, fake, env, fails):
    """The weights are added by the last kernel: a call that fails has not
    added any, and leaves no error for the next."""
    L, base, _ = env
    fake.fake_fail_launch(fails)
    assert attend(lmc, fake, L, base, weights=True, max_length=1900, cols=30) == lmc.LMC_ERR_CUDA
    assert fake.fake_last_error() == 0
    names = [x[0] for x in launches(fake)]
    assert len(names) == fails and not any("weights" in n for n in names)
    fake.fake_reset()
    assert attend(lmc, fake, L, base, weights=True, max_length=1900, cols=30) == lmc.LMC_OK
    names = [x[0] for x in launches(fake)]
    assert len(names) == 3 and "join" in names[1] and "weights" in names[2]


def test_a_failed_limit_leaves_no_error(lmc, fake_lib, env, tmp_path):
    """The largest shared memory is asked for once per kernel; in a fresh
    process the request fails, is reported, and leaves no error behind."""
    import sys
    code = f"""
import ctypes, sys
sys.path[:0] = [{ROOT!r}, {HERE!r}]
import state_cache_paging_gb300 as lmc
import test_tokens_launches_cpu as t
import workloads as W
lib = ctypes.CDLL({fake_lib._name!r})
for name in ("lmc_select_tokens", "lmc_attend", "lmc_attend_workspace"):
    getattr(lib, name).argtypes = getattr(lmc._lib, name).argtypes
L = lmc.lmc_layout_build([W.kda(768, 3, 4, 64), W.mla(1152)], 64, False, 1 << 28)
base = 1 << 20
lib.fake_fail_attributes(1)
for call in (lambda: t.select(lib, base), lambda: t.attend(lmc, lib, L, base)):
    assert call() == lmc.LMC_ERR_CUDA
    assert lib.fake_last_error() == 0, "left behind"
    assert lib.fake_launches() == 0
lib.fake_fail_attributes(0)
for call in (lambda: t.select(lib, base), lambda: t.attend(lmc, lib, L, base)):
    assert call() == call() == lmc.LMC_OK
assert lib.fake_attributes() == 4  # two that failed, then one for each kernel
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_attend_weights_grid_is_bounded(lmc, fake, env):
    """The tokens' weights of short requests in a batch that could hold long
    ones: no block for every 256 tokens that there might be."""
    L, base, _ = env
    for requests, max_length in ((256, 131_072), (1, 131_072), (65_535, 64 * 40), (3, 10)):
        fake.fake_reset()
        assert attend(lmc, fake, L, base, requests=requests, heads=2, max_length=max_length, cols=-(-max_length // 64),
                      weights=True) == lmc.LMC_OK
        name, grid, _, _ = launches(fake)[-1]
        assert "weights" in name and grid[1] == requests
        assert 1 <= grid[0] <= max(1, -(-64 * 152 // requests)) and grid[0] <= max_length // 256 + 1


def test_attend_refuses_scales_whose_product_is_infinite(lmc, fake, env):
    """Logits are scaled by one binary32 number; an infinite one would make NaN
    of logits that are 0."""
    L, base, _ = env
    assert attend(lmc, fake, L, base, scale=3e38) == lmc.LMC_ERR_INVALID_ARG
    assert attend(lmc, fake, L, base, scale=-3e38) == lmc.LMC_ERR_INVALID_ARG
    fp8 = dict(layer=3, dtype=lmc.LMC_E_E4M3)
    assert attend(lmc, fake, L, base, scale=1e20, entry_scale=1e20, **fp8) == lmc.LMC_ERR_INVALID_ARG
    assert not launches(fake)
    for kw in (dict(scale=2e38), dict(scale=1e20, entry_scale=1e18, **fp8), dict(scale=1e20, entry_scale=1e-20, **fp8)):
        assert attend(lmc, fake, L, base, **kw) == lmc.LMC_OK
