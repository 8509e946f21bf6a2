"""What the host code of linear attention and of the rotations launches, without
a GPU: their own translation units linked with a fake of the CUDA calls they
make (tests/fake_cuda.cpp)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import test_linear_cpu as C
import workloads as W
from test_tokens_launches_cpu import CSRC, CUDA, HERE, ROOT, launches


@pytest.fixture(scope="module")
def fake_lib(lmc, tmp_path_factory):
    nvcc = os.environ.get("NVCC", "nvcc")
    if shutil.which(nvcc) is None or shutil.which("g++") is None or CUDA is None:
        pytest.skip("the CUDA compiler is not available")
    d = tmp_path_factory.mktemp("fake")
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    cmds = [[nvcc, "-O1", "-std=c++17", "-gencode", "arch=compute_103a,code=compute_103a", "-Xcompiler", "-fPIC", *inc,
             "-c", os.path.join(CSRC, f"{u}.cu"), "-o", str(d / f"{u}.o")] for u in ("tokens", "rotate", "linear")]
    cmds += [["g++", "-O1", "-std=c++17", "-fPIC", *inc, "-I", os.path.join(CUDA, "include"), "-c", src, "-o",
              str(d / (os.path.basename(src)[:-4] + ".o"))]
             for src in (os.path.join(CSRC, "layout.cpp"), os.path.join(CSRC, "checks.cpp"),
                         os.path.join(HERE, "fake_cuda.cpp"))]
    procs = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for c in cmds]
    for c, p in zip(cmds, procs):
        out, _ = p.communicate()
        assert p.returncode == 0, f"{' '.join(c)}\n{out}"
    so = d / "libfake.so"
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", str(so), *map(str, sorted(d.glob("*.o")))], check=True,
                   capture_output=True, text=True)
    lib = ctypes.CDLL(str(so))
    lib.fake_launch.restype = ctypes.c_char_p
    for name in ("lmc_rotate", "lmc_append_rotated", "lmc_linear_step", "lmc_linear_scan", "lmc_linear_scan_workspace"):
        getattr(lib, name).argtypes = getattr(lmc._lib, name).argtypes
    return lib


@pytest.fixture()
def fake(fake_lib):
    fake_lib.fake_reset()
    return fake_lib


@pytest.fixture()
def env(lmc):
    layers = [W.kda(768, 3, 4, 64), W.mla(1152), W.swa(64, 128), W.kda(4, 1, 4, 64)]
    L = lmc.lmc_layout_build(layers, 64, False, 1 << 24)
    buf = np.zeros(8192, dtype=np.uint8)
    return L, (buf.ctypes.data + 255) // 256 * 256, buf


class Fake:
    """The binding's names over another library."""

    def __init__(self, lmc, lib):
        self._lmc, self._lib = lmc, lib

    def __getattr__(self, name):
        return getattr(self._lmc, name)


CALLS = {
    "rotate": lambda f, L, base: C._rotate(f, base),
    "rotate odd": lambda f, L, base: C._rotate(f, base, xr=517, xh=129),
    "append": lambda f, L, base: C._append(f, L, base),
    "append odd": lambda f, L, base: C._append(f, L, base, stride=577),
    "step": lambda f, L, base: C._step(f, L, base),
    "scan": lambda f, L, base: C._scan(f, L, base),
    "long scan": lambda f, L, base: C._scan(f, L, base, n=1 << 20),
}
KERNELS = {"rotate": ["eights"], "rotate odd": ["rotate_kernel"], "append": ["long"], "append odd": ["rotate_kernel"],
           "step": ["step"], "scan": ["scan"], "long scan": ["scan", "join", "scan"]}


@pytest.mark.parametrize("name", CALLS)
def test_each_calls_launches(lmc, fake, env, name):
    L, base, _ = env
    f = Fake(lmc, fake)
    assert CALLS[name](f, L, base) == lmc.LMC_OK
    got = launches(fake)
    assert len(got) == len(KERNELS[name]) and all(k in g[0] for k, g in zip(KERNELS[name], got)), got


@pytest.mark.parametrize("name", CALLS)
def test_a_failed_launch_is_reported_and_nothing_follows(lmc, fake, env, name):
    L, base, _ = env
    f = Fake(lmc, fake)
    for at in range(len(KERNELS[name])):
        fake.fake_reset()
        fake.fake_fail_launch(at)
        assert CALLS[name](f, L, base) == lmc.LMC_ERR_CUDA
        assert len(launches(fake)) == at
        assert fake.fake_last_error() == 0  # it has been taken, and is not the next call's
        fake.fake_fail_launch(-1)
        assert CALLS[name](f, L, base) == lmc.LMC_OK


@pytest.mark.parametrize("name", CALLS)
def test_an_error_of_an_earlier_call_is_not_this_ones(lmc, fake, env, name):
    L, base, _ = env
    fake.fake_set_last_error(700)
    assert CALLS[name](Fake(lmc, fake), L, base) == lmc.LMC_OK


@pytest.mark.parametrize("R,n", [(1, 1), (5, 400), (1, 600), (3, 5000), (1 << 20, 1 << 20), (1, (1 << 31) - 1),
                                 (200, 3_000_000)])
def test_scan_covers_every_segment_within_its_workspace(lmc, fake, env, R, n):
    """A thread block for every head of every segment that requests of n tokens may
    have; the workspace holds a state and a decay for each but the last."""
    L, base, _ = env
    H, rec = 4, 4 * 64 * 64 * 4
    need = ctypes.c_int64(0)
    assert fake.lmc_linear_scan_workspace(L.handle, 0, R, n, H, ctypes.byref(need)) == lmc.LMC_OK
    segment = max(512, -(-(-(-n * H // 152)) // 64) * 64)
    cuts = n // segment
    assert cuts <= min(n // 512, 152 // H)
    most = min(n // 512, 152 // H) * (rec + H * 4)
    assert most <= need.value <= most + 1024
    f = Fake(lmc, fake)
    far = dict(out=base + (1 << 60))
    assert C._scan(f, L, base, R=R, n=n, ws_bytes=need.value - 1, **far) == lmc.LMC_ERR_INVALID_ARG
    assert launches(fake) == []
    assert C._scan(f, L, base, R=R, n=n, ws_bytes=need.value, **far) == lmc.LMC_OK
    got = launches(fake)
    assert got[-1][1] == ((cuts + R) * H, 1, 1)
    assert len(got) == 1 + (cuts >= 2) + (cuts >= 3)
    if cuts >= 2:
        assert got[0][1] == (cuts * H, 1, 1)


def test_grids_past_31_bits_are_refused(lmc, fake, env):
    layers = [W.kda(64, 1, 65535, 8)]
    L = lmc.lmc_layout_build(layers, 64, False, 1 << 30)
    _, base, _ = env
    f = Fake(lmc, fake)
    kw = dict(R=1 << 17, H=65535, K=1, dk=8, dv=8, qr=8, kr=8, vr=65535 * 8, vh=8, outr=65535 * 8, outh=8, dr=0, dh=0,
              out=base + (1 << 60))
    assert C._step(f, L, base, **kw) == lmc.LMC_ERR_OVERFLOW
    assert C._scan(f, L, base, n=1, **kw) == lmc.LMC_ERR_OVERFLOW
    assert launches(fake) == []


@pytest.mark.parametrize("H", [1, 4, 5, 8, 64, 153])
def test_a_workspace_for_the_largest_call_serves_smaller_ones(lmc, H):
    """Segments are of whole tiles, so calls of fewer tokens may have more of them."""
    L = lmc.lmc_layout_build([W.kda(64, 1, H, 8)], 64, False, 1 << 24)
    sizes = [lmc.lmc_linear_scan_workspace(L, 0, 3, n, H) for n in [0, 1, *range(500, 200_000, 333), 1 << 20, (1 << 31) - 1]]
    assert sizes == sorted(sizes)


def test_a_call_takes_the_workspace_of_a_larger_one(lmc, fake, env):
    L, base, _ = env
    need = ctypes.c_int64(0)
    assert fake.lmc_linear_scan_workspace(L.handle, 0, 8, 131072, 4, ctypes.byref(need)) == lmc.LMC_OK
    for n in range(64, 131072, 1000):
        assert C._scan(Fake(lmc, fake), L, base, n=n, ws_bytes=need.value, out=base + (1 << 60)) == lmc.LMC_OK
