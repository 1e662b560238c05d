"""What the library asks of the CUDA runtime, without a GPU: its objects are
linked against the stand-in in fake_cudart.cpp, which keeps every kernel's
shared-memory opt-in and every launch."""

import ctypes
import glob
import os
import shutil
import subprocess

import pytest

from shared_kv_caches_b200 import build as B
from shared_kv_caches_b200 import kvattn as K

HERE = os.path.dirname(os.path.abspath(__file__))
FAKE = 1 << 20

#: shared memory that the kernels declare themselves (bytes, as ptxas reports
#: them): it counts against the 48 KB of a launch without an opt-in
DECLARED = {"build_tables_kernel": 272, "plan_kernel": 4352}


class Runtime:
    def __init__(self, path):
        self.lib = ctypes.CDLL(path)
        self.lib.fake_lines.restype = ctypes.c_char_p
        self.lib.fake_fail.argtypes = [ctypes.c_char_p, ctypes.c_int]
        self.lib.fake_fixed.argtypes = [ctypes.c_char_p, ctypes.c_int]
        for name, n in DECLARED.items():
            self.lib.fake_fixed(name.encode(), n)

    def clear(self):
        self.lib.fake_clear()
        self.lib.fake_fail(b"", 0)
        self.lib.fake_last_error(0)

    def lines(self, what, kernel):
        rows = [x.split() for x in self.lib.fake_lines().decode().splitlines()]
        return [r for r in rows if r[0] == what and kernel in r[1]]

    def opt_ins(self, kernel):
        return [int(r[2]) for r in self.lines("opt_in", kernel)]

    def launches(self, kernel):
        return [dict(grid=int(r[2]), block=int(r[3]), shared=int(r[4]), cluster=int(r[5])) for r in self.lines("launch", kernel)]


def linked(folder):
    """The library's objects and the stand-in, in a library of their own: a
    process has each kernel's opt-in from the start."""
    B.build()
    names = [os.path.basename(s)[:-3] for s in glob.glob(os.path.join(B.CSRC, "*.cu"))]
    objs = [os.path.join(B.BUILD, n + ".o") for n in names]
    if not all(os.path.exists(o) and os.path.getmtime(o) <= os.path.getmtime(B.LIB) + 1 for o in objs):
        B.build(force=True)
    out = os.path.join(folder, "libkvattn_fake.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(B.NVCC)), "include")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-O1", "-I", cuda, "-Wl,-Bsymbolic",
                    os.path.join(HERE, "fake_cudart.cpp")] + objs + ["-o", out], check=True)
    return out


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    return linked(str(tmp_path_factory.mktemp("fake")))


@pytest.fixture
def rt(library, tmp_path, monkeypatch):
    """A runtime that has seen no call yet, and the Python names bound to it."""
    path = str(tmp_path / "libkvattn_fake.so")
    shutil.copy(library, path)
    monkeypatch.setattr(K, "LIB_PATH", path)
    monkeypatch.setattr(K, "_lib", None)
    return Runtime(path)


# ------------------------------------------------------------------ tables

def tables(batch, tokens=64, in_place=False):
    lens = FAKE if in_place else 2 * FAKE
    return K.kvattn_build_tables(batch, 8, 100, tokens, FAKE, FAKE + 4, FAKE + 8, FAKE + 12, FAKE + 16, lens, lens + 12, *[FAKE] * 5)


@pytest.mark.parametrize("batch", [1, 4072, 4073, 4074, 4095, 4096, 4097, 16384])
def test_tables_of_any_batch_fit_their_shared_memory(rt, batch):
    """The sums take 12 bytes a request beside what the kernel declares: a
    first call near the 48 KB of a launch without an opt-in goes through."""
    assert tables(batch) == 0
    assert rt.launches("build_tables_kernel")[-1]["shared"] == 12 * batch + 8
