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


# ------------------------------------- opt-ins that calls at once may share

def sizes_asked(rt, kernel):
    """The opt-ins of a kernel and the shared memory of its launches.  An
    opt-in is the kernel's, on its device, for every host thread: were it one
    call's own, another call could lower it before this one's launch."""
    return set(rt.opt_ins(kernel)), {x["shared"] for x in rt.launches(kernel)}


def check_sizes(rt, kernel):
    opt_ins, shared = sizes_asked(rt, kernel)
    assert len(shared) > 1 and len(opt_ins) == 1 and max(shared) <= max(opt_ins)


def expand(d_c, batch=2, n=50000):
    p = K.make_params(batch, 16, 1, d_c, 64, 4, 9, 0)
    return K.kvattn_expand_kv(K.KVATTN_MLA, p, FAKE, FAKE, FAKE, n, 128, 128, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40, None, None)


def prefill(batch=2, n=50000, d=128):
    p = K.kvattn_prefill_params(batch, 8, 8, d, 0, 128, n, n, 1, 0, 0)
    return K.kvattn_prefill(p, FAKE, None, FAKE, None, FAKE, FAKE, FAKE, 0.1, FAKE, None, FAKE, 1 << 40, None, None)


def test_one_opt_in_for_tables_of_every_size(rt):
    for batch in (16384, 5000, 10000):
        assert tables(batch) == 0
    check_sizes(rt, "build_tables_kernel")


def test_one_opt_in_for_expansions_of_every_width(rt):
    for d_c in (512, 64, 256, 128):
        assert expand(d_c) == 0
    check_sizes(rt, "expand_kernel")


def test_one_opt_in_for_lists_of_every_length(rt):
    for batch in (16384, 12000, 11000):
        assert expand(128, batch) == 0 and prefill(batch) == 0
    check_sizes(rt, "plan_kernel")


def decode(variant, heads, kv, dn, dr, splits=0, pages=4096, batch=1):
    p = K.make_params(batch, heads, kv, dn, dr, pages, pages * batch, pages * 64, splits)
    return K.kvattn_decode(variant, p, FAKE, FAKE if dr else None, FAKE, FAKE, FAKE, 0.1, FAKE, None, FAKE, K.kvattn_workspace_size(variant, p), None)


def test_one_opt_in_for_generic_decodes_of_every_width(rt):
    for dn, dr in ((512, 128), (264, 8), (64, 0)):
        assert decode(K.KVATTN_MLA, 4, 1, dn, dr) == 0
    check_sizes(rt, "generic_decode_kernel")


def test_one_opt_in_for_merges_of_every_number_of_parts(rt):
    for branches in (16, 13, 14):
        assert decode(K.KVATTN_MLRA, 16, branches, 64, 8, splits=1024) == 0
    check_sizes(rt, "combine_kernel")


def test_merges_near_48_kb_go_through(rt):
    """The merge declares 2 KB of its own."""
    rt.lib.fake_fixed(b"combine_kernel", 2048)
    assert decode(K.KVATTN_MLRA, 16, 12, 64, 8, splits=1024) == 0
    assert rt.launches("combine_kernel")[-1]["shared"] == 48 * 1024


def test_one_opt_in_for_projections_of_every_depth(rt):
    for k in (512, 64, 128):
        assert K.kvattn_head_proj(FAKE, FAKE, FAKE, 0, 4, 200, k, 64, None, None) == 0
    for kernel in {r[1] for r in rt.lines("launch", "head_proj_kernel")}:
        check_sizes(rt, kernel)


# ------------------------------------------------ errors of calls before

def append(n=4):
    p = K.make_params(1, 16, 1, 512, 64, 4, 9, 0)
    return K.kvattn_append_slots(K.KVATTN_MLA, p, FAKE, n, FAKE, FAKE, FAKE, 1e4, None, None)


@pytest.mark.parametrize("call", [append, lambda: expand(512), prefill, lambda: tables(4)],
                         ids=["append", "expand", "prefill", "tables"])
def test_an_error_left_by_another_call_is_not_this_ones(rt, call):
    """The runtime keeps the last error until someone asks for it: a launch's
    own status counts, not what an earlier call of the process left."""
    rt.lib.fake_last_error(1)
    assert call() == 0


@pytest.mark.parametrize("where", ["cudaFuncSetAttribute", "launch"])
@pytest.mark.parametrize("call", [append, lambda: expand(512), prefill, lambda: tables(16384)],
                         ids=["append", "expand", "prefill", "tables"])
def test_a_failed_call_takes_its_error_with_it(rt, call, where):
    rt.lib.fake_fail(where.encode(), 1)
    st = call()
    assert st == (0 if call is append and where != "launch" else K.KVATTN_ERR_CUDA)
    assert rt.lib.fake_peek() == 0


# -------------------------------------------------------- calls that fail once

def test_prefill_asks_again_where_its_registers_could_not_be_read(rt):
    rt.lib.fake_fail(b"cudaFuncGetAttributes", 1)
    assert prefill() == K.KVATTN_ERR_CUDA and not rt.launches("prefill_kernel")
    assert prefill() == 0 and len(rt.launches("prefill_kernel")) == 1


def test_tensor_maps_are_asked_for_again_where_the_driver_did_not_answer(rt):
    rt.lib.fake_fail(b"cudaGetDriverEntryPoint", 1)
    assert prefill() != 0 and not rt.launches("prefill_kernel") and rt.lib.fake_peek() == 0
    assert prefill() == 0 and len(rt.launches("prefill_kernel")) == 1
