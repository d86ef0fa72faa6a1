"""Host code of the attention over pages on a stand-in for the CUDA runtime
(fake_cudart.cpp): which kernels a call launches, how its work is cut for which
device.  No GPU needed; the buffer addresses are never followed."""
import ctypes as C
import os
import subprocess

import pytest

from prefill_kv_shared_gb300 import build
from prefill_kv_shared_gb300.binding import PF_E_ARG, PF_OK

HERE = os.path.dirname(os.path.abspath(__file__))
Q, K, V, OUT, WORK, TABLE = (0x10000 * (i + 1) for i in range(6))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    build.build()
    objs = [os.path.join(build.BUILD, f + ".cu.o") for f in ("attention_paged", "attention_runs")]
    if not all(os.path.exists(o) for o in objs):
        build.build(force=True)
    so = str(tmp_path_factory.mktemp("fake") / "paged_on_fake_runtime.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    # -Bsymbolic: the stand-in's functions, also where a CUDA runtime is loaded
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I" + cuda, "-Wl,-Bsymbolic", "-o", so,
                    os.path.join(HERE, "fake_cudart.cpp"), *objs], check=True)
    lib = C.CDLL(so)
    lib.fake_log.restype = C.c_char_p
    lib.pfop_attention_paged_work_bytes.restype = C.c_int64
    return lib


class _Run(C.Structure):
    _fields_ = [("n_rows", C.c_int32), ("pos0", C.c_int32), ("cell0", C.c_int32)]


def _call(lib, runs, heads=(8, 1, 256), device=0, sms=(152, 152), short=0):
    """(status, [(CTAs, threads) of each launch], scratch bytes)"""
    lib.fake_reset(device, *sms, 0)
    arr = (_Run * len(runs))(*[_Run(*r) for r in runs])
    need = lib.pfop_attention_paged_work_bytes(*heads, arr, len(runs))
    p = C.c_void_p
    rc = lib.pfop_attention_paged(p(Q), p(K), p(V), 100000, 16, *heads, arr, len(runs), p(TABLE), C.c_int64(1 << 20), None,
                                  0, p(OUT), p(WORK), C.c_int64(need - short), None)
    log = [w for w in lib.fake_log().decode().split() if w.startswith("launch")]
    return rc, [tuple(int(x) for x in w.split(":")[1].split("x")) for w in log], need


def test_single_tokens_take_the_kernel_of_few_rows(lib):
    for heads, few, threads in (((8, 1, 256), 1, 256), ((32, 4, 64), 2, 256)):
        rc, grids, need = _call(lib, [(1, 9000, 0)] * 64, heads)
        assert rc == PF_OK and grids[0][0] <= 152 * few and grids[0][1] == threads
        # a chunk among them: all of them on the other kernel
        rc, grids, _ = _call(lib, [(1, 9000, 0)] * 64 + [(300, 0, 0)], heads)
        assert rc == PF_OK and grids[0][1] in (256, 384)


def test_an_item_a_cta_where_that_is_even(lib):
    rc, grids, need = _call(lib, [(1, 600, 0)] * 128, (8, 1, 256))
    assert rc == PF_OK and grids == [(128, 256)] and need >= 4096
    rc, grids, need = _call(lib, [(1, 32768, 0)], (8, 1, 256))
    assert rc == PF_OK and len(grids) == 2 and 100 < grids[0][0] <= 152 and need > 4096  # cut, and joined


def test_the_cut_is_that_of_the_current_device(lib):
    rc, big, big_need = _call(lib, [(1, 32768, 0)], sms=(152, 20))
    rc2, small, small_need = _call(lib, [(1, 32768, 0)], device=1, sms=(152, 20))
    assert rc == rc2 == PF_OK and 100 < big[0][0] <= 152 and small[0][0] == 20 and small_need < big_need
    assert _call(lib, [(1, 32768, 0)], sms=(152, 20)) == (rc, big, big_need)


@pytest.mark.parametrize("runs", [[(1, 32768, 0)], [(1, 100, 0)], [(40, 9000, 0), (1, 20, 0)], [(2, 5000, 0)] * 100])
@pytest.mark.parametrize("heads", [(8, 1, 256), (8, 2, 256), (32, 4, 64)])
def test_a_scratch_too_small_launches_nothing(lib, runs, heads):
    rc, grids, need = _call(lib, runs, heads)
    assert rc == PF_OK and grids
    rc, grids, _ = _call(lib, runs, heads, short=need - 4095)
    assert rc == PF_E_ARG and grids == []
