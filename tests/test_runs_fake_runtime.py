"""Host code of the attention over runs on a stand-in for the CUDA runtime
(fake_cudart.cpp): the order of its calls and what it asks of which device.
No GPU needed; the buffer addresses are never followed."""
import ctypes as C
import os
import subprocess

import pytest

from prefill_kv_shared_gb300 import build
from prefill_kv_shared_gb300.binding import PF_E_DEVICE_TIMEOUT, PF_OK

HERE = os.path.dirname(os.path.abspath(__file__))
WORK = 0x50000


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    build.build()
    obj = os.path.join(build.BUILD, "attention_runs.cu.o")
    if not os.path.exists(obj):
        build.build(force=True)
    so = str(tmp_path_factory.mktemp("fake") / "runs_on_fake_runtime.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    # -Bsymbolic: the stand-in's functions, also where a CUDA runtime is loaded
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I" + cuda, "-Wl,-Bsymbolic", "-o", so,
                    os.path.join(HERE, "fake_cudart.cpp"), obj], check=True)
    lib = C.CDLL(so)
    lib.fake_log.restype = C.c_char_p
    lib.pfop_attention_status.argtypes = [C.c_void_p, C.c_void_p]
    return lib


def _log(lib):
    return lib.fake_log().decode().split()


def test_status_without_an_error_waits_once(lib):
    lib.fake_reset(0, 152, 152, 0)
    assert lib.pfop_attention_status(WORK, None) == PF_OK
    assert _log(lib) == ["copy", "sync"]


def test_status_after_an_error_returns_with_the_scratch_cleared(lib):
    """A call that follows on another stream is not ordered behind the
    clearing, so that has to be over when the status returns."""
    lib.fake_reset(0, 152, 152, 4)
    assert lib.pfop_attention_status(WORK, None) == PF_E_DEVICE_TIMEOUT
    assert _log(lib) == ["copy", "sync", "set:0x4096", "sync"]


class _Run(C.Structure):
    _fields_ = [("n_rows", C.c_int32), ("pos0", C.c_int32), ("cell0", C.c_int32)]


def _launches(lib, device, sms0, sms1, rows, past, heads=(8, 1, 256)):
    """The grids of a call on `device`, and the scratch it needs."""
    lib.fake_reset(device, sms0, sms1, 0)
    runs = (_Run * 1)(_Run(rows, past, 0))
    lib.pfop_attention_work_bytes.restype = C.c_int64
    need = lib.pfop_attention_work_bytes(*heads, runs, 1)
    p = C.c_void_p
    rc = lib.pfop_attention_packed(p(0x10000), p(0x20000), p(0x30000), C.c_int64(rows + past), *heads, runs, 1,
                                   p(0x40000), p(WORK), C.c_int64(need), None)
    assert rc == PF_OK
    return [int(w.split(":")[1].split("x")[0]) for w in _log(lib) if w.startswith("launch")], need


def test_the_cut_is_that_of_the_current_device(lib):
    """Each call's share of the work is cut for the multiprocessors of the
    device that is current, whichever device the first call was made on."""
    big, big_need = _launches(lib, 0, 152, 20, 25, 30000)
    small, small_need = _launches(lib, 1, 152, 20, 25, 30000)
    assert 100 < big[0] <= 152 and small[0] == 20
    assert small_need < big_need
    assert _launches(lib, 0, 152, 20, 25, 30000) == (big, big_need)
