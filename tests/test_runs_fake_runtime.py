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
