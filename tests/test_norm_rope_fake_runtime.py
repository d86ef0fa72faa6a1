"""What norm and rotation hand to their kernel, on a stand-in for the CUDA
runtime.  No GPU needed; the buffer addresses are never followed."""
import ctypes as C
import os
import subprocess

import pytest

from prefill_kv_shared_gb300 import build
from prefill_kv_shared_gb300.binding import PF_OK

HERE = os.path.dirname(os.path.abspath(__file__))
Q, K, V, POS, SLOTS, OUT, KC, VC = (0x10000 * (i + 1) for i in range(8))
Q_GAIN, K_GAIN = 0x7b51_0000_1230, 0x7b52_0000_4560


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    build.build()
    obj = os.path.join(build.BUILD, "norm_rope.cu.o")
    if not os.path.exists(obj):
        build.build(force=True)
    so = str(tmp_path_factory.mktemp("fake") / "norm_rope_on_fake_runtime.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I" + cuda, "-Wl,-Bsymbolic", "-o", so,
                    os.path.join(HERE, "fake_cudart_args.cpp"), obj], check=True)
    lib = C.CDLL(so)
    lib.fake_first_arg.restype = C.POINTER(C.c_uint8 * 112)
    return lib


@pytest.mark.parametrize("itype", [0, 1])
@pytest.mark.parametrize("hd", [64, 256])
def test_without_keys_their_gain_is_not_handed_on(lib, itype, hd):
    """It may be any address then: the call has not looked at it."""
    p, i64, f = C.c_void_p, C.c_int64, C.c_float

    def handed(hkv, k_gain):
        lib.fake_reset(0, 152, 152, 0)
        rc = lib.pfop_qk_norm_rope(itype, p(Q), i64(8 * hd), p(K), i64(2 * hd), p(V), i64(2 * hd), 3, 8, hkv, hd, p(POS),
                                   p(SLOTS), p(Q_GAIN), p(k_gain), f(1e-6), f(1e4), p(OUT), p(KC), p(VC), i64(64), None)
        assert rc == PF_OK
        words = bytes(lib.fake_first_arg().contents)
        return Q_GAIN.to_bytes(8, "little") in words, k_gain.to_bytes(8, "little") in words

    assert handed(2, K_GAIN) == (True, True)
    assert handed(0, K_GAIN) == (True, False)
    assert handed(0, K_GAIN + 1) == (True, False)  # no float's address
