"""Host code of the drafts' verification on a stand-in for the CUDA runtime
(fake_cudart.cpp).  No GPU needed; the buffer addresses are never followed."""
import ctypes as C
import os
import subprocess

import pytest

from prefill_kv_shared_gb300 import build
from prefill_kv_shared_gb300.binding import PF_E_ARG, PF_OK

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    build.build()
    obj = os.path.join(build.BUILD, "verify_draft.cu.o")
    if not os.path.exists(obj):
        build.build(force=True)
    so = str(tmp_path_factory.mktemp("fake") / "verify_on_fake_runtime.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I" + cuda, "-Wl,-Bsymbolic", "-o", so,
                    os.path.join(HERE, "fake_cudart.cpp"), obj], check=True)
    lib = C.CDLL(so)
    lib.fake_log.restype = C.c_char_p
    lib.pfop_verify_draft_work_bytes.restype = C.c_int64
    return lib


@pytest.mark.parametrize("ltype,of_chunk", [(0, 512), (1, 1024)])
@pytest.mark.parametrize("rows,n_seq,draft,chunks,fits", [
    (1 << 20, 1, False, 2047, True), (1 << 20, 1, False, 2048, False), (1 << 11, 1, False, 1 << 20, False),
    ((1 << 11) - 1, 1, False, 1 << 20, True), (1 << 20, 0, False, 2048, True),
    (1 << 20, 1 << 19, True, 1365, True), (1 << 20, 1 << 19, True, 1366, False), (1 << 10, 1, True, (1 << 20) - 1, True),
    (1 << 10, 1, True, 1 << 20, True), ((1 << 10) + 1, 1, True, 1 << 20, False),
])
def test_chunks_in_all_rows(lib, ltype, of_chunk, rows, n_seq, draft, chunks, fits):
    """Up to 2^31 - 1 of them, a row's last one whole."""
    vocab = chunks * of_chunk - of_chunk + 1  # one logit into the last
    if vocab >= 1 << 30:
        vocab, chunks = (1 << 30) - 1, (1 << 30) // of_chunk
        fits = chunks * (rows + (rows - n_seq if draft else 0)) < 1 << 31
    fits = fits or n_seq == 0
    p, i64 = C.c_void_p, C.c_int64
    lib.fake_reset(0, 152, 152, 0)
    rc = lib.pfop_verify_draft(ltype, p(0x1000), i64(vocab), p(0x2000) if draft else None, i64(vocab), rows, n_seq, vocab,
                               p(0x3000), p(0x4000), p(0x5000), p(0x6000), p(0x7000), p(0x8000), None, p(0x9000),
                               i64(lib.pfop_verify_draft_work_bytes(rows, n_seq)), None)
    assert rc == (PF_OK if fits else PF_E_ARG)
    assert (lib.fake_log().decode().count("launch") == 2) == (fits and n_seq > 0)
