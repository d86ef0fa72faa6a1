"""Refusals of the paged serving step's operators (attention over pages, norm
and rotation into the cache, verification of drafts), all made on the host
before any CUDA call: no GPU needed.  The buffer addresses are never followed."""
import ctypes as C

import pytest

from prefill_kv_shared_gb300 import binding
from prefill_kv_shared_gb300.binding import AttnRun, PF_E_ARG, PF_OK

BUF = [0x10000 * (i + 1) for i in range(12)]
Q, K, V, OUT, WORK, MASK, TABLE = BUF[:7]
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from prefill_kv_shared_gb300 import build
    build.build()
    return binding.load()


def _paged(lib, runs, pages=10, page=16, heads=(8, 2, 64), q=Q, k=K, v=V, out=OUT, work=WORK, nbytes=BIG, table=TABLE,
           entries=100, mask=None, words=0):
    arr = (AttnRun * max(1, len(runs)))(*[AttnRun(*r) for r in runs])
    return lib.pfop_attention_paged(q, k, v, pages, page, *heads, arr, len(runs), table, entries, mask, words, out, work,
                                    nbytes, None)


@pytest.mark.parametrize("page", [0, -16, 1, 4, 7, 12, 24, 100, (1 << 30) + 1, -(1 << 31)])
def test_page_sizes(lib, page):
    assert _paged(lib, [(4, 0, 0)], page=page) == PF_E_ARG
    assert b"page_size" in lib.pfop_last_error()


@pytest.mark.parametrize("pages,page", [(-1, 16), (1 << 27, 16), ((1 << 31) - 1, 8), (2, 1 << 30), (0, 16)])
def test_page_counts(lib, pages, page):
    assert _paged(lib, [(4, 0, 0)], pages=pages, page=page) == PF_E_ARG


@pytest.mark.parametrize("run,entries", [
    ((4, 0, 0), 0), ((16, 0, 0), 0), ((17, 0, 0), 1), ((1, 16, 0), 1), ((4, 0, 5), 5), ((4, 0, 100), 100),
    ((1, 1600, 0), 100), ((4, 0, (1 << 31) - 1), 1 << 20), ((-1, 0, 0), 100), ((4, -1, 0), 100), ((4, 0, -1), 100),
    ((4, (1 << 30) - 3, 0), 1 << 40), ((4, 0, 0), -1), ((17, 0, (1 << 31) - 2), 1 << 40),
    ((1, 16, (1 << 31) - 2), 1 << 33),
])
def test_runs_outside_the_table(lib, run, entries):
    assert _paged(lib, [run], entries=entries) == PF_E_ARG


@pytest.mark.parametrize("heads", [(8, 2, 128), (6, 4, 64), (24, 8, 64), (0, 1, 64), (2048, 128, 64)])
def test_head_layouts(lib, heads):
    assert _paged(lib, [(4, 0, 0)], heads=heads) == PF_E_ARG
    assert lib.pfop_attention_paged_work_bytes(*heads, (AttnRun * 1)(AttnRun(4, 0, 0)), 1) == PF_E_ARG


def test_buffers(lib):
    one = [(4, 0, 0)]
    for name in ("q", "k", "v", "out"):
        for bad in (None, 0x10008) + ((0x10010,) if name == "out" else ()):
            assert _paged(lib, one, **{name: bad}) == PF_E_ARG, name
    assert _paged(lib, one, work=None) == PF_E_ARG
    assert _paged(lib, one, work=WORK + 16) == PF_E_ARG
    assert _paged(lib, one, nbytes=4095) == PF_E_ARG
    assert _paged(lib, one, table=None) == PF_E_ARG
    assert _paged(lib, one, table=TABLE + 2) == PF_E_ARG
    assert _paged(lib, one, mask=MASK + 4, words=1) == PF_E_ARG
    assert lib.pfop_attention_paged_status(None, None) == PF_E_ARG


@pytest.mark.parametrize("words,rows", [(0, 1), (5, 1), (-1, 1), (1, 65), (2, 129), (4, 257)])
def test_mask_words(lib, words, rows):
    assert _paged(lib, [(rows, 0, 0)], mask=MASK, words=words) == PF_E_ARG


def test_nothing_to_do(lib):
    assert _paged(lib, [], q=None, work=None, nbytes=0, table=None, pages=0) == PF_OK
    assert _paged(lib, [(0, 5, 7), (0, 0, 0)], q=None, work=None, nbytes=0, entries=0) == PF_OK
    assert _paged(lib, [(1, 0, 0)] * 129) == PF_E_ARG
    assert lib.pfop_attention_paged_work_bytes(8, 2, 64, (AttnRun * 1)(), 0) == 4096


@pytest.mark.parametrize("heads", [(8, 1, 256), (8, 2, 256), (32, 4, 64), (16, 16, 64), (16, 1, 256)])
@pytest.mark.parametrize("runs", [[(1, 0, 0)], [(25, 32768, 0)], [(512, 0, 0)], [(16, 500 + i, 0) for i in range(64)],
                                  [(1, 4000 * i, 0) for i in range(128)]])
def test_scratch_sizes(lib, heads, runs):
    """The size serves the calls over cells too (one AttnRuns for both)."""
    arr = (AttnRun * len(runs))(*[AttnRun(*r) for r in runs])
    need = lib.pfop_attention_paged_work_bytes(*heads, arr, len(runs))
    assert lib.pfop_attention_work_bytes(*heads, arr, len(runs)) <= need < 1 << 30


def _rope(lib, itype=0, q=Q, q_ld=512, k=K, k_ld=128, v=V, v_ld=128, rows=3, hq=8, hkv=2, hd=64, pos=MASK, slots=TABLE,
          qg=None, kg=None, eps=1e-6, base=1e4, qo=OUT, kc=WORK, vc=BUF[8], cells=100):
    return lib.pfop_qk_norm_rope(itype, q, q_ld, k, k_ld, v, v_ld, rows, hq, hkv, hd, pos, slots, qg, kg, eps, base, qo,
                                 kc, vc, cells, None)


@pytest.mark.parametrize("kw", [
    dict(itype=2), dict(itype=-1), dict(hd=128), dict(hd=0), dict(rows=-1), dict(rows=(1 << 24) + 1), dict(hq=0),
    dict(hq=1025), dict(hkv=-1), dict(hkv=1025), dict(q_ld=511), dict(q_ld=514), dict(k_ld=127), dict(v_ld=127),
    dict(v_ld=130), dict(itype=1, q_ld=516), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(base=0.5), dict(base=float("nan")), dict(base=float("inf")), dict(cells=-1), dict(cells=1 << 31),
    dict(q=None), dict(k=None), dict(v=None), dict(pos=None), dict(slots=None), dict(qo=None), dict(kc=None),
    dict(vc=None), dict(q=Q + 8), dict(k=K + 4), dict(v=V + 8), dict(qo=OUT + 8), dict(kc=WORK + 8),
    dict(vc=BUF[8] + 2), dict(pos=MASK + 2), dict(slots=TABLE + 1), dict(qg=BUF[9] + 2), dict(kg=BUF[9] + 1),
])
def test_norm_rope_refusals(lib, kw):
    assert _rope(lib, **kw) == PF_E_ARG
    assert lib.pfop_last_error()


def test_norm_rope_of_no_rows(lib):
    assert _rope(lib, rows=0, q=None, k=None, pos=None) == PF_OK


def _verify(lib, ltype=0, t=Q, t_ld=100, d=K, d_ld=100, rows=5, n=2, vocab=100, tok=V, first=OUT, u=WORK, noise=MASK,
            na=TABLE, token=BUF[8], pa=BUF[9], work=BUF[10], nbytes=1 << 20):
    return lib.pfop_verify_draft(ltype, t, t_ld, d, d_ld, rows, n, vocab, tok, first, u, noise, na, token, pa, work,
                                 nbytes, None)


@pytest.mark.parametrize("kw", [
    dict(ltype=2), dict(ltype=-1), dict(rows=-1), dict(rows=(1 << 20) + 1), dict(n=-1), dict(n=6), dict(vocab=0),
    dict(vocab=1 << 30, t_ld=1 << 30, d_ld=1 << 30), dict(t_ld=99), dict(d_ld=99), dict(t=None), dict(tok=None),
    dict(first=None), dict(u=None), dict(noise=None), dict(na=None), dict(token=None), dict(work=None),
    dict(t=Q + 2), dict(d=K + 2), dict(ltype=1, t=Q + 1), dict(tok=V + 2), dict(first=OUT + 1), dict(u=WORK + 2),
    dict(noise=MASK + 2), dict(na=TABLE + 2), dict(token=BUF[8] + 1), dict(pa=BUF[9] + 3), dict(work=BUF[10] + 128),
    dict(nbytes=0), dict(nbytes=300),
])
def test_verify_refusals(lib, kw):
    assert _verify(lib, **kw) == PF_E_ARG
    assert lib.pfop_last_error()


def test_verify_of_no_sequences(lib):
    assert _verify(lib, rows=0, n=0, t=None, tok=None) == PF_OK
    assert lib.pfop_verify_draft_work_bytes(0, 0) >= 0
    for rows, n in ((-1, 0), (4, 5), (4, -1), ((1 << 20) + 1, 0)):
        assert lib.pfop_verify_draft_work_bytes(rows, n) == PF_E_ARG
    assert lib.pfop_verify_draft_work_bytes(1 << 20, 1) > 0


def test_wrappers_refuse_host_tensors_and_types():
    torch = pytest.importorskip("torch")
    q = torch.zeros(4, 8, 64)
    with pytest.raises(ValueError, match="CUDA"):
        binding.qk_norm_rope(q, None, None)
    with pytest.raises(ValueError, match="element type"):
        binding.qk_norm_rope(q.half(), None, None)
    with pytest.raises(ValueError, match="element type"):
        binding.verify_draft(torch.zeros(2, 10, dtype=torch.float16), *[None] * 8)
    runs = object.__new__(binding.AttnRuns)
    with pytest.raises(ValueError, match="page size"):
        binding.attention_paged(q, torch.zeros(4, 8, 64), torch.zeros(4, 8, 64), runs, None, None)
    with pytest.raises(ValueError, match="32 bits"):
        binding.VerifyWork(1 << 32, 1)
