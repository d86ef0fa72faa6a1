"""Refusals of the several-sequence operators (attention over runs, token log
probabilities), all made on the host before any CUDA call: no GPU needed.
The buffer addresses here are never followed."""
import ctypes as C

import pytest

from prefill_kv_shared_gb300 import binding
from prefill_kv_shared_gb300.binding import AttnRun, PF_E_ARG, PF_OK

Q, K, V, OUT, WORK, MASK = (0x10000 * (i + 1) for i in range(6))
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from prefill_kv_shared_gb300 import build
    build.build()
    return binding.load()


def _runs(*runs):
    return (AttnRun * max(1, len(runs)))(*[AttnRun(*r) for r in runs]), len(runs)


def _packed(lib, runs, cells=1000, heads=(8, 2, 64), q=Q, k=K, v=V, out=OUT, work=WORK, nbytes=BIG):
    arr, n = _runs(*runs)
    return lib.pfop_attention_packed(q, k, v, cells, *heads, arr, n, out, work, nbytes, None)


def _tree(lib, runs, cells=1000, heads=(8, 2, 64), mask=MASK, words=1, work=WORK, nbytes=BIG):
    arr, n = _runs(*runs)
    return lib.pfop_attention_tree(Q, K, V, cells, *heads, arr, n, mask, words, OUT, work, nbytes, None)


@pytest.mark.parametrize("heads", [(8, 2, 128), (8, 2, 0), (6, 4, 64), (24, 8, 64), (0, 1, 64), (8, 0, 64),
                                   (2048, 128, 64), (32, 1, 64)])
def test_head_layouts(lib, heads):
    assert _packed(lib, [(4, 0, 0)], heads=heads) == PF_E_ARG
    assert _tree(lib, [(4, 0, 0)], heads=heads) == PF_E_ARG
    arr, n = _runs((4, 0, 0))
    assert lib.pfop_attention_work_bytes(*heads, arr, n) == PF_E_ARG


@pytest.mark.parametrize("run,cells", [
    ((-1, 0, 0), 1000), ((4, -1, 0), 1000), ((4, 0, -1), 1000),
    ((4, 0, 997), 1000), ((4, 997, 0), 1000), ((1001, 0, 0), 1000), ((1, 0, 0), 0),
    ((4, (1 << 30) - 3, 0), (1 << 31) - 1024), ((4, (1 << 31) - 1, (1 << 31) - 1), 1000),
    (((1 << 20) + 1, 0, 0), (1 << 31) - 1024),
])
def test_runs_outside_the_cache(lib, run, cells):
    assert _packed(lib, [run], cells=cells) == PF_E_ARG
    assert _tree(lib, [run], cells=cells, words=4) == PF_E_ARG


def test_cell_counts(lib):
    for cells in (-1, (1 << 31) - 1023, 1 << 40):
        assert _packed(lib, [(4, 0, 0)], cells=cells) == PF_E_ARG


def test_run_counts(lib):
    assert _packed(lib, [(1, 0, i) for i in range(129)]) == PF_E_ARG
    assert lib.pfop_attention_packed(Q, K, V, 10, 8, 2, 64, None, 1, OUT, WORK, BIG, None) == PF_E_ARG
    assert lib.pfop_attention_packed(Q, K, V, 10, 8, 2, 64, None, -1, OUT, WORK, BIG, None) == PF_E_ARG
    # nothing to do: no rows, whatever the buffers
    assert _packed(lib, [], q=None, work=None, nbytes=0) == PF_OK
    assert _packed(lib, [(0, 5, 7), (0, 0, 0)], q=None, work=None, nbytes=0) == PF_OK
    assert _tree(lib, [(0, 5, 7)], mask=None, work=None, nbytes=0) == PF_OK


@pytest.mark.parametrize("words,rows", [(0, 1), (5, 1), (-1, 1), (1, 65), (2, 129), (4, 257)])
def test_mask_words(lib, words, rows):
    assert _tree(lib, [(rows, 0, 0)], words=words) == PF_E_ARG


def test_buffers(lib):
    one = [(4, 0, 0)]
    for name in ("q", "k", "v", "out"):
        for bad in (None, 0x10008) + ((0x10010,) if name == "out" else ()):
            assert _packed(lib, one, **{name: bad}) == PF_E_ARG, name
    assert _packed(lib, one, work=None) == PF_E_ARG
    assert _packed(lib, one, work=WORK + 16) == PF_E_ARG
    assert _tree(lib, one, mask=None) == PF_E_ARG
    assert _tree(lib, one, mask=MASK + 4) == PF_E_ARG
    assert lib.pfop_attention_status(None, None) == PF_E_ARG


@pytest.mark.parametrize("heads", [(8, 1, 256), (8, 2, 256), (32, 4, 64), (16, 16, 64)])
@pytest.mark.parametrize("runs", [[(1, 0, 0)], [(25, 32768, 0)], [(512, 0, 0)], [(16, 500 + i, 0) for i in range(64)]])
def test_scratch_sizes(lib, heads, runs):
    """The size covers both calls; a scratch of the header alone is refused
    where states have to be kept, one below the header always."""
    arr, n = _runs(*runs)
    need = lib.pfop_attention_work_bytes(*heads, arr, n)
    assert 4096 <= need < 1 << 30
    assert lib.pfop_attention_work_bytes(*heads, arr, 0) == 4096
    assert _packed(lib, runs, cells=1 << 20, heads=heads, nbytes=4095) == PF_E_ARG
    if runs[0][0] <= 256:
        assert _tree(lib, runs, cells=1 << 20, heads=heads, words=4, nbytes=4095) == PF_E_ARG


def _logprobs(lib, ltype=0, logits=Q, ld=100, rows=2, vocab=100, tok=K, n_top=0, logp=V, ent=OUT, tid=None, tlp=None):
    return lib.pfop_logprobs(ltype, logits, ld, rows, vocab, tok, n_top, logp, ent, tid, tlp, None)


@pytest.mark.parametrize("kw", [
    dict(ltype=2), dict(ltype=-1), dict(rows=-1), dict(vocab=0), dict(vocab=1 << 30, ld=1 << 30), dict(ld=99),
    dict(n_top=33, tid=WORK, tlp=MASK), dict(n_top=-1), dict(n_top=5, vocab=4, ld=4, tid=WORK, tlp=MASK),
    dict(n_top=5), dict(n_top=5, tid=WORK), dict(logits=None), dict(tok=None), dict(logp=None),
    dict(logits=Q + 2), dict(ltype=1, logits=Q + 1), dict(logp=V + 2), dict(ent=OUT + 1), dict(tok=K + 2),
    dict(n_top=5, tid=WORK + 1, tlp=MASK),
])
def test_logprob_refusals(lib, kw):
    assert _logprobs(lib, **kw) == PF_E_ARG
    assert lib.pfop_last_error()


def test_logprobs_of_no_rows(lib):
    assert _logprobs(lib, rows=0, logits=None, tok=None, logp=None, ent=None) == PF_OK


def test_wrappers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="CUDA"):
        binding.logprobs(torch.zeros(2, 10))
    with pytest.raises(ValueError, match="element type"):
        binding.logprobs(torch.zeros(2, 10, dtype=torch.float16))
    with pytest.raises(ValueError, match="dense rows"):
        binding.logprobs(torch.zeros(10, 2).T)
    with pytest.raises(ValueError, match="go together"):
        binding.logprobs(torch.zeros(2, 10), tokens=torch.zeros(2, dtype=torch.int32))
