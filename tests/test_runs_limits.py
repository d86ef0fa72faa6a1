"""How much work one call of attention over runs takes: a call is refused only
where its real work passes the limit that include/prefill_ops.h states.  Host
only: no GPU needed."""
import pytest

from prefill_kv_shared_gb300 import binding
from prefill_kv_shared_gb300.binding import AttnRun, PF_E_ARG

LIMIT = 1 << 30


@pytest.fixture(scope="module")
def lib():
    from prefill_kv_shared_gb300 import build
    build.build()
    return binding.load()


def _work(heads, runs, block):
    """The units of the header, block by block: for every KV head and block
    of `block` MMA rows of a run the 128-key chunks that its last row reaches,
    and 3 (head_dim 256) or 4."""
    hq, hkv, hd = heads
    step = block // (hq // hkv)  # a block's rows of the run
    total = 0
    for n, pos0, _ in runs:
        for first in range(0, n, step):
            keys = pos0 + min(n, first + step)
            total += (keys + 127) // 128 + (3 if hd == 256 else 4)
    return total * hkv


def _need(lib, heads, runs):
    return lib.pfop_attention_work_bytes(*heads, (AttnRun * len(runs))(*[AttnRun(*r) for r in runs]), len(runs))


@pytest.mark.parametrize("heads,block", [((32, 8, 64), 256), ((8, 1, 256), 256), ((16, 1, 256), 256), ((48, 3, 256), 256)])
def test_the_longest_prompts_are_taken(lib, heads, block):
    runs = [(1 << 20, 0, 0)]
    assert _work(heads, runs, block) < LIMIT
    assert _need(lib, heads, runs) >= 4096


@pytest.mark.parametrize("heads", [(64, 64, 64), (64, 16, 256), (1024, 64, 64)])
@pytest.mark.parametrize("pos0", [0, 100_001])
def test_just_below_and_above_the_limit(lib, heads, pos0):
    """The largest prompt that fits, and the next one.  (A tree over the same
    rows would see more keys; runs of more than 256 rows are no trees.)"""
    lo, hi = 1, 1 << 20
    assert _work(heads, [(hi, pos0, 0)], 256) >= LIMIT
    while hi - lo > 1:
        mid = (lo + hi) // 2
        if _work(heads, [(mid, pos0, 0)], 256) < LIMIT:
            lo = mid
        else:
            hi = mid
    assert _need(lib, heads, [(lo, pos0, 0)]) >= 4096
    assert _need(lib, heads, [(hi, pos0, 0)]) == PF_E_ARG
    assert b"more work" in lib.pfop_last_error()


def test_many_runs_below_and_above(lib):
    """One row of 64 KV heads behind 2^24 keys is 64 (2^17 + 4) units or more."""
    heads, run = (64, 64, 64), (256, (1 << 24) - 256, 0)
    each = _work(heads, [run], 256)
    assert _need(lib, heads, [run] * ((LIMIT - 1) // each)) >= 4096
    assert _need(lib, heads, [run] * ((LIMIT - 1) // each + 1)) == PF_E_ARG


@pytest.mark.parametrize("run", [(1 << 20, (1 << 30) - (1 << 20), 0), (1 << 19, 1 << 29, 0)])
@pytest.mark.parametrize("heads", [(8, 1, 64), (16, 1, 256), (1024, 1024, 64)])
def test_far_above_the_limit(lib, heads, run):
    """Work that passes 2^32 units."""
    assert _need(lib, heads, [run]) == PF_E_ARG
    assert _need(lib, heads, [run] * 2) == PF_E_ARG
