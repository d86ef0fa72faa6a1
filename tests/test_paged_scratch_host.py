"""The scratch of attention over pages, to the byte, on a stand-in for the CUDA
runtime: no GPU needed."""
import pytest

from prefill_kv_shared_gb300.binding import PF_E_ARG, PF_OK
from tests.test_paged_fake_runtime import _call, lib  # noqa: F401 (a fixture)


@pytest.mark.parametrize("heads,runs", [
    ((8, 1, 256), [(1, 32768, 0)]), ((8, 2, 256), [(4, 9000, 0)] * 3), ((32, 4, 64), [(1, 32768, 0), (1, 5, 0)]),
    ((32, 4, 64), [(3, 700, 0)] * 50 + [(1, 20000, 0)]), ((8, 1, 256), [(40, 9000, 0), (1, 20, 0)]),
    ((32, 4, 64), [(25, 30000, 0)]),
])
def test_cut_work_needs_all_of_it(lib, heads, runs):  # noqa: F811
    """The header alone, or a byte too few: refused, with no launch."""
    rc, grids, need = _call(lib, runs, heads)
    assert rc == PF_OK and len(grids) == 2 and need > 4096  # cut, and joined
    # (the size serves the calls over cells too, and may be more than this one needs)
    least = next(s for s in range(need, 0, -256) if _call(lib, runs, heads, short=need - s)[0] != PF_OK)
    assert least >= 4096
    for short in (need - 4096, need - 4096 - 256, need - least):
        rc, grids, _ = _call(lib, runs, heads, short=short)
        assert rc == PF_E_ARG and grids == []
