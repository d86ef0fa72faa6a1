"""Prefill attention (pfop_attention, mode 0) of row blocks that lie across the
first border between two groups of key chunks.  The rows before the border
have all their keys in group 0, whose CTA writes them; the CTA of group 1
holds the same block for the rows behind the border, has seen no key of the
others (sum 0) and must leave them alone.  Reference and tolerance are those
of test_gpu_attention_runs.py (fp16 probabilities, bf16 output)."""
import pytest

from prefill_kv_shared_gb300 import binding
from tests.gpu_util import need_gpu, torch
from tests.test_gpu_attention_runs import _check, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    need_gpu()
    from prefill_kv_shared_gb300 import build
    build.build()
    return binding.load()


# a group holds max(4, ceil(chunks / groups)) chunks of 64 keys: the first
# border is at position 256 up to 1024 keys, at 512 for 2048 keys
@pytest.mark.parametrize("heads,rows,pos,kv_len", [
    ((8, 1, 256), 32, 250, 282), ((8, 1, 256), 2, 255, 257), ((8, 2, 256), 40, 240, 280),
    ((32, 4, 64), 32, 250, 282), ((4, 4, 64), 128, 130, 258), ((4, 4, 64), 100, 200, 300),
    ((16, 1, 64), 16, 249, 265), ((8, 1, 256), 64, 500, 2048), ((4, 1, 64), 300, 300, 2048),
])
def test_blocks_across_the_first_group_border(lib, heads, rows, pos, kv_len):
    hq, hkv, hd = heads
    runs = [(rows, pos, 0)]
    q, k, v, out = _inputs(heads, runs, kv_len, rows + pos, gap=0.0)
    first = None
    for _ in range(20):
        out.fill_(7)
        binding.check_op(lib.pfop_attention(0, q.data_ptr(), k.data_ptr(), v.data_ptr(), rows, hq, hkv, hd, pos,
                                            kv_len, out.data_ptr(), None))
        if first is None:
            first = out.clone()
            _check(heads, runs, q, k, v, out)
        assert torch.equal(out, first)
