"""Attention over runs with scores as large as fp16 queries and keys allow:
2^35 and more in the exponent, where the product of the running maximum and
log2(e) / sqrt(hd), rounded to fp32, is off by hundreds.  The probabilities are
still those of the differences to the maximum.

All queries are f 24576 with f = 1 or -1 by row and head, all keys 24576 but
for what a case changes, in steps of 16 (fp16's there).  A score is then a sum
of multiples of 2^14 below 2^38, exact in fp32 in any order.  Reference and
tolerance are those of test_gpu_attention_runs.py."""
import pytest

from prefill_kv_shared_gb300 import binding
from tests.gpu_util import need_gpu, torch
from tests.test_gpu_attention_runs import _check, _inputs, _layout, _packed, _random_tree
from tests.test_gpu_attention_runs_scores import CUTS

pytestmark = pytest.mark.gpu

BIG = 24576.0


@pytest.fixture(scope="module", autouse=True)
def lib():
    need_gpu()
    from prefill_kv_shared_gb300 import build
    build.build()
    return binding.load()


@pytest.mark.parametrize("kind", ["equal", "one higher", "climbing"])
@pytest.mark.parametrize("heads,rows,past", CUTS[:-1] + [((4, 1, 64), [1], [0]), ((8, 1, 256), [70], [0])])
def test_large_scores(heads, rows, past, kind):
    runs, cells = _layout(rows, past)
    q, k, v, out = _inputs(heads, runs, cells, 91)
    row = torch.arange(q.shape[0], device="cuda")[:, None]
    f = 1 - 2 * ((row + torch.arange(heads[0], device="cuda")) % 2)
    q[:] = (BIG * f).half()[:, :, None]
    for n, p, c in runs:
        k[c:c + p + n] = BIG
        if kind == "one higher":   # 2^14 24 above the others: a row with f = 1 takes it alone, one with -1 all others
            k[c + (p + n) // 2, :, 0] += 16
        elif kind == "climbing":   # a step every 50 keys
            k[c:c + p + n, :, 0] += (16 * (torch.arange(p + n, device="cuda") // 50)).half()[:, None]
    plan = _packed(heads, runs, q, k, v, out)
    _check(heads, runs, q, k, v, out)
    mask_np = _random_tree(runs, 2, 5)
    out.fill_(7)
    binding.attention_tree(q, k, v, plan, torch.from_numpy(mask_np.view("int64")).cuda(), out)
    plan.check()
    _check(heads, runs, q, k, v, out, mask_np)
