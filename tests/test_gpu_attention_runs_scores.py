"""Attention over runs where scores decide how the sums are kept: running
maxima that climb, chunk after chunk, by more than the 2^8 that the kernels
let a probability exceed 1 before they rescale what has been summed.

A row's query is f e_0 with f of (1, 0, -1, 1/2) by row and head, so that in a
warp some rows climb, some stay and some fall; key j of a sequence has j a in
dim 0, with a such that a step of one key is a log2(e) / sqrt(hd) = 0.09 in
the exponent: 11.5 a chunk of 128 keys (f = 1) and 5.8 (f = 1/2, which climbs
past 2^8 every second chunk).  Scores are products of two fp16 numbers, exact in
fp32; the exponent m c of up to 2800 is rounded to fp32, off by at most 2^-13,
the same for all of a segment's keys.  That adds 2^-13 ln 2 < 2^-13 of A where
segments are joined, twice, within the 2^-12 A that the module whose reference
and tolerance are used here (test_gpu_attention_runs.py) leaves for the scale
and the sums: scores there are rounded, here they are exact, which leaves
2^-10 A more."""
import pytest

from prefill_kv_shared_gb300 import binding
from tests.gpu_util import need_gpu, torch
from tests.test_gpu_attention_runs import _check, _inputs, _layout, _packed, _random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    need_gpu()
    from prefill_kv_shared_gb300 import build
    build.build()
    return binding.load()


# items of 8 or more chunks: one segment each, cut in two, cut in three or
# more; for CTA pairs and (head_dim 64, the first three) CTAs that work alone
CUTS = [
    ((8, 1, 256), [40] * 20, [900] * 20),
    ((8, 1, 256), [64] * 40, [900 + 7 * i for i in range(40)]),
    ((8, 1, 256), [64] * 12, [2000 + 200 * i for i in range(12)]),
    ((8, 2, 256), [64] * 40, [900 + 7 * i for i in range(40)]),
    ((32, 4, 64), [16] * 30, [900] * 30),
    ((32, 4, 64), [40] * 20, [900] * 20),
    ((32, 4, 64), [16] * 8, [4000] * 8),
    ((32, 4, 64), [64] * 40, [900 + 7 * i for i in range(40)]),
    ((32, 4, 64), [64] * 20, [1000] * 19 + [30000]),
]


def _climbing(heads, runs, q, k):
    hq, _, hd = heads
    q.zero_()
    row = torch.arange(q.shape[0], device="cuda")[:, None]
    f = torch.tensor([1.0, 0.0, -1.0, 0.5], device="cuda")
    q[:, :, 0] = f[(3 * row + torch.arange(hq, device="cuda")) % 4].half()
    for n, p, c in runs:
        k[c:c + p + n, :, 0] = (torch.arange(p + n, device="cuda") * (1.0 if hd == 256 else 0.5)).half()[:, None]


@pytest.mark.parametrize("heads,rows,past", CUTS)
def test_climbing_scores(heads, rows, past):
    runs, cells = _layout(rows, past)
    q, k, v, out = _inputs(heads, runs, cells, 89)
    _climbing(heads, runs, q, k)
    plan = _packed(heads, runs, q, k, v, out)
    _check(heads, runs, q, k, v, out)
    mask_np = _random_tree(runs, 1, 5)
    out.fill_(7)
    binding.attention_tree(q, k, v, plan, torch.from_numpy(mask_np.view("int64")).cuda(), out)
    plan.check()
    _check(heads, runs, q, k, v, out, mask_np)
