"""Attention over pages and over cells where queries or keys are no numbers:
they reach the rows that they belong to, or that see them, and no others, however
the call is cut.  And rows that see no key at all."""
import numpy as np
import pytest

from prefill_kv_shared_gb300 import binding
from tests.gpu_util import need_gpu, torch
from tests.test_gpu_attention_paged import Paged
from tests.test_gpu_attention_runs import _random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    need_gpu()
    from prefill_kv_shared_gb300 import build
    build.build()
    return binding.load()


# whole items, items cut in two and in many, on the kernel of few rows and on the chunks'
CALLS = [([1, 1, 1], [40, 700, 3]), ([1], [20000]), ([1] * 40, [1500] * 40), ([2, 1], [9000, 16]), ([70, 90], [1500, 800]),
         ([25], [30000]), ([20, 5], [100, 6000]), ([300], [0])]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("heads", [(8, 1, 256), (8, 2, 256), (32, 4, 64), (4, 4, 64)])
@pytest.mark.parametrize("rows,past", CALLS)
def test_queries_that_are_no_numbers(heads, rows, past, bad):
    """They make their own row and head NaN, and touch no other."""
    c = Paged(heads, 16, rows, past, 101)
    c.go()
    first = c.out.clone()
    row, head = c.total - 1, heads[0] // 2
    # NaN, or infinite in two dims where the keys have both signs: every score is NaN, or one infinity is
    c.q[row, head, 3], c.q[row, head, heads[2] - 1] = bad, bad
    c.go()
    c.plan.check()
    assert torch.isnan(c.out[row, head]).all()
    c.out[row, head] = first[row, head]
    assert torch.equal(c.out, first)


@pytest.mark.parametrize("heads", [(8, 1, 256), (8, 2, 256), (32, 4, 64), (4, 4, 64)])
@pytest.mark.parametrize("rows,past", CALLS)
@pytest.mark.parametrize("part", ["key", "all keys"])
def test_keys_that_are_no_numbers(heads, rows, past, part):
    """The rows of their run and KV head that see them are NaN, all others as they were."""
    c = Paged(heads, 16, rows, past, 103)
    c.go()
    first = c.out.clone()
    hq, hkv, hd = heads
    cells = c.cells(0)
    n, p, _ = c.runs[0]
    # the run's last token's key, which only its last row sees; or every key of the run
    at = cells[-1:] if part == "key" else cells
    c.k.view(-1, hkv, hd)[at, hkv - 1, 5] = float("nan")
    c.go()
    c.plan.check()
    seen = c.out[n - 1:n] if part == "key" else c.out[:n]
    g = hq // hkv
    assert torch.isnan(seen[:, hq - g:]).all()
    seen[:, hq - g:] = (first[n - 1:n] if part == "key" else first[:n])[:, hq - g:]
    assert torch.equal(c.out, first)


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64)])
@pytest.mark.parametrize("rows,past", [([25], [30000]), ([20, 5], [100, 6000]), ([300], [0]), ([1, 70], [5000, 900])])
def test_queries_that_are_no_numbers_over_cells(heads, rows, past):
    """The same over a contiguous cache, causal and as a tree."""
    hq, hkv, hd = heads
    g = torch.Generator(device="cuda").manual_seed(107)
    runs, at = [], 0
    for n, p in zip(rows, past):
        runs.append((n, p, at))
        at += n + p
    total = sum(rows)
    q = (1.5 * torch.randn(total, hq, hd, generator=g, device="cuda")).half()
    k, v = (torch.randn(at, hkv, hd, generator=g, device="cuda").half() for _ in range(2))
    plan = binding.AttnRuns(runs, *heads)
    mask = None
    for tree in (False, True):
        if tree and max(rows) > 256:
            continue
        if tree:
            mask = torch.from_numpy(_random_tree(runs, 2, 3).view(np.int64)).cuda()
        out = torch.empty(total, hq, hd, dtype=torch.bfloat16, device="cuda")

        def go():
            if tree:
                binding.attention_tree(q, k, v, plan, mask, out)
            else:
                binding.attention_packed(q, k, v, plan, out)
            plan.check()
            return out.clone()

        first, kept = go(), q.clone()
        q[total - 2, 1, 9] = float("nan")
        got = go()
        q.copy_(kept)
        assert torch.isnan(got[total - 2, 1]).all()
        got[total - 2, 1] = first[total - 2, 1]
        assert torch.equal(got, first)


@pytest.mark.parametrize("heads", [(8, 1, 256), (8, 2, 256), (32, 4, 64), (4, 4, 64)])
@pytest.mark.parametrize("words", [1, 3])
@pytest.mark.parametrize("rows,past", [([1, 2, 1, 1], [0, 0, 7, 0]), ([1, 1, 2], [0, 40000, 0]), ([1] * 100, [0, 700] * 50)])
def test_masks_that_leave_nothing_in_calls_of_few_rows(heads, words, rows, past):
    """Rows without any key give zeros on the kernel of few rows too, in
    items of their own and between parts of others; every second one sees
    itself."""
    c = Paged(heads, 16, rows, past, 109)
    mask = np.zeros((c.total, words), np.uint64)
    row, empty = 0, []
    for i, (n, p) in enumerate(zip(rows, past)):
        for t in range(n):
            if i % 4 == 3:
                mask[row, 0] = 1 << t
            elif p == 0:
                empty.append(row)
            row += 1
    c.go(np.concatenate([mask, np.zeros((3, words), np.uint64)]))
    c.plan.check()
    c.check(mask)
    assert empty and (c.out[empty] == 0).all()
