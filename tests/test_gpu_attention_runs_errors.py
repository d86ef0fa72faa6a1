"""What attention over runs does after a call that gave up a wait: the status
call reports it, makes the scratch as good as new, and later calls in that
scratch are right on any stream.  Reference and tolerance are those of
test_gpu_attention_runs.py.

The scratch's header (include/prefill_ops.h: 4096 bytes, zero before the first
call) holds the error word first and from word 64 the flags of items cut in
two; the tests write there what a call that gave up leaves."""
import pytest

from prefill_kv_shared_gb300 import binding
from tests.gpu_util import need_gpu, torch
from tests.test_gpu_attention_runs import _check, _inputs, _layout, _random_tree

pytestmark = pytest.mark.gpu

# (rows, past): cut in two, in a few, in many, and a pair (or CTA) per item
RUNS = [([64] * 40, [900 + 7 * i for i in range(40)]), ([40] * 20, [900] * 20), ([16, 17, 1], [500, 4000, 6000]),
        ([25], [9000]), ([64], [100])]


@pytest.fixture(scope="module", autouse=True)
def lib():
    need_gpu()
    from prefill_kv_shared_gb300 import build
    build.build()
    return binding.load()


def _job(heads, rows, past, seed=83):
    runs, cells = _layout(rows, past)
    q, k, v, out = _inputs(heads, runs, cells, seed)
    mask_np = _random_tree(runs, 1, 3)
    return runs, q, k, v, out, mask_np, torch.from_numpy(mask_np.view("int64")).cuda(), binding.AttnRuns(runs, *heads)


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64)])
@pytest.mark.parametrize("rows,past", RUNS)
def test_status_makes_the_scratch_as_good_as_new(heads, rows, past):
    runs, q, k, v, out, mask_np, mask, plan = _job(heads, rows, past)
    side = torch.cuda.Stream()
    for _ in range(3):
        header = plan.work[:4096].view(torch.int32)
        header[0] = 4           # a wait given up
        header[64:64 + 960] = 1  # parts that were counted and never joined
        with pytest.raises(binding.PrefillError, match="gave up"):
            plan.check()
        with torch.cuda.stream(side):  # not ordered behind the status call's stream
            assert not plan.work[:4096].any()
            out.fill_(7)
            binding.attention_packed(q, k, v, plan, out)
        plan.check(side)
        _check(heads, runs, q, k, v, out)
        binding.attention_tree(q, k, v, plan, mask, out)
        plan.check()
        _check(heads, runs, q, k, v, out, mask_np)


# both lists hold items that are cut in two, for CTA pairs and (head_dim 64, 40
# rows) for CTAs that work alone
@pytest.mark.parametrize("heads,rows,past", [((8, 1, 256), *RUNS[0]), ((32, 4, 64), *RUNS[0]), ((32, 4, 64), *RUNS[1])])
def test_a_wait_that_runs_out(heads, rows, past):
    """Flags that never count to what the second parts wait for: their waits
    end after their bound (about 2 s), the kernel returns, the status says
    so, and the scratch is good again."""
    runs, q, k, v, out, mask_np, mask, plan = _job(heads, rows, past)
    plan.work[:4096].view(torch.int32)[64:64 + 960] = -1000
    binding.attention_packed(q, k, v, plan, out)
    with pytest.raises(binding.PrefillError, match="gave up") as e:
        plan.check()
    assert e.value.code == binding.PF_E_DEVICE_TIMEOUT
    for _ in range(2):
        out.fill_(7)
        binding.attention_packed(q, k, v, plan, out)
        plan.check()
        _check(heads, runs, q, k, v, out)
        binding.attention_tree(q, k, v, plan, mask, out)
        plan.check()
        _check(heads, runs, q, k, v, out, mask_np)


@pytest.mark.parametrize("heads", [(8, 1, 256), (8, 2, 256), (32, 4, 64)])
@pytest.mark.parametrize("rows,past", RUNS + [([128] * 30, [5000] * 30)])
def test_calls_behind_one_that_gave_up(heads, rows, past):
    """Calls that find the error word set, as those do that were enqueued
    behind a call that gave up: all roles leave at whatever wait they look at
    it in, with copies and MMAs on their way.  Their results are invalid; they
    end, the status says so, and the scratch is good again."""
    runs, q, k, v, out, mask_np, _, plan = _job(heads, rows, past)
    mask_np = _random_tree(runs, 2, 3)
    mask = torch.from_numpy(mask_np.view("int64")).cuda()
    for _ in range(3):
        plan.work[:4096].view(torch.int32)[0] = 4
        for _ in range(4):
            binding.attention_packed(q, k, v, plan, out)
            binding.attention_tree(q, k, v, plan, mask, out)
        with pytest.raises(binding.PrefillError, match="gave up"):
            plan.check()
        out.fill_(7)
        binding.attention_packed(q, k, v, plan, out)
        plan.check()
        _check(heads, runs, q, k, v, out)
        binding.attention_tree(q, k, v, plan, mask, out)
        plan.check()
    _check(heads, runs, q, k, v, out, mask_np)
