"""Attention of several sequences in one call (pfop_attention_packed,
pfop_attention_tree) against the formula in float64, one (row, head) at a
time over exactly the keys it sees.

Tolerance of an output o = sum p v / sum p, with A = sum p|v| / sum p:
  - o is rounded to bf16: half a step, 2^-8 |o|;
  - p is rounded to fp16 before P V: 2^-11 of each p, at most 2^-11 A in the
    numerator and 2^-11 |o| <= 2^-11 A where the sum takes the unrounded p;
    a p below fp16's normal range (2^-14) is off by at most 2^-25, over a sum
    of at least 1: keys * 2^-25 * max|v|;
  - a score is a sum of hd products in fp32, off by at most
    hd 2^-24 sum|q k| / sqrt(hd); with q ~ 1.5 N(0,1), k ~ N(0,1) that is
    below 256 * 2^-24 * 256 * 1.5 / 16 < 2^-11 and acts on numerator and sum,
    2 * 2^-11 A;
  - the base-2 exponential (2^-22), the scale and the fp32 sums add under
    2^-12 A.
Together 2^-8 |o| + 2^-9 (1 + 1/8) A + keys 2^-25 max|v|."""
import numpy as np
import pytest

from prefill_kv_shared_gb300 import binding
from tests.gpu_util import need_gpu, torch

pytestmark = pytest.mark.gpu

HEADS = [(8, 1, 256), (8, 2, 256), (32, 4, 64), (4, 1, 64), (4, 4, 64), (16, 1, 256), (2, 2, 256), (16, 1, 64)]


@pytest.fixture(scope="module", autouse=True)
def lib():
    need_gpu()
    from prefill_kv_shared_gb300 import build
    build.build()
    return binding.load()


def _inputs(heads, runs, n_cells, seed, extra_rows=0, gap=float("nan")):
    """q, k, v, out; cells that no run uses hold `gap`, out holds a mark."""
    hq, hkv, hd = heads
    g = torch.Generator(device="cuda").manual_seed(seed)
    total = sum(r[0] for r in runs)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    q = (1.5 * normal(total + extra_rows, hq, hd)).half()
    k, v = normal(n_cells, hkv, hd).half(), normal(n_cells, hkv, hd).half()
    used = torch.zeros(n_cells, dtype=torch.bool, device="cuda")
    for n, pos0, cell0 in runs:
        if n:
            used[cell0:cell0 + pos0 + n] = True
    k[~used] = gap
    v[~used] = gap
    out = torch.full((total + extra_rows, hq, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    return q, k, v, out


def _chain(runs, words):
    """Masks that make a tree call causal: row i sees drafted tokens 0 .. i."""
    rows = []
    for n, _, _ in runs:
        for i in range(n):
            bits = (1 << (i + 1)) - 1
            rows.append([(bits >> (64 * w)) & (2**64 - 1) for w in range(words)])
    return np.array(rows, dtype=np.uint64).reshape(-1, words)


def _check(heads, runs, q, k, v, out, mask=None):
    hq, hkv, hd = heads
    row0 = 0
    for n, pos0, cell0 in runs:
        if n == 0:
            continue
        keys = pos0 + n
        kk = k[cell0:cell0 + keys].double().repeat_interleave(hq // hkv, 1)
        vv = v[cell0:cell0 + keys].double().repeat_interleave(hq // hkv, 1)
        for t0 in range(0, n, 512):
            t1 = min(n, t0 + 512)
            s = torch.einsum("thd,khd->thk", q[row0 + t0:row0 + t1].double(), kk) / hd ** 0.5
            if mask is None:
                vis = torch.arange(keys)[None, :] <= pos0 + torch.arange(t0, t1)[:, None]
            else:
                vis = torch.ones(t1 - t0, keys, dtype=torch.bool)
                for i in range(t0, t1):
                    w = [int(x) for x in mask[row0 + i]]
                    for j in range(n):
                        vis[i - t0, pos0 + j] = bool(w[j // 64] >> (j % 64) & 1)
            s = s.masked_fill(~vis.to(s.device)[:, None, :], float("-inf"))
            p = torch.nan_to_num(torch.softmax(s, -1))
            want = torch.einsum("thk,khd->thd", p, vv)
            a = torch.einsum("thk,khd->thd", p, vv.abs())
            tol = 2 ** -8 * want.abs() + 2 ** -9 * 1.125 * a + keys * 2 ** -25 * vv.abs().max()
            got = out[row0 + t0:row0 + t1].double()
            assert torch.isfinite(got).all()
            over = ((got - want).abs() / tol.clamp(min=1e-30))
            over[(got == want)] = 0
            assert over.max() <= 1, f"run {(n, pos0, cell0)} rows {t0}..: {float(over.max())} of the tolerance"
        row0 += n


def _packed(heads, runs, q, k, v, out, **kw):
    plan = binding.AttnRuns(runs, *heads)
    binding.attention_packed(q, k, v, plan, out, **kw)
    plan.check()
    return plan


def _tree(heads, runs, q, k, v, mask, out):
    plan = binding.AttnRuns(runs, *heads)
    binding.attention_tree(q, k, v, plan, torch.from_numpy(mask.view(np.int64)).cuda(), out)
    plan.check()
    return plan


def _layout(rows, past, gap=3):
    runs, c = [], gap
    for n, p in zip(rows, past):
        runs.append((n, p, c))
        c += n + p + gap
    return runs, c


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("rows,past", [
    ([1], [0]), ([1], [127]), ([1], [128]), ([25], [0]), ([129], [0]),
    ([0, 1, 0, 5, 0], [9, 0, 0, 130, 0]),
    ([127, 128, 1, 2, 63], [0, 0, 255, 256, 1]),
    ([257, 31, 16, 300], [100, 1000, 0, 0]),
])
def test_packed(heads, rows, past):
    runs, cells = _layout(rows, past)
    q, k, v, out = _inputs(heads, runs, cells, len(rows) + sum(past), extra_rows=5)
    _packed(heads, runs, q, k, v, out)
    _check(heads, runs, q, k, v, out)
    assert (out[sum(rows):] == 7).all()


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64)])
def test_packed_long_keys(heads):
    runs, cells = _layout([3, 40, 600], [5000, 2049, 1500])
    q, k, v, out = _inputs(heads, runs, cells, 5)
    _packed(heads, runs, q, k, v, out)
    _check(heads, runs, q, k, v, out)


@pytest.mark.parametrize("heads", [(8, 2, 256), (32, 4, 64)])
def test_packed_long_prompts(heads):
    """More row blocks than fit the GPU at once."""
    runs, cells = _layout([2500, 1, 1800, 1023], [0, 0, 200, 0])
    q, k, v, out = _inputs(heads, runs, cells, 6)
    _packed(heads, runs, q, k, v, out)
    _check(heads, runs, q, k, v, out)


@pytest.mark.parametrize("heads", [(8, 1, 256), (4, 1, 64)])
def test_packed_128_runs_in_any_order(heads):
    rng = np.random.default_rng(3)
    rows = rng.integers(0, 20, 128).tolist()
    past = rng.integers(0, 300, 128).tolist()
    runs, cells = _layout(rows, past)
    # the sequences' cells in another order than their rows
    order = rng.permutation(128)
    runs = [(rows[i], past[i], runs[j][2]) if rows[i] + past[i] <= runs[j][0] + runs[j][1] else (0, 0, 0)
            for i, j in enumerate(order)]
    q, k, v, out = _inputs(heads, runs, cells, 7)
    _packed(heads, runs, q, k, v, out)
    _check(heads, runs, q, k, v, out)


def _random_tree(runs, words, seed, forest=True):
    rng = np.random.default_rng(seed)
    rows = []
    for n, _, _ in runs:
        bits = []
        for j in range(n):
            p = int(rng.integers(-1 if forest else 0, j)) if j else -1
            bits.append((bits[p] if p >= 0 else 0) | (1 << j))
        rows += [[(b >> (64 * w)) & (2**64 - 1) for w in range(words)] for b in bits]
    return np.array(rows, dtype=np.uint64).reshape(-1, words)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("rows,past,words", [
    ([1], [0], 1), ([1], [63], 1), ([5], [532], 1), ([64], [100], 1), ([16, 1, 33, 8], [127, 128, 129, 0], 1),
    ([65, 0, 128], [62, 5, 300], 2), ([256, 200, 1], [1, 190, 64], 4),
])
def test_tree(heads, rows, past, words):
    runs, cells = _layout(rows, past)
    q, k, v, out = _inputs(heads, runs, cells, 11 + sum(rows), extra_rows=2)
    mask = _random_tree(runs, words, 1)
    padded = np.concatenate([mask, np.zeros((2, words), np.uint64)])
    _tree(heads, runs, q, k, v, padded, out)
    _check(heads, runs, q, k, v, out, mask)
    assert (out[sum(rows):] == 7).all()


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64)])
def test_tree_long_contexts(heads):
    runs, cells = _layout([25, 3, 64, 1], [9000, 4097, 700, 2047])
    q, k, v, out = _inputs(heads, runs, cells, 13)
    mask = _random_tree(runs, 1, 2)
    _tree(heads, runs, q, k, v, mask, out)
    _check(heads, runs, q, k, v, out, mask)


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64)])
def test_tree_masks_that_leave_nothing(heads):
    """Rows without any key give zeros; any bits are taken as they are (a row
    that does not see itself, one that sees a later token)."""
    runs, cells = _layout([40, 70, 3], [0, 0, 64])
    q, k, v, out = _inputs(heads, runs, cells, 17)
    rng = np.random.default_rng(5)
    mask = rng.integers(0, 2**63, (113, 2), dtype=np.uint64)
    mask[0] = 0
    mask[17] = 0
    mask[110] = 0            # sees its context only
    mask[3] = [1 << 39, 0]   # a later token only
    mask[50] = [0, 1 << 5]   # token 69 of the second run only
    _tree(heads, runs, q, k, v, mask, out)
    want = mask.copy()
    want[:40, 0] &= np.uint64((1 << 40) - 1)
    want[:40, 1] = 0
    _check(heads, runs, q, k, v, out, mask)
    assert (out[0] == 0).all() and (out[17] == 0).all()
    again = torch.zeros_like(out)
    _tree(heads, runs, q, k, v, want, again)  # the bits past n_rows change nothing
    assert torch.equal(out[:40], again[:40])


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64)])
def test_tree_of_chains_is_causal(heads):
    runs, cells = _layout([64, 10, 1], [200, 3000, 77])
    q, k, v, out = _inputs(heads, runs, cells, 19)
    _tree(heads, runs, q, k, v, _chain(runs, 1), out)
    _check(heads, runs, q, k, v, out)


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64)])
def test_peaky_and_growing_scores(heads):
    """Scores whose running maximum grows from chunk to chunk by more than the
    exponent range of one fp16 probability, and rows with one dominant key.
    Keys and values are chosen so that the formula's answer is near-exact: the
    score tolerance of the module's derivation scales with |q k|, so |q| is
    kept small here and the growth comes from the keys."""
    runs, cells = _layout([70, 5], [700, 1300])
    q, k, v, out = _inputs(heads, runs, cells, 23)
    hd = heads[2]
    ramp = torch.zeros(cells, device="cuda")
    for n, p, c in runs:
        ramp[c:c + p + n] = torch.arange(p + n, device="cuda") / 32.0
    q.zero_()
    q[:, :, 0] = 1.0
    k.zero_()
    k[:, :, 0] = ramp[:, None].half()     # scores j / 32 / sqrt(hd): exact steps of the fp16 ramp
    if hd == 256:
        k[:, :, 0] *= 4
    _packed(heads, runs, q, k, v, out)
    _check(heads, runs, q, k, v, out)
    k[:, :, 0] = -k[:, :, 0]              # falling: the first key stays the maximum
    _packed(heads, runs, q, k, v, out)
    _check(heads, runs, q, k, v, out)


@pytest.mark.parametrize("tree", [False, True])
def test_repeats_and_other_runs_values(tree):
    """The same bits on a repeat, and whatever the other runs hold."""
    heads = (8, 2, 256)
    runs, cells = _layout([40, 64, 7], [900, 2000, 100])
    q, k, v, out = _inputs(heads, runs, cells, 29)
    plan = binding.AttnRuns(runs, *heads)
    mask = torch.from_numpy(_random_tree(runs, 1, 3).view(np.int64)).cuda()

    def go(o):
        if tree:
            binding.attention_tree(q, k, v, plan, mask, o)
        else:
            binding.attention_packed(q, k, v, plan, o)
        plan.check()

    go(out)
    for _ in range(3):
        again = torch.zeros_like(out)
        go(again)
        assert torch.equal(out, again)
    n, p, c = runs[1]
    k[c:c + p + n] = 1.0
    v[c:c + p + n] = -2.0
    q[40:104] = 0.5
    again = torch.zeros_like(out)
    go(again)
    assert torch.equal(out[:40], again[:40]) and torch.equal(out[104:], again[104:])


def test_offsets_past_32_bits():
    """A cache whose elements (and bytes) pass 2^31 and 2^32."""
    heads = (8, 2, 256)
    cells = 4_400_000
    k = torch.empty(cells, 2, 256, dtype=torch.float16, device="cuda")
    v = torch.empty(cells, 2, 256, dtype=torch.float16, device="cuda")
    runs = [(30, 500, cells - 530), (5, 3, 0), (64, 90, cells // 2)]
    g = torch.Generator(device="cuda").manual_seed(31)
    for n, p, c in runs:
        k[c:c + p + n] = torch.randn(p + n, 2, 256, generator=g, device="cuda").half()
        v[c:c + p + n] = torch.randn(p + n, 2, 256, generator=g, device="cuda").half()
    q = (1.5 * torch.randn(99, 8, 256, generator=g, device="cuda")).half()
    out = torch.zeros(99, 8, 256, dtype=torch.bfloat16, device="cuda")
    _packed(heads, runs, q, k, v, out)
    _check(heads, runs, q, k, v, out)
    mask = _random_tree(runs, 1, 4)
    _tree(heads, runs, q, k, v, mask, out)
    _check(heads, runs, q, k, v, out, mask)


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64)])
def test_recorded_and_replayed(heads):
    """Both calls in one graph, replayed on new values."""
    runs, cells = _layout([50, 9], [800, 40])
    q, k, v, out = _inputs(heads, runs, cells, 37)
    out2 = torch.zeros_like(out)
    plan = binding.AttnRuns(runs, *heads)
    mask_np = _random_tree(runs, 1, 5)
    mask = torch.from_numpy(mask_np.view(np.int64)).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        binding.attention_packed(q, k, v, plan, out)
        binding.attention_tree(q, k, v, plan, mask, out2)
    for seed in (41, 43):
        q2, k2, v2, _ = _inputs(heads, runs, cells, seed)
        q.copy_(q2), k.copy_(k2), v.copy_(v2)
        graph.replay()
        torch.cuda.synchronize()
        plan.check()
        _check(heads, runs, q, k, v, out)
        _check(heads, runs, q, k, v, out2, mask_np)


def test_two_streams_at_once():
    """Two calls with a scratch each, overlapping on two streams, inputs made
    on those streams."""
    heads = (8, 1, 256)
    jobs = []
    for i in range(2):
        runs, cells = _layout([64 + i, 9], [3000, 500 * i])
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            q, k, v, out = _inputs(heads, runs, cells, 47 + i)
            plan = binding.AttnRuns(runs, *heads)
        jobs.append((s, runs, q, k, v, out, plan))
    for _ in range(4):
        for s, runs, q, k, v, out, plan in jobs:
            with torch.cuda.stream(s):
                binding.attention_packed(q, k, v, plan, out)
    torch.cuda.synchronize()
    for s, runs, q, k, v, out, plan in jobs:
        plan.check(s)
        _check(heads, runs, q, k, v, out)


@pytest.mark.parametrize("rows,past", [
    ([16], [130]), ([17], [130]), ([16], [20000]), ([1], [30000]), ([16] * 5, [3000, 10, 700, 0, 9000]),
    ([16, 17, 1], [500, 4000, 6000]), ([1] * 100, [37 * i for i in range(100)]),
    ([4, 0, 12, 1] * 10, [100 + 150 * i for i in range(40)]),
])
def test_few_rows_a_run(rows, past):
    """Up to 128 MMA rows a run and more, whole, cut in two and cut in many;
    a tree's and a prompt's masks."""
    heads = (32, 4, 64)
    runs, cells = _layout(rows, past)
    q, k, v, out = _inputs(heads, runs, cells, 67)
    plan = _packed(heads, runs, q, k, v, out)
    _check(heads, runs, q, k, v, out)
    mask_np = _random_tree(runs, 1, 3)
    out.fill_(7)
    binding.attention_tree(q, k, v, plan, torch.from_numpy(mask_np.view(np.int64)).cuda(), out)
    plan.check()
    _check(heads, runs, q, k, v, out, mask_np)


@pytest.mark.parametrize("rows,past", [
    ([700, 33, 900], [0, 2000, 50]), ([40] * 20, [10] * 20), ([40] * 20 + [33], [10] * 20 + [40000]),
    ([160, 17] * 12, [1000, 0] * 12),
])
def test_many_rows_at_head_dim_64(rows, past):
    """Items of up to 256 MMA rows, more of them than SMs, whole, cut in two
    and in many, and recorded; the tree's masks where its rows allow them."""
    heads = (32, 4, 64)
    runs, cells = _layout(rows, past)
    q, k, v, out = _inputs(heads, runs, cells, 71)
    plan = _packed(heads, runs, q, k, v, out)
    _check(heads, runs, q, k, v, out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        binding.attention_packed(q, k, v, plan, out)
    first = out.clone()
    out.fill_(7)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    plan.check()
    assert torch.equal(out, first)
    if max(rows) > 256:
        return
    mask_np = _random_tree(runs, 3, 3)
    binding.attention_tree(q, k, v, plan, torch.from_numpy(mask_np.view(np.int64)).cuda(), out)
    plan.check()
    _check(heads, runs, q, k, v, out, mask_np)


@pytest.mark.parametrize("heads", [(1024, 64, 64), (1024, 1024, 64), (64, 64, 256), (256, 16, 256)])
def test_many_heads(heads):
    runs, cells = _layout([3, 20, 1], [40, 0, 300])
    q, k, v, out = _inputs(heads, runs, cells, 79)
    plan = _packed(heads, runs, q, k, v, out)
    _check(heads, runs, q, k, v, out)
    mask_np = _random_tree(runs, 1, 7)
    binding.attention_tree(q, k, v, plan, torch.from_numpy(mask_np.view(np.int64)).cuda(), out)
    plan.check()
    _check(heads, runs, q, k, v, out, mask_np)


@pytest.mark.parametrize("heads", [(8, 2, 256), (32, 4, 64)])
def test_runs_that_share_cells(heads):
    """Several sequences over the same prefix, and one over another's cells."""
    runs = [(5, 300, 0), (9, 300, 0), (1, 0, 0), (40, 100, 37), (1, 308, 0)]
    q, k, v, out = _inputs(heads, runs, 320, 73)
    _packed(heads, runs, q, k, v, out)
    _check(heads, runs, q, k, v, out)


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64)])
def test_runs_made_on_one_stream_used_on_another(heads):
    """A scratch that is made behind long work of one stream, in memory that
    held other values, is ready for a call on another stream."""
    runs, cells = _layout([40, 300, 7], [2500, 100, 9000])
    q, k, v, out = _inputs(heads, runs, cells, 59)
    marked = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del marked  # the next allocations get its memory
    torch.cuda._sleep(20_000_000)
    plan = binding.AttnRuns(runs, *heads)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        binding.attention_packed(q, k, v, plan, out)
    plan.check(side)
    _check(heads, runs, q, k, v, out)


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64)])
def test_one_scratch_for_changing_runs(heads):
    """Calls one after another in one scratch, their items whole, cut in two
    and cut in many."""
    sizes = [([3, 3], [10, 20]), ([70, 90, 33, 200], [1500, 800, 3000, 0]), ([20], [20000]),
             ([64, 1, 128], [600, 6000, 0])]
    jobs = []
    for i, (rows, past) in enumerate(sizes):
        runs, cells = _layout(rows, past)
        q, k, v, out = _inputs(heads, runs, cells, 61 + i)
        mask_np = _random_tree(runs, 4, i)
        jobs.append((runs, q, k, v, out, out.clone(), binding.AttnRuns(runs, *heads), mask_np,
                     torch.from_numpy(mask_np.view(np.int64)).cuda()))
    big = max((j[6] for j in jobs), key=lambda p: p.work_bytes)
    for _ in range(3):
        for runs, q, k, v, out, out2, plan, _, mask in jobs:
            plan.work, plan.work_at, plan.work_bytes = big.work, big.work_at, big.work_bytes
            binding.attention_packed(q, k, v, plan, out)
            binding.attention_tree(q, k, v, plan, mask, out2)
    big.check()
    for runs, q, k, v, out, out2, _, mask_np, _ in jobs:
        _check(heads, runs, q, k, v, out)
        _check(heads, runs, q, k, v, out2, mask_np)


def test_wrappers_refuse_what_does_not_fit():
    heads = (8, 2, 64)
    runs = [(4, 10, 0)]
    q, k, v, out = _inputs(heads, runs, 20, 53)
    plan = binding.AttnRuns(runs, *heads)
    mask = torch.zeros(4, 1, dtype=torch.int64, device="cuda")
    for bad in (dict(q=q.float()), dict(q=q[:3].contiguous()), dict(k=k[:, :1]), dict(k=k.cpu()), dict(v=v[:19]),
                dict(out=out.half()), dict(out=out[:3]), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(q=q[:, 0]), dict(out=out.flatten()), dict(k=k[0, 0, 0]), dict(v=v[:, :, :32].contiguous())):
        a = dict(q=q, k=k, v=v, out=out)
        a.update(bad)
        with pytest.raises(ValueError):
            binding.attention_packed(a["q"], a["k"], a["v"], plan, a["out"])
    for bad in (mask[:3], mask.int(), mask[:, 0], mask.cpu(), mask.repeat(1, 2)[:, :1]):
        with pytest.raises(ValueError):
            binding.attention_tree(q, k, v, plan, bad, out)
    with pytest.raises(binding.PrefillError):  # a run past the cache
        binding.attention_packed(q, k[:13], v[:13], plan, out)
    with pytest.raises(binding.PrefillError):
        binding.AttnRuns([(4, -1, 0)], *heads)
