"""Attention over a paged cache (pfop_attention_paged) against the formula in
float64 over exactly the keys each row sees.  Tolerances as derived in
test_gpu_attention_runs (whose check is used on the sequences' pages, laid end
to end): the same roundings are made here."""
import numpy as np
import pytest

from prefill_kv_shared_gb300 import binding
from tests.gpu_util import need_gpu, torch
from tests.test_gpu_attention_runs import HEADS, _check, _random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    need_gpu()
    from prefill_kv_shared_gb300 import build
    build.build()
    return binding.load()


class Paged:
    """Sequences of `rows` new tokens behind `past` cached ones in pages that
    lie anywhere; unused pages and the rest of last pages hold `gap`, table
    entries behind a sequence's pages are no page ids."""

    def __init__(self, heads, page, rows, past, seed, gap=float("nan"), extra_rows=3):
        hq, hkv, hd = self.heads = heads
        self.page = page
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        need = [-(-(n + p) // page) if n else 0 for n, p in zip(rows, past)]
        width = max(need) + 1
        n_pages = sum(need) + 4
        ids = rng.permutation(n_pages)
        table = np.full((len(rows), width), -7, np.int32)
        at = 0
        for r, n in enumerate(need):
            table[r, :n] = ids[at:at + n]
            at += n
        self.table = torch.from_numpy(table).cuda()
        self.runs = [(n, p, r * width) for r, (n, p) in enumerate(zip(rows, past))]
        self.total = sum(rows)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        self.q = (1.5 * normal(self.total + extra_rows, hq, hd)).half()
        self.k = torch.full((n_pages, page, hkv, hd), gap, dtype=torch.float16, device="cuda")
        self.v = self.k.clone()
        self.fill(normal)
        self.out = torch.full((self.total + extra_rows, hq, hd), 7.0, dtype=torch.bfloat16, device="cuda")
        self.plan = binding.AttnRuns(self.runs, *heads)

    def cells(self, r):
        """Flat cells of sequence r's positions."""
        n, p, e = self.runs[r]
        pos = torch.arange(n + p, device="cuda")
        pages = self.table.flatten()[e + pos // self.page].long()
        return pages * self.page + pos % self.page

    def fill(self, normal):
        hkv, hd = self.k.shape[2:]
        for r, (n, p, _) in enumerate(self.runs):
            if n:
                c = self.cells(r)
                self.k.view(-1, hkv, hd)[c] = normal(n + p, hkv, hd).half()
                self.v.view(-1, hkv, hd)[c] = normal(n + p, hkv, hd).half()

    def go(self, mask=None, **kw):
        m = None if mask is None else torch.from_numpy(mask.view(np.int64)).cuda()
        binding.attention_paged(self.q, self.k, self.v, self.plan, self.table, self.out, mask=m, **kw)

    def check(self, mask=None):
        hkv, hd = self.k.shape[2:]
        ks, vs, runs, at = [], [], [], 0
        for r, (n, p, _) in enumerate(self.runs):
            runs.append((n, p, at))
            if n:
                c = self.cells(r)
                ks.append(self.k.view(-1, hkv, hd)[c])
                vs.append(self.v.view(-1, hkv, hd)[c])
                at += n + p
        _check(self.heads, runs, self.q, torch.cat(ks), torch.cat(vs), self.out, mask)
        assert (self.out[self.total:] == 7).all()


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("page", [8, 16, 64, 128, 512])
@pytest.mark.parametrize("rows,past", [
    ([1], [0]), ([1], [15]), ([1, 1, 1], [127, 128, 129]), ([25], [0]), ([0, 1, 0, 5, 0], [9, 0, 0, 130, 0]),
    ([127, 128, 1, 2, 63], [0, 0, 255, 256, 1]), ([257, 31, 16, 300], [100, 1000, 0, 0]),
])
def test_causal(heads, page, rows, past):
    c = Paged(heads, page, rows, past, 1 + sum(past) + page)
    c.go()
    c.plan.check()
    c.check()


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("page", [8, 32, 256])
@pytest.mark.parametrize("rows,past", [
    ([1], [40000]), ([1, 1], [5000, 3]), ([1] * 128, [37 * i for i in range(128)]), ([1] * 20, [4096] * 20),
    ([2] * 30, [129 * i for i in range(30)]), ([5, 1, 9], [3000, 8191, 20000]),
])
def test_few_rows_over_long_contexts(heads, page, rows, past):
    c = Paged(heads, page, rows, past, 2 + page)
    c.go()
    c.plan.check()
    c.check()


@pytest.mark.parametrize("heads", HEADS)
def test_a_single_token_at_every_length(heads):
    """1 to 128 keys in one call, then 129 to 512 four at a time."""
    c = Paged(heads, 16, [1] * 128, list(range(128)), 3)
    c.go()
    c.plan.check()
    c.check()
    c = Paged(heads, 8, [1] * 96, list(range(128, 512, 4)), 4)
    c.go()
    c.plan.check()
    c.check()


@pytest.mark.parametrize("heads", [(8, 2, 256), (32, 4, 64), (8, 1, 256), (16, 16, 64)])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("rows,past,words", [
    ([1], [63], 1), ([5], [532], 1), ([16, 1, 33, 8], [127, 128, 129, 0], 1), ([65, 0, 128], [62, 5, 300], 2),
    ([256, 200, 1], [1, 190, 64], 4), ([25, 3, 64, 1], [9000, 4097, 700, 2047], 1), ([1] * 40, [500] * 40, 1),
])
def test_trees(heads, page, rows, past, words):
    c = Paged(heads, page, rows, past, 5 + sum(rows))
    mask = _random_tree(c.runs, words, 1)
    c.go(np.concatenate([mask, np.zeros((3, words), np.uint64)]))
    c.plan.check()
    c.check(mask)


@pytest.mark.parametrize("heads,rows", [((8, 1, 256), 2), ((8, 2, 256), 4), ((8, 2, 256), 3), ((16, 1, 256), 1),
                                        ((16, 16, 256), 16), ((32, 4, 64), 2), ((4, 4, 64), 16), ((16, 1, 64), 1),
                                        ((32, 4, 64), 3), ((4, 1, 64), 6), ((4, 2, 64), 11), ((32, 4, 64), 5)])
@pytest.mark.parametrize("page", [8, 64])
def test_up_to_24_columns_over_much_work(heads, rows, page):
    """Runs of up to 24 (row, head) pairs a KV head (and of 40), as many keys as a large
    batch has: causal, and each row with its own mask."""
    n = 70 if heads[1] < 16 else 6
    c = Paged(heads, page, [rows] * n, [1100 + 37 * i for i in range(n)], 83 + rows)
    c.go()
    c.plan.check()
    c.check()
    mask = _random_tree(c.runs, 1, 3)
    c.out[:c.total] = 7
    c.go(np.concatenate([mask, np.zeros((3, 1), np.uint64)]))
    c.plan.check()
    c.check(mask)


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64), (4, 4, 64)])
def test_masks_that_leave_nothing(heads):
    """Rows without any key give zeros, single tokens among them."""
    c = Paged(heads, 16, [1, 40, 1, 3, 1], [0, 0, 7, 64, 0], 17)
    mask = np.random.default_rng(5).integers(0, 2**63, (46, 1), dtype=np.uint64)
    mask[0] = 0       # nothing
    mask[1] = 0       # nothing
    mask[41] = 0      # its context only
    mask[45] = 1      # itself only
    c.go(mask)
    c.plan.check()
    c.check(mask)
    assert (c.out[0] == 0).all() and (c.out[1] == 0).all()


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64)])
def test_mixed_step(heads):
    c = Paged(heads, 32, [700] + [1] * 15 + [5, 5], [3584] + [601 * i for i in range(15)] + [8191, 10], 19)
    c.go()
    c.plan.check()
    c.check()


@pytest.mark.parametrize("heads", [(8, 2, 256), (32, 4, 64)])
@pytest.mark.parametrize("rows", [1, 4, 150])
def test_sequences_that_share_pages(heads, rows):
    """The same prefix's pages in several sequences' tables."""
    c = Paged(heads, 16, [rows] * 6, [64 + 5 * i for i in range(6)], 23)
    c.table[1:, :4] = c.table[0, :4]
    c.go()
    c.plan.check()
    c.check()


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64), (16, 1, 256)])
@pytest.mark.parametrize("rows", [1, 3, 40])
def test_large_values_and_growing_scores(heads, rows):
    """Scores whose maximum climbs from page to page, and one dominant key."""
    c = Paged(heads, 16, [rows, rows], [700, 2300], 29)
    hkv, hd = heads[1:]
    c.q.zero_()
    c.q[:, :, 0] = 1.0
    for sign in (1, -1):
        for r, (n, p, _) in enumerate(c.runs):
            ramp = torch.zeros(n + p, hkv, hd, device="cuda")
            ramp[:, :, 0] = sign * (4 if hd == 256 else 1) * torch.arange(n + p, device="cuda")[:, None] / 32.0
            c.k.view(-1, hkv, hd)[c.cells(r)] = ramp.half()
        c.go()
        c.plan.check()
        c.check()


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64)])
@pytest.mark.parametrize("rows", [1, 30])
def test_scores_as_large_as_fp16_allows(heads, rows):
    """All scores equal at about 2^24 and more: the answer is the mean of v."""
    c = Paged(heads, 32, [rows], [300], 31)
    hkv, hd = heads[1:]
    c.q[:] = 60000.0
    c.k.view(-1, hkv, hd)[c.cells(0)] = 60000.0
    c.go()
    c.plan.check()
    v = c.v.view(-1, hkv, hd)[c.cells(0)].double()
    for i in range(rows):
        want = v[:301 + i].mean(0).repeat_interleave(heads[0] // hkv, 0)
        a = v[:301 + i].abs().mean(0).repeat_interleave(heads[0] // hkv, 0)
        # every score is the same number: p is 1 throughout, only the sums and the last rounding are left
        assert ((c.out[i].double() - want).abs() <= 2 ** -8 * want.abs() + 2 ** -11 * a).all()


@pytest.mark.parametrize("rows", [1, 3, 60])
@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64)])
def test_ids_outside_the_cache(heads, rows):
    """They stand for zeros, are reported, and touch no other sequence."""
    c = Paged(heads, 16, [rows, rows, rows], [100, 90, 1500], 37)
    c.go()
    c.plan.check()
    first = c.out.clone()
    for bad in (-1, c.k.shape[0], (1 << 31) - 1, -(1 << 31)):
        kept = int(c.table[1, 2])
        c.table[1, 2] = bad
        c.go()
        with pytest.raises(binding.PrefillError, match="page id"):
            c.plan.check()
        c.plan.check()  # reported once
        assert torch.equal(c.out[:rows], first[:rows]) and torch.equal(c.out[2 * rows:], first[2 * rows:])
        # the same as a page of zeros
        got = c.out.clone()
        k0, v0 = c.k[kept].clone(), c.v[kept].clone()
        c.table[1, 2] = kept
        c.k[kept], c.v[kept] = 0.0, 0.0
        c.go()
        c.plan.check()
        c.check()
        assert torch.equal(got, c.out)
        c.k[kept], c.v[kept] = k0, v0


@pytest.mark.parametrize("rows,past", [([1] * 9, [700 * i for i in range(9)]), ([40, 64, 7], [900, 2000, 100])])
def test_repeats_and_other_sequences_values(rows, past):
    """The same bits on a repeat, and whatever the other sequences hold."""
    c = Paged((8, 2, 256), 64, rows, past, 41)
    c.go()
    first = c.out.clone()
    for _ in range(3):
        c.out.fill_(7)
        c.go()
        assert torch.equal(c.out, first)
    cells = c.cells(1)
    c.k.view(-1, 2, 256)[cells] = 1.0
    c.v.view(-1, 2, 256)[cells] = -2.0
    c.go()
    c.plan.check()
    a, b = rows[0], rows[0] + rows[1]
    assert torch.equal(c.out[:a], first[:a]) and torch.equal(c.out[b:], first[b:])


@pytest.mark.parametrize("rows", [1, 6])
def test_offsets_past_32_bits(rows):
    """A cache whose elements (and bytes) pass 2^31 and 2^32."""
    heads, page = (8, 2, 256), 64
    n_pages = 70_000
    c = Paged(heads, page, [rows, rows], [500, 90], 43)
    small_k, small_v, small = c.k, c.v, c.table.clone()
    c.k = torch.empty(n_pages, page, 2, 256, dtype=torch.float16, device="cuda")
    c.v = torch.empty(n_pages, page, 2, 256, dtype=torch.float16, device="cuda")
    far = small.clone()
    real = small >= 0
    far[real] = n_pages - 1 - small[real] * 1000
    c.k[far[real].long()], c.v[far[real].long()] = small_k[small[real].long()], small_v[small[real].long()]
    c.table = far
    c.go()
    c.plan.check()
    c.check()


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64)])
@pytest.mark.parametrize("rows,past", [([1] * 10, [333 * i for i in range(10)]), ([50, 9], [800, 40])])
def test_recorded_and_replayed(heads, rows, past):
    """Replayed on new values and new pages."""
    c = Paged(heads, 16, rows, past, 47)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.go()
    for seed in (1, 2, 3):
        d = Paged(heads, 16, rows, past, 47 + seed)
        c.q.copy_(d.q), c.k.copy_(d.k), c.v.copy_(d.v), c.table.copy_(d.table)
        graph.replay()
        torch.cuda.synchronize()
        c.plan.check()
        c.check()


def test_two_streams_at_once():
    jobs = []
    for i in range(2):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            jobs.append((s, Paged((8, 1, 256), 16, [1] * (20 + i), [200 * j for j in range(20 + i)], 53 + i)))
    for _ in range(4):
        for s, c in jobs:
            with torch.cuda.stream(s):
                c.go()
    torch.cuda.synchronize()
    for s, c in jobs:
        c.plan.check(s)
        c.check()


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64)])
def test_one_scratch_for_changing_runs(heads):
    """Calls one after another in one scratch: single tokens, chunks and
    trees, whole, cut in two and cut in many."""
    sizes = [([1, 1], [10, 20]), ([70, 90, 33, 200], [1500, 800, 3000, 0]), ([1], [30000]), ([1] * 64, [900] * 64),
             ([64, 1, 128], [600, 6000, 0]), ([1] * 3, [5000] * 3)]
    jobs = [Paged(heads, 16, rows, past, 61 + i) for i, (rows, past) in enumerate(sizes)]
    big = max((c.plan for c in jobs), key=lambda p: p.work_bytes)
    for c in jobs:
        c.plan.work, c.plan.work_at, c.plan.work_bytes = big.work, big.work_at, big.work_bytes
    for _ in range(3):
        for c in jobs:
            c.out[:c.total] = 7
            c.go()
    big.check()
    for c in jobs:
        c.check()


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64), (16, 16, 64)])
@pytest.mark.parametrize("words", [2, 4])
def test_wide_masks_over_few_rows(heads, words):
    """A single word would do: the others are skipped, whatever they hold."""
    c = Paged(heads, 16, [2, 1, 2, 0, 1], [700, 33, 0, 5, 2000], 89)
    mask = np.concatenate([_random_tree(c.runs, 1, 3)] + [np.full((6, 1), 2**64 - 1, np.uint64)] * (words - 1), 1)
    c.go(np.concatenate([mask, np.zeros((3, words), np.uint64)]))
    c.plan.check()
    c.check(mask)


@pytest.mark.parametrize("page", [1024, 4096])
@pytest.mark.parametrize("rows", [1, 70])
def test_large_pages(page, rows):
    c = Paged((8, 2, 256), page, [rows] * 3, [5000, 10, 4096], 97)
    c.go()
    c.plan.check()
    c.check()


def test_no_rows():
    c = Paged((8, 2, 64), 16, [4], [10], 71)
    for runs in ([], [(0, 0, 0), (0, 30, 5)]):
        plan = binding.AttnRuns(runs, 8, 2, 64)
        binding.attention_paged(c.q[:0], c.k, c.v, plan, c.table, c.out)
        plan.check()
    assert (c.out == 7).all()


@pytest.mark.parametrize("heads", [(1024, 64, 64), (1024, 1024, 64), (64, 64, 256), (256, 16, 256)])
def test_many_heads(heads):
    for rows, past in (([3, 20, 1], [40, 0, 300]), ([1, 1], [40, 2000])):
        c = Paged(heads, 16, rows, past, 67)
        c.go()
        c.plan.check()
        c.check()


def test_wrapper_refuses_what_does_not_fit():
    c = Paged((8, 2, 64), 16, [4], [10], 71)
    mask = torch.zeros(4, 1, dtype=torch.int64, device="cuda")

    def call(**bad):
        a = dict(q=c.q, k=c.k, v=c.v, runs=c.plan, pages=c.table, out=c.out)
        a.update(bad)
        binding.attention_paged(**a)

    for bad in (dict(q=c.q.float()), dict(q=c.q[:3]), dict(k=c.k[:, :, :1]), dict(k=c.k.cpu()), dict(v=c.v[:1]),
                dict(out=c.out.half()), dict(out=c.out[:3]), dict(k=c.k[:, 0], v=c.v[:, 0]),
                dict(k=c.k[:, :8], v=c.v[:, :8]), dict(pages=c.table.long()), dict(pages=c.table.cpu()),
                dict(pages=c.table.repeat(2, 2)[:, :3]), dict(mask=mask[:3]), dict(mask=mask.int()),
                dict(mask=mask.cpu()), dict(mask=mask[:, :0]), dict(mask=mask.repeat(1, 5))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(binding.PrefillError):  # a table too short
        call(pages=c.table[:, :0])
    k12 = torch.zeros(4, 12, 2, 64, dtype=torch.float16, device="cuda")
    with pytest.raises(binding.PrefillError, match="page_size"):
        call(k=k12, v=k12)
