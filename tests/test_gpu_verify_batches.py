"""Verification of drafted tokens in batches as a server forms them, with slots
that have no rows, and rows in which target and draft agree.  Definition and
margins as in test_gpu_verify_draft; here every decision has to have its margin
(the seeds are such), so that all of them are compared."""
import pytest

from prefill_kv_shared_gb300 import binding
from tests.gpu_util import need_gpu, torch
from tests.test_gpu_verify_draft import CLOSE, Draft, _expected

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    need_gpu()
    from prefill_kv_shared_gb300 import build
    build.build()
    return binding.load()


def _slots(lens, vocab, seed, model, dtype=torch.float32):
    """A batch whose sequence s has lens[s] rows, none where it is 0."""
    c = Draft([n - 1 for n in lens if n], vocab, dtype, seed, model=model)
    first = [0]
    for n in lens:
        first.append(first[-1] + n)
    c.first = torch.tensor(first, dtype=torch.int32, device="cuda")
    n = len(lens)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    c.noise = torch.empty(n, vocab, device="cuda").exponential_(generator=g).clamp_min_(1e-30)
    c.n_accept = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    c.token = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    c.work = binding.VerifyWork(first[-1], n)
    if model:
        c.draft = c.draft[:first[-1] - n]
    return c


def _check(c, refused=()):
    """Every sequence against the definition; `refused` and empty ones give -1,
    and no share is written for their rows."""
    t, d = c.target.cpu(), None if c.draft is None else c.draft.cpu()
    tok, first, u, noise = c.tokens.tolist(), c.first.tolist(), c.u.tolist(), c.noise.cpu()
    share = c.p_accept.tolist()
    for s, (r0, r1) in enumerate(zip(first, first[1:])):
        got = (int(c.n_accept[s]), int(c.token[s]))
        if r0 == r1 or s in refused:
            assert got == (-1, -1), (s, got)
            assert share[r0:r1] == [-9.0] * (r1 - r0)
            continue
        n, token, shares, sure = _expected(t, d, tok, first, u, noise, s)
        assert sure, s
        assert got == (n, token), (s, got, n, token)
        for r, p in enumerate(shares, r0):
            assert abs(share[r] - p) <= CLOSE * p + 1e-37, (s, r)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens", [[5, 0], [0, 5], [0, 0, 5, 0], [3, 0, 4, 0, 1, 0], [0, 1, 0, 1, 2, 0, 0, 6], [2, 0]])
def test_slots_without_rows(lens, dtype):
    """No draft model: each sequence for itself, whatever the others have."""
    c = _slots(lens, 900, 5 + sum(lens), False, dtype)
    c.go()
    _check(c)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens,refused", [
    ([4, 0, 1], (0,)), ([3, 0], (0,)), ([0, 3], (1,)), ([1, 0, 1, 3], (3,)), ([2, 3, 0, 0, 1], (1,)), ([0, 0, 5, 0], (2,)),
    ([3, 1, 0, 2], ()), ([1, 0, 1, 1, 2, 1, 1], (4,)), ([2, 1, 1, 0, 1], (0,)), ([2, 0], (0,)), ([0, 2], (1,)),
])
def test_slots_without_rows_with_a_draft_model(lens, refused, dtype):
    """Draft row r - s of row r: refused are the sequences of which that lies
    outside the draft's rows, and no others; a sequence without drafts needs
    none."""
    c = _slots(lens, 900, 7 + sum(lens), True, dtype)
    assert len(c.draft) == sum(lens) - len(lens)
    c.go()
    _check(c, refused)


@pytest.mark.parametrize("drafts,vocab", [([3], 32000), ([2] * 5, 50257), ([1, 0, 4], 131072), ([2] * 90, 9001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0.0, 0.5])
def test_a_refused_draft_whose_rows_agree(drafts, vocab, dtype, shift):
    """w is 0 throughout where p and q are alike (or a shift apart, which a
    softmax does not see): drawn from p.  The two rows' sums are formed in
    other orders, so that they differ by their roundings; u of 2 refuses all
    the same."""
    c = Draft(drafts, vocab, dtype, 11 + vocab, near=0.0)
    if dtype is torch.float32:
        c.target.copy_((c.target * 64).round() / 64)  # (so that the shift rounds nothing)
        c.draft.copy_(c.target[[r for r in range(len(c.target)) if r + 1 not in c.first.tolist()]] + shift)
    c.u[:] = 2.0
    c.go()
    p = torch.softmax(c.target.double(), -1)
    first = c.first.tolist()
    for s, r in enumerate(first[:-1]):
        score = p[r] / c.noise[s].double()
        best, second = score.topk(2).values.tolist()
        assert best > second * (1 + 4 * CLOSE)
        assert (int(c.n_accept[s]), int(c.token[s])) == (0, int(score.argmax())), s


@pytest.mark.parametrize("vocab", [32000, 50257])
@pytest.mark.parametrize("sequences", [1, 3, 60])
def test_all_of_p_on_the_refused_draft(vocab, sequences):
    """Without a draft model: nothing is left but the drafted token, which is p
    itself; few sequences share their rows among several CTAs."""
    c = Draft([2] * sequences, vocab, torch.float32, 13 + vocab, model=False)
    c.target[:] = float("-inf")
    c.target[torch.arange(3 * sequences - 1), c.tokens[1:].long()] = 1.0
    c.target[3 * sequences - 1, 5] = 1.0
    c.u[:] = 2.0
    c.go()
    assert (c.n_accept == 0).all() and torch.equal(c.token, c.tokens[1::3])


def test_a_scratch_serves_every_batch_of_no_more_rows():
    """Fewer rows, and fewer or more sequences than it was made for."""
    work = binding.VerifyWork(64, 64)
    for drafts in ([0] * 64, [4] * 8, [31, 30], [63], [62], [0, 0, 0]):
        c = Draft(drafts, 500, torch.float32, 19 + len(drafts))
        c.work = work
        c.go()
        c.check()
    c = Draft([64], 500, torch.float32, 23)
    c.work = work
    with pytest.raises(binding.PrefillError, match="scratch"):
        c.go()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("model", [True, False])
@pytest.mark.parametrize("drafts,vocab", [([0], 7), ([1], 1000), ([4], 32000), ([33], 300), ([100], 5000), ([5, 0], 50257)])
def test_few_sequences_all_compared(drafts, vocab, dtype, model):
    """Ten batches of one or two sequences: nine in ten decisions have their
    margin, and those are compared."""
    sure_of = 0
    for seed in range(10):
        c = Draft(drafts, vocab, dtype, 1000 + seed, model=model, near=0.3)
        c.go()
        t, d = c.target.cpu(), None if c.draft is None else c.draft.cpu()
        tok, first, u, noise = c.tokens.tolist(), c.first.tolist(), c.u.tolist(), c.noise.cpu()
        for s in range(len(drafts)):
            n, token, _, sure = _expected(t, d, tok, first, u, noise, s)
            if sure:
                assert (int(c.n_accept[s]), int(c.token[s])) == (n, token), (seed, s)
                sure_of += 1
    assert sure_of >= 9 * len(drafts)
