"""Verification of drafted tokens (pfop_verify_draft) against its definition in
float64.

The share p(d) / q(d) comes from two softmax values: exp of a difference
(2^-22 and its argument's 2^-24 |x - m|, |x - m| below 2^5 for tokens that were
drafted), two sums of exponentials of 2^-22 terms in fp32 (2^-20) and three
roundings: below 2^-17 relative.  Whether a draft is accepted and which token
is drawn are whole numbers: they are compared wherever the definition's own
margin is above the same 2^-17 (relative, of p where p - q is drawn from), and
all but a few of a test's decisions have to be."""
import numpy as np
import pytest

from prefill_kv_shared_gb300 import binding
from tests.gpu_util import need_gpu, torch

pytestmark = pytest.mark.gpu

CLOSE = 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def lib():
    need_gpu()
    from prefill_kv_shared_gb300 import build
    build.build()
    return binding.load()


def _softmax(x):
    x = x.double()
    m = x.max()
    if not torch.isfinite(m):
        return None  # a NaN, +inf or only -inf
    e = torch.exp(x - m)
    return e / e.sum()


def _expected(target, draft, tokens, first, u, noise, s):
    """(n_accept, token, shares, sure) of sequence s; sure: every decision on
    the way has a margin."""
    vocab = target.shape[1]
    r0, r1 = int(first[s]), int(first[s + 1])
    shares, n, tok, sure, done = [], 0, -1, True, False
    for r in range(r0, r1):
        p = _softmax(target[r])
        q = None
        if r == r1 - 1:
            shares.append(0.0)
            if done:
                break
            if p is not None:
                w, scale = p, p
        else:
            d = int(tokens[r + 1])
            known = 0 <= d < vocab
            if draft is not None:
                q = _softmax(draft[r - s])
            if p is None or (draft is not None and q is None):
                shares.append(float("nan"))
                if done:
                    continue
                done = True
                continue
            pd = float(p[d]) if known else 0.0
            qd = (float(q[d]) if known else 1.0) if q is not None else 1.0
            shares.append(1.0 if pd >= qd and pd > 0 else 0.0 if pd == 0 else pd / qd)
            if done:
                continue
            lhs = float(u[r]) * qd
            if abs(lhs - pd) <= CLOSE * pd and lhs != pd:
                sure = False
            if lhs < pd:
                n += 1
                continue
            done = True
            scale = p
            if q is not None:
                w = (p - q).clamp(min=0)
            else:
                w = p.clone()
                if known:
                    w[d] = 0
            if not bool((w > 0).any()):
                w = p
        if r == r1 - 1 and p is None:
            return n, -1, shares, sure
        score = w / noise[s].double()
        best = int(score.argmax())
        tok = int((score == score[best]).nonzero()[0])
        off = CLOSE * (scale + (q if q is not None and r < r1 - 1 else 0)) / noise[s].double()
        rivals = score + off >= score[tok] - off[tok]
        rivals[tok] = False
        if bool((rivals & (w > 0)).any()) and bool((score[rivals & (w > 0)] != score[tok]).any()):
            sure = False
        done = True
        if r == r1 - 1:
            break
    return n, tok, shares, sure


class Draft:
    def __init__(self, drafts, vocab, dtype, seed, model=True, scale=3.0, near=1.0, pad=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n, rows = len(drafts), sum(drafts) + len(drafts)
        nd = rows - n

        def strided(r):
            t = torch.full((r, vocab + pad), float("nan"), dtype=dtype, device="cuda")
            return t[:, pad // 2:pad // 2 + vocab] if pad else t

        self.target = strided(rows)
        x = torch.randn(rows, vocab, generator=g, device="cuda") * scale
        self.target.copy_(x)
        self.first = torch.tensor(np.concatenate([[0], np.cumsum(np.array(drafts) + 1)]).astype(np.int32), device="cuda")
        judges = torch.tensor([r for s in range(n) for r in range(int(self.first[s]), int(self.first[s + 1]) - 1)],
                              dtype=torch.long, device="cuda")
        self.draft = None
        y = x[judges] + near * torch.randn(nd, vocab, generator=g, device="cuda")
        if model:
            self.draft = strided(nd)
            self.draft.copy_(y)
            y = self.draft.float()
        self.tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
        if nd:
            e = torch.empty(nd, vocab, device="cuda").exponential_(generator=g)
            self.tokens[judges + 1] = (y - e.log()).argmax(-1).to(torch.int32)
        self.u = torch.rand(rows, generator=g, device="cuda")
        self.noise = torch.empty(n, vocab, device="cuda").exponential_(generator=g).clamp_min_(1e-30)
        self.n_accept = torch.full((n,), -9, dtype=torch.int32, device="cuda")
        self.token = torch.full((n,), -9, dtype=torch.int32, device="cuda")
        self.p_accept = torch.full((rows,), -9.0, device="cuda")
        self.work = binding.VerifyWork(rows, n)

    def go(self, **kw):
        binding.verify_draft(self.target, self.tokens, self.first, self.u, self.noise, self.n_accept, self.token,
                             self.p_accept, self.work, draft=self.draft, **kw)

    def check(self, least=0.99):
        t, tok, first, u = self.target.cpu(), self.tokens.tolist(), self.first.tolist(), self.u.tolist()
        d = None if self.draft is None else self.draft.cpu()
        noise, sure_of = self.noise.cpu(), 0
        got_n, got_t, got_p = self.n_accept.tolist(), self.token.tolist(), self.p_accept.tolist()
        n = len(got_n)
        for s in range(n):
            want_n, want_t, shares, sure = _expected(t, d, tok, first, u, noise, s)
            for r, p in enumerate(shares, first[s]):
                if np.isnan(p):
                    assert np.isnan(got_p[r]), (s, r)
                else:
                    assert abs(got_p[r] - p) <= CLOSE * p + 1e-37, (s, r, got_p[r], p)
            if sure:
                assert (got_n[s], got_t[s]) == (want_n, want_t), (s, got_n[s], got_t[s], want_n, want_t)
                sure_of += 1
        assert sure_of >= least * n - 1


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("model", [True, False])
@pytest.mark.parametrize("vocab", [1, 2, 7, 64, 1000, 1023, 4096, 32000])
@pytest.mark.parametrize("drafts", [[0], [1], [4], [0, 3, 0, 1, 5]])
def test_small(dtype, model, vocab, drafts):
    c = Draft(drafts, vocab, dtype, 1 + vocab + sum(drafts), model=model)
    c.go()
    c.check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("model", [True, False])
@pytest.mark.parametrize("n,vocab", [(40, 1025), (150, 512), (300, 333), (20, 50257)])
def test_batches(dtype, model, n, vocab):
    c = Draft([(5 * i) % 7 for i in range(n)], vocab, dtype, 3, model=model, near=0.5, scale=2.0)
    c.go()
    c.check()


@pytest.mark.parametrize("drafts", [[33], [31, 32, 64, 1], [100]])
def test_long_drafts(drafts):
    """Beyond a warp's lanes, mostly accepted."""
    c = Draft(drafts, 300, torch.float32, 5, near=0.02)
    c.u *= 0.5
    c.go()
    c.check()
    assert int(c.n_accept.max()) > 25
    c.u[0] = 0.999999
    c.tokens[1] = int(c.target[0].argmin())
    c.go()
    c.check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad", [1, 3, 6, 17])
def test_strided_rows(dtype, pad):
    """Rows of any alignment within wider ones, whose rest is NaN."""
    c = Draft([3, 0, 2], 1234, dtype, 7, pad=pad)
    c.go()
    c.check()


def test_all_accepted_and_all_refused():
    c = Draft([4] * 10, 500, torch.float32, 11)
    c.draft.copy_(c.target[[r for s in range(10) for r in range(5 * s, 5 * s + 4)]])
    c.go()
    assert (c.n_accept == 4).all()
    c.check()
    c = Draft([4] * 10, 500, torch.float32, 13)
    c.target[torch.arange(49), c.tokens[1:].long()] = float("-inf")
    c.go()
    assert (c.n_accept == 0).all()
    c.check()


def test_nothing_left_to_draw_from():
    """u of 1 refuses a draft although p and q are alike: drawn from p."""
    c = Draft([2, 3], 700, torch.float32, 17)
    c.draft.copy_(c.target[[0, 1, 3, 4, 5]])
    c.u[:] = 1.0
    c.go()
    assert (c.n_accept == 0).all()
    c.check()
    # all of p on the drafted token, refused: p itself again
    c = Draft([1], 50, torch.float32, 19, model=False)
    c.target[0] = float("-inf")
    c.target[0, 7] = 2.0
    c.tokens[1] = 7
    c.u[:] = 1.0
    c.go()
    assert c.n_accept.tolist() == [0] and c.token.tolist() == [7]


def test_equal_scores_take_the_lowest_token():
    for model in (False, True):
        c = Draft([0, 2], 5000, torch.float32, 23, model=model)
        c.target.zero_()
        if model:
            c.draft.zero_()
            c.draft[:, 9] = 3.0  # q everywhere below p but on token 9
        c.noise.fill_(1.0)
        c.tokens[2:] = 9
        c.u[:] = 0.99
        c.go()
        assert c.n_accept.tolist() == [0, 0] and c.token.tolist() == [0, 0]


def test_ruled_out_tokens():
    """-inf and the type's lowest value, in target and draft."""
    for low in (float("-inf"), torch.finfo(torch.float32).min):
        c = Draft([3, 1, 4, 0], 3000, torch.float32, 29)
        out = torch.rand(3000, device="cuda") < 0.5
        out[:50] = False
        c.target[:, out] = low
        c.draft[:, out.flip(0)] = low
        c.go()
        c.check()
        assert not out[c.token.long()].any()


def test_rows_without_a_distribution():
    nan, inf = float("nan"), float("inf")
    c = Draft([3] * 8, 900, torch.float32, 31, near=0.01)
    c.u *= 0.1
    c.target[0] = -inf          # sequence 0's first row
    c.target[4 + 1, 5] = nan    # the second of sequence 1
    c.target[8 + 3, 7] = inf    # the last of sequence 2
    c.draft[9 + 2, 0] = nan     # sequence 3's third draft
    c.draft[12] = -inf          # sequence 4's first
    c.draft[15, 899] = inf      # sequence 5's first
    c.go()
    assert c.n_accept.tolist()[:6] == [0, 1, 3, 2, 0, 0] and c.token.tolist()[:6] == [-1] * 6
    c.check()


def test_tokens_outside_the_vocabulary():
    c = Draft([2, 2, 2], 400, torch.float32, 37, near=0.01)
    c.u *= 0.1
    c.tokens[1], c.tokens[5], c.tokens[7] = -1, 400, (1 << 31) - 1
    c.go()
    assert c.n_accept.tolist() == [0, 1, 0]
    assert c.p_accept.tolist()[0] == 0 and ((c.token >= 0) & (c.token < 400)).all()
    c.check()


def test_rows_that_do_not_fit():
    """first[] from the device: sequences outside the rows are refused, each
    for itself."""
    c = Draft([2, 2, 2, 2], 100, torch.float32, 41)
    for bad in ([0, 3, 3, 9, 12], [-3, 3, 6, 9, 12], [0, 3, 6, 9, 13], [0, 12, 6, 9, 12],
                [0, 3, 6, (1 << 31) - 1, 12], [0, 3, -(1 << 31), 9, 12]):
        c.first.copy_(torch.tensor(bad, dtype=torch.int32))
        c.go()
        torch.cuda.synchronize()
        for s in range(4):
            a, b = bad[s], bad[s + 1]
            if not (0 <= a < b <= 12):
                assert int(c.n_accept[s]) == -1 and int(c.token[s]) == -1, (bad, s)
            elif [a, b] == [3 * s, 3 * s + 3]:
                assert 0 <= int(c.n_accept[s]) <= 2 and 0 <= int(c.token[s]) < 100


def test_without_shares_and_without_drafts():
    c = Draft([0] * 7, 2000, torch.float32, 43)
    c.p_accept = None
    c.go()
    p = torch.softmax(c.target.double(), -1)
    assert torch.equal(c.token.long(), (p / c.noise.double()).argmax(-1)) and (c.n_accept == 0).all()


def test_the_answers_are_distributed_as_the_target():
    """8192 times the same step: the first token after the prompt, accepted or
    drawn, has the target's distribution.  Counts of n p (1 - p) variance: 5
    standard deviations."""
    n, vocab = 8192, 6
    for model in (True, False):
        c = Draft([2] * n, vocab, torch.float32, 47, model=model)
        c.target.copy_(c.target[:3].repeat(n, 1))
        if model:
            c.draft.copy_(c.draft[:2].repeat(n, 1))
            g = torch.Generator(device="cuda").manual_seed(1)
            e = torch.empty(2 * n, vocab, device="cuda").exponential_(generator=g)
            drawn = (c.draft - e.log()).argmax(-1).to(torch.int32).view(n, 2)
        else:
            drawn = torch.tensor([[2, 4]], dtype=torch.int32, device="cuda").repeat(n, 1)
        c.tokens.view(n, 3)[:, 1:] = drawn
        c.go()
        got = torch.where(c.n_accept > 0, drawn[:, 0], c.token)
        p = torch.softmax(c.target[0].double(), -1).cpu()
        counts = torch.bincount(got.long(), minlength=vocab).double().cpu()
        assert ((counts - n * p).abs() <= 5 * (n * p * (1 - p)).sqrt() + 1).all(), (counts / n, p)


def test_offsets_past_32_bits():
    """Logits of more than 2^32 bytes; rows more than 2^31 elements apart."""
    c = Draft([3, 2], 500, torch.bfloat16, 53)
    rows = c.target.shape[0]
    wide = torch.empty(rows, (1 << 29) + 8, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:508] = c.target
    c.target = wide[:, 8:508]
    c.go()
    c.check()


def test_recorded_and_replayed():
    c = Draft([3, 1, 0, 4], 2500, torch.float32, 59)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.go()
    for seed in (61, 67):
        d = Draft([1, 4, 3, 0], 2500, torch.float32, seed)
        for name in ("target", "draft", "tokens", "first", "u", "noise"):
            getattr(c, name).copy_(getattr(d, name))
        graph.replay()
        torch.cuda.synchronize()
        c.check()


def test_repeats_and_streams():
    jobs = []
    for i in range(2):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            jobs.append((s, Draft([4] * (9 + i), 8000, torch.float32, 71 + i)))
    for _ in range(3):
        for s, c in jobs:
            with torch.cuda.stream(s):
                c.go()
    torch.cuda.synchronize()
    for s, c in jobs:
        c.check()
        first = (c.n_accept.clone(), c.token.clone(), c.p_accept.clone())
        c.go()
        for a, b in zip(first, (c.n_accept, c.token, c.p_accept)):
            assert torch.equal(a, b)


def test_no_sequences():
    c = Draft([1], 100, torch.float32, 79)
    binding.verify_draft(c.target[:0], c.tokens[:0], c.first[:1], c.u[:0], c.noise[:0], c.n_accept[:0], c.token[:0],
                         c.p_accept[:0], c.work, draft=c.draft[:0])
    torch.cuda.synchronize()
    assert c.n_accept.tolist() == [-9]


def test_more_sequences_than_fit_the_gpu_at_once():
    c = Draft([1, 0, 2] * 400, 700, torch.bfloat16, 83, near=0.5, scale=2.0)
    c.go()
    c.check()


def test_wrapper_refuses_what_does_not_fit():
    c = Draft([2, 1], 100, torch.float32, 73)

    def call(**bad):
        a = dict(target=c.target, tokens=c.tokens, first=c.first, u=c.u, noise=c.noise, n_accept=c.n_accept,
                 token=c.token, p_accept=c.p_accept, work=c.work, draft=c.draft)
        a.update(bad)
        binding.verify_draft(**a)

    for bad in (dict(target=c.target[0]), dict(target=c.target.cpu()), dict(target=c.target.T.contiguous().T),
                dict(draft=c.draft[:2]), dict(draft=c.draft.bfloat16()), dict(draft=c.draft.cpu()),
                dict(tokens=c.tokens.long()), dict(tokens=c.tokens[:4]), dict(first=c.first.long()),
                dict(first=c.first[:0]), dict(u=c.u.double()), dict(u=c.u[:4]), dict(noise=c.noise[:1]),
                dict(noise=c.noise.half()), dict(n_accept=c.n_accept[:1]), dict(token=c.token.long()),
                dict(p_accept=c.p_accept[:4]), dict(p_accept=c.p_accept.double())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(binding.PrefillError, match="scratch"):
        call(work=binding.VerifyWork(2, 2))
