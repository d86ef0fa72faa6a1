"""Token log probabilities, entropy and top alternatives (pfop_logprobs)
against the definition in float64.

Tolerances, with u = 2^-24, d = x - max, s = sum e^d, h = sum e^d d / s:
  - s: a term's exponent d log2(e) is rounded (|d| 1.45 u of e^d in relative
    terms, and e^d |d| <= 1/e, so at most u s over the sum of one-sided
    terms bounded by (1 + |h|) u), the exponential is good to 4 u, and the
    longest chain of additions is vocab / 256 + 64 long:
    rel(s) <= (vocab / 256 + 72 + |h|) u =: E;
  - logp = d - log s: rounding of d, log s and their difference, and E:
    E + 2 u (|d| + |log s|) + u |logp|;
  - entropy = log s - h: E for log s, and for h its own sum and s:
    E + 2 E |h| + 3 u (|log s| + |h|)."""
import numpy as np
import pytest

from prefill_kv_shared_gb300 import binding
from tests.gpu_util import need_gpu, torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def lib():
    need_gpu()
    from prefill_kv_shared_gb300 import build
    build.build()
    return binding.load()


def _run(x, tokens, n_top):
    r = x.shape[0]
    nan = float("nan")
    out = dict(logp=torch.full((r,), nan, device="cuda"), entropy=torch.full((r,), nan, device="cuda"),
               top_id=torch.full((r, n_top), -7, dtype=torch.int32, device="cuda"),
               top_logp=torch.full((r, n_top), nan, device="cuda"))
    binding.logprobs(x, tokens, **out)
    return out


def _check(x, tokens, n_top, out):
    xd = x.double()
    vocab = x.shape[1]
    m = xd.amax(-1, keepdim=True)
    d = xd - m
    e = d.exp()
    s = e.sum(-1, keepdim=True)
    h = torch.where(e > 0, e * d, torch.zeros_like(e)).sum(-1, keepdim=True) / s
    log_s = s.log()
    rel = (vocab / 256 + 72 + h.abs()) * U

    def close(got, want, tol):
        got = got.double()
        same = got == want  # infinities
        assert (same | ((got - want).abs() <= tol)).all(), float(((got - want).abs() / tol)[~same].max())

    dt = torch.gather(d, 1, tokens.long()[:, None])
    want = dt - log_s
    close(out["logp"][:, None], want, rel + 2 * U * (dt.abs() + log_s.abs()) + U * want.abs())
    close(out["entropy"][:, None], log_s - h, rel + 2 * rel * h.abs() + 3 * U * (log_s.abs() + h.abs()))
    if n_top:
        order = torch.sort(x.double(), dim=-1, descending=True, stable=True)[1][:, :n_top]
        assert torch.equal(out["top_id"].long(), order)
        dt = torch.gather(d, 1, order)
        want = dt - log_s
        close(out["top_logp"], want, rel + 2 * U * (dt.abs() + log_s.abs()) + U * want.abs())


def _logits(rows, vocab, dtype, seed, scale=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * scale).to(dtype)
    return x, torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab,n_top", [
    (1, 1, 1), (3, 2, 2), (2, 7, 5), (5, 31, 31), (2, 33, 32), (1, 255, 0), (4, 1000, 20), (1, 4097, 32),
    (7, 32000, 5), (1, 32768, 5), (300, 1024, 1), (130, 32768, 8), (700, 5001, 20), (2, 131073, 32), (1, 262144, 20),
    (40, 50257, 3),
])
def test_values(dtype, rows, vocab, n_top):
    x, tokens = _logits(rows, vocab, dtype, rows + vocab)
    _check(x, tokens, n_top, _run(x, tokens, n_top))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(1, 32768), (3, 6000), (200, 3001)])
@pytest.mark.parametrize("kind", ["equal", "two values", "rising", "falling", "blocks", "one high", "lowest masks",
                                  "infinite masks", "all but one masked", "large"])
def test_ties_orders_and_masks(dtype, rows, vocab, kind):
    x, tokens = _logits(rows, vocab, torch.float32, 5)
    i = torch.arange(vocab, device="cuda", dtype=torch.float32)
    low = torch.finfo(dtype).min
    if kind == "equal":
        x.fill_(-3.25)
    elif kind == "two values":
        x = (x > 2).float()
    elif kind == "rising":
        x[:] = i / 64
    elif kind == "falling":
        x[:] = -i / 64
    elif kind == "blocks":     # the largest values lie side by side
        x[:, vocab // 2:vocab // 2 + 64] += 40
    elif kind == "one high":
        x[:, vocab - 1] = 100
    elif kind == "lowest masks":
        x[:, ::3] = low
        x[:, 100:2000] = low
    elif kind == "infinite masks":
        x[:, ::3] = float("-inf")
        x[:, 100:2000] = float("-inf")
    elif kind == "all but one masked":
        x[:] = float("-inf")
        x[:, 1234] = 2.0
        tokens[:] = 1234
    elif kind == "large":
        x *= 1e4
    x = x.to(dtype)
    _check(x, tokens, 32, _run(x, tokens, 32))


def test_rows_without_a_distribution():
    x, tokens = _logits(6, 5000, torch.float32, 9)
    x[1, 77] = float("nan")
    x[2, 4999] = float("inf")
    x[3] = float("-inf")
    x[4, 0] = -float("nan")
    out = _run(x, tokens, 4)
    for r in (1, 2, 3, 4):
        assert torch.isnan(out["logp"][r]) and torch.isnan(out["entropy"][r])
        assert torch.isnan(out["top_logp"][r]).all() and (out["top_id"][r] == -1).all()
    keep = [0, 5]
    _check(x[keep], tokens[keep], 4, {k: v[keep] for k, v in out.items()})


def test_tokens_outside_the_vocabulary():
    x, tokens = _logits(4, 300, torch.float32, 10)
    tokens[1], tokens[2] = -1, 300
    out = _run(x, tokens, 2)
    assert torch.isnan(out["logp"][1]) and torch.isnan(out["logp"][2])
    assert torch.isfinite(out["logp"][[0, 3]]).all() and torch.isfinite(out["entropy"]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [3, 400])
def test_strided_and_unaligned_rows(dtype, rows):
    """A view of wider rows, starting off any vector boundary; what lies
    between the rows is never used."""
    wide, _ = _logits(rows, 2100, dtype, 12)
    wide[:] = float("nan")
    vals, tokens = _logits(rows, 2043, dtype, 13)
    x = wide[:, 5:5 + 2043]
    x.copy_(vals)
    _check(vals, tokens, 7, _run(x, tokens, 7))


def test_parts_left_out():
    x, tokens = _logits(5, 777, torch.float32, 14)
    want = _run(x, tokens, 3)
    logp, ent = torch.zeros(5, device="cuda"), torch.zeros(5, device="cuda")
    binding.logprobs(x, tokens, logp)
    binding.logprobs(x, entropy=ent)
    assert torch.equal(logp, want["logp"]) and torch.equal(ent, want["entropy"])
    tid, tlp = torch.zeros_like(want["top_id"]), torch.zeros_like(want["top_logp"])
    binding.logprobs(x, top_id=tid, top_logp=tlp)
    assert torch.equal(tid, want["top_id"]) and torch.equal(tlp, want["top_logp"])
    binding.logprobs(x)


def test_repeats_and_many_rows():
    """The same bits on a repeat; more rows than a grid dimension of 65535."""
    x, tokens = _logits(70_000, 40, torch.float32, 15)
    a, b = _run(x, tokens, 4), _run(x, tokens, 4)
    for k in a:
        assert torch.equal(a[k], b[k])
    _check(x, tokens, 4, a)


def test_offsets_past_32_bits():
    rows, vocab = 20_000, 131_072
    x = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    x[-1] = _logits(1, vocab, torch.bfloat16, 16)[0][0]
    tokens = torch.full((rows,), 5, dtype=torch.int32, device="cuda")
    out = _run(x, tokens, 2)
    _check(x[-1:], tokens[-1:], 2, {k: v[-1:] for k, v in out.items()})
    _check(x[:2], tokens[:2], 2, {k: v[:2] for k, v in out.items()})


@pytest.mark.parametrize("rows", [1, 300])
def test_recorded_and_replayed(rows):
    x, tokens = _logits(rows, 32000, torch.float32, 17)
    out = dict(logp=torch.zeros(rows, device="cuda"), entropy=torch.zeros(rows, device="cuda"),
               top_id=torch.zeros(rows, 5, dtype=torch.int32, device="cuda"), top_logp=torch.zeros(rows, 5, device="cuda"))
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        binding.logprobs(x, tokens, **out)
    for seed in (18, 19):
        x.copy_(_logits(rows, 32000, torch.float32, seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        _check(x, tokens, 5, out)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [3, 700])
@pytest.mark.parametrize("vocab", [32, 127, 512, 1023, 2000, 2057, 4095, 4096, 6151, 8200, 12289, 16383, 16385])
def test_small_slices(dtype, rows, vocab):
    """Rows that fill the warps' copies in part, for CTAs of either size,
    the rows' starts on and off 16-byte boundaries; with masked logits too."""
    x, tokens = _logits(rows, vocab, dtype, vocab)
    _check(x, tokens, 32, _run(x, tokens, 32))
    x[:, ::3] = float("-inf")
    x[:, -1] = 0.5
    _check(x, torch.full_like(tokens, vocab - 1), 5, _run(x, torch.full_like(tokens, vocab - 1), 5))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(1, 32768), (700, 9000)])
def test_alternatives_close_together(dtype, rows, vocab):
    """All alternatives in one thread's step, in several steps of one thread,
    and at a row's ragged ends."""
    x, tokens = _logits(rows, vocab, dtype, 5)
    g = torch.Generator(device="cuda").manual_seed(6)
    high = (40 + torch.arange(24, device="cuda")).to(dtype)
    for r in range(min(rows, 40)):
        start = int(torch.randint(0, vocab - 24, (1,), generator=g, device="cuda")) if r % 4 else (0, vocab - 24)[r // 4 % 2]
        span = (vocab - start - 1) // 24
        at = start + torch.arange(24, device="cuda") * (1, 8, 32, max(1, span))[r // 4 % 4]
        at = at[at < vocab]
        x[r, at] = high[torch.randperm(24, generator=g, device="cuda")][:len(at)]
    _check(x, tokens, 20, _run(x, tokens, 20))
