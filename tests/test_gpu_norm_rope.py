"""Norm and rotation of queries and keys, K and V into the cache
(pfop_qk_norm_rope) against the formula in float64.

Tolerance of an output y = a cos t - b sin t (a, b the normed pair):
  - y is rounded to fp16: half a step, 2^-11 |y|, and 2^-25 below fp16's
    normal range;
  - the mean of squares is a sum of hd positive fp32 products over chains of at
    most 21 additions: 21 * 2^-24 relative, half of that in its root; the
    reciprocal root 2^-22, the products and 1 + g 3 * 2^-24: together below
    2^-20 of a and of b;
  - sine and cosine of an angle that is off by the rounding of its half turns
    to fp32 (pi 2^-24) and by the turn's own (pos 2^-53 2 pi), themselves 2^-22:
    below 2^-20 + pos 2^-50 in all;
  - two products and a sum: 3 * 2^-24.
Together 2^-11 |y| + 2^-25 + (|a| + |b|) (2^-18 + pos 2^-50), the last term
also for the float64 angle of the check itself."""
import numpy as np
import pytest

from prefill_kv_shared_gb300 import binding
from tests.gpu_util import need_gpu, torch

pytestmark = pytest.mark.gpu

HEADS = [(8, 1, 256), (8, 2, 256), (32, 4, 64), (4, 1, 64), (3, 3, 64), (1, 1, 256), (5, 2, 256), (17, 1, 64)]


@pytest.fixture(scope="module", autouse=True)
def lib():
    need_gpu()
    from prefill_kv_shared_gb300 import build
    build.build()
    return binding.load()


def _normed(x, gain, eps):
    y = x.double()
    if gain is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * (1 + gain.double())
    return y


def _check(got, x, gain, pos, eps=1e-6, base=10000.0):
    hd = x.shape[-1]
    y = _normed(x, gain, eps)
    a, b = y[..., :hd // 2], y[..., hd // 2:]
    t = pos.double()[:, None] * base ** (-2.0 * torch.arange(hd // 2, device="cuda", dtype=torch.float64) / hd)
    cos, sin = torch.cos(t)[:, None], torch.sin(t)[:, None]
    want = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    size = torch.cat([a.abs() + b.abs()] * 2, -1)
    tol = 2 ** -11 * want.abs() + 2 ** -25 + size * (2 ** -18 + pos.double().abs()[:, None, None] * 2 ** -50)
    over = (got.double() - want).abs() / tol
    assert float(over.max()) <= 1, f"{float(over.max())} of the tolerance"


class Step:
    def __init__(self, heads, rows, dtype, seed, norm=True, page=16, far=4096, wide=False, scale=2.0):
        hq, hkv, hd = heads
        g = torch.Generator(device="cuda").manual_seed(seed)
        # parts of one projection's rows, or apart
        qkv = (torch.randn(rows, hq + 2 * hkv, hd, generator=g, device="cuda") * scale).to(dtype)
        self.q, self.k, self.v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        if wide:
            self.q, self.k, self.v = self.q.contiguous(), self.k.contiguous(), self.v.contiguous()
        self.gains = (None, None)
        if norm:
            self.gains = tuple(torch.randn(hd, generator=g, device="cuda") * 0.3 for _ in range(2))
        self.pos = torch.randint(0, far, (rows,), generator=g, device="cuda", dtype=torch.int32)
        n_pages = -(-rows // page) + 2
        self.slots = torch.from_numpy(np.random.default_rng(seed).permutation(n_pages * page)[:rows].astype(np.int32)).cuda()
        self.q_out = torch.full((rows, hq, hd), 7.0, dtype=torch.float16, device="cuda")
        self.kc = torch.full((n_pages, page, hkv, hd), 5.0, dtype=torch.float16, device="cuda")
        self.vc = torch.full((n_pages, page, hkv, hd), 3.0, dtype=torch.float16, device="cuda")

    def go(self, **kw):
        binding.qk_norm_rope(self.q, self.pos, self.q_out, self.k, self.v, self.slots, self.kc, self.vc,
                             q_gain=self.gains[0], k_gain=self.gains[1], **kw)

    def check(self, **kw):
        hkv, hd = self.kc.shape[2:]
        _check(self.q_out, self.q, self.gains[0], self.pos, **kw)
        cells_k, cells_v = self.kc.view(-1, hkv, hd), self.vc.view(-1, hkv, hd)
        here = (self.slots >= 0) & (self.slots < len(cells_k))
        at = self.slots[here].long()
        _check(cells_k[at], self.k[here], self.gains[1], self.pos[here], **kw)
        assert torch.equal(cells_v[at], self.v[here].half())
        rest = torch.ones(len(cells_k), dtype=torch.bool, device="cuda")
        rest[at] = False
        assert (cells_k[rest] == 5).all() and (cells_v[rest] == 3).all()


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("rows", [1, 2, 37])
def test_step(heads, dtype, norm, rows):
    c = Step(heads, rows, dtype, 1 + rows, norm=norm)
    c.go()
    c.check()


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [513, 5000])
def test_many_rows(heads, dtype, rows):
    c = Step(heads, rows, dtype, 3, wide=True)
    c.go()
    c.check()


@pytest.mark.parametrize("heads", [(8, 1, 256), (32, 4, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [1, 300])
def test_queries_only(heads, dtype, rows):
    """A KV-shared layer's rows: no keys, no values."""
    c = Step(heads, rows, dtype, 5)
    binding.qk_norm_rope(c.q, c.pos, c.q_out, q_gain=c.gains[0])
    _check(c.q_out, c.q, c.gains[0], c.pos)
    assert (c.kc == 5).all() and (c.vc == 3).all()


@pytest.mark.parametrize("hd", [64, 256])
def test_far_positions(hd):
    c = Step((4, 2, hd), 64, torch.float32, 7)
    c.pos = torch.tensor([0, 1, (1 << 17) - 1, 1 << 20, (1 << 24) + 1, (1 << 30) - 1, (1 << 31) - 1, -5] * 8,
                         dtype=torch.int32, device="cuda")
    c.go()
    c.check()
    # position 0 turns nothing
    zero = c.pos == 0
    y = _normed(c.q[zero], c.gains[0], 1e-6)
    assert ((c.q_out[zero].double() - y).abs() <= 2 ** -11 * y.abs() + 2 ** -25 + 2 ** -18 * y.abs()).all()


@pytest.mark.parametrize("base", [1.0, 500000.0, 1e6])
@pytest.mark.parametrize("eps", [0.0, 1e-5, 0.5])
def test_bases_and_eps(base, eps):
    for hd in (64, 256):
        c = Step((4, 1, hd), 20, torch.float32, 11)
        c.go(rope_base=base, eps=eps)
        c.check(base=base, eps=eps)


def test_rows_of_no_cell():
    """Slots outside the cache: the row's queries only."""
    c = Step((8, 2, 256), 60, torch.bfloat16, 13)
    c.slots[::3] = -1
    c.slots[1::6] = c.kc.shape[0] * c.kc.shape[1]
    c.slots[4] = -(1 << 31)
    c.slots[7] = (1 << 31) - 1
    c.go()
    c.check()


def test_a_cache_of_cells_and_strided_rows():
    c = Step((32, 4, 64), 9, torch.float32, 17)
    wide = torch.zeros(9, 41, 64, device="cuda")
    wide[:, 1:33] = c.q
    c.q = wide[:, 1:33]
    c.kc, c.vc = c.kc.flatten(0, 1), c.vc.flatten(0, 1)
    c.go()
    c.kc, c.vc = c.kc[:, None], c.vc[:, None]
    c.check()


def test_zeros_and_values_past_fp16():
    c = Step((4, 1, 64), 4, torch.float32, 19)
    c.q[0] = 0.0
    c.k[1] = 0.0
    c.v[2] = 1e6
    c.q[3] = 1e15  # the norm brings it back
    c.go()
    assert (c.q_out[0] == 0).all()
    cells = c.vc.view(-1, 1, 64)
    assert torch.isinf(cells[c.slots[2].long()]).all()
    _check(c.q_out[3:], c.q[3:], c.gains[0], c.pos[3:])


def test_offsets_past_32_bits():
    """A cache, and rows, whose bytes pass 2^32."""
    heads, rows, cells = (4, 2, 256), 40, 9_000_000
    c = Step(heads, rows, torch.float32, 23)
    c.kc = torch.full((cells, 2, 256), 5.0, dtype=torch.float16, device="cuda")
    c.vc = torch.full((cells, 2, 256), 3.0, dtype=torch.float16, device="cuda")
    c.slots = (cells - 1 - 200_000 * torch.arange(rows, device="cuda")).to(torch.int32)
    wide = torch.empty(rows, 1 << 25, device="cuda")   # 128 MB from a row to the next
    wide[:, :1024] = c.q.reshape(rows, -1)
    c.q = wide[:, :1024].unflatten(1, (4, 256))
    c.go()
    at = c.slots.long()
    _check(c.q_out, c.q, c.gains[0], c.pos)
    _check(c.kc[at], c.k, c.gains[1], c.pos)
    assert torch.equal(c.vc[at], c.v.half())
    assert (c.kc[at - 1] == 5).all() and (c.vc[at - 1] == 3).all()


def test_recorded_and_on_another_stream():
    c = Step((8, 1, 256), 50, torch.bfloat16, 29)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.go()
    d = Step((8, 1, 256), 50, torch.bfloat16, 31)
    c.q.copy_(d.q), c.k.copy_(d.k), c.v.copy_(d.v), c.pos.copy_(d.pos), c.slots.copy_(d.slots)
    c.kc.fill_(5), c.vc.fill_(3)
    graph.replay()
    torch.cuda.synchronize()
    c.check()
    with torch.cuda.stream(s):
        e = Step((8, 1, 256), 50, torch.bfloat16, 37)
        e.go()
    s.synchronize()
    e.check()


def test_no_rows_and_many_heads():
    c = Step((8, 2, 64), 0, torch.float32, 47)
    c.go()
    assert (c.kc == 5).all()
    for heads, dtype in (((1024, 8, 64), torch.float32), ((128, 1024, 64), torch.bfloat16), ((33, 7, 256), torch.bfloat16)):
        c = Step(heads, 3, dtype, 53)
        c.go()
        c.check()


def test_two_bases_in_turn():
    for _ in range(2):
        for base in (10000.0, 1e6):
            c = Step((4, 1, 64), 5, torch.float32, 41)
            c.go(rope_base=base)
            c.check(base=base)


def test_wrapper_refuses_what_does_not_fit():
    c = Step((8, 2, 64), 4, torch.float32, 43)

    def call(**bad):
        a = dict(q=c.q, pos=c.pos, q_out=c.q_out, k=c.k, v=c.v, slots=c.slots, k_cache=c.kc, v_cache=c.vc,
                 q_gain=c.gains[0], k_gain=c.gains[1])
        a.update(bad)
        binding.qk_norm_rope(**a)

    for bad in (dict(q=c.q[:, 0]), dict(q=c.q.transpose(0, 1)), dict(k=c.k.bfloat16()), dict(v=c.v[:, :1]),
                dict(k=c.k[:3]), dict(pos=c.pos.long()), dict(pos=c.pos[:3]), dict(pos=c.pos.cpu()),
                dict(slots=None), dict(slots=c.slots.long()), dict(q_out=c.q_out.float()), dict(q_out=c.q_out[:3]),
                dict(k_cache=c.kc.float()), dict(k_cache=c.kc[..., :32]), dict(v_cache=c.vc[:1]), dict(k_cache=None),
                dict(q_gain=c.gains[0][:32]), dict(k_gain=c.gains[1].half()), dict(k=None), dict(v=c.v.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(binding.PrefillError):
        call(q=c.q[..., ::1][:, :, :32].contiguous(), q_out=c.q_out[:, :, :32].contiguous(),
             k=c.k[:, :, :32].contiguous(), v=c.v[:, :, :32].contiguous(), k_cache=c.kc[..., :32].contiguous(),
             v_cache=c.vc[..., :32].contiguous(), q_gain=None, k_gain=None)
    # a row that does not start on 16 bytes
    wide = torch.zeros(4, 8 * 64 + 2, device="cuda")
    with pytest.raises(binding.PrefillError):
        call(q=wide[:, 2:].unflatten(1, (8, 64)))
