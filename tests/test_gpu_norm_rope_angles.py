"""Angles of norm and rotation: where a pair's two products cancel, and bases
of several host threads.

A rotated pair (a, b) without a norm: y = a cos t - b sin t.  The angle is a
32-bit part of a turn, made a float and multiplied by 2 pi 2^-32, itself
rounded: 3 * 2^-24 pi; sine and cosine are the approximate instructions, 2^-20.5
on it; a product and a fused sum 3 * 2^-24 at most.  Together
(9.5 + 11.4 + 3) 2^-24 (|a| + |b|) < 2^-19 (|a| + |b|), and pos 2^-50 for the
turn's own rounding and the check's angle, before y is rounded to fp16 (2^-11
|y|, 2^-25 below its normal range)."""
import threading

import pytest

from prefill_kv_shared_gb300 import binding
from tests.gpu_util import need_gpu, torch
from tests.test_gpu_norm_rope import Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    need_gpu()
    from prefill_kv_shared_gb300 import build
    build.build()
    return binding.load()


def _within(got, x, pos, base):
    hd = x.shape[-1]
    a, b = x[..., :hd // 2].double(), x[..., hd // 2:].double()
    t = pos.double()[:, None] * base ** (-2.0 * torch.arange(hd // 2, device="cuda", dtype=torch.float64) / hd)
    cos, sin = torch.cos(t)[:, None], torch.sin(t)[:, None]
    want = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    size = torch.cat([a.abs() + b.abs()] * 2, -1)
    tol = 2 ** -11 * want.abs() + 2 ** -25 + size * (2 ** -19 + pos.double()[:, None, None] * 2 ** -50)
    over = float(((got.double() - want).abs() / tol).max())
    assert over <= 1, over


@pytest.mark.parametrize("hd", [64, 256])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("far", [50, 4096, 1 << 20])
def test_pairs_that_cancel(hd, dtype, far):
    """Pairs along and across their own angle: one of the two results is as
    small as the inputs' rounding leaves it."""
    heads, rows, base = (6, 2, hd), 500, 10000.0
    c = Step(heads, rows, dtype, 61, norm=False, far=far, wide=True)
    t = c.pos.double()[:, None] * base ** (-2.0 * torch.arange(hd // 2, device="cuda", dtype=torch.float64) / hd)
    sin, cos = torch.sin(t), torch.cos(t)
    for x in (c.q, c.k):
        for h in range(x.shape[1]):
            scale = 2.0 ** (3 * h - 6)
            pair = (sin, cos) if h % 2 == 0 else (cos, -sin)
            x[:, h] = (scale * torch.cat(pair, -1)).to(dtype)
    c.go()
    _within(c.q_out, c.q, c.pos, base)
    hkv = heads[1]
    _within(c.kc.view(-1, hkv, hd)[c.slots.long()], c.k, c.pos, base)


def test_bases_of_several_threads():
    """Each host thread keeps the turns of its last base: two alternating in
    each of four threads, no two alike."""
    failed = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for j in range(20):
                    hd, base = (64, 256)[j // 2 % 2], 1000.0 * (1 + i) + 500.0 * (j % 2)
                    c = Step((4, 1, hd), 7, torch.float32, 67 + i, norm=False)
                    c.go(rope_base=base)
                    torch.cuda.current_stream().synchronize()
                    _within(c.q_out, c.q, c.pos, base)
        except BaseException as e:  # noqa: BLE001 (told by the test's own thread)
            failed.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
