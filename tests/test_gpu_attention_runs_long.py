"""Attention over runs of the longest kind: one prompt of 2^20 - 1 rows of 16
heads, whose launch takes longer (about 6 s) than the bound of a single wait
(about 2 s of SM clock).  A wait that lasts while a CTA pair works through its
share must not be cut off by that bound.

Sampled rows against the formula in float64.  Tolerance as in
test_gpu_attention_runs.py, with two changes for the length: scores are kept
small (q ~ N(0, 1/4), so of 2^20 scores all lie within 3 of the largest and
no probability is below fp16's normal range), and the fp32 accumulator takes
keys / 16 products in a row, each addition off by at most 2^-23 of what has
been summed: 2^-8 |o| + 2^-9 (1 + 1/8) A + keys / 16 * 2^-23 A."""
import pytest

from prefill_kv_shared_gb300 import binding
from tests.gpu_util import need_gpu, torch

pytestmark = pytest.mark.gpu


def test_a_prompt_of_a_million_rows():
    need_gpu()
    from prefill_kv_shared_gb300 import build
    build.build()
    hq, hd, n = 16, 256, (1 << 20) - 1  # an odd length: the run's last chunk of V is cleared behind its end
    g = torch.Generator(device="cuda").manual_seed(97)
    q = torch.empty(n, hq, hd, dtype=torch.float16, device="cuda").normal_(0, 0.25, generator=g)
    k = torch.empty(n, 1, hd, dtype=torch.float16, device="cuda").normal_(0, 1, generator=g)
    v = torch.empty(n, 1, hd, dtype=torch.float16, device="cuda").normal_(0, 1, generator=g)
    v += (torch.arange(n, device="cuda") / n)[:, None, None].half()
    out = torch.full((n, hq, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    plan = binding.AttnRuns([(n, 0, 0)], hq, 1, hd)
    binding.attention_packed(q, k, v, plan, out)
    plan.check()
    kd, vd = k[:, 0].double(), v[:, 0].double()
    for t in (0, 1, 127, 128, 4095, 70_000, n // 2, n - 129, n - 128, n - 2, n - 1):
        p = torch.softmax(q[t].double() @ kd[:t + 1].T / hd ** 0.5, -1)
        want, a = p @ vd[:t + 1], p @ vd[:t + 1].abs()
        tol = 2 ** -8 * want.abs() + (2 ** -9 * 1.125 + (t + 1) / 16 * 2 ** -23) * a
        over = float(((out[t].double() - want).abs() / tol).max())
        assert over <= 1, f"row {t}: {over} of the tolerance"
