"""The paged serving step's operators run together, as a server uses them: a
prompt's rows normed, turned and written into pages chunk by chunk, attention
over them, then drafted tokens verified; against the same steps in float64."""
import numpy as np
import pytest

from prefill_kv_shared_gb300 import binding, synth
from tests.gpu_util import need_gpu, torch
from tests.test_gpu_attention_runs import _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    need_gpu()
    from prefill_kv_shared_gb300 import build
    build.build()
    return binding.load()


@pytest.mark.parametrize("model", ["tiny", "e2b", "tinyllama"])
def test_prompt_chunks_drafts_and_verification(model):
    cfg = synth.config(model)
    hq, hkv, hd = cfg["n_head"], cfg["n_head_kv"], cfg["head_dim"]
    page, lengths, chunk, drafts = 16, [130, 70, 1], 64, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    total = [n + drafts for n in lengths]
    need = [-(-n // page) for n in total]
    n_pages = sum(need) + 2
    ids = np.random.default_rng(1).permutation(n_pages)[:sum(need)].astype(np.int32)
    width = max(need)
    table = torch.full((len(lengths), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = torch.from_numpy(ids[at:at + n])
        at += n
    k_cache = torch.full((n_pages, page, hkv, hd), float("nan"), dtype=torch.float16, device="cuda")
    v_cache = k_cache.clone()
    qkv = [torch.randn(n, hq + 2 * hkv, hd, generator=g, device="cuda") for n in total]
    gains = [torch.randn(hd, generator=g, device="cuda") * 0.2 for _ in range(2)]
    done = [0] * len(lengths)
    q_all = [torch.empty(n, hq, hd, dtype=torch.float16, device="cuda") for n in total]
    out_all = [torch.empty(n, hq, hd, dtype=torch.bfloat16, device="cuda") for n in total]

    def step(rows):
        """One call of each operator over rows[s] new rows of every sequence."""
        pos = torch.cat([torch.arange(done[s], done[s] + n) for s, n in enumerate(rows)]).int().cuda()
        slots = torch.cat([table[s, torch.arange(done[s], done[s] + n) // page].cpu() * page +
                           torch.arange(done[s], done[s] + n) % page for s, n in enumerate(rows)]).int().cuda()
        part = torch.cat([qkv[s][done[s]:done[s] + n] for s, n in enumerate(rows)])
        q = torch.empty(len(part), hq, hd, dtype=torch.float16, device="cuda")
        binding.qk_norm_rope(part[:, :hq], pos, q, part[:, hq:hq + hkv], part[:, hq + hkv:], slots, k_cache, v_cache,
                             q_gain=gains[0], k_gain=gains[1], eps=cfg["rms_eps"], rope_base=cfg["rope_base"])
        plan = binding.AttnRuns([(n, done[s], s * width) for s, n in enumerate(rows)], hq, hkv, hd)
        out = torch.empty(len(part), hq, hd, dtype=torch.bfloat16, device="cuda")
        binding.attention_paged(q, k_cache, v_cache, plan, table, out)
        plan.check()
        r = 0
        for s, n in enumerate(rows):
            q_all[s][done[s]:done[s] + n], out_all[s][done[s]:done[s] + n] = q[r:r + n], out[r:r + n]
            done[s] += n
            r += n
        return out

    while any(d < n for d, n in zip(done, lengths)):
        step([min(chunk, n - d) for d, n in zip(done, lengths)])
    # the last token of each prompt again with its four drafts: rows of a verification
    for s in range(len(lengths)):
        done[s] -= 1
    last = step([drafts + 1] * len(lengths))

    # every row of every sequence, against the formula over its rotated keys
    i = torch.arange(hd // 2, device="cuda", dtype=torch.float64)
    ks, vs = [], []
    for s, n in enumerate(total):
        x = qkv[s][:, hq:hq + hkv].double()
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + cfg["rms_eps"]) * (1 + gains[1].double())
        t = torch.arange(n, device="cuda").double()[:, None] * cfg["rope_base"] ** (-2 * i / hd)
        a, b, c, sn = y[..., :hd // 2], y[..., hd // 2:], torch.cos(t)[:, None], torch.sin(t)[:, None]
        want = torch.cat([a * c - b * sn, a * sn + b * c], -1)
        cells = table[s, torch.arange(n, device="cuda") // page].long() * page + torch.arange(n, device="cuda") % page
        got = k_cache.view(-1, hkv, hd)[cells]
        size = torch.cat([a.abs() + b.abs()] * 2, -1)
        assert ((got.double() - want).abs() <= 2 ** -11 * want.abs() + 2 ** -25 + 2 ** -18 * size).all()
        ks.append(got), vs.append(v_cache.view(-1, hkv, hd)[cells])
        assert torch.equal(vs[-1], qkv[s][:, hq + hkv:].half())
    runs, cell = [], 0
    for n in total:
        runs.append((n, 0, cell))
        cell += n
    _check((hq, hkv, hd), runs, torch.cat(q_all), torch.cat(ks), torch.cat(vs), torch.cat(out_all))

    # logits of the verification's rows (a projection of the attention's output), and their verification
    vocab = cfg["vocab"]
    head = torch.randn(hq * hd, vocab, generator=g, device="cuda") / (hq * hd) ** 0.5 * 8
    logits = last.flatten(1).float() @ head
    rows, n_seq = len(logits), len(lengths)
    first = torch.arange(0, rows + 1, drafts + 1, dtype=torch.int32, device="cuda")
    judges = torch.tensor([r for r in range(rows) if (r + 1) % (drafts + 1)], device="cuda")
    draft = logits[judges] + 0.3 * torch.randn(len(judges), vocab, generator=g, device="cuda")
    tokens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    tokens[judges + 1] = (draft - torch.empty_like(draft).exponential_(generator=g).log()).argmax(-1).int()
    u = torch.rand(rows, generator=g, device="cuda")
    noise = torch.empty(n_seq, vocab, device="cuda").exponential_(generator=g)
    n_accept = torch.empty(n_seq, dtype=torch.int32, device="cuda")
    token = torch.empty_like(n_accept)
    p_accept = torch.empty(rows, device="cuda")
    binding.verify_draft(logits, tokens, first, u, noise, n_accept, token, p_accept, binding.VerifyWork(rows, n_seq),
                         draft=draft)
    p, q = torch.softmax(logits.double(), -1), torch.softmax(draft.double(), -1)
    for s in range(n_seq):
        taken = 0
        while taken < drafts:
            r = s * (drafts + 1) + taken
            d = int(tokens[r + 1])
            if not float(u[r]) * float(q[r - s, d]) < float(p[r, d]):
                break
            taken += 1
        r = s * (drafts + 1) + taken
        w = (p[r] - q[r - s]).clamp(min=0) if taken < drafts else p[r]
        assert int(n_accept[s]) == taken and int(token[s]) == int((w / noise[s].double()).argmax())
    # and their log probabilities agree with the verification's shares
    lp = torch.empty(len(judges), device="cuda")
    binding.logprobs(logits[judges].contiguous(), tokens[judges + 1].contiguous(), lp)
    share = (lp.double().exp() / q.gather(1, tokens[judges + 1].long()[:, None])[:, 0]).clamp(max=1)
    assert ((share - p_accept[judges].double()).abs() <= 1e-4 * share).all()
