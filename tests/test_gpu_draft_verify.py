"""The several-sequence operators run together, as a serving loop uses them:
a model's prompt prefilled into the cache, attention of the prompt's rows and
of a drafted tree over the model's own cached K/V, then the log probabilities
of the drafted tokens."""
import numpy as np
import pytest

import oracle
from prefill_kv_shared_gb300 import binding, synth
from tests.gpu_util import need_gpu, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    need_gpu()
    from prefill_kv_shared_gb300 import build
    build.build()
    return binding.load()


def test_prompt_cache_tree_and_scores(lib):
    cfg = synth.config("tiny")
    w = synth.make_weights(cfg)
    n = 150
    tok = synth.make_tokens(cfg, n)
    ctx = binding.PrefillContext(w, max_ctx=256, ubatch_max=256)
    logits = torch.empty(cfg["vocab"], dtype=torch.float32, device="cuda")
    ctx.ubatch(tok, 0, True, logits)
    ctx.sync()
    nbytes = ctx.kv_image_bytes(n)
    image = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    ctx.kv_save(image, nbytes)
    ctx.sync()
    hq, hkv, hd = cfg["n_head"], cfg["n_head_kv"], cfg["head_dim"]
    body = image[16:].view(torch.float16).view(2, ctx.n_layers_written, n, hkv, hd)
    k, v = body[0, 1].contiguous(), body[1, 1].contiguous()
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(n, hq, hd, generator=g, device="cuda").half()

    # the whole prompt's rows, against the oracle and the one-sequence kernel
    plan = binding.AttnRuns([(n, 0, 0)], hq, hkv, hd)
    out = torch.empty(n, hq, hd, dtype=torch.bfloat16, device="cuda")
    binding.attention_packed(q, k, v, plan, out)
    plan.check()
    want = oracle.attention(q.float().cpu().numpy(), k.float().cpu().numpy(), v.float().cpu().numpy(), np.arange(n))
    one = torch.empty_like(out)
    binding.check_op(lib.pfop_attention(0, q.data_ptr(), k.data_ptr(), v.data_ptr(), n, hq, hkv, hd, 0, n,
                                        one.data_ptr(), None))
    assert np.abs(out.float().cpu().numpy() - want).max() <= 1e-2
    # two bf16 roundings of values at most max|v|, and the fp16 probabilities of both
    assert (out.float() - one.float()).abs().max() <= (2 ** -7 + 2 ** -8) * v.float().abs().max()

    # the prompt's last ten tokens taken as a drafted tree over the first 140:
    # two branches, 0-1-2-3-4 and 0-5-6-7-8-9
    parents = [-1, 0, 1, 2, 3, 0, 5, 6, 7, 8]
    bits = []
    for j, p in enumerate(parents):
        bits.append((bits[p] if p >= 0 else 0) | (1 << j))
    mask = torch.tensor(bits, dtype=torch.int64, device="cuda")[:, None].contiguous()
    tree = binding.AttnRuns([(10, 140, 0)], hq, hkv, hd)
    tout = torch.empty(10, hq, hd, dtype=torch.bfloat16, device="cuda")
    binding.attention_tree(q[140:].contiguous(), k, v, tree, mask, tout)
    tree.check()
    kn, vn = k.float().cpu().numpy(), v.float().cpu().numpy()
    for j in range(10):
        cells = list(range(140)) + [140 + i for i in range(10) if bits[j] >> i & 1]
        ref = oracle.attention(q[140 + j:141 + j].float().cpu().numpy(), kn[cells], vn[cells],
                               np.array([len(cells) - 1]))
        assert np.abs(tout[j].float().cpu().numpy() - ref[0]).max() <= 1e-2

    # the model's own logits: what it gives the next tokens
    lp, ent = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    tid, tlp = torch.empty(1, 5, dtype=torch.int32, device="cuda"), torch.empty(1, 5, device="cuda")
    drafted = torch.tensor([int(tok[0])], dtype=torch.int32, device="cuda")
    binding.logprobs(logits[None], drafted, lp, ent, tid, tlp)
    x = logits.double().cpu()
    ref = torch.log_softmax(x, -1)
    assert abs(float(lp) - float(ref[int(tok[0])])) < 1e-5
    assert abs(float(ent) - float(-(ref.exp() * ref).sum())) < 1e-5
    assert tid[0].tolist() == torch.sort(x, descending=True, stable=True)[1][:5].tolist()
    assert int(tid[0, 0]) == int(torch.argmax(logits))
    ctx.close()
