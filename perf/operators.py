"""Workloads of the library's multi-sequence operators, with their plain forms.

  packed    causal grouped-query attention of several sequences' rows in one
            call (whole prompts, or rows that continue a cached prefix)
  tree      attention of drafted token trees over the sequences' caches
  logprobs  log probabilities of given tokens, entropy and top alternatives
            of a batch of logits rows

`own` false: elementary torch operations in 32 bits, rounded once at the end.
`own` true: the library's entry points (prefill_kv_shared_gb300.binding).
Head layouts, lengths and vocabularies are those of the package's synthetic
models (synth.CONFIGS) and of its benchmark.
"""
import math

import numpy as np
import torch

own = False

# (query heads, KV heads, head dim) of the package's models
HEADS = {"e2b": (8, 1, 256), "e4b": (8, 2, 256), "tinyllama": (32, 4, 64), "tiny": (4, 1, 64)}


# ---------------------------------------------------------------------------
# cases


def listed():
    """`rows`: rows of each sequence in the call; `past`: cached positions before them."""
    return [
        # the command line's default prompt on the TinyLlama shape: one short prompt, latency
        dict(name="packed tinyllama 25", op="packed", heads="tinyllama", rows="25", past="0"),
        # the benchmark's first workload: one prompt of one ubatch
        dict(name="packed e2b 512", op="packed", heads="e2b", rows="512", past="0"),
        # suffixes of 32 tokens behind a restored 500-token system prefix, 64 requests at once
        dict(name="packed tinyllama 64x32", op="packed", heads="tinyllama",
             rows=",".join(["32"] * 64), past=",".join(["500"] * 64)),
        # a server's prompts of very different lengths in one call, one of a single token
        dict(name="packed e4b ragged 16k", op="packed", heads="e4b", rows="8192,4093,2048,1000,511,1",
             past="0,0,0,0,0,0"),
        # a chain of four drafted tokens after a short prompt: the smallest verification step
        dict(name="tree tinyllama 1x5", op="tree", heads="tinyllama", rows="5", past="532"),
        # one long chat: 25 drafted tokens over the longest prompt of the benchmark
        dict(name="tree e2b 1x25 32k", op="tree", heads="e2b", rows="25", past="32768"),
        # a batch at ragged contexts, from one token (plain decoding) to 64-token trees
        dict(name="tree e4b 12 ragged", op="tree", heads="e4b", rows="64,1,16,25,40,64,8,33,16,1,61,16",
             past="8192,16000,4096,8191,12345,2048,0,500,8192,7,10000,6000"),
        # 64 short contexts with 16 drafted tokens each
        dict(name="tree tinyllama 64x16", op="tree", heads="tinyllama", rows=",".join(["16"] * 64),
             past=",".join(str(500 + 13 * i) for i in range(64))),
        # after one decoding step: one row, the choices shown to a user
        dict(name="logprobs 1x32768", op="logprobs", rows=1, vocab=32768, dtype="float32", top=5, masked=False),
        # the rows of a verification step, vocabulary 32000
        dict(name="logprobs 64x32000", op="logprobs", rows=64, vocab=32000, dtype="float32", top=20, masked=False),
        # scoring one ubatch of a prompt
        dict(name="logprobs 512x32768", op="logprobs", rows=512, vocab=32768, dtype="float32", top=1, masked=False),
        # scoring a long prompt from 16-bit logits, part of the vocabulary ruled out
        dict(name="logprobs 4096x32768 bf16", op="logprobs", rows=4096, vocab=32768, dtype="bfloat16", top=8,
             masked=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["packed", "tree", "logprobs"])
    if op == "logprobs":
        vocab = _log_int(rng, 1024, 131072)
        rows = _log_int(rng, 1, max(1, min(4096, (1 << 26) // vocab)))
        return dict(op=op, rows=rows, vocab=vocab, dtype=rng.choice(["float32", "bfloat16"]),
                    top=rng.choice([0, 1, 5, 8, 20, 32]), masked=rng.random() < 0.3)
    heads = rng.choice(sorted(HEADS))
    if op == "packed":
        longest = _log_int(rng, 1, 4096)
        past_max = rng.choice([0, 0, _log_int(rng, 1, 4096)])
        n = _log_int(rng, 1, max(1, min(64, 16384 // (longest + past_max))))
        rows = [longest] + [rng.randint(0, longest) for _ in range(n - 1)]
        past = [rng.randint(0, past_max) for _ in range(n)]
    else:
        longest = _log_int(rng, 1, 120)
        past_max = _log_int(rng, 16, 32768)
        n = _log_int(rng, 1, max(1, min(64, 65536 // past_max)))
        rows = [longest] + [rng.randint(1, longest) for _ in range(n - 1)]
        past = [past_max] + [rng.randint(0, past_max) for _ in range(n - 1)]
    return dict(op=op, heads=heads, rows=",".join(map(str, rows)), past=",".join(map(str, past)))


def _lists(case):
    return [int(x) for x in case["rows"].split(",")], [int(x) for x in case["past"].split(",")]


# ---------------------------------------------------------------------------
# inputs


def _tree_masks(rows, words, rng):
    """Random trees: bit j of a row's words is set where drafted token j of the
    same sequence is the row's token or one of its ancestors."""
    out = []
    for n in rows:
        parents = [int(rng.integers(-1, j)) if j else -1 for j in range(n)]
        bits = []
        for j, p in enumerate(parents):
            bits.append((bits[p] if p >= 0 else 0) | (1 << j))
        out += [[(b >> (64 * w)) & 0xFFFFFFFFFFFFFFFF for w in range(words)] for b in bits]
    return np.array(out, dtype=np.uint64).reshape(-1, words).view(np.int64)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, scale=1.0, dtype=torch.float16):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    if case["op"] == "logprobs":
        r, vocab, top = case["rows"], case["vocab"], case["top"]
        logits = normal(r, vocab, scale=3.0, dtype=getattr(torch, case["dtype"]))
        tokens = torch.randint(0, vocab, (r,), generator=g, device="cuda", dtype=torch.int32)
        if case["masked"]:
            ruled_out = torch.rand(vocab, generator=g, device="cuda") < 0.3
            ruled_out[:64] = False
            logits.masked_fill_(ruled_out, float("-inf"))
            tokens[ruled_out[tokens.long()]] = 7
        return dict(case=case, logits=logits, tokens=tokens,
                    logp=torch.empty(r, device="cuda"), entropy=torch.empty(r, device="cuda"),
                    top_id=torch.empty(r, top, device="cuda", dtype=torch.int32),
                    top_logp=torch.empty(r, top, device="cuda"))
    hq, hkv, hd = HEADS[case["heads"]]
    rows, past = _lists(case)
    # the unified cache: every sequence has the same number of cells
    per_seq = max(n + p for n, p in zip(rows, past))
    cells = per_seq * len(rows)
    total = sum(rows)
    runs = [(n, p, i * per_seq) for i, (n, p) in enumerate(zip(rows, past))]
    st = dict(case=case, runs=runs, sizes=torch.tensor(runs, device="cuda").T.contiguous(),
              q=normal(total, hq, hd, scale=1.5), k=normal(cells, hkv, hd), v=normal(cells, hkv, hd),
              out=torch.empty(total, hq, hd, device="cuda", dtype=torch.bfloat16))
    if case["op"] == "tree":
        words = -(-max(rows) // 64)
        rng = np.random.default_rng(int(seed))
        st["mask"] = torch.from_numpy(_tree_masks(rows, words, rng)).cuda()
    return st


# ---------------------------------------------------------------------------
# one pass


def run(state):
    if own:
        return _run_own(state)
    if state["case"]["op"] == "logprobs":
        return _plain_logprobs(state)
    return _plain_attention(state)


def _run_own(state):
    from prefill_kv_shared_gb300 import binding

    op = state["case"]["op"]
    if op == "logprobs":
        binding.logprobs(state["logits"], state["tokens"], state["logp"], state["entropy"], state["top_id"],
                         state["top_logp"])
        return {k: state[k] for k in ("logp", "entropy", "top_id", "top_logp")}
    q, k, v, out = state["q"], state["k"], state["v"], state["out"]
    if "plan" not in state:  # kept by a program for as long as the sequences' shapes stay
        state["plan"] = binding.AttnRuns(state["runs"], q.shape[1], k.shape[1], q.shape[2])
    if op == "packed":
        binding.attention_packed(q, k, v, state["plan"], out)
    else:
        binding.attention_tree(q, k, v, state["plan"], state["mask"], out)
    return out


def _plain_attention(state):
    """All sequences as one padded batch."""
    q, k, v = state["q"], state["k"], state["v"]
    dev = q.device
    total, hq, hd = q.shape
    hkv = k.shape[1]
    n, past, cell0 = state["sizes"]
    r, n_max, l_max = len(n), int(max(x[0] for x in state["runs"])), int(max(x[0] + x[1] for x in state["runs"]))
    out = torch.zeros(total, hq, hd, device=dev, dtype=torch.bfloat16)
    i = torch.arange(n_max, device=dev)
    j = torch.arange(l_max, device=dev)
    real = i[None, :] < n[:, None]                                      # [r, n_max]
    row = ((torch.cumsum(n, 0) - n)[:, None] + i[None, :])[real]        # packed row of each real (r, i)
    qp = torch.zeros(r, n_max, hq, hd, device=dev)
    qp[real] = q[row].float()
    cell = (cell0[:, None] + j[None, :]).clamp(max=k.shape[0] - 1)
    kp, vp = k[cell].float(), v[cell].float()                           # [r, l_max, hkv, hd]
    qp = qp.view(r, n_max, hkv, hq // hkv, hd).permute(0, 2, 1, 3, 4).reshape(r, hkv, -1, hd)
    s = qp @ kp.permute(0, 2, 3, 1) / math.sqrt(hd)                     # [r, hkv, n_max * group, l_max]
    s = s.view(r, hkv, n_max, -1, l_max)
    if "mask" in state:
        seen = torch.zeros(r, n_max, l_max, device=dev, dtype=torch.bool)
        d = j[None, :] - past[:, None]                                  # drafted token at key j
        w = (d.clamp(min=0) // 64).clamp(max=state["mask"].shape[1] - 1)
        words = torch.zeros(r, n_max, state["mask"].shape[1], device=dev, dtype=torch.int64)
        words[real] = state["mask"][row]
        bit = torch.gather(words, 2, w[:, None, :].expand(r, n_max, l_max)) >> (d.clamp(min=0) % 64)[:, None, :] & 1
        seen = (d < 0)[:, None, :] | ((bit == 1) & (d >= 0)[:, None, :] & (d < n[:, None])[:, None, :])
    else:
        seen = j[None, None, :] <= past[:, None, None] + i[None, :, None]
    s = s.masked_fill(~seen[:, None, :, None, :], float("-inf"))
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m == float("-inf"), torch.zeros_like(m), m))
    del s
    l = e.sum(-1, keepdim=True)
    e = e / torch.where(l == 0, torch.ones_like(l), l)
    o = e.view(r, hkv, -1, l_max) @ vp.permute(0, 2, 1, 3)
    o = o.view(r, hkv, n_max, hq // hkv, hd).permute(0, 2, 1, 3, 4).reshape(r, n_max, hq, hd)
    out[row] = o[real].to(torch.bfloat16)
    return out


def _plain_logprobs(state):
    x = state["logits"].float()
    m = x.amax(-1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    z = e.sum(-1, keepdim=True)
    log_z = torch.log(z)
    logp = torch.gather(d, 1, state["tokens"].long()[:, None]) - log_z
    entropy = log_z - torch.where(e > 0, e * d, torch.zeros_like(e)).sum(-1, keepdim=True) / z
    top = state["case"]["top"]
    value, index = torch.sort(x, dim=-1, descending=True, stable=True)  # ties: the lowest index first
    return {"logp": logp[:, 0], "entropy": entropy[:, 0], "top_id": index[:, :top].to(torch.int32),
            "top_logp": value[:, :top] - m - log_z}


# ---------------------------------------------------------------------------
# work and exact values


def work(case):
    if case["op"] == "logprobs":
        n = case["rows"] * case["vocab"]
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": n * size + case["rows"] * (12 + 8 * case["top"]), "flops": 5 * n}
    hq, hkv, hd = HEADS[case["heads"]]
    rows, past = _lists(case)
    if case["op"] == "packed":
        pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(rows, past))
        mask = 0
    else:
        # a drafted token sees its context, itself and its ancestors: about log2 of the tree's size of them
        pairs = sum(int(n * (p + 1 + math.log(max(1, n)))) for n, p in zip(rows, past))
        mask = sum(rows) * 8 * -(-max(rows) // 64)
    keys = sum(n + p for n, p in zip(rows, past) if n)
    return {"bytes": sum(rows) * hq * hd * 4 + keys * hkv * hd * 4 + mask, "flops": 4 * hd * hq * pairs}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "logprobs":
        return _exact_logprobs(st)
    if work(case)["flops"] > 1e13:
        return None
    return _exact_attention(st)


def _exact_logprobs(st):
    parts = []
    top = st["case"]["top"]
    for at in range(0, st["logits"].shape[0], 256):
        x = st["logits"][at:at + 256].double()
        lp = torch.log_softmax(x, -1)
        p = lp.exp()
        h = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(-1)
        # the order of the values, the lower index first where two are equal
        order = torch.argsort(-x, dim=-1, stable=True)[:, :top]
        parts.append((lp[torch.arange(len(x), device=x.device), st["tokens"][at:at + 256].long()], h,
                      order.to(torch.int32), torch.gather(lp, 1, order)))
    a, b, c, d = (torch.cat(t) for t in zip(*parts))
    return {"logp": a, "entropy": b, "top_id": c, "top_logp": d}


def _exact_attention(st):
    """Sequence by sequence and query head by query head, in float64."""
    q, k, v = st["q"], st["k"], st["v"]
    hq, hkv, hd = q.shape[1], k.shape[1], q.shape[2]
    out = torch.zeros(q.shape, device=q.device, dtype=torch.float64)
    row0 = 0
    for n, past, cell0 in st["runs"]:
        for t0 in range(0, n, 1024):
            t1 = min(n, t0 + 1024)
            keys = past + (n if "mask" in st else t1)
            pos = torch.arange(keys, device=q.device)
            t = torch.arange(t0, t1, device=q.device)[:, None]
            if "mask" in st:
                words = st["mask"][row0 + t0:row0 + t1].cpu().numpy().view(np.uint64)
                bits = np.unpackbits(words.astype("<u8").view(np.uint8), axis=1, bitorder="little")[:, :n]
                vis = torch.ones(t1 - t0, keys, dtype=torch.bool, device=q.device)
                vis[:, past:] = torch.from_numpy(bits.astype(bool)).to(q.device)
            else:
                vis = pos[None, :] <= past + t
            for h in range(hq):
                kh = k[cell0:cell0 + keys, h * hkv // hq].double()
                vh = v[cell0:cell0 + keys, h * hkv // hq].double()
                a = q[row0 + t0:row0 + t1, h].double() @ kh.T * hd ** -0.5
                a = a.masked_fill(~vis, -math.inf).softmax(-1)
                out[row0 + t0:row0 + t1, h] = torch.nan_to_num(a) @ vh
        row0 += n
    return out
