"""Workloads of the library's paged serving step, with their plain forms.

  paged     attention of new tokens (a chunk of a prompt, single tokens,
            drafted tokens) over a paged K/V cache
  rope      per-head RMS norm of queries and keys, rotation by position, and
            K and V written to their cells of the cache
  verify    drafted tokens accepted or refused against the target's
            probabilities, from given random numbers

`own` false: elementary torch operations in 32 bits, rounded once at the end
(angles, and probabilities that decide between tokens, in 64).
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
ROPE_BASE, EPS = 10000.0, 1e-6


# ---------------------------------------------------------------------------
# cases


def listed():
    """`rows`: rows of each sequence in the call; `past`: cached positions before them."""
    return [
        # one chat on the TinyLlama shape: a single new token behind the command line's default prompt
        dict(name="paged tinyllama 1 token", op="paged", heads="tinyllama", rows="1", past="532", page=16, tree=False),
        # a batch of chats generating, a token each at ragged contexts
        dict(name="paged tinyllama 64 tokens", op="paged", heads="tinyllama", rows=",".join(["1"] * 64),
             past=",".join(str(500 + 13 * i) for i in range(64)), page=16, tree=False),
        # one long chat: a token behind the longest prompt of the benchmark
        dict(name="paged e2b 1 token 32k", op="paged", heads="e2b", rows="1", past="32768", page=64, tree=False),
        # drafted trees of 16 tokens over the same chats, each row seeing its own branch
        dict(name="paged tinyllama 64 trees", op="paged", heads="tinyllama", rows=",".join(["16"] * 64),
             past=",".join(str(500 + 13 * i) for i in range(64)), page=16, tree=True),
        # a server's mixed step: a chunk of one prompt, single tokens, and two chains of drafted tokens
        dict(name="paged e4b mixed", op="paged", heads="e4b", rows="512,1,1,1,1,1,1,1,1,5,5,1,1,1,1,1",
             past="3584,8192,16000,500,7,2048,4093,6000,12345,8191,1000,333,64,15,9999,0", page=32, tree=False),
        # a chunk of a long prompt behind the chunks before it
        dict(name="paged e4b chunk 4096 behind 28672", op="paged", heads="e4b", rows="4096", past="28672", page=128,
             tree=False),
        # one token of one sequence: the smallest step's projections
        dict(name="rope tinyllama 1", op="rope", heads="tinyllama", rows=1, dtype="float32", norm=True, shared=False,
             far=2048),
        # the benchmark's first prompt through a KV-shared layer: queries only
        dict(name="rope e2b 512 queries", op="rope", heads="e2b", rows=512, dtype="float32", norm=True, shared=True,
             far=2048),
        # many prompts' chunks in one step, from 16-bit projections, at positions up to 128k
        dict(name="rope e2b 16384", op="rope", heads="e2b", rows=16384, dtype="bfloat16", norm=True, shared=False,
             far=131072),
        # one chat's chain of four drafted tokens, with the draft model's logits
        dict(name="verify 1x4 32768", op="verify", drafts="4", vocab=32768, dtype="float32", model=True),
        # a batch of chats, up to five drafted tokens each, some none, on the TinyLlama vocabulary
        dict(name="verify 64 ragged 32000", op="verify", drafts=",".join(str((3 * i) % 6) for i in range(64)),
             vocab=32000, dtype="float32", model=True),
        # a large batch with tokens found by looking back in the text (no draft model), 16-bit logits
        dict(name="verify 256x4 32768 bf16", op="verify", drafts=",".join(["4"] * 256), vocab=32768,
             dtype="bfloat16", model=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["paged", "rope", "verify"])
    if op == "rope":
        return dict(op=op, heads=rng.choice(["e2b", "tinyllama", "tiny"]), rows=_log_int(rng, 1, 16384),
                    dtype=rng.choice(["float32", "bfloat16"]), norm=rng.random() < 0.7, shared=rng.random() < 0.3,
                    far=_log_int(rng, 16, 131072))
    if op == "verify":
        vocab = _log_int(rng, 1024, 131072)
        most = rng.randint(0, 8)
        n = _log_int(rng, 1, max(1, min(256, (1 << 24) // (vocab * (2 * most + 2)))))
        return dict(op=op, drafts=",".join(str(rng.randint(0, most)) for _ in range(n)), vocab=vocab,
                    dtype=rng.choice(["float32", "bfloat16"]), model=rng.random() < 0.7)
    heads = rng.choice(sorted(HEADS))
    page = rng.choice([8, 16, 16, 32, 64, 128, 256])
    kind = rng.choice(["tokens", "chunk", "drafts", "mixed"])
    past_max = _log_int(rng, 16, 32768)
    n = 1 if kind == "chunk" else _log_int(rng, 1, max(1, min(64, 65536 // past_max)))
    longest = {"tokens": 1, "chunk": _log_int(rng, 1, 4096), "drafts": _log_int(rng, 1, 120),
               "mixed": _log_int(rng, 1, 512)}[kind]
    rows = [longest] + [1 if kind == "mixed" else rng.randint(1, longest) for _ in range(n - 1)]
    past = [min(past_max, 28672)] + [rng.randint(0, past_max) for _ in range(n - 1)]
    return dict(op=op, heads=heads, rows=",".join(map(str, rows)), past=",".join(map(str, past)), page=page,
                tree=kind == "drafts")


def _ints(text):
    return [int(x) for x in text.split(",")]


# ---------------------------------------------------------------------------
# inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    return {"paged": _prepare_paged, "rope": _prepare_rope, "verify": _prepare_verify}[case["op"]](case, g, rng)


def _normal(g, *shape, scale=1.0, dtype=torch.float16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _prepare_paged(case, g, rng):
    hq, hkv, hd = HEADS[case["heads"]]
    rows, past, page = _ints(case["rows"]), _ints(case["past"]), case["page"]
    need = [-(-(n + p) // page) for n, p in zip(rows, past)]
    n_pages = sum(need) + 3                     # a pool with some pages to spare, handed out in no order
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(rows), max(need)), -1, np.int32)   # what lies behind a sequence's pages is no page
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    runs = [(n, p, r * max(need)) for r, (n, p) in enumerate(zip(rows, past))]
    total = sum(rows)
    st = dict(case=case, runs=runs, sizes=torch.tensor(runs, device="cuda").T.contiguous(),
              table=torch.from_numpy(table).cuda(), q=_normal(g, total, hq, hd, scale=1.5),
              k=_normal(g, n_pages, page, hkv, hd), v=_normal(g, n_pages, page, hkv, hd),
              out=torch.empty(total, hq, hd, device="cuda", dtype=torch.bfloat16))
    if case["tree"]:
        # bit j of a row's words is set where drafted token j of its run is the row's token or one of its ancestors
        bits = []
        words = -(-max(rows) // 64)
        for n in rows:
            own_bits = []
            for j in range(n):
                p = int(rng.integers(-1, j)) if j else -1
                own_bits.append((own_bits[p] if p >= 0 else 0) | (1 << j))
            bits += [[(b >> (64 * w)) & 0xFFFFFFFFFFFFFFFF for w in range(words)] for b in own_bits]
        st["mask"] = torch.from_numpy(np.array(bits, dtype=np.uint64).reshape(-1, words).view(np.int64)).cuda()
    return st


def _prepare_rope(case, g, rng):
    hq, hkv, hd = HEADS[case["heads"]]
    t = case["rows"]
    dtype = getattr(torch, case["dtype"])
    kv = 0 if case["shared"] else hkv
    # queries, keys and values as one projection leaves them
    qkv = _normal(g, t, hq + 2 * kv, hd, scale=2.0, dtype=dtype)
    st = dict(case=case, q=qkv[:, :hq], q_out=torch.empty(t, hq, hd, device="cuda", dtype=torch.float16),
              pos=torch.randint(0, case["far"], (t,), generator=g, device="cuda", dtype=torch.int32),
              q_gain=None, k_gain=None, k=None, v=None, k_cache=None, v_cache=None, slots=None)
    if case["norm"]:
        st["q_gain"] = torch.randn(hd, generator=g, device="cuda") * 0.2
        st["k_gain"] = torch.randn(hd, generator=g, device="cuda") * 0.2
    if kv:
        page = 16
        n_pages = -(-t // page) + 2
        st["k"], st["v"] = qkv[:, hq:hq + kv], qkv[:, hq + kv:]
        st["k_cache"], st["v_cache"] = _normal(g, n_pages, page, kv, hd), _normal(g, n_pages, page, kv, hd)
        slots = rng.permutation(n_pages)[np.arange(t) // page] * page + np.arange(t) % page
        slots[rng.random(t) < 0.02] = -1        # rows of a padded batch that belong to no sequence
        st["slots"] = torch.from_numpy(slots.astype(np.int32)).cuda()
    return st


def _prepare_verify(case, g, rng):
    drafts, vocab = _ints(case["drafts"]), case["vocab"]
    dtype = getattr(torch, case["dtype"])
    n, rows = len(drafts), sum(drafts) + len(drafts)
    target = torch.randn(rows, vocab, generator=g, device="cuda") * 3.0
    first = np.concatenate([[0], np.cumsum(np.array(drafts) + 1)]).astype(np.int32)
    seq = np.repeat(np.arange(n), np.array(drafts) + 1)
    drafted = np.ones(rows, bool)
    drafted[first[1:] - 1] = False              # the rows before which a token was drafted: not the last
    d_rows = torch.from_numpy(np.flatnonzero(drafted)).cuda()
    # the draft model agrees in part; its tokens are sampled from its logits
    near = (target[d_rows] + torch.randn(len(d_rows), vocab, generator=g, device="cuda")).to(dtype)
    gumbel = -torch.log(torch.empty(len(d_rows), vocab, device="cuda").exponential_(generator=g))
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    if len(d_rows):
        tokens[d_rows + 1] = (near.float() + gumbel).argmax(-1).to(torch.int32)
    noise = torch.empty(n, vocab, device="cuda").exponential_(generator=g).clamp_min_(1e-30)
    return dict(case=case, target=target.to(dtype), draft=near if case["model"] else None, tokens=tokens,
                first=torch.from_numpy(first).cuda(), seq=torch.from_numpy(seq).cuda(), d_rows=d_rows,
                host_first=first.tolist(), u=torch.rand(rows, generator=g, device="cuda"), noise=noise,
                n_accept=torch.empty(n, device="cuda", dtype=torch.int32),
                token=torch.empty(n, device="cuda", dtype=torch.int32), p_accept=torch.empty(rows, device="cuda"))


# ---------------------------------------------------------------------------
# one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return {"paged": _own_paged, "rope": _own_rope, "verify": _own_verify}[op](state)
    return {"paged": _plain_paged, "rope": _plain_rope, "verify": _plain_verify}[op](state)


def _own_paged(st):
    from prefill_kv_shared_gb300 import binding

    q, k = st["q"], st["k"]
    if "plan" not in st:  # kept by a program for as long as the sequences' shapes stay
        st["plan"] = binding.AttnRuns(st["runs"], q.shape[1], k.shape[2], q.shape[2])
    binding.attention_paged(q, k, st["v"], st["plan"], st["table"], st["out"], mask=st.get("mask"))
    return st["out"]


def _own_rope(st):
    from prefill_kv_shared_gb300 import binding

    binding.qk_norm_rope(st["q"], st["pos"], st["q_out"], st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"],
                         q_gain=st["q_gain"], k_gain=st["k_gain"], eps=EPS, rope_base=ROPE_BASE)
    return _rope_outputs(st)


def _rope_outputs(st):
    out = {"q": st["q_out"]}
    if st["k"] is not None:
        out["k_cache"], out["v_cache"] = st["k_cache"], st["v_cache"]
    return out


def _own_verify(st):
    from prefill_kv_shared_gb300 import binding

    if "work" not in st:
        st["work"] = binding.VerifyWork(st["target"].shape[0], len(st["noise"]))
    binding.verify_draft(st["target"], st["tokens"], st["first"], st["u"], st["noise"], st["n_accept"], st["token"],
                         st["p_accept"], st["work"], draft=st["draft"])
    return {k: st[k] for k in ("n_accept", "token", "p_accept")}


def _plain_paged(st):
    """All sequences as one padded batch, their pages gathered."""
    q, k, v, page = st["q"], st["k"], st["v"], st["case"]["page"]
    dev = q.device
    total, hq, hd = q.shape
    hkv = k.shape[2]
    n, past, _ = st["sizes"]
    r, n_max, l_max = len(n), int(max(x[0] for x in st["runs"])), int(max(x[0] + x[1] for x in st["runs"]))
    out = torch.zeros(total, hq, hd, device=dev, dtype=torch.bfloat16)
    i = torch.arange(n_max, device=dev)
    j = torch.arange(l_max, device=dev)
    real = i[None, :] < n[:, None]                                      # [r, n_max]
    row = ((torch.cumsum(n, 0) - n)[:, None] + i[None, :])[real]        # packed row of each real (r, i)
    qp = torch.zeros(r, n_max, hq, hd, device=dev)
    qp[real] = q[row].float()
    cell = st["table"].long()[:, j // page].clamp(min=0) * page + j % page
    kp, vp = k.view(-1, hkv, hd)[cell].float(), v.view(-1, hkv, hd)[cell].float()   # [r, l_max, hkv, hd]
    qp = qp.view(r, n_max, hkv, hq // hkv, hd).permute(0, 2, 1, 3, 4).reshape(r, hkv, -1, hd)
    s = qp @ kp.permute(0, 2, 3, 1) / math.sqrt(hd)                     # [r, hkv, n_max * group, l_max]
    s = s.view(r, hkv, n_max, -1, l_max)
    if "mask" in st:
        d = j[None, :] - past[:, None]                                  # drafted token at key j
        w = (d.clamp(min=0) // 64).clamp(max=st["mask"].shape[1] - 1)
        words = torch.zeros(r, n_max, st["mask"].shape[1], device=dev, dtype=torch.int64)
        words[real] = st["mask"][row]
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


def _plain_rope(st):
    hd = st["q"].shape[2]
    i = torch.arange(hd // 2, device="cuda", dtype=torch.float64)
    angle = st["pos"].double()[:, None] * ROPE_BASE ** (-2.0 * i / hd)
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turned(x, gain):
        x = x.float()
        if gain is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * (1.0 + gain)
        a, b = x[..., :hd // 2], x[..., hd // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1).to(torch.float16)

    st["q_out"].copy_(turned(st["q"], st["q_gain"]))
    if st["k"] is not None:
        here = st["slots"] >= 0
        at = st["slots"][here].long()
        st["k_cache"].view(-1, *st["k"].shape[1:])[at] = turned(st["k"], st["k_gain"])[here]
        st["v_cache"].view(-1, *st["v"].shape[1:])[at] = st["v"][here].to(torch.float16)
    return _rope_outputs(st)


def _plain_verify(st):
    """Which token is taken hangs on values next to a border: in 64 bits."""
    def softmax(x):
        x = x.double()
        e = torch.exp(x - x.amax(-1, keepdim=True))
        return e / e.sum(-1, keepdim=True)

    n, rows = len(st["noise"]), len(st["tokens"])
    first, d_rows = st["first"].long(), st["d_rows"]
    p = softmax(st["target"])
    token = st["tokens"].long()[d_rows + 1] if len(d_rows) else torch.zeros(0, dtype=torch.long, device="cuda")
    pd = torch.gather(p[d_rows], 1, token[:, None])[:, 0]
    if st["draft"] is not None:
        q = softmax(st["draft"]) if len(d_rows) else st["draft"].double()
        qd = torch.gather(q, 1, token[:, None])[:, 0]
    else:
        q, qd = None, torch.ones_like(pd)
    p_accept = torch.zeros(rows, device="cuda", dtype=torch.float64)
    p_accept[d_rows] = torch.where((pd >= qd) & (pd > 0), torch.ones_like(pd),
                                   pd / torch.where(qd > 0, qd, torch.ones_like(qd)))
    yes = torch.zeros(rows, device="cuda", dtype=torch.bool)
    yes[d_rows] = st["u"].double()[d_rows] * qd < pd
    # a sequence's row of the first refusal, or its last row
    index = torch.arange(rows, device="cuda")
    stop = torch.where(yes, torch.full_like(index, rows), index)
    at = torch.full((n,), rows, device="cuda").scatter_reduce(0, st["seq"], stop, "amin")
    w = p[at]
    refused = at < first[1:] - 1
    d_at = (at - torch.arange(n, device="cuda")).clamp(max=max(0, len(d_rows) - 1))   # its row of the draft's
    if len(d_rows):
        if q is not None:
            less = (w - q[d_at]).clamp(min=0)
        else:
            less = w.scatter(1, token[d_at][:, None], 0.0)
        less = torch.where((less > 0).any(-1, keepdim=True), less, w)
        w = torch.where(refused[:, None], less, w)
    best = (w / st["noise"].double()).argmax(-1)
    return {"n_accept": (at - first[:-1]).to(torch.int32), "token": best.to(torch.int32), "p_accept": p_accept.float()}


# ---------------------------------------------------------------------------
# work and exact values


def work(case):
    if case["op"] == "rope":
        hq, hkv, hd = HEADS[case["heads"]]
        kv = 0 if case["shared"] else hkv
        size = 4 if case["dtype"] == "float32" else 2
        n = case["rows"] * (hq + 2 * kv) * hd
        return {"bytes": n * (size + 2) + case["rows"] * 8, "flops": 8 * n}
    if case["op"] == "verify":
        drafts, vocab = _ints(case["drafts"]), case["vocab"]
        size = 4 if case["dtype"] == "float32" else 2
        rows = sum(drafts) + len(drafts) + (sum(drafts) if case["model"] else 0)
        return {"bytes": rows * vocab * size + len(drafts) * vocab * 4, "flops": 4 * rows * vocab}
    hq, hkv, hd = HEADS[case["heads"]]
    rows, past = _ints(case["rows"]), _ints(case["past"])
    if case["tree"]:
        # a drafted token sees its context, itself and its ancestors: about log2 of the tree's size of them
        pairs = sum(int(n * (p + 1 + math.log(max(1, n)))) for n, p in zip(rows, past))
    else:
        pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(rows, past))
    keys = sum(n + p for n, p in zip(rows, past))
    return {"bytes": sum(rows) * hq * hd * 4 + keys * hkv * hd * 4 + 4 * keys // case["page"],
            "flops": 4 * hd * hq * pairs}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "paged" and work(case)["flops"] > 1e13:
        return None
    return {"paged": _exact_paged, "rope": _exact_rope, "verify": _exact_verify}[case["op"]](st)


def _exact_paged(st):
    """Sequence by sequence and query head by query head, in float64."""
    q, page = st["q"], st["case"]["page"]
    hq, hkv, hd = q.shape[1], st["k"].shape[2], q.shape[2]
    out = torch.zeros(q.shape, device=q.device, dtype=torch.float64)
    row0 = 0
    for r, (n, past, _) in enumerate(st["runs"]):
        pages = st["table"][r, :-(-(n + past) // page)].long()
        ks = st["k"][pages].reshape(-1, hkv, hd)[:n + past]
        vs = st["v"][pages].reshape(-1, hkv, hd)[:n + past]
        for t0 in range(0, n, 1024):
            t1 = min(n, t0 + 1024)
            if "mask" in st:
                words = st["mask"][row0 + t0:row0 + t1].cpu().numpy().view(np.uint64)
                bits = np.unpackbits(words.astype("<u8").view(np.uint8), axis=1, bitorder="little")[:, :n]
                vis = torch.ones(t1 - t0, n + past, dtype=torch.bool, device=q.device)
                vis[:, past:] = torch.from_numpy(bits.astype(bool)).to(q.device)
            else:
                vis = torch.arange(n + past, device=q.device) <= past + torch.arange(t0, t1, device=q.device)[:, None]
            for h in range(hq):
                a = q[row0 + t0:row0 + t1, h].double() @ ks[:, h * hkv // hq].double().T * hd ** -0.5
                a = a.masked_fill(~vis, -math.inf).softmax(-1)
                out[row0 + t0:row0 + t1, h] = torch.nan_to_num(a) @ vs[:, h * hkv // hq].double()
        row0 += n
    return out


def _exact_rope(st):
    """The rotation as a product of complex numbers."""
    hd = st["q"].shape[2]
    turn = torch.exp(torch.arange(hd // 2, device="cuda", dtype=torch.float64) * (-2.0 * math.log(ROPE_BASE) / hd))
    angle = torch.outer(st["pos"].double(), turn)
    unit = torch.polar(torch.ones_like(angle), angle)[:, None, :]

    def turned(x, gain):
        y = x.double()
        if gain is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * (1.0 + gain.double())
        z = torch.complex(y[..., :hd // 2].contiguous(), y[..., hd // 2:].contiguous()) * unit
        return torch.cat([z.real, z.imag], -1)

    out = {"q": turned(st["q"], st["q_gain"])}
    if st["k"] is not None:
        heads = st["k"].shape[1:]
        for name, rows in (("k_cache", turned(st["k"], st["k_gain"])), ("v_cache", st["v"].double())):
            cells = st[name].double().reshape(-1, *heads)
            for at in range(0, len(rows), 4096):
                here = (st["slots"][at:at + 4096] >= 0).nonzero()[:, 0]
                cells[st["slots"][at:at + 4096][here].long()] = rows[at:at + 4096][here]
            out[name] = cells.view(st[name].shape)
    return out


def _exact_verify(st):
    """Sequence by sequence, token by token, in float64."""
    drafts = _ints(st["case"]["drafts"])
    n_accept, tokens = [], []
    p_accept = torch.zeros(len(st["tokens"]), dtype=torch.float64)
    token_of, u = st["tokens"].tolist(), st["u"].double().tolist()
    d0 = 0
    for s, count in enumerate(drafts):
        r0 = st["host_first"][s]
        p = torch.softmax(st["target"][r0:r0 + count + 1].double(), -1)
        q = torch.softmax(st["draft"][d0:d0 + count].double(), -1) if st["draft"] is not None else None
        d0 += count
        weights, taken, stopped = p[count], count, False
        if count:
            wanted = torch.tensor(token_of[r0 + 1:r0 + 1 + count], device="cuda")[:, None]
            of_p = p[:count].gather(1, wanted)[:, 0].tolist()
            of_q = q.gather(1, wanted)[:, 0].tolist() if q is not None else [1.0] * count
        for i in range(count):
            p_accept[r0 + i] = min(1.0, of_p[i] / of_q[i]) if of_q[i] > 0 else float(of_p[i] > 0)
            if not stopped and not u[r0 + i] * of_q[i] < of_p[i]:
                stopped, taken = True, i
                weights = p[i].clone()
                if q is not None:
                    weights = torch.relu(weights - q[i])
                else:
                    weights[token_of[r0 + i + 1]] = 0.0
                if not bool((weights > 0).any()):
                    weights = p[i]
        n_accept.append(taken)
        tokens.append(int(torch.argmax(weights / st["noise"][s].double())))
    return {"n_accept": torch.tensor(n_accept, dtype=torch.int32, device="cuda"),
            "token": torch.tensor(tokens, dtype=torch.int32, device="cuda"), "p_accept": p_accept.cuda()}
