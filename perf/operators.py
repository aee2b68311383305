"""The operators of a speculative decode step next to an Engram layer, as
measured cases: the product in 8-bit integers (of float rows, quantised per
token on the way, or of codes at hand), token probabilities from logits, the
verification of drafted tokens, and the commit of a drafted chunk into a
layer's decode state.

With `own` false, run() computes each operator in its plain form from
elementary torch operations; with `own` true it calls the library's entry
points.  Both start from what prepare() returns.
"""
from types import SimpleNamespace

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SPAN_OF = {"w4": (4, 3), "w3": (3, 2), "w2": (2, 1)}   # conv taps, dilation


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one sequence decoding: its final hidden state against the whole vocabulary, bound by reading W
        {"name": "product_one_token_vocab", "op": "product", "rows": 1, "cols": 1024, "out": 128000,
         "from": "bf16", "to": "f32"},
        # Step 5 of a decode batch of 256 sequences (W_V and W_K of one branch): a few microseconds of work
        {"name": "product_decode_step5", "op": "product", "rows": 256, "cols": 1024, "out": 2048,
         "from": "bf16", "to": "bf16"},
        # Step 5 of the four-branch layer over 8 x 4096 tokens, less a ragged tail; codes at hand
        {"name": "product_prefill_step5", "op": "product", "rows": 32763, "cols": 1024, "out": 5120,
         "from": "i8", "to": "bf16"},
        # the vocabulary product of the drafted chunks of 256 sequences, 7 tokens on average
        {"name": "product_draft_vocab", "op": "product", "rows": 1795, "cols": 1024, "out": 128000,
         "from": "bf16", "to": "bf16"},
        # the probabilities of one sequence's chunk, odd vocabulary
        {"name": "probs_one_chunk", "op": "probs", "seqs": 1, "per": 5, "vocab": 32001, "from": "f32",
         "greedy": 0.0, "masked": 0.01},
        # the probabilities of 256 sequences' chunks of 8, some of them greedy
        {"name": "probs_batch", "op": "probs", "seqs": 256, "per": 8, "vocab": 128000, "from": "bf16",
         "greedy": 0.1, "masked": 0.01},
        # one sequence with 4 drafts: two passes over one short row, latency
        {"name": "verify_one", "op": "verify", "seqs": 1, "drafts": 4, "vocab": 32001, "from": "f32",
         "sampled": True, "ragged": False},
        # 48 sequences whose drafts come from a lookup (no draft probabilities), ragged
        {"name": "verify_lookup", "op": "verify", "seqs": 48, "drafts": 5, "vocab": 98561, "from": "f32",
         "sampled": False, "ragged": True},
        # 256 sequences with up to 7 sampled drafts each
        {"name": "verify_batch", "op": "verify", "seqs": 256, "drafts": 7, "vocab": 128000, "from": "f32",
         "sampled": True, "ragged": True},
        # one sequence's chunk into a single-branch layer's state
        {"name": "commit_one", "op": "commit", "seqs": 1, "chunk": 5, "d": 1024, "branches": 1, "conv": "w4"},
        # 256 sequences' chunks of 8 into a four-branch layer's state
        {"name": "commit_batch", "op": "commit", "seqs": 256, "chunk": 8, "d": 1024, "branches": 4, "conv": "w4"},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["product", "product", "probs", "verify", "verify", "commit"])
    if op == "product":
        c = {"op": op, "rows": _log(rng, 1, 32768), "cols": _log(rng, 48, 4096), "out": _log(rng, 64, 128000),
             "from": rng.choice(["bf16", "f32", "i8"]), "to": rng.choice(["bf16", "f32"])}
        if rng.random() < 0.5:
            c["cols"] = max(64, c["cols"] // 64 * 64)
        while c["rows"] * c["cols"] * c["out"] > 1795 * 1024 * 128000 or c["rows"] * c["out"] > 1795 * 128000:
            c["rows"] = max(1, c["rows"] // 2)
        return c
    if op == "probs":
        c = {"op": op, "seqs": _log(rng, 1, 256), "per": rng.randint(1, 8), "vocab": _log(rng, 1000, 128000),
             "from": rng.choice(["bf16", "f32"]), "greedy": rng.choice([0.0, 0.2]), "masked": rng.choice([0.0, 0.5])}
        return c
    if op == "verify":
        return {"op": op, "seqs": _log(rng, 1, 256), "drafts": rng.randint(1, 7), "vocab": _log(rng, 1000, 128000),
                "from": rng.choice(["f32", "f32", "bf16"]), "sampled": rng.random() < 0.6, "ragged": rng.random() < 0.5}
    return {"op": op, "seqs": _log(rng, 1, 256), "chunk": rng.randint(1, 12), "d": 64 * _log(rng, 1, 24),
            "branches": rng.randint(1, 4), "conv": rng.choice(["w4", "w4", "w3", "w2"])}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _softmax(x):
    return torch.softmax(x, -1)   # of inputs being made, not of an operator


def prepare(case, seed):
    g = _gen(seed)
    return {"product": _prepare_product, "probs": _prepare_probs, "verify": _prepare_verify,
            "commit": _prepare_commit}[case["op"]](case, g)


def _prepare_product(c, g):
    n, k, o = c["rows"], c["cols"], c["out"]
    # hidden states differ in size from token to token; rows of W are near one another in size
    x = _normal(g, n, k) * torch.exp(_normal(g, n, 1))
    w = _normal(g, o, k)
    ws = w.abs().amax(1) / 127.0
    wq = torch.round(w / ws[:, None]).clamp(-127, 127).to(torch.int8)
    s = {"op": "product", "to": c["to"], "w": wq, "w_scale": ws / k ** 0.5}
    if c["from"] == "i8":
        xs = x.abs().amax(1) / 127.0
        s["x"] = torch.round(x / xs[:, None]).clamp(-127, 127).to(torch.int8)
        s["x_scale"] = xs
    else:
        s["x"] = x.to(TYPES[c["from"]])
        s["x_scale"] = None
    return s


def _prepare_probs(c, g):
    rows = c["seqs"] * c["per"]
    logits = torch.empty(rows, c["vocab"], device=DEV, dtype=TYPES[c["from"]])
    for i in range(0, rows, 256):
        x = 3.0 * _normal(g, min(256, rows - i), c["vocab"])
        if c["masked"]:
            x = torch.where(torch.rand(x.shape, generator=g, device=DEV) < c["masked"], float("-inf"), x)
        logits[i:i + 256] = x.to(logits.dtype)
    t = 0.5 + torch.rand(c["seqs"], generator=g, device=DEV)
    t = torch.where(torch.rand(c["seqs"], generator=g, device=DEV) < c["greedy"], 0.0, t)
    return {"op": "probs", "logits": logits.view(c["seqs"], c["per"], c["vocab"]), "temperature": t}


def _prepare_verify(c, g):
    s_, n, v, dt = c["seqs"], c["drafts"], c["vocab"], TYPES[c["from"]]
    target = torch.empty(s_, n + 1, v, device=DEV, dtype=dt)
    draft = torch.empty(s_, n, v, device=DEV, dtype=dt) if c["sampled"] else None
    drafted = torch.empty(s_, n, device=DEV, dtype=torch.int32)
    step = max(1, (1 << 25) // ((n + 1) * v))
    for i in range(0, s_, step):
        m = min(step, s_ - i)
        x = 2.5 * _normal(g, m, n + 1, v)
        p = _softmax(x)
        target[i:i + m] = p.to(dt)
        # the draft model is near the target; a lookup proposes one of the likelier tokens
        q = _softmax(x[:, :n] + 0.5 * _normal(g, m, n, v))
        if draft is not None:
            draft[i:i + m] = q.to(dt)
            pick = torch.rand(m, n, 1, generator=g, device=DEV, dtype=torch.float64)
            c_ = q.double().cumsum(-1)
            drafted[i:i + m] = torch.searchsorted(c_, pick * c_[..., -1:]).clamp(max=v - 1)[..., 0].to(torch.int32)
        else:
            drafted[i:i + m] = q.argmax(-1).to(torch.int32)
    if draft is None:
        # a lookup is right more often than a single token's probability says
        u = torch.rand(s_, n, generator=g, device=DEV) * 0.02
    else:
        u = torch.rand(s_, n, generator=g, device=DEV)
    count = torch.randint(0, n + 1, (s_,), generator=g, device=DEV, dtype=torch.int32) if c["ragged"] else None
    return {"op": "verify", "target": target, "draft": draft, "drafted": drafted, "n_draft": count, "u_accept": u,
            "u_sample": torch.rand(s_, generator=g, device=DEV)}


def _prepare_commit(c, g):
    b, t, d, m = c["seqs"], c["chunk"], c["d"], c["branches"]
    w, dil = SPAN_OF[c["conv"]]
    span, vocab, vocab_c, max_n = (w - 1) * dil, 128000, 98560, 3
    proj = torch.randint(0, vocab_c, (vocab,), generator=g, device=DEV, dtype=torch.int32)
    s = {"op": "commit", "span": span, "proj": proj,
         "tokens": torch.randint(0, vocab, (b, t), generator=g, device=DEV, dtype=torch.int32),
         "v": _normal(g, b * t, d), "gamma": torch.rand(b * t, m, generator=g, device=DEV),
         "n_accepted": torch.randint(0, t, (b,), generator=g, device=DEV, dtype=torch.int32),
         "ids0": torch.randint(0, vocab_c, (b, max_n - 1), generator=g, device=DEV, dtype=torch.int32),
         "pos0": torch.randint(0, 100000, (b,), generator=g, device=DEV, dtype=torch.int32),
         "conv": _normal(g, b, m, span, d)}
    if own:
        from hashed_gram_embedding_amd import engram as eg
        # the layer as its descriptors say it is, with tables of the smallest size
        primes = np.array([2, 3], dtype=np.uint32)
        hp = SimpleNamespace(vocab=vocab, vocab_c=vocab_c, max_n=max_n, heads=1, proj=proj.cpu().numpy(),
                             mult=np.ones((max_n - 1, 1, max_n), dtype=np.uint64), prime=primes)
        dim = 32
        tab = SimpleNamespace(row_offset=np.array([0, 2]), n_rows=primes.astype(np.int64), total_rows=5, dim=dim,
                              dtype="bf16", rows=np.zeros((5, dim), dtype=np.uint16), scale=None)
        li = SimpleNamespace(hash=hp, tables=tab, w=np.zeros(((1 + m) * d, 2 * dim), dtype=np.uint16),
                             conv_w=np.zeros((m, d, w), dtype=np.float32), d=d, branches=m, kernel_w=w, dilation=dil,
                             eps=1e-6)
        s["layer"] = eg.Layer(li, "bf16", DEV)
        s["state"] = eg.DecodeState(b, max_n, m, span, d, DEV)
        s["state"].conv.copy_(s["conv"])
        s["chunk"] = eg.Draft(b, t, s["layer"], DEV, v=s["v"], gamma=s["gamma"])
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    return {"product": _run_product, "probs": _run_probs, "verify": _run_verify, "commit": _run_commit}[state["op"]](state)


def _run_product(s):
    if own:
        from hashed_gram_embedding_amd import engram as eg
        return eg.project_i8(s["x"], s["w"], s["w_scale"], e_scale=s["x_scale"], out_dtype=s["to"])
    if s["x_scale"] is None:
        # codes are the nearest whole numbers of 127 x / max |x| (ties to even): next to a border 32 bits are not enough
        x = s["x"].double()
        top = x.abs().amax(1, keepdim=True)
        q = torch.where(top > 0, torch.round(x * 127.0 / top), 0.0).float()
        xs = s["x"].float().abs().amax(1) / 127.0
    else:
        q, xs = s["x"].float(), s["x_scale"]
    return ((q @ s["w"].float().t()) * xs[:, None] * s["w_scale"][None, :]).to(TYPES[s["to"]])


def _run_probs(s):
    if own:
        from hashed_gram_embedding_amd import engram as eg
        return eg.token_probs(s["logits"], s["temperature"])
    x = s["logits"].float()
    t = s["temperature"][:, None, None]
    top = x.amax(-1, keepdim=True)
    e = torch.exp((x - top) / torch.where(t > 0, t, 1.0))
    p = torch.where(top == float("-inf"), 0.0, e / e.sum(-1, keepdim=True))
    at = torch.arange(x.shape[-1], device=x.device)
    first = torch.where(x == top, at, x.shape[-1]).amin(-1, keepdim=True)   # the lowest index of the largest logit
    one = ((at == first) & (top > float("-inf"))).float()
    return torch.where(t > 0, p, one)


def _run_verify(s):
    if own:
        from hashed_gram_embedding_amd import engram as eg
        return eg.verify_drafts(s["target"], s["draft"], s["drafted"], s["u_accept"], s["u_sample"],
                                n_draft=s["n_draft"])
    p, q, x = s["target"], s["draft"], s["drafted"].long()
    b, n = x.shape
    count = torch.full((b,), n, device=x.device) if s["n_draft"] is None else s["n_draft"].long()
    px = p[:, :n].gather(2, x[..., None])[..., 0].double()
    qx = torch.ones_like(px) if q is None else q.gather(2, x[..., None])[..., 0].double()
    slots = torch.arange(n, device=x.device)
    ok = (s["u_accept"].double() * qx < px) & (slots < count[:, None])
    a = ok.long().cumprod(1).sum(1)                       # drafts accepted before the first refusal
    each = torch.arange(b, device=x.device)
    row = p[each, a].double()                             # the row that the next token is drawn from
    refused = a < count
    at = a.clamp(max=n - 1)
    if q is None:
        rest = row.scatter(1, x[each, at][:, None], 0.0)
    else:
        rest = (row - q[each, at].double()).clamp(min=0.0)
    rest = torch.where((refused & (rest.sum(1) > 0))[:, None], rest, row)
    c = rest.cumsum(1)
    picked = torch.searchsorted(c, s["u_sample"].double()[:, None] * c[:, -1:], right=True)[:, 0]
    out = torch.full((b, n + 1), -1, dtype=torch.int32, device=x.device)
    out[:, :n] = torch.where(slots < a[:, None], x, -1).to(torch.int32)
    out.scatter_(1, a[:, None], picked[:, None].to(torch.int32))
    return out, a.to(torch.int32)


def _run_commit(s):
    if own:
        from hashed_gram_embedding_amd import engram as eg
        st = s["state"]
        st.ids.copy_(s["ids0"])   # the state as it was before the chunk
        st.pos.copy_(s["pos0"])
        eg.commit_draft(s["tokens"], s["layer"], s["chunk"], s["n_accepted"], st)
        return st.ids, st.conv, st.pos
    b, t = s["tokens"].shape
    conv, span = s["conv"], s["span"]
    m, d = conv.shape[1], conv.shape[3]
    keep = (s["n_accepted"].long() + 1).clamp(0, t)
    pos0 = s["pos0"].long()
    last = (pos0 + keep - 1)[:, None]
    slot = torch.arange(span, device=conv.device)[None]
    at = last - (last - slot) % span - pos0[:, None]      # the chunk's token that belongs in each slot, if >= 0
    each = torch.arange(b, device=conv.device)[:, None]
    tok = at.clamp(min=0)
    u = s["v"].view(b, t, d)[each, tok][:, None] * s["gamma"].view(b, t, m)[each, tok].transpose(1, 2)[..., None]
    new = torch.where((at >= 0)[:, None, :, None], u, conv)
    known = torch.cat([s["ids0"], s["proj"][s["tokens"].long()]], 1)
    n1 = s["ids0"].shape[1]
    ids = known.gather(1, keep[:, None] + torch.arange(n1, device=conv.device)[None])
    return ids, new, (pos0 + keep).to(torch.int32)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "i8": 1}
    if c["op"] == "product":
        n, k, o = c["rows"], c["cols"], c["out"]
        return {"bytes": n * k * size[c["from"]] + o * k + 4 * o + n * o * size[c["to"]], "flops": 2 * n * k * o}
    if c["op"] == "probs":
        n = c["seqs"] * c["per"] * c["vocab"]
        return {"bytes": n * (size[c["from"]] + 4), "flops": 4 * n}
    if c["op"] == "verify":
        # one row of the target for each sequence, and the draft's where a draft is refused
        rows = c["seqs"] * (1.8 if c["sampled"] else 1.0)
        return {"bytes": rows * c["vocab"] * size[c["from"]], "flops": 2 * rows * c["vocab"]}
    w, dil = SPAN_OF[c["conv"]]
    kept = c["seqs"] * min((c["chunk"] + 1) / 2, (w - 1) * dil)
    return {"bytes": kept * c["d"] * 4 * (1 + c["branches"]) + 32 * c["seqs"], "flops": kept * c["d"] * c["branches"]}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "product":
        x, w, sw = s["x"].double(), s["w"].double(), s["w_scale"].double()
        if s["x_scale"] is None:
            big = torch.linalg.vector_norm(x, float("inf"), dim=1, keepdim=True)
            code = torch.round(127.0 * x / big)
            code[big[:, 0] == 0] = 0
            return (code @ w.t()) * (big / 127.0) * sw
        return (x @ w.t()) * s["x_scale"].double()[:, None] * sw
    if case["op"] == "probs":
        out = torch.empty(s["logits"].shape, dtype=torch.float64, device=DEV)
        for i in range(case["seqs"]):
            x, t = s["logits"][i].double(), float(s["temperature"][i])
            for j in range(case["per"]):
                if t > 0:
                    out[i, j] = torch.exp(x[j] / t - torch.logsumexp(x[j] / t, 0))
                else:
                    out[i, j] = 0
                    out[i, j, int(torch.nonzero(x[j] == x[j].max())[0, 0])] = 1
        return out
    if case["op"] == "verify":
        b, n = case["seqs"], case["drafts"]
        xs, us, vs = s["drafted"].cpu().numpy(), s["u_accept"].double().cpu().numpy(), s["u_sample"].double().cpu().numpy()
        out, acc = np.full((b, n + 1), -1, dtype=np.int32), np.zeros(b, dtype=np.int32)
        for i in range(b):
            m = n if s["n_draft"] is None else int(s["n_draft"][i])
            a = 0
            while a < m:
                qx = 1.0 if s["draft"] is None else float(s["draft"][i, a, xs[i, a]])
                if not us[i, a] * qx < float(s["target"][i, a, xs[i, a]]):
                    break
                out[i, a] = xs[i, a]
                a += 1
            r = s["target"][i, a].double().cpu().numpy()
            if a < m:
                left = r.copy()
                if s["draft"] is None:
                    left[xs[i, a]] = 0
                else:
                    left = np.maximum(left - s["draft"][i, a].double().cpu().numpy(), 0)
                r = left if left.sum() > 0 else r
            acc[i] = a
            below = np.cumsum(r)
            out[i, a] = int(np.argmax(below > vs[i] * below[-1]))
        return torch.from_numpy(out).to(DEV), torch.from_numpy(acc).to(DEV)
    ids, conv, pos = s["ids0"].cpu().numpy().copy(), s["conv"].double().cpu().numpy().copy(), s["pos0"].cpu().numpy().copy()
    tok, proj = s["tokens"].cpu().numpy(), s["proj"].cpu().numpy()
    v, gm, acc = s["v"].double().cpu().numpy(), s["gamma"].double().cpu().numpy(), s["n_accepted"].cpu().numpy()
    t = case["chunk"]
    for i in range(case["seqs"]):
        for j in range(min(int(acc[i]) + 1, t)):           # token by token, as it would have been without drafts
            conv[i, :, pos[i] % s["span"]] = gm[i * t + j][:, None] * v[i * t + j][None]
            ids[i] = np.append(ids[i][1:], proj[tok[i, j]])
            pos[i] += 1
    return torch.from_numpy(ids).to(DEV), torch.from_numpy(conv).to(DEV), torch.from_numpy(pos).to(DEV)
