"""The operators around an Engram layer in a model that serves many requests
and is fine-tuned, as measured cases: the lookup of token embeddings with
scaling and its gradient by sorted tokens, Step 5's product with each
request's low-rank adapter beside the shared W, and the drawing of the next
token with temperature, top-k, top-p and min-p from given random numbers.

With `own` false, run() computes each operator in its plain form from
elementary torch operations; with `own` true it calls the library's entry
points.  Both start from what prepare() returns.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # the sampled tokens of a decode batch back into the first hidden states: latency
        {"name": "embed_decode", "op": "embed", "n": 256, "vocab": 128000, "dim": 1024, "branches": 1, "from": "bf16",
         "to": "bf16"},
        # a prefill of 8 x 4096 tokens, less a ragged tail, into the hidden states of a four-branch model
        {"name": "embed_prefill", "op": "embed", "n": 32763, "vocab": 128000, "dim": 1024, "branches": 4, "from": "bf16",
         "to": "bf16"},
        # the gradient of a small model's table: a short sequence, odd vocabulary
        {"name": "grad_small", "op": "grad", "n": 509, "vocab": 32001, "dim": 256, "branches": 1, "from": "f32", "to": "f32"},
        # one hashed table of an Engram layer (64 columns, 646,400 rows) after a sequence of 4096 tokens
        {"name": "grad_hashed_table", "op": "grad", "n": 4096, "vocab": 646400, "dim": 64, "branches": 1, "from": "bf16",
         "to": "f32"},
        # the vocabulary's table after a training batch of 8 x 4096 tokens, four branches' gradients joined
        {"name": "grad_batch", "op": "grad", "n": 32763, "vocab": 128000, "dim": 1024, "branches": 4, "from": "bf16",
         "to": "f32"},
        # one sequence decoding with its adapter: reads W once, latency
        {"name": "adapt_one", "op": "adapt", "n": 1, "cols": 1024, "out": 2048, "rank": 16, "adapters": 4, "per": 1,
         "from": "bf16", "to": "f32"},
        # a decode batch of 256 requests over 64 adapters in a four-branch layer
        {"name": "adapt_decode", "op": "adapt", "n": 256, "cols": 1024, "out": 5120, "rank": 16, "adapters": 64, "per": 1,
         "from": "bf16", "to": "f32"},
        # a float32 layer of the small test configuration's kind: four requests' prompts
        {"name": "adapt_f32", "op": "adapt", "n": 251, "cols": 512, "out": 1024, "rank": 8, "adapters": 3, "per": 64,
         "from": "f32", "to": "f32"},
        # eight requests' prompts of 4096 tokens, less a ragged tail, each with its own adapter
        {"name": "adapt_prefill", "op": "adapt", "n": 32763, "cols": 1024, "out": 5120, "rank": 32, "adapters": 16,
         "per": 4096, "from": "bf16", "to": "bf16"},
        # one sequence's next token, odd vocabulary: latency
        {"name": "sample_one", "op": "sample", "seqs": 1, "per": 1, "vocab": 32001, "from": "f32", "filters": "kpm",
         "greedy": 0.0, "masked": 0.01},
        # a decode batch of 256 requests, each with settings of its own, some of them greedy
        {"name": "sample_batch", "op": "sample", "seqs": 256, "per": 1, "vocab": 128000, "from": "bf16", "filters": "mixed",
         "greedy": 0.1, "masked": 0.01},
        # chunks of 8 rows of 256 sequences (a draft model's proposals), nucleus sampling alone
        {"name": "sample_chunks", "op": "sample", "seqs": 256, "per": 8, "vocab": 128000, "from": "bf16", "filters": "p",
         "greedy": 0.0, "masked": 0.0},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["embed", "grad", "grad", "adapt", "adapt", "adapt", "sample", "sample", "sample"])
    if op in ("embed", "grad"):
        c = {"op": op, "n": _log(rng, 1, 32768), "vocab": _log(rng, 1000, 128000), "dim": 8 * _log(rng, 4, 160),
             "branches": rng.randint(1, 4), "from": rng.choice(["f32", "bf16"]),
             "to": rng.choice(["f32", "bf16"])}
        while c["n"] * c["dim"] * c["branches"] * (2 if c["from"] == "f32" or c["to"] == "f32" else 1) > 32763 * 1024 * 4:
            c["n"] //= 2
        while op == "grad" and c["vocab"] * c["dim"] > 128000 * 1024:
            c["vocab"] //= 2
        return c
    if op == "adapt":
        c = {"op": op, "n": _log(rng, 1, 32768), "cols": 64 * _log(rng, 2, 32), "out": 64 * _log(rng, 2, 80),
             "rank": 8 * rng.randint(1, 8), "adapters": _log(rng, 1, 64), "per": rng.choice([1, 1, 7, 256, 4096]),
             "from": "bf16", "to": rng.choice(["f32", "bf16"])}
        if rng.random() < 0.2:
            c["from"] = c["to"] = "f32"
            c["n"] = min(c["n"], 1024)
            c["cols"] = min(c["cols"], 1024)
        while c["n"] * c["out"] * (4 if c["to"] == "f32" else 2) > 32763 * 5120 * 2 or \
                c["n"] * c["out"] * c["cols"] > 32763 * 5120 * 1024:
            c["n"] //= 2
        return c
    return {"op": op, "seqs": _log(rng, 1, 256), "per": rng.choice([1, 1, 2, 5, 8]), "vocab": _log(rng, 1000, 128000),
            "from": rng.choice(["f32", "bf16"]), "filters": rng.choice(["none", "k", "p", "m", "kpm", "mixed"]),
            "greedy": rng.choice([0.0, 0.2]), "masked": rng.choice([0.0, 0.5])}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    return {"embed": _prepare_embed, "grad": _prepare_grad, "adapt": _prepare_adapt,
            "sample": _prepare_sample}[case["op"]](case, g)


def _tokens(c, g):
    """Tokens by Zipf's law over a shuffled vocabulary, one in a hundred a
    padding id (-1)."""
    u = _uniform(g, c["n"]).double()
    rank = (torch.exp(u * math.log(c["vocab"] + 1.0)).long() - 1).clamp(0, c["vocab"] - 1)
    ids = torch.randperm(c["vocab"], generator=g, device=DEV)[rank]
    return torch.where(_uniform(g, c["n"]) < 0.01, -1, ids).to(torch.int32)


def _prepare_embed(c, g):
    table = torch.empty(c["vocab"], c["dim"], device=DEV, dtype=TYPES[c["from"]])
    table.copy_(_normal(g, c["vocab"], c["dim"]) / c["dim"] ** 0.5)
    return {"op": "embed", "ids": _tokens(c, g), "table": table, "scale": c["dim"] ** 0.5, "branches": c["branches"],
            "to": c["to"]}


def _prepare_grad(c, g):
    # gradients differ in size from token to token
    d = _normal(g, c["n"], c["branches"], c["dim"]) * torch.exp(_normal(g, c["n"], 1, 1)) * 1e-3
    return {"op": "grad", "ids": _tokens(c, g), "dout": d.to(TYPES[c["from"]]), "vocab": c["vocab"],
            "scale": c["dim"] ** 0.5, "to": c["to"]}


def _prepare_adapt(c, g):
    n, k, o, r, a = c["n"], c["cols"], c["out"], c["rank"], c["adapters"]
    dt = TYPES[c["from"]]
    s = {"op": "adapt", "per": c["per"], "to": c["to"],
         "e": _normal(g, n, k).to(dt), "w": (_normal(g, o, k) / k ** 0.5).to(dt),
         "a": (_normal(g, a, r, k) / k ** 0.5).to(dt), "b": (0.3 * _normal(g, a, o, r) / r ** 0.5).to(dt),
         "scale": 0.5 + 1.5 * _uniform(g, a)}
    seqs = (n + c["per"] - 1) // c["per"]
    which = torch.randint(0, a, (seqs,), generator=g, device=DEV)
    if seqs > 1:   # some requests have no adapter
        which = torch.where(_uniform(g, seqs) < 0.1, -1, which)
    s["which"] = which.to(torch.int32)
    if own:
        from hashed_gram_embedding_amd import engram as eg
        s["adapters"] = eg.Adapters(s["a"], s["b"], s["scale"])
    return s


def _prepare_sample(c, g):
    rows, seqs = c["seqs"] * c["per"], c["seqs"]
    logits = torch.empty(rows, c["vocab"], device=DEV, dtype=TYPES[c["from"]])
    for i in range(0, rows, 256):
        x = 3.0 * _normal(g, min(256, rows - i), c["vocab"])
        if c["masked"]:
            x = torch.where(_uniform(g, *x.shape) < c["masked"], float("-inf"), x)
        logits[i:i + 256] = x.to(logits.dtype)
    t = 0.5 + _uniform(g, seqs)
    t = torch.where(_uniform(g, seqs) < c["greedy"], 0.0, t)
    k = torch.randint(1, 201, (seqs,), generator=g, device=DEV)
    p = 0.5 + 0.5 * _uniform(g, seqs)
    m = 0.2 * _uniform(g, seqs)
    f = c["filters"]
    if f == "mixed":   # each request switches each filter on or off
        k = torch.where(_uniform(g, seqs) < 0.5, 0, k)
        p = torch.where(_uniform(g, seqs) < 0.5, 1.0, p)
        m = torch.where(_uniform(g, seqs) < 0.5, 0.0, m)
        f = "kpm"
    return {"op": "sample", "logits": logits.view(seqs, c["per"], c["vocab"]), "temperature": t,
            "top_k": k.to(torch.int32) if "k" in f else None, "top_p": p if "p" in f else None,
            "min_p": m if "m" in f else None, "u": _uniform(g, seqs, c["per"])}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    return {"embed": _run_embed, "grad": _run_grad, "adapt": _run_adapt, "sample": _run_sample}[state["op"]](state)


def _run_embed(s):
    if own:
        from hashed_gram_embedding_amd import engram as eg
        return eg.embed(s["ids"], s["table"], scale=s["scale"], branches=s["branches"], out_dtype=s["to"])
    ids = s["ids"].long()
    x = s["table"][ids.clamp(min=0)].float() * s["scale"]
    x = torch.where((ids >= 0)[:, None], x, 0.0).to(TYPES[s["to"]])
    return x[:, None].expand(-1, s["branches"], -1).contiguous()


def _run_grad(s):
    if own:
        from hashed_gram_embedding_amd import engram as eg
        return eg.embed_backward(s["ids"], s["dout"], s["vocab"], scale=s["scale"], out_dtype=s["to"])
    ids = s["ids"].long()
    d = s["dout"].float().sum(1) * s["scale"]
    d = torch.where((ids >= 0)[:, None], d, 0.0)
    out = torch.zeros(s["vocab"], d.shape[1], device=d.device)
    return out.index_add_(0, ids.clamp(min=0), d).to(TYPES[s["to"]])


def _run_adapt(s):
    if own:
        from hashed_gram_embedding_amd import engram as eg
        return eg.project_adapted(s["e"], s["w"], s["adapters"], s["which"], per=s["per"], out_dtype=s["to"])
    e, n = s["e"].float(), s["e"].shape[0]
    a, b = s["a"].float(), s["b"].float()
    na, r, k = a.shape
    which = s["which"].long()[torch.arange(n, device=e.device) // s["per"]]
    mine = (which[:, None] == torch.arange(na, device=e.device)).float() * s["scale"]     # [n, adapters]
    h = (e @ a.reshape(na * r, k).t()).view(n, na, r) * mine[..., None]
    out = e @ s["w"].float().t() + h.reshape(n, na * r) @ b.transpose(1, 2).reshape(na * r, -1)
    return out.to(TYPES[s["to"]])


def _run_sample(s):
    if own:
        from hashed_gram_embedding_amd import engram as eg
        return eg.sample_tokens(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                                min_p=s["min_p"], want_logprob=True)
    x, t = s["logits"].double(), s["temperature"].double()[:, None, None]
    v = x.shape[-1]
    x, order = x.sort(dim=-1, descending=True, stable=True)   # ties: the lowest index first
    e = torch.exp((x - x[..., :1]) / torch.where(t > 0, t, 1.0))
    at = torch.arange(v, device=x.device)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None, None]
        e = torch.where((k <= 0) | (at < k), e, 0.0)
    keep = e > 0
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None, None]
        c = e.cumsum(-1)
        before = torch.cat([torch.zeros_like(c[..., :1]), c[..., :-1]], -1)
        keep &= (p >= 1) | (before < p * c[..., -1:])
    if s["min_p"] is not None:
        keep &= e >= s["min_p"].double()[:, None, None]
    keep &= (t > 0) | (at == 0)
    e = torch.where(keep, e, 0.0)
    w = torch.zeros_like(e).scatter_(-1, order, e)        # back in the vocabulary's order
    c = w.cumsum(-1)
    total = c[..., -1:]
    token = torch.searchsorted(c, s["u"].double()[..., None] * total, right=True)
    logprob = torch.log(w.gather(-1, token) / total)
    return token[..., 0].to(torch.int32), logprob[..., 0].float()


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c = case
    size = {"f32": 4, "bf16": 2}
    if c["op"] == "embed":
        # rows of tokens that come again are read once: so many differ on average
        v = np.arange(c["vocab"])
        share = 0.99 * np.log((v + 2.0) / (v + 1.0)) / math.log(c["vocab"] + 1.0)
        differ = float((1.0 - (1.0 - share) ** c["n"]).sum())
        return {"bytes": 4 * c["n"] + differ * c["dim"] * size[c["from"]] + c["n"] * c["branches"] * c["dim"] * size[c["to"]],
                "flops": c["n"] * c["dim"]}
    if c["op"] == "grad":
        d = c["n"] * c["branches"] * c["dim"]
        return {"bytes": 4 * c["n"] + d * size[c["from"]] + c["vocab"] * c["dim"] * size[c["to"]], "flops": 2 * d}
    if c["op"] == "adapt":
        n, k, o, r = c["n"], c["cols"], c["out"], c["rank"]
        seqs = (n + c["per"] - 1) // c["per"]
        used = c["adapters"] * (1 - (1 - 1 / c["adapters"]) ** seqs)
        return {"bytes": (n * k + o * k + used * r * (k + o)) * size[c["from"]] + n * o * size[c["to"]],
                "flops": 2 * n * k * o + 2 * n * r * (k + o)}
    n = c["seqs"] * c["per"] * c["vocab"]
    return {"bytes": n * size[c["from"]] + 20 * c["seqs"] * c["per"], "flops": 3 * n}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embed":
        out = torch.zeros(case["n"], case["branches"], case["dim"], dtype=torch.float64, device=DEV)
        has = torch.nonzero(s["ids"] >= 0)[:, 0]
        out[has] = (s["table"].double() * s["scale"]).index_select(0, s["ids"][has].long())[:, None]
        return out
    if case["op"] == "grad":
        ids = s["ids"].long()
        has = torch.nonzero(ids >= 0)[:, 0]
        out = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device=DEV)
        for part in has.split(4096):
            out.index_put_((ids[part],), s["dout"][part].double().sum(1), accumulate=True)
        return out.mul_(s["scale"])
    if case["op"] == "adapt":
        e, w = s["e"].double(), s["w"].double()
        out = e @ w.t()
        which = s["which"].cpu().numpy()
        owner = which[np.arange(case["n"]) // case["per"]]
        for i in np.unique(owner):
            if i < 0:
                continue
            rows = torch.from_numpy(np.nonzero(owner == i)[0]).to(DEV)
            h = e[rows] @ s["a"][i].double().t()
            out[rows] += float(s["scale"][i]) * (h @ s["b"][i].double().t())
        return out
    seqs, per, v = s["logits"].shape
    tokens = torch.empty(seqs, per, dtype=torch.int32, device=DEV)
    logprob = torch.empty(seqs, per, dtype=torch.float64, device=DEV)
    for i in range(seqs):
        t = float(s["temperature"][i])
        for j in range(per):
            x = s["logits"][i, j].double()
            if t <= 0:
                tokens[i, j] = int(torch.nonzero(x == x.max())[0, 0])
                logprob[i, j] = 0.0
                continue
            w = torch.softmax(x / t, 0)
            by = torch.argsort(x, descending=True, stable=True)
            kept = v
            if s["top_k"] is not None and int(s["top_k"][i]) > 0:
                kept = min(v, int(s["top_k"][i]))
            inside = w[by[:kept]]
            if s["min_p"] is not None:
                kept = min(kept, int((inside >= float(s["min_p"][i]) * inside[0]).sum()))
            if s["top_p"] is not None and float(s["top_p"][i]) < 1:
                run_ = inside.cumsum(0)
                kept = min(kept, 1 + int((run_ < float(s["top_p"][i]) * run_[-1]).sum()))
            chosen = by[:kept].sort()[0]
            run_ = w[chosen].cumsum(0)
            pick = int((run_ <= float(s["u"][i, j]) * run_[-1]).sum())
            tokens[i, j] = chosen[pick].to(torch.int32)
            logprob[i, j] = torch.log(w[chosen[pick]] / run_[-1])
    return tokens, logprob
