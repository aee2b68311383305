"""GPU: the operators around the layer on more than 2^31 elements, and where a
call takes more than one launch; chosen rows against float64, with the
tolerances of the operators' own tests."""
import numpy as np
import pytest
import torch

import plain_around as plain
from hashed_gram_embedding_amd import engram as eg
from parity import log

pytestmark = pytest.mark.gpu

DEV = "cuda"
UNIT = 2.0 ** -23


def _f64(t):
    return t.double().cpu().numpy()


def test_embed_in_several_launches():
    """A launch takes 2^23 tokens of a row this long."""
    log("embed in several launches")
    n, dim = (1 << 23) + 5, 1032
    table = torch.arange(7, device=DEV).float()[:, None].expand(7, dim).bfloat16().contiguous()
    ids = (torch.arange(n, device=DEV) % 7).int()
    out = eg.embed(ids, table)
    at = torch.tensor([0, 1, (1 << 23) - 1, 1 << 23, (1 << 23) + 1, n - 1], device=DEV)
    assert torch.equal(out[at, 0].float(), (at % 7).float()[:, None].expand(-1, dim))
    assert torch.equal(out[:, 0, 0].float(), ids.float()) and torch.equal(out[:, 0, -1].float(), ids.float())


def test_embed_backward_past_32_bits():
    """A gradient of more than 2^31 elements going in."""
    log("embed_backward past 32 bits")
    n, V, dim = (1 << 18) + 301, 977, 8200
    g = torch.Generator(device=DEV).manual_seed(3)
    ids = torch.randint(-1, V, (n,), generator=g, device=DEV, dtype=torch.int32)
    d = torch.empty(n, 1, dim, dtype=torch.bfloat16, device=DEV)
    for i in range(0, n, 1 << 15):
        d[i:i + (1 << 15)] = torch.randn(d[i:i + (1 << 15)].shape, generator=g, device=DEV)
    assert d.numel() > 1 << 31
    grad = eg.embed_backward(ids, d, V, scale=0.5)
    for v in (0, 1, V // 2, V - 1):
        terms = _f64(d[ids == v][:, 0])
        ref, size = 0.5 * terms.sum(0), 0.5 * np.abs(terms).sum(0)
        assert (np.abs(_f64(grad[v]) - ref) <= (len(terms) + 1) * 2.0 ** -24 * size + 2.0 ** -126).all()


@pytest.mark.parametrize("dtype,n,K,out,out_t", [
    ("bf16", (1 << 20) + 77, 2112, 2176, "bf16"),    # tokens and outputs past 2^31 elements
    ("f32", (1 << 24) + 33, 64, 192, "f32"),         # an adapter of its own for each token; outputs past 2^31
    ("bf16", (1 << 24) + 33, 64, 192, "f32")])
def test_project_adapted_past_32_bits(dtype, n, K, out, out_t):
    log(f"project_adapted past 32 bits {dtype} {n} {K} {out}")
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator(device=DEV).manual_seed(K)
    e = torch.empty(n, K, dtype=dt, device=DEV)
    for i in range(0, n, 1 << 18):
        e[i:i + (1 << 18)] = torch.randn(e[i:i + (1 << 18)].shape, generator=g, device=DEV)
    w = (torch.randn(out, K, generator=g, device=DEV) / K ** 0.5).to(dt)
    ad = eg.Adapters((torch.randn(100, 8, K, generator=g, device=DEV) / K ** 0.5).to(dt), torch.randn(100, out, 8, generator=g, device=DEV).to(dt))
    which = torch.randint(-1, 100, (n,), generator=g, device=DEV, dtype=torch.int32)
    got = eg.project_adapted(e, w, ad, which, out_dtype=out_t)
    rows = torch.tensor([0, 31, 32, (1 << 31) // K, (1 << 31) // K + 1, (1 << 32) // K, (1 << 31) // out, (1 << 31) // out + 1,
                         (1 << 32) // out, n // 2, n - 34, n - 2, n - 1], device=DEV)
    rows = rows[rows < n]
    ref, size, carried = plain.project_adapted(_f64(e[rows]), _f64(w), _f64(ad.a), _f64(ad.b), None, which[rows].cpu().numpy())
    tol = (K + 10) * UNIT * size + (2.0 ** -17 * carried if dtype == "bf16" else 0.0) + (2.0 ** -8 * np.abs(ref) if out_t == "bf16" else 0.0)
    assert (np.abs(_f64(got[rows]) - ref) <= tol).all()


def _check_rows(got, e, w, ad, which, out_t):
    K = e.shape[1]
    ref, size, carried = plain.project_adapted(_f64(e), _f64(w), _f64(ad.a), _f64(ad.b), None, which.cpu().numpy())
    tol = (K + ad.rank + 2) * UNIT * size + 2.0 ** -17 * carried + (2.0 ** -8 * np.abs(ref) if out_t == "bf16" else 0.0)
    assert (np.abs(_f64(got) - ref) <= tol).all()


def test_project_adapted_of_many_tokens():
    """More workgroups than one launch has work-items for: 2^20 tokens again and again, and the first ones once more."""
    log("project_adapted of 2^29 tokens")
    torch.cuda.empty_cache()
    n, again, turns, K = 33, 1 << 20, 512, 64
    g = torch.Generator(device=DEV).manual_seed(29)
    bf16 = torch.bfloat16
    e = torch.empty(turns * again + n, K, dtype=bf16, device=DEV)
    which = torch.empty(turns * again + n, dtype=torch.int32, device=DEV)
    e[:again] = torch.randn(again, K, generator=g, device=DEV)
    which[:again] = torch.randint(-1, 3, (again,), generator=g, device=DEV)
    for t in (e, which):
        t[again:turns * again].view(turns - 1, again, *t.shape[1:]).copy_(t[None, :again])
        t[turns * again:] = t[:n]
    w = (torch.randn(64, K, generator=g, device=DEV) / 8).to(bf16)
    ad = eg.Adapters((torch.randn(3, 8, K, generator=g, device=DEV) / 8).to(bf16), torch.randn(3, 64, 8, generator=g, device=DEV).to(bf16))
    got = eg.project_adapted(e, w, ad, which, out_dtype="bf16")
    rows = torch.arange(0, again, 4099, device=DEV)
    _check_rows(got[rows], e[rows], w, ad, which[rows], "bf16")
    for i in range(1, turns):
        assert torch.equal(got[i * again:(i + 1) * again], got[:again]), i
    assert torch.equal(got[turns * again:], got[:n])


@pytest.mark.parametrize("out_t", ["f32", "bf16"])
def test_project_adapted_of_many_outputs(out_t):
    """2^27 outputs and more of few tokens: rows of W and B again and again."""
    log(f"project_adapted of 2^27 outputs {out_t}")
    torch.cuda.empty_cache()
    more, again, turns, K, n = 64, 1 << 20, 128, 64, 3
    g = torch.Generator(device=DEV).manual_seed(27)
    bf16 = torch.bfloat16
    out = turns * again + more
    w, b = torch.empty(out, K, dtype=bf16, device=DEV), torch.empty(1, out, 8, dtype=bf16, device=DEV)
    for t in (w, b[0]):
        t[:again] = torch.randn(again, t.shape[1], generator=g, device=DEV) / 8
        t[again:turns * again].view(turns - 1, again, -1).copy_(t[None, :again])
        t[turns * again:] = t[:more]
    ad = eg.Adapters((torch.randn(1, 8, K, generator=g, device=DEV) / 8).to(bf16), b)
    e = torch.randn(n, K, generator=g, device=DEV).to(bf16)
    which = torch.tensor([0, -1, 0], dtype=torch.int32, device=DEV)
    got = eg.project_adapted(e, w, ad, which, out_dtype=out_t)
    _check_rows(got[:, :again:4099], e, w[:again:4099], eg.Adapters(ad.a, b[:, :again:4099].contiguous()), which, out_t)
    for i in range(1, turns):
        assert torch.equal(got[:, i * again:(i + 1) * again], got[:, :again]), i
    assert torch.equal(got[:, turns * again:], got[:, :more])


@pytest.mark.parametrize("per", [1, 5, 1 << 20, (1 << 21) + 9])
def test_sample_in_several_launches(per):
    """A launch takes 2^21 rows: more of them, with settings of one row, of a few, and of more rows than a launch's."""
    log(f"sample_tokens in several launches {per}")
    S = 2 if per > 1 << 21 else -(-((1 << 22) + 7) // per)
    rows = S * per
    i = torch.arange(rows, device=DEV)
    x = torch.zeros(rows, 8, dtype=torch.bfloat16, device=DEV)
    x[i, i % 8] = 1.0
    keep = (torch.arange(S, device=DEV) % 3 + 1).int()      # the largest, then the lowest indexes
    u = torch.full((rows,), 0.999, device=DEV)
    tokens, lp = eg.sample_tokens(x.view(S, per, 8), u.view(S, per), top_k=keep, want_logprob=True)
    k = keep.repeat_interleave(per)
    top = i % 8
    last = torch.where(k == 1, top, torch.maximum(top, torch.where(top < k - 1, k - 1, k - 2)))
    assert torch.equal(tokens.view(-1).long(), last)
    weight = torch.where(last == top, torch.e, 1.0).double() / (torch.e + k - 1)
    assert (lp.view(-1).double() - weight.log()).abs().max() <= 2.0 ** -22


@pytest.mark.parametrize("top_p", [-0.125, -0.25, -1.0, -3e38, float("-inf"), 0.0])
def test_sample_negative_top_p_in_a_long_row(top_p):
    """Weights of more than 2^30 entries are multiples of 2^-31, so the largest is 2^31 units: a top_p of 0 and less keeps
    the first entry, whatever the low bits of top_p times the total are."""
    log(f"sample_tokens long row, top_p {top_p}")
    V = (1 << 30) + 8
    x = torch.full((1, V), float("-inf"), dtype=torch.bfloat16, device=DEV)
    x[0, torch.tensor([5, 77, 1 << 20, V - 1], device=DEV)] = 1.0
    tokens, lp = eg.sample_tokens(x, torch.tensor([0.9], device=DEV), top_p=torch.tensor([top_p], device=DEV), want_logprob=True)
    assert tokens.tolist() == [5] and lp.tolist() == [0.0]
