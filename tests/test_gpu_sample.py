"""GPU: tokens drawn with temperature, top-k, top-p and min-p against float64.

A token has to equal the reference's unless the random number (or top_p) lies
within 2^-30 of the total from the border between two tokens: weights are
multiples of 2^-F, F >= 44 at the sizes here, so that V 2^-45 is the furthest a
border moves.  Such rows are counted; with the seeds used there are none.
A log-probability is one float32 rounding (2^-24) of a double, beside the
total's error (below 2^-27 of it)."""
import numpy as np
import pytest
import torch

import plain_around as plain
from hashed_gram_embedding_amd import engram as eg
from parity import log

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
NEAR = 2.0 ** -30


def _dev(a, dtype):
    return None if a is None else torch.tensor(a, dtype=dtype, device=DEV)


def _check(logits, u, t=None, k=None, p=None, m=None):
    """logits [S, R, V] on the device, u [S, R], the rest one a sequence or None."""
    tokens, lp = eg.sample_tokens(logits, u, temperature=_dev(t, torch.float32), top_k=_dev(k, torch.int32),
                                  top_p=_dev(p, torch.float32), min_p=_dev(m, torch.float32), want_logprob=True)
    again, none = eg.sample_tokens(logits, u, temperature=_dev(t, torch.float32), top_k=_dev(k, torch.int32),
                                   top_p=_dev(p, torch.float32), min_p=_dev(m, torch.float32))
    assert torch.equal(tokens, again) and none is None
    x, us = logits.float().cpu().numpy(), u.cpu().numpy()
    f32 = np.float32
    for s in range(x.shape[0]):
        for r in range(x.shape[1]):
            with np.errstate(over="ignore"):
                args = [float(f32(1.0 if t is None else t[s])), 0 if k is None else k[s],
                        float(f32(1.0 if p is None else p[s])), float(f32(0.0 if m is None else m[s]))]
            want, logprob, near = plain.sample(x[s, r], *args, float(us[s, r]))
            assert near > NEAR, f"row {s},{r} is at a border: {near}"
            assert int(tokens[s, r]) == want, (s, r, int(tokens[s, r]), want, args, us[s, r])
            got = float(lp[s, r])
            assert got == logprob or abs(got - logprob) <= 2.0 ** -24 * abs(logprob) + 2.0 ** -26, (s, r, got, logprob)


def _logits(S, R, V, dtype, seed, spread=3.0, masked=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = spread * torch.randn(S, R, V, generator=g, device=DEV)
    if masked:
        x = torch.where(torch.rand(x.shape, generator=g, device=DEV) < masked, float("-inf"), x)
    return x.to(TYPES[dtype]), torch.rand(S, R, generator=g, device=DEV)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 3, 4, 5, 63, 257, 1000, 2048, 2049, 8191, 8193, 32001, 32769, 65536, 65537, 131072, 131073,
                               200003])
def test_filters(V, dtype):
    """Each filter alone, all together, none, greedy; every size of the row's registers and the ones behind."""
    log(f"sample_tokens {dtype} V={V}")
    x, u = _logits(8, 2, V, dtype, V, masked=0.1 if V > 10 else 0.0)
    _check(x, u)
    _check(x, u, t=[1.0, 0.7, 1.3, 0.0, 0.05, 30.0, -1.0, 1.0],
           k=[0, 5, 1, 7, 50, V // 2 + 1, V, 3000], p=[1.0, 0.9, 0.5, 0.1, 0.99, 0.7, 1.5, 0.95],
           m=[0.0, 0.0, 0.1, 0.5, 0.02, 0.9, -1.0, 1e-4])
    _check(x, u, p=[0.95, 0.5, 0.999, 0.1, 1e-6, 0.0, -1.0, 0.8])
    _check(x, u, k=[1, 2, 40, 64, 1000, 5000, 2 ** 31 - 1, -3])
    _check(x, u, m=[0.05, 0.5, 1.0, 2.0, 1e-30, 0.001, 0.9, 0.0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [70, 9000, 40000, 140000])
def test_equal_logits(V, dtype):
    """Few different values: cuts fall inside groups of equal logits, which are larger than the list of one bin."""
    log(f"sample_tokens equal logits {dtype} V={V}")
    g = torch.Generator(device=DEV).manual_seed(V)
    x = torch.randint(0, 3, (6, 1, V), generator=g, device=DEV).float().to(TYPES[dtype])
    x[5] = 1.25
    x[4, 0, : V // 2] = -0.0
    u = torch.rand(6, 1, generator=g, device=DEV)
    _check(x, u, k=[1, V // 4, V // 2 + 3, V - 1, 7, V // 3])
    _check(x, u, p=[0.3, 0.61, 0.9, 0.123, 0.77, 0.51])
    _check(x, u, k=[V // 2, V // 4, V // 2 + 3, V - 1, 7, V // 3], p=[0.3, 0.61, 0.9, 0.123, 0.77, 0.51], m=[0.3, 0.2, 0.0, 0.1, 0.5, 1.0])


@pytest.mark.parametrize("V", [6, 3000, 70000])
def test_special_rows(V):
    """Nothing but -inf, a NaN, infinities, a single entry; the smallest and largest temperatures; logits further apart
    than float32 reaches."""
    log(f"sample_tokens special rows V={V}")
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(9, 1, V, device=DEV)
    x[0] = -inf
    x[1, 0, V - 1] = nan
    x[2, 0, 4] = inf
    x[3] = -inf
    x[3, 0, V - 2] = -5.0
    x[4, 0, ::2], x[4, 0, 1::2] = 3e38, -3e38
    x[5, 0, 1] = 1e-38
    x[6, 0, 0] = -inf
    x[7, 0, 2:] = -3e38
    x[8, 0, 3] = -1e30
    u = torch.full((9, 1), 0.623, device=DEV)
    for t in (1.0, 0.0, 1e-38, 1e-45, 1e30, 3e38, inf, nan):
        _check(x, u, t=[t] * 9)
        _check(x, u, t=[t] * 9, k=[3] * 9, p=[0.9] * 9, m=[0.5] * 9)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_random_numbers_at_the_ends(dtype):
    """u of 0, just below 1, and outside [0, 1): the first and the last entry that stays."""
    log(f"sample_tokens u at the ends {dtype}")
    V = 5003
    x, _ = _logits(1, 7, V, dtype, 4)
    x[..., :3] = float("-inf")
    x[..., -2:] = float("-inf")
    u = torch.tensor([[0.0, 1.0 - 2.0 ** -24, 1.0, 5.0, -1.0, float("nan"), float("inf")]], device=DEV)
    tokens, _ = eg.sample_tokens(x, u)
    assert tokens[0].tolist() == [3, V - 3, V - 3, V - 3, 3, 3, V - 3]
    stays = torch.topk(x[0].float(), 2, dim=1)[1].sort(1)[0]
    tokens, _ = eg.sample_tokens(x, u, top_k=torch.tensor([2], dtype=torch.int32, device=DEV))
    for r, at in enumerate([0, 1, 1, 1, 0, 0, 1]):
        assert int(tokens[0, r]) == int(stays[r, at])


def test_strided_rows_and_surroundings():
    """Rows at a stride that leaves them unaligned, [S, V] and [S, R, V], and what lies around the outputs."""
    log("sample_tokens strides")
    for dtype in ("f32", "bf16"):
        for V, ld in ((1001, 1003), (4099, 4099)):
            base, u = _logits(1, 12, ld, dtype, ld)
            x = base.view(6, 2, ld)[..., 1:1 + min(V, ld - 1)]
            _check(x, u.view(6, 2), p=[0.9] * 6)
            _check(x.reshape(12, -1)[:, None], u.view(12, 1), k=[9] * 12)
            flat = base[0][:, 1:V - 1]
            one, _ = eg.sample_tokens(flat, u[0])
            three, _ = eg.sample_tokens(flat[:, None], u.view(12, 1))
            assert torch.equal(one, three[:, 0])


def test_draws_follow_the_weights():
    """A grid of random numbers visits each token in proportion to its weight: the number of its grid points is its
    share of the grid, up to one at either border."""
    log("sample_tokens distribution")
    V, n = 11, 4096
    x = torch.randn(1, 1, V, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2)).expand(n, 1, V).contiguous()
    u = ((torch.arange(n, device=DEV) + 0.5) / n).view(n, 1)
    tokens, _ = eg.sample_tokens(x, u, temperature=torch.full((n,), 0.8, device=DEV))
    share = torch.softmax(x[0, 0].double() / float(np.float32(0.8)), 0) * n
    count = torch.bincount(tokens[:, 0].long(), minlength=V).double()
    assert ((count - share).abs() <= 1.0 + 1e-9 * n).all()


def test_more_rows_than_temperatures():
    log("sample_tokens rows of a sequence")
    x, u = _logits(5, 7, 300, "bf16", 9)
    _check(x, u, t=[0.5, 1.0, 2.0, 0.0, 0.9], k=[3, 0, 40, 9, 1], p=[0.9, 0.5, 1.0, 0.2, 0.7])


def test_row_past_32_bits():
    """Rows whose elements lie past 2^31, and a row longer than 2^24."""
    log("sample_tokens past 32 bits")
    V = (1 << 24) + 7
    x = torch.full((260, V), float("-inf"), dtype=torch.bfloat16, device=DEV)
    at = torch.arange(260, device=DEV) * 60000 + 5
    x[torch.arange(260, device=DEV), at] = 1.0
    x[torch.arange(260, device=DEV), V - 1 - at] = 1.0
    u = torch.full((260,), 0.25, device=DEV)
    tokens, lp = eg.sample_tokens(x, u, want_logprob=True)
    assert torch.equal(tokens.long(), torch.minimum(at, V - 1 - at)) and torch.allclose(lp, torch.full_like(lp, -0.6931472))
    tokens, _ = eg.sample_tokens(x, u + 0.5, top_p=torch.full((260,), 0.75, device=DEV))
    assert torch.equal(tokens.long(), torch.maximum(at, V - 1 - at))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [4095, 4097, 8189, 8192, 8193])
def test_many_rows(V, dtype):
    """More rows than the GPU has places for, each with settings of its own."""
    log(f"sample_tokens many rows {V} {dtype}")
    S = 300
    x, u = _logits(S, 1, V, dtype, V, masked=0.2)
    g = np.random.default_rng(V)
    t = np.where(g.random(S) < 0.1, 0.0, 0.3 + g.random(S)).astype(np.float32)
    k = np.where(g.random(S) < 0.5, 0, g.integers(1, 400, S))
    p = np.where(g.random(S) < 0.4, 1.0, g.random(S)).astype(np.float32)
    m = np.where(g.random(S) < 0.6, 0.0, 0.3 * g.random(S)).astype(np.float32)
    _check(x, u, t.tolist(), k.tolist(), p.tolist(), m.tolist())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5003, 70001])
def test_rows_up_to_zero(V, dtype):
    """Logits less their largest, rows of zeros of both signs (all of the row, more and less than half of it), and rows
    whose largest is tiny, below the smallest normal number or far below zero."""
    log(f"sample_tokens rows up to zero {dtype} {V}")
    x, u = _logits(12, 1, V, dtype, V, spread=2.0, masked=0.05)
    x = (x.float() - x.float().amax(-1, keepdim=True)).to(TYPES[dtype])
    at = torch.arange(V, device=DEV)
    x[1] = 0.0
    x[2] = -0.0
    x[3, 0, at % 3 > 0] = 0.0
    x[4, 0, at % 3 == 0] = -0.0
    x[5] = torch.where(at % 2 == 0, 0.0, -0.0)
    x[6, 0, 17] = 2.0 ** -126
    x[7] = torch.where(x[7] == 0, 2.0 ** -115, x[7].float())
    x[8] = torch.where(at % 5 == 0, 0.0, -(at % 7).float() * 2.0 ** -112)
    x[9] -= 300.0
    x[10] = torch.where(at % 3 == 0, 0.0, 2.0 ** -9)
    x[11] = torch.where(at == V - 2, 0.0, float("-inf"))
    S = x.shape[0]
    _check(x, u)
    _check(x, u, p=[0.9] * S)
    _check(x, u, k=[1500] * S)
    _check(x, u, t=[0.7] * S, k=[3000] * S, p=[0.83] * S, m=[0.01] * S)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [8192, 7001])
def test_equal_logits_of_many_rows(V, dtype):
    """More than 256 rows of few different logits, up to 8192 entries each: more equal ones than the smallest workgroup's
    list holds, cut by a top_k that is collected and one that is binned, by top_p, and by both."""
    log(f"sample_tokens equal logits of many rows {dtype} {V}")
    S = 260
    g = torch.Generator(device=DEV).manual_seed(V)
    often = torch.rand(S, 1, 1, generator=g, device=DEV)             # of the largest: few of a row to all of it
    x = torch.where(torch.rand(S, 1, V, generator=g, device=DEV) < often, 1.5,
                    torch.randint(0, 2, (S, 1, V), generator=g, device=DEV).float()).to(TYPES[dtype])
    x[7] = 0.75
    assert int((x == 1.5).sum(-1).max()) > 5120
    u = torch.rand(S, 1, generator=g, device=DEV)
    r = np.random.default_rng(V)
    small, large = 2 * r.integers(0, 60, S) + 1, 2 * r.integers(100, V // 2, S) + 1
    p = (0.05 + 0.9 * r.random(S)).tolist()
    _check(x, u, k=small.tolist())
    _check(x, u, k=large.tolist())
    _check(x, u, p=p)
    _check(x, u, k=large.tolist(), p=p)
    _check(x, u, m=[0.3, 0.7] * (S // 2))
