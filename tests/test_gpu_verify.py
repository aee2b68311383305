"""GPU: token probabilities and the verification of drafted tokens.

Probabilities: the exponent (l - max) log2(e) / T is formed with four
roundings (difference, the factor's constant, division and product), so the
exponential is off by ln 2 * 4 * 2^-24 * |exponent| and by the two units of
the hardware's exp2; the sum by the length of its longest chain of additions
(at most V / 64 + 32 of them); reciprocal and product by 2 * 2^-24.  Results
below the smallest normal number may be flushed.

Verification is exact: accepted counts and tokens are equal."""
import math

import numpy as np
import pytest
import torch

from hashed_gram_embedding_amd import engram as eg
from oracle import engram_oracle as orc

from parity import log

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
INF, NAN = float("inf"), float("nan")


def _check_probs(p, logits, temps):
    x, got = logits.double().cpu().numpy(), p.double().cpu().numpy()
    S, R, V = x.shape
    for s in range(S):
        t = 1.0 if temps is None else float(temps[s])
        for r in range(R):
            ref = orc.token_probs(x[s, r], t)
            assert np.array_equal(np.isnan(ref), np.isnan(got[s, r])), (s, r)
            if np.isnan(ref).any():
                continue
            if t > 0 and np.isfinite(x[s, r].max()):
                arg = np.where(np.isfinite(x[s, r]), (x[s, r].max() - x[s, r]) / t / math.log(2), 0.0)
                # the exponentials' error enters each term, and through the sum the weighted mean of it
                own = 2.0 ** -24 * (4 * math.log(2) * arg + 4)
                rel = own + np.sum(ref * own) + 2.0 ** -24 * (V / 64 + 32 + 2)
            else:
                rel = 0.0
            err = np.abs(got[s, r] - ref)
            assert np.all(err <= rel * ref + 2.0 ** -125), (s, r, float(np.max(err - rel * ref)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 3, 5), (1, 5, 1000), (3, 2, 4096), (2, 2, 4097), (1, 4, 32001),
                                   (40, 8, 2049), (1, 1, 128000), (300, 1, 515), (2, 1, 300001)])
def test_probs(dtype, shape):
    log(f"token_probs {dtype} {shape}")
    g = torch.Generator(device=DEV).manual_seed(3)
    x = (4 * torch.randn(shape, generator=g, device=DEV)).to(TYPES[dtype])
    t = 0.3 + torch.rand(shape[0], generator=g, device=DEV)
    if shape[0] > 1:
        t[0] = 0.0
    _check_probs(eg.token_probs(x, t), x, t)
    if x.numel() < 1 << 18:
        _check_probs(eg.token_probs(x), x, None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [3, 700, 9000, 40000])
def test_probs_of_masked_and_bad_rows(dtype, V):
    """Rows that a mask leaves empty or with one entry, the type's lowest value as a mask, infinities, NaN, ties."""
    log(f"token_probs masked {dtype} V={V}")
    x = torch.randn(2, 9, V, device=DEV).to(TYPES[dtype])
    x[:, 0] = -INF
    x[:, 1] = -INF
    x[:, 1, V - 1] = -5.0
    x[:, 2] = torch.finfo(TYPES[dtype]).min
    x[:, 3, V // 2:] = torch.finfo(TYPES[dtype]).min
    x[:, 4, 1] = INF
    x[:, 5, V - 1] = NAN
    x[:, 6] = 2.5                            # all tied
    x[:, 7, 2] = 1000.0
    x[:, 8, 0] = -INF
    t = torch.tensor([0.7, 0.0], device=DEV)
    p = eg.token_probs(x, t)
    _check_probs(p, x, t)
    assert (p[:, 0] == 0).all() and torch.isnan(p[:, 5]).all() and torch.isnan(p[0, 4]).all()
    assert p[1, 4, 1] == 1 and p[1, 6, 0] == 1 and p[0, 1, V - 1] == 1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [700, 40000, 200000])
def test_probs_at_the_ends_of_the_temperature(dtype, V):
    """The smallest temperatures (their reciprocal is past float32) leave the
    largest logit, the largest ones every entry that is not masked; NaN counts as 0."""
    log(f"token_probs temperatures {dtype} V={V}")
    t = torch.tensor([2.0 ** -149, 1e-39, 1e-20, 1e30, 3e38, INF, NAN, -INF], device=DEV)
    for rows in (1, 9):                      # 9: more rows than are split over workgroups
        x = torch.randn(8, rows, V, device=DEV).to(TYPES[dtype])
        x[:, :, V // 2] = 20.0
        x[:, :, 5:9] = -INF
        p = eg.token_probs(x, t).double().cpu().numpy()
        one = np.zeros(V)
        one[V // 2] = 1
        flat = np.full(V, 1 / (V - 4))
        flat[5:9] = 0
        for s in range(8):
            want = flat if 3 <= s <= 5 else one
            assert np.all(np.abs(p[s] - want) <= want * 2.0 ** -24 * (V / 64 + 32 + 4)), (s, rows)


@pytest.mark.parametrize("S,R,V", [(2 ** 24 + 3, 1, 3), (5, 2 ** 22 - 1, 4), (1, 2 ** 24 + 5, 3), (3, 2 ** 23 + 7, 2)])
def test_probs_of_the_most_rows(S, R, V):
    """More rows than one launch can have: each with its own sequence's temperature."""
    log(f"token_probs {S} x {R} rows")
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(S, R, V, generator=g, device=DEV)
    t = 0.25 + torch.rand(S, generator=g, device=DEV)
    p = eg.token_probs(x, t)
    worst = 0.0
    for part in range(0, S * R, 1 << 22):
        rows = slice(part, min(part + (1 << 22), S * R))
        seq = torch.arange(rows.start, rows.stop, device=DEV) // R
        a = x.view(S * R, V)[rows].double()
        ref = torch.softmax(a / t.double()[seq, None], -1)
        arg = (a.max(-1, keepdim=True).values - a) / t.double()[seq, None] / math.log(2)
        own = 2.0 ** -24 * (4 * math.log(2) * arg + 4)
        rel = own + (ref * own).sum(-1, keepdim=True) + 2.0 ** -24 * (32 + 2)
        worst = max(worst, float(((p.view(S * R, V)[rows].double() - ref).abs() / (rel * ref)).max()))
    assert worst <= 1.0, worst


def test_every_launch_of_a_call_is_timed():
    """Stage timing names each kernel that the calls launch, in order: one for
    rows that a workgroup takes, two where they are split over workgroups."""
    log("stages of token_probs and verify_drafts")
    x = torch.randn(3, 2, 40000, device=DEV)
    many = torch.randn(70, 1, 40000, device=DEV)
    p, q, d, ua, us = _case(2, 1, 60000, "f32", True)
    short = _case(2, 1, 6000, "f32", True)
    calls = [(lambda: eg.quantize_i8(x.view(6, 40000)), ["quantize_i8_kernel"]),
             (lambda: eg.token_probs(x), ["token_probs_segments_kernel", "token_probs_join_kernel"]),
             (lambda: eg.token_probs(many), ["token_probs_kernel"]),
             (lambda: eg.verify_drafts(p, q, d, ua, us), ["verify_parts_kernel", "verify_drafts_kernel"]),
             (lambda: eg.verify_drafts(*short[:5]), ["verify_drafts_kernel"])]
    try:
        for call, names in calls:
            eg.profile_enable(1)
            call()
            got = eg.profile_read()
            assert [n for n, _ in got] == names and all(ms > 0 for _, ms in got), got
    finally:
        eg.profile_enable(False)


def _chain(V):
    """Longest chain of additions in the sum of a row that one workgroup takes
    (1024 threads, quads: up to V / 4096 of them a thread, three more in a quad
    and for the tail, 6 over the wavefront and 15 over the workgroup), and for
    rows past the registers the rescalings, one per 8 quads, of 4 units each."""
    return V / 4096 + 1 + 3 + 6 + 15 + 4 * (V / 32768 + 2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V", [(1, 700), (9, 40000), (12, 9000), (12, 200003)])
def test_probs_of_logits_further_apart_than_their_type(dtype, rows, V):
    """Logits at both ends of their type's range, whose difference leaves it: at
    the largest temperatures they still have a share."""
    log(f"token_probs far logits {dtype} {rows} x {V}")
    t = torch.tensor([3.4e38, 1e38, 2.0 ** 120, 1e30, 0.5, INF], device=DEV)
    g = torch.Generator(device=DEV).manual_seed(7)
    x = (torch.finfo(TYPES[dtype]).max * (2 * torch.rand(len(t), rows, V, generator=g, device=DEV, dtype=torch.float64) - 1)).to(TYPES[dtype])
    x[..., 3] = torch.finfo(TYPES[dtype]).max
    x[..., V - 1] = torch.finfo(TYPES[dtype]).min
    x[..., 5] = -INF
    p = eg.token_probs(x, t)
    a, got, temps = x.double().cpu().numpy(), p.double().cpu().numpy(), t.double().cpu().numpy()
    for s, temp in enumerate(temps):
        for r in range(rows):
            row = a[s, r]
            arg = np.zeros(V)
            arg[np.isfinite(row)] = (row.max() - row[np.isfinite(row)]) / temp / math.log(2)
            ref = np.where(np.isfinite(row), np.exp2(-arg), 0.0)
            ref /= ref.sum()
            own = 2.0 ** -24 * (4 * math.log(2) * arg + 4)
            rel = own + np.sum(ref * own) + 2.0 ** -24 * (_chain(V) + 2)
            err = np.abs(got[s, r] - ref)
            assert np.all(err <= rel * ref + 2.0 ** -125), (temp, r, float(np.max(err / np.maximum(rel * ref, 1e-300))))


@pytest.mark.parametrize("dtype,V", [("bf16", 40001), ("bf16", 65536), ("bf16", 65537), ("bf16", 100003), ("bf16", 128000),
                                     ("bf16", 131075), ("bf16", 262145), ("f32", 32770), ("f32", 65535), ("f32", 65539),
                                     ("f32", 200003)])
def test_probs_of_a_batch_of_long_rows(dtype, V):
    """More rows than are split over workgroups, at ordinary temperatures: the
    forms that hold a long row in registers and the one that reads it twice.
    Rows of zeros, with NaN or +inf, masked and tied ones, greedy ones, and rows
    whose weight lies in the entries behind the last four."""
    log(f"token_probs batch {dtype} V={V}")
    g = torch.Generator(device=DEV).manual_seed(V)
    x = (3 * torch.randn(3, 25, V, generator=g, device=DEV)).to(TYPES[dtype])
    low = torch.finfo(TYPES[dtype]).min
    x[:, 0] = -INF
    x[:, 1] = -INF
    x[:, 1, V - 1] = -5.0
    x[:, 2, 17] = NAN
    x[:, 3, V - 1] = NAN
    x[:, 4, V - 1] = INF
    x[:, 5] = low
    x[:, 6, V // 3:] = low
    x[:, 7] = -2.5                           # all tied
    x[:, 8] = x[:, 8].sort(dim=-1).values    # the running maximum moves all the way
    x[:, 9] = x[:, 9].sort(dim=-1, descending=True).values
    x[:, 10, V - V % 4 - 1:] = 24.0          # most of the weight at the very end
    x[:, 11, V - 1] = 22.0
    x[:, 12, :V - 1] = -INF
    x[:, 13] = -INF
    x[:, 13, ::4096] = 0.0
    x[:, 14, V - 2:] = x[:, 14].max(dim=-1, keepdim=True).values
    x[:, 15, 40:] = -INF
    t = torch.tensor([0.7, 0.0, 1.9], device=DEV)
    p = eg.token_probs(x, t)
    a, got = x.double().cpu().numpy(), p.double().cpu().numpy()
    for s in range(3):
        temp = float(t[s])
        for r in range(25):
            ref, row = orc.token_probs(a[s, r], temp), a[s, r]
            assert np.array_equal(np.isnan(ref), np.isnan(got[s, r])), (s, r)
            if np.isnan(ref).any():
                continue
            rel = 0.0
            if temp > 0 and np.isfinite(row.max()):
                arg = np.where(np.isfinite(row), (row.max() - row) / temp / math.log(2), 0.0)
                own = 2.0 ** -24 * (4 * math.log(2) * arg + 4)
                rel = own + np.sum(ref * own) + 2.0 ** -24 * (_chain(V) + 2)
            err = np.abs(got[s, r] - ref)
            assert np.all(err <= rel * ref + 2.0 ** -125), (s, r, float(np.max(err - rel * ref)))


def test_the_longest_rows():
    """V = 2^31 - 1, the documented limit of both calls: entries at the very end
    of a row, found through offsets past 32 bits."""
    log("token_probs and verify_drafts longest rows")
    n = 2 ** 31 - 1
    x = torch.full((2, 1, n), -INF, dtype=torch.bfloat16, device=DEV)
    x[:, 0, n - 1] = 1.0
    x[:, 0, n - 2] = 1.0
    x[:, 0, 11] = 0.0
    p = eg.token_probs(x, torch.tensor([1.0, 0.0], device=DEV))
    z = 2 * math.e + 1
    got = [float(p[0, 0, c]) for c in (11, n - 2, n - 1)]
    assert all(abs(g - w) <= w * 2.0 ** -20 for g, w in zip(got, (1 / z, math.e / z, math.e / z)))
    assert float(p[1, 0, n - 2]) == 1.0
    p[0, 0, 11] = p[0, 0, n - 2] = p[0, 0, n - 1] = p[1, 0, n - 2] = 0
    assert not any(bool(c.any()) for r in p[:, 0] for c in r.split(1 << 28))
    del x, p

    t = torch.zeros((1, 3, n), dtype=torch.bfloat16, device=DEV)
    t[0, 0, n - 1] = 1.0
    t[0, 1, n - 3] = 0.25
    t[0, 1, n - 1] = 0.5
    t[0, 1, 3] = 0.25
    drafted = torch.tensor([[n - 1, 5]], dtype=torch.int32, device=DEV)
    ua = torch.zeros(1, 2, device=DEV)
    for u, want in ((0.1, 3), (0.3, n - 3), (0.49, n - 3), (0.5, n - 1), (0.99, n - 1)):
        tok, acc = eg.verify_drafts(t, None, drafted, ua, torch.tensor([u], device=DEV))
        assert acc.tolist() == [1] and tok.tolist() == [[n - 1, want, -1]], u


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_batches_past_32_bits(dtype):
    """More than 2^31 (and 2^32) entries: the last rows and sequences as alone."""
    log(f"token_probs and verify_drafts past 32 bits {dtype}")
    V, G = 128000, 8
    g = torch.Generator(device=DEV).manual_seed(11)
    S = 3800 if dtype == "bf16" else 2000
    x = torch.empty((S, G + 1, V), dtype=TYPES[dtype], device=DEV)
    for part in x.split(200):
        part.normal_(generator=g)
    t = torch.rand(S, generator=g, device=DEV) + 0.5
    p = eg.token_probs(x, t)
    for a in (0, S // 2, S - 3):
        assert torch.equal(p[a:a + 3], eg.token_probs(x[a:a + 3].repeat(3, 1, 1), t[a:a + 3].repeat(3))[:3]), a   # (81 rows: the same form)
    d = torch.randint(0, V, (S, G), generator=g, device=DEV, dtype=torch.int32)
    ua, us = 1e-7 * torch.rand(S, G, generator=g, device=DEV), torch.rand(S, generator=g, device=DEV)
    for q in (None, x[:, :G].contiguous()):
        tgt = x if q is None else p.to(TYPES[dtype])
        if q is not None:
            q.abs_()
        tok, acc = eg.verify_drafts(tgt, q, d, ua, us)
        for a in (0, S // 2, S - 3):
            rows = slice(a, a + 3)
            et, ea = eg.verify_drafts(tgt[rows].clone(), None if q is None else q[rows].clone(), d[rows].clone(), ua[rows].clone(),
                                      us[rows].clone())
            assert torch.equal(tok[rows], et) and torch.equal(acc[rows], ea), a
        assert int(acc.max()) > 0


def test_probs_of_padded_rows():
    """Rows of a padded vocabulary: the padding is not read, whatever it holds."""
    log("token_probs padded")
    for V, ld in ((515, 520), (4099, 4100), (32001, 32064)):
        x = torch.full((2, 3, ld), NAN, device=DEV)
        x[..., :V] = torch.randn(2, 3, V, device=DEV)
        t = torch.tensor([0.8, 0.0], device=DEV)
        assert torch.equal(eg.token_probs(x[..., :V], t), eg.token_probs(x[..., :V].contiguous(), t))


def _verify_both(p, q, drafted, ua, us, n=None):
    tok, acc = eg.verify_drafts(p, q, drafted, ua, us, n_draft=n)
    p64 = p.double().cpu().numpy()
    q64 = None if q is None else q.double().cpu().numpy()
    S, G = drafted.shape
    d, a64, s64 = drafted.cpu().numpy(), ua.double().cpu().numpy(), us.double().cpu().numpy()
    for s in range(S):
        rt, ra = orc.verify_drafts(p64[s], None if q64 is None else q64[s], d[s], a64[s], s64[s],
                                   G if n is None else int(n[s]))
        assert int(acc[s]) == ra, s
        assert np.array_equal(tok[s].cpu().numpy(), rt), (s, tok[s], rt)
    return tok, acc


def _case(S, G, V, dtype, sampled, seed=0, sharp=2.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = sharp * torch.randn(S, G + 1, V, generator=g, device=DEV)
    p = torch.softmax(x, -1).to(TYPES[dtype])
    q = torch.softmax(x[:, :G] + 0.5 * torch.randn(S, G, V, generator=g, device=DEV), -1).to(TYPES[dtype])
    drafted = torch.multinomial(q.float().view(S * G, V), 1, generator=g).view(S, G).to(torch.int32) if G else \
        torch.empty((S, 0), dtype=torch.int32, device=DEV)
    ua = torch.rand(S, G, generator=g, device=DEV)
    if not sampled:
        ua = ua * 0.02
    return p, (q if sampled else None), drafted, ua, torch.rand(S, generator=g, device=DEV)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("size", [(1, 1, 1), (3, 2, 5), (1, 4, 32001), (7, 7, 4095), (5, 3, 4096), (5, 3, 4097), (64, 5, 1000),
                                  (300, 2, 777), (2, 64, 130), (2, 1, 128000), (3, 0, 900), (1, 2, 600011)])
def test_verify(size, sampled, dtype):
    log(f"verify {size} sampled={sampled} {dtype}")
    S, G, V = size
    p, q, d, ua, us = _case(S, G, V, dtype, sampled, seed=S + G)
    _verify_both(p, q, d, ua, us)
    n = torch.randint(-1, G + 3, (S,), device=DEV, dtype=torch.int32)
    _verify_both(p, q, d, ua, us, n)


@pytest.mark.parametrize("V", [6, 5000, 70000])
@pytest.mark.parametrize("S", [4, 200])
def test_verify_borders(V, S):
    """Random numbers at both ends, one-hot and dyadic rows, drafts outside the vocabulary, rows that leave nothing."""
    log(f"verify borders V={V} S={S}")
    top = 1.0 - 2.0 ** -24
    for us_v in (0.0, 0.5, top):
        us = torch.full((S,), us_v, device=DEV)
        p = torch.zeros(S, 3, V, device=DEV)
        p[:, 0, V - 1] = 0.5                                   # two equal halves at both ends
        p[:, 0, 0] = 0.5
        p[:, 1, V // 2] = 1.0
        p[:, 2, V // 3] = 0.25
        p[:, 2, V - 2] = 0.75
        q = torch.zeros(S, 2, V, device=DEV)
        q[:, :, 0] = 1.0
        d = torch.zeros(S, 2, dtype=torch.int32, device=DEV)
        d[1, 0], d[2, 0], d[3, 0] = V, -1, V - 1
        for ua_v in (0.0, 0.5, top):
            ua = torch.full((S, 2), ua_v, device=DEV)
            _verify_both(p, q, d, ua, us)
            _verify_both(p, None, d, ua, us)
            _verify_both(p, 2 * p[:, :2].contiguous(), torch.full_like(d, V // 2), ua, us)   # p - q leaves nothing
        z = torch.zeros_like(p)
        tok, acc = _verify_both(z, q, d, ua, us)               # rows of zeros: no token
        assert (tok == -1).all() and (acc == 0).all()
        z[:, :, 2] = NAN
        z[:, :, 4] = 0.125
        tok, _ = _verify_both(z, None, d, ua, us)              # a NaN counts as nothing
        assert (tok[:, 0] == 4).all()
        z[:, :, 3] = INF
        assert (eg.verify_drafts(z, None, d, ua, us)[0][:, 0] == -1).all()


def test_verify_in_a_graph_and_on_another_stream():
    log("verify graph")
    for S, V in ((1, 32001), (300, 4000)):
        p, q, d, ua, us = _case(S, 4, V, "f32", True)
        x = torch.randn(S, 5, V, device=DEV)
        t = torch.rand(S, device=DEV) + 0.5
        eg.verify_drafts(p, q, d, ua, us)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            probs = eg.token_probs(x, t)
            tok, acc = eg.verify_drafts(probs, q, d, ua, us)
        for i in range(4):
            x.copy_(torch.log(p) + 0.3 * torch.randn(S, 5, V, device=DEV))
            us.copy_(torch.rand(S, device=DEV))
            g.replay()
            torch.cuda.synchronize()
            et, ea = eg.verify_drafts(eg.token_probs(x, t), q, d, ua, us)
            assert torch.equal(tok, et) and torch.equal(acc, ea), i
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        st, sa = eg.verify_drafts(eg.token_probs(x, t, stream=side), q, d, ua, us, stream=side)
        side.synchronize()
        assert torch.equal(st, et) and torch.equal(sa, ea)


def test_verified_tokens_follow_the_target():
    """Over many random numbers the next token is distributed as the target says, accepted or not."""
    log("verify distribution")
    V, n = 7, 60000
    g = torch.Generator(device=DEV).manual_seed(9)
    p1 = torch.softmax(torch.randn(2, V, generator=g, device=DEV), -1)
    q1 = torch.softmax(torch.randn(1, V, generator=g, device=DEV), -1)
    p, q = p1.expand(n, 2, V).contiguous(), q1.expand(n, 1, V).contiguous()
    d = torch.multinomial(q1.expand(n, V), 1, generator=g).to(torch.int32)
    tok, _ = eg.verify_drafts(p, q, d, torch.rand(n, 1, generator=g, device=DEV), torch.rand(n, generator=g, device=DEV))
    got = torch.bincount(tok[:, 0].long(), minlength=V).double().cpu() / n
    # six standard deviations of each share
    assert (got - p1[0].double().cpu()).abs().max() < 6 * math.sqrt(0.25 / n)
