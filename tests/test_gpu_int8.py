"""GPU: rows and products in 8-bit integers.  Codes and scales are exact; the
product's sum is exact, so an output is off by the float32 conversion of the
sum and two multiplications (3 * 2^-24, second-order terms within a fourth),
and by half a bf16 step (2^-8) more where it is stored in bf16."""
import dataclasses

import numpy as np
import pytest
import torch

from hashed_gram_embedding_amd import engram as eg
from hashed_gram_embedding_amd import inputs
from oracle import engram_oracle as orc

from parity import check_bf16_layer, check_f32_layer, log, to_f64

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
TINY = 2.0 ** -126


def _bound(ref, out_dtype):
    rel = 4 * 2.0 ** -24 + (2.0 ** -8 if out_dtype == "bf16" else 0.0)
    return rel * np.abs(ref) + 2 * TINY


def _rows(rng, n, k, dtype):
    x = (rng.standard_normal((n, k)) * np.exp2(rng.integers(-20, 20, (n, 1)))).astype(np.float32)
    t = torch.from_numpy(x).to(DEV).to(TYPES[dtype])
    return t, t.double().cpu().numpy()


def _check_rows(q, s, x64):
    rq, rs = orc.quantize_i8(x64)
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (5, 64), (70, 256), (9, 1000), (33, 1024), (2, 2048), (3, 2049),
                                   (4, 5003), (1, 16384)])
def test_quantize_exact(dtype, shape):
    log(f"quantize_i8 {dtype} {shape}")
    rng = np.random.default_rng(1)
    x, x64 = _rows(rng, *shape, dtype)
    _check_rows(*eg.quantize_i8(x), x64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_borders(dtype):
    """Ties, equal magnitudes, subnormal rows, zeros, infinities and NaN."""
    log(f"quantize_i8 borders {dtype}")
    rng = np.random.default_rng(2)
    x = rng.standard_normal((12, 130)).astype(np.float32)
    for r in range(3):                       # x = max / 2 is the tie 63.5 for every max
        x[r, :] = np.float32(1.0 + r * 0.375) * 0.5
        x[r, 5] = np.float32(1.0 + r * 0.375)
        x[r, 6] = -x[r, 5]
    x[3, :] = np.arange(130) * 0.5           # max 64.5: many near borders
    x[4, :] = 0.0
    x[5, :] = 2.0 ** -133 * np.arange(130)   # subnormal in both types
    x[6, :] = 0.0
    x[6, 9] = 2.0 ** -149 if dtype == "f32" else 2.0 ** -133
    x[7, 3] = np.inf
    x[8, 4] = np.nan
    x[9, 5] = -np.inf
    x[9, 6] = np.nan
    x[10, :] = 3.0e38
    x[11, :] = np.arange(130) + 125.0        # 254 = 2 * 127: whole and half codes
    t = torch.from_numpy(x).to(DEV).to(TYPES[dtype])
    x64 = t.double().cpu().numpy()
    q, s = eg.quantize_i8(t)
    _check_rows(q, s, x64)
    assert torch.isnan(s[7:10]).all() and (q[7:10] == 0).all() and s[4] == 0


def test_quantize_the_longest_row():
    """2^31 - 1 columns, the documented limit: the last ones are reached, nothing behind them."""
    log("quantize_i8 longest row")
    n = 2 ** 31 - 1
    x = torch.zeros(1, n, dtype=torch.bfloat16, device=DEV)
    at = [0, 5, 2 ** 30, n - 2049, n - 9, n - 8, n - 2, n - 1]
    for i, c in enumerate(at):
        x[0, c] = (i + 1) * (-1) ** i
    x[0, n - 3] = 127.0
    q, s = eg.quantize_i8(x)
    assert float(s) == 1.0 and [int(q[0, c]) for c in at] == [(i + 1) * (-1) ** i for i in range(len(at))]
    assert int(q[0, n - 3]) == 127
    q[0, at + [n - 3]] = 0
    assert not any(bool(p.any()) for p in q[0].split(1 << 28))


@pytest.mark.parametrize("rows,cols,dtype", [(2 ** 26 + 5, 4, "bf16"), (2 ** 26 + 5, 9, "f32"), (2 ** 20 + 3, 4097, "bf16"),
                                             (2 ** 19 + 9, 8203, "bf16")])
def test_quantize_the_most_rows(rows, cols, dtype):
    """More rows than one launch can have, more codes than 32 bits count."""
    log(f"quantize_i8 {rows} rows")
    g = torch.Generator(device=DEV).manual_seed(6)
    pattern = torch.randn(4099, cols, generator=g, device=DEV).to(TYPES[dtype])
    times = -(-rows // 4099)
    x = pattern.repeat(times, 1)[:rows].contiguous()
    q, s = eg.quantize_i8(x)
    del x
    rq, rs = orc.quantize_i8(pattern.double().cpu().numpy())
    rq, rs = torch.from_numpy(rq).to(DEV), torch.from_numpy(rs).to(DEV)
    whole = rows // 4099 * 4099
    assert (q[:whole].view(-1, 4099, cols) == rq).all() and (s[:whole].view(-1, 4099) == rs).all()
    assert torch.equal(q[whole:], rq[:rows - whole]) and torch.equal(s[whole:], rs[:rows - whole])


@pytest.mark.parametrize("source", ["i8", "bf16"])
def test_the_most_outputs_of_short_rows(source):
    """Fewer than 16 columns and more outputs than one launch can have threads."""
    log(f"project_i8 short rows, past 2^32 outputs, {source}")
    n, k, o = 70001, 5, 61441
    g = torch.Generator(device=DEV).manual_seed(8)
    w = torch.randint(-127, 128, (o, k), generator=g, dtype=torch.int8, device=DEV)
    ws = torch.rand(o, generator=g, device=DEV)
    e, s = torch.randn(n, k, generator=g, device=DEV).to(torch.bfloat16), None
    if source == "i8":
        e, s = eg.quantize_i8(e)
    out = eg.project_i8(e, w, ws, e_scale=s)
    for a in [*range(0, n - 5, 7919), n - 5]:
        part = eg.project_i8(e[a:a + 5].clone(), w, ws, e_scale=None if s is None else s[a:a + 5].clone())
        assert torch.equal(out[a:a + 5], part), a
    for a in range(0, n, 4096):   # every output, to the rounding of its type
        qf, sf = (e[a:a + 4096], s[a:a + 4096]) if s is not None else eg.quantize_i8(e[a:a + 4096].clone())
        ref = (qf.float() @ w.float().t()) * sf[:, None] * ws
        assert ((out[a:a + 4096].float() - ref).abs() <= (2.0 ** -8 + 2.0 ** -20) * ref.abs() + 2 * TINY).all(), a


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 2823, 700), (3, 4099, 77), (9, 1025, 515), (15, 3001, 40), (20, 4097, 515), (8, 3842, 330),
                                  (5, 4101, 8192), (32, 4349, 8193), (2, 9997, 21)])
def test_few_tokens_of_long_odd_rows(size, out_dtype):
    """Rows of W at every alignment, longer than a wavefront's loads in flight
    and few enough for a workgroup's wavefronts to share each: every code is its
    own, so a column out of place shows."""
    n, k, o = size
    log(f"project_i8 shared odd rows {size} {out_dtype}")
    rng = np.random.default_rng(n * 7 + k * 3 + o)
    w, q = rng.integers(-128, 128, (o, k), dtype=np.int8), rng.integers(-128, 128, (n, k), dtype=np.int8)
    ws, s = np.exp2(rng.uniform(-9, 3, o)).astype(np.float32), np.exp2(rng.uniform(-9, 3, n)).astype(np.float32)
    out = eg.project_i8(torch.from_numpy(q).to(DEV), torch.from_numpy(w).to(DEV), torch.from_numpy(ws).to(DEV),
                        e_scale=torch.from_numpy(s).to(DEV), out_dtype=out_dtype)
    ref = orc.project_i8(q, s, w, ws)
    err = np.abs(to_f64(out) - ref)
    assert np.all(err <= _bound(ref, out_dtype)), float(np.max(err - _bound(ref, out_dtype)))
    if n <= 8:                                # float rows, quantised by the product itself
        x, x64 = _rows(rng, n, k, "bf16")
        rq, rs = orc.quantize_i8(x64)
        out = eg.project_i8(x, torch.from_numpy(w).to(DEV), torch.from_numpy(ws).to(DEV), out_dtype=out_dtype)
        ref = orc.project_i8(rq, rs, w, ws)
        assert np.all(np.abs(to_f64(out) - ref) <= _bound(ref, out_dtype))


SIZES = [(1, 16, 1), (1, 1024, 2000), (2, 64, 64), (3, 48, 65), (5, 17, 33), (16, 1024, 4100), (31, 15, 7), (33, 1, 5),
         (64, 1024, 256), (65, 128, 129), (130, 1000, 515), (200, 2823, 103), (257, 1024, 512), (300, 4096, 192),
         (1000, 320, 1031), (513, 2048, 2048), (33, 513, 66),
         (70, 601, 130), (300, 1001, 259), (40, 4099, 70), (18, 1009, 5)]


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("source", ["i8", "bf16", "f32"])
@pytest.mark.parametrize("size", SIZES)
def test_product(size, source, out_dtype):
    n, k, o = size
    log(f"project_i8 {size} {source} -> {out_dtype}")
    rng = np.random.default_rng(n * 7 + k * 3 + o)
    w = rng.integers(-128, 128, (o, k), dtype=np.int8)
    ws = np.exp2(rng.uniform(-9, 3, o)).astype(np.float32)
    if source == "i8":
        q = rng.integers(-128, 128, (n, k), dtype=np.int8)
        s = np.exp2(rng.uniform(-9, 3, n)).astype(np.float32)
        e, e_scale = torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV)
    else:
        e, x64 = _rows(rng, n, k, source)
        e_scale = None
        q, s = orc.quantize_i8(x64)
    out = eg.project_i8(e, torch.from_numpy(w).to(DEV), torch.from_numpy(ws).to(DEV), e_scale=e_scale,
                        out_dtype=out_dtype)
    ref = orc.project_i8(q, s, w, ws)
    assert out.dtype == TYPES[out_dtype] and tuple(out.shape) == (n, o)
    err = np.abs(to_f64(out) - ref)
    assert np.all(err <= _bound(ref, out_dtype)), float(np.max(err - _bound(ref, out_dtype)))


@pytest.mark.parametrize("n", [1, 20, 300])
def test_product_full_sums(n):
    """All codes at -128 with the most columns that fit: the sum is 2^31 - 2^14."""
    log(f"project_i8 full sums n={n}")
    k, o = 131071, 40
    e = torch.full((n, k), -128, dtype=torch.int8, device=DEV)
    w = torch.full((o, k), -128, dtype=torch.int8, device=DEV)
    one = torch.ones(max(n, o), device=DEV)
    out = eg.project_i8(e, w, one[:o], e_scale=one[:n], out_dtype="f32")
    assert (out.double() == float(np.float32(131071 * 16384))).all()


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k", [17, 64, 1024, 1000, 1001, 1002])
def test_product_into_a_view(k, out_dtype):
    """Outputs that start at any element, operands that end with their
    allocations' last byte: nothing beside the output is written."""
    log(f"project_i8 views k={k} {out_dtype}")
    rng = np.random.default_rng(5)
    for n, o in ((1, 70), (20, 37), (40, 71), (300, 130), (4200, 4100)):
        q = rng.integers(-128, 128, (n, k), dtype=np.int8)
        w = rng.integers(-128, 128, (o, k), dtype=np.int8)
        buf = torch.full((n * o + 2,), 7.0, device=DEV, dtype=TYPES[out_dtype])
        out = buf[1:1 + n * o].view(n, o)
        eg.project_i8(torch.from_numpy(q).to(DEV), torch.from_numpy(w).to(DEV), torch.ones(o, device=DEV),
                      e_scale=torch.ones(n, device=DEV), out_dtype=out_dtype, out=out)
        ref = torch.from_numpy(q.astype(np.float32)).to(DEV).double() @ torch.from_numpy(w.astype(np.float32)).to(DEV).double().t()
        assert torch.equal(out, ref.float().to(TYPES[out_dtype])), (n, o)
        assert buf[0] == 7.0 and buf[-1] == 7.0


@pytest.mark.parametrize("k,n_out,out_dtype", [(32, 120000, "bf16"), (40, 119999, "f32")])
def test_outputs_past_32_bits(k, n_out, out_dtype):
    """More than 2^31 outputs: rows at both ends against the same rows multiplied alone."""
    log(f"project_i8 {k} x {n_out} past 32 bits")
    n = 20001
    q = torch.randint(-127, 128, (n, k), dtype=torch.int8, device=DEV)
    w = torch.randint(-127, 128, (n_out, k), dtype=torch.int8, device=DEV)
    qs, ws = torch.rand(n, device=DEV), torch.rand(n_out, device=DEV)
    out = eg.project_i8(q, w, ws, e_scale=qs, out_dtype=out_dtype)
    for a, b in ((0, 5), (17890, 17900), (n - 7, n)):
        assert torch.equal(out[a:b], eg.project_i8(q[a:b].clone(), w, ws, e_scale=qs[a:b].clone(), out_dtype=out_dtype)), a


@pytest.mark.parametrize("n,k,o", [(3, 16384, 140001), (20, 16383, 140001), (300, 16384, 140001), (300, 16385, 140001), (140001, 16384, 70),
                                   (140001, 16385, 70)])
def test_operands_past_32_bits(n, k, o):
    """Operands of more than 2^31 bytes: outputs at both ends and around the
    border against the same rows multiplied alone."""
    log(f"project_i8 {n} x {k} x {o}")
    g = torch.Generator(device=DEV).manual_seed(3)
    q = torch.randint(-127, 128, (n, k), generator=g, dtype=torch.int8, device=DEV)
    w = torch.randint(-127, 128, (o, k), generator=g, dtype=torch.int8, device=DEV)
    qs, ws = torch.rand(n, generator=g, device=DEV), torch.rand(o, generator=g, device=DEV)
    out = eg.project_i8(q, w, ws, e_scale=qs, out_dtype="f32")
    for t in {0, max(n - 40, 0)}:
        for a in {0, min(131050, o - 64), o - 64}:
            tt = slice(t, min(t + 40, n))
            part = eg.project_i8(q[tt].clone(), w[a:a + 64].clone(), ws[a:a + 64].clone(), e_scale=qs[tt].clone(), out_dtype="f32")
            assert torch.equal(out[tt, a:a + 64], part), (t, a)
    if n > 131072:
        a = slice(131060, 131090)
        assert torch.equal(out[a], eg.project_i8(q[a].clone(), w, ws, e_scale=qs[a].clone(), out_dtype="f32"))


@pytest.mark.parametrize("k,o,source", [(17, 3, "bf16"), (32, 2, "bf16"), (17, 2, "i8"), (9, 2, "f32")])
def test_product_of_the_most_tokens(k, o, source):
    """More tokens than one launch quantises, W's odd rows copied beside the
    first of them: every output against those of the pattern that repeats."""
    log(f"project_i8 2^26 tokens x {k} x {o} {source}")
    n, g = 2 ** 26 + 5, torch.Generator(device=DEV).manual_seed(12)
    pattern = torch.randn(4099, k, generator=g, device=DEV).to(TYPES["f32" if source == "f32" else "bf16"])
    w = torch.randint(-127, 128, (o, k), generator=g, dtype=torch.int8, device=DEV)
    ws = torch.rand(o, generator=g, device=DEV)
    times, e_scale = -(-n // 4099), None
    want = eg.project_i8(pattern, w, ws, out_dtype="f32")
    if source == "i8":
        pattern, s = eg.quantize_i8(pattern)
        e_scale = s.repeat(times)[:n].contiguous()
    e = pattern.repeat(times, 1)[:n].contiguous()
    out = eg.project_i8(e, w, ws, e_scale=e_scale, out_dtype="f32")
    whole = n // 4099 * 4099
    assert (out[:whole].view(-1, 4099, o) == want).all() and torch.equal(out[whole:], want[:n - whole])


def test_unaligned_operands_are_refused():
    log("project_i8 unaligned operands")
    b = torch.zeros(40 * 64 + 16, dtype=torch.int8, device=DEV)
    one = torch.ones(40, device=DEV)
    good, bad = b[:40 * 64].view(40, 64), b[8:8 + 40 * 64].view(40, 64)
    for e, w in ((bad, good), (good, bad)):
        with pytest.raises(eg.EngramError, match="16-byte"):
            eg.project_i8(e, w, one, e_scale=one)


@pytest.mark.parametrize("n", [1, 2, 40, 300])
def test_product_of_bad_rows(n):
    """A row with an infinity or a NaN gives NaN in its outputs and in no other row; a row of zeros gives zeros."""
    log(f"project_i8 bad rows n={n}")
    x = torch.randn(n + 3, 256, device=DEV)
    x[0, 3] = float("inf")
    x[1, 255] = float("nan")
    x[2] = 0
    w = torch.randint(-127, 128, (90, 256), dtype=torch.int8, device=DEV)
    out = eg.project_i8(x, w, torch.ones(90, device=DEV), out_dtype="f32")
    assert torch.isnan(out[:2]).all() and (out[2] == 0).all() and torch.isfinite(out[2:]).all()
    if n == 1:
        solo = eg.project_i8(x[:1].contiguous(), w, torch.ones(90, device=DEV), out_dtype="bf16")
        assert torch.isnan(solo).all()


def test_empty_products():
    log("project_i8 empty")
    w, s = torch.ones((8, 32), dtype=torch.int8, device=DEV), torch.ones(8, device=DEV)
    assert eg.project_i8(torch.empty((0, 32), device=DEV), w, s).shape == (0, 8)
    q, sc = eg.quantize_i8(torch.empty((0, 32), device=DEV))
    assert q.shape == (0, 32) and sc.shape == (0,)


def _layer_case(config, hdtype, **kw):
    w = inputs.make_config(config, rows_per_table=None if config == 0 else 997, **kw)
    lay = w.layers[0]
    L = eg.Layer(lay, hdtype, DEV)
    return w, lay, L, eg.Int8Weights(L)


@pytest.mark.parametrize("config,hdtype,kw", [(0, "f32", {}), (1, "bf16", dict(B=2, T=90)), (1, "bf16", dict(B=1, T=1)),
                                              (2, "bf16", dict(B=2, T=33)), (3, "bf16", dict(B=16, T=1, layers=1))])
def test_layer_matches_oracle(config, hdtype, kw):
    """The layer with Step 5 in 8-bit integers against the oracle's."""
    log(f"forward_i8 config {config} {kw}")
    w, lay, L, w8 = _layer_case(config, hdtype, **kw)
    H = eg.to_device(w.H, hdtype, DEV)
    alpha, y = eg.forward_i8(torch.from_numpy(w.tokens).to(DEV), H, L, w8, want_alpha=True, want_y=True)
    ref = orc.forward(w.tokens, w.H, lay, hdtype, gemm="int8")
    check, h_in = (check_bf16_layer, orc.bf16_to_f64(w.H)) if hdtype == "bf16" else (check_f32_layer, w.H.astype(np.float64))
    check(to_f64(alpha), ref["alpha"], to_f64(y), ref["Y"], to_f64(H), h_in, tag=f"int8 config {config}")


@pytest.mark.parametrize("config,kw", [(1, dict(B=2, T=600)), (1, dict(B=3, T=7, table_dim=32, heads=1, d=128)),
                                       (1, dict(B=2, T=40, d=192)), (1, dict(B=1, T=33, d=4096)),
                                       (2, dict(B=1, T=3300)), (2, dict(B=1, T=8100, d=384)), (3, dict(B=600, T=1, layers=1))])
def test_layer_forms(config, kw):
    """Every form of the product with the gate's sums, ragged in tokens, at
    widths that the sums' runs divide or not, and the unfused one."""
    log(f"forward_i8 form {config} {kw}")
    w, lay, L, w8 = _layer_case(config, "bf16", **kw)
    H = eg.to_device(w.H, "bf16", DEV)
    alpha, y = eg.forward_i8(torch.from_numpy(np.ascontiguousarray(w.tokens)).to(DEV), H, L, w8, want_alpha=True, want_y=True)
    ref = orc.forward(w.tokens, w.H, lay, "bf16", gemm="int8")
    check_bf16_layer(to_f64(alpha), ref["alpha"], to_f64(y), ref["Y"], to_f64(H), orc.bf16_to_f64(w.H), tag=f"int8 {config} {kw}")


@pytest.mark.parametrize("config,kw", [(1, dict(B=3, T=37)), (1, dict(B=1, T=700, heads=4)), (1, dict(B=2, T=5, heads=16)),
                                       (1, dict(B=3, T=11, heads=5, table_dim=32)), (3, dict(B=9, T=1, layers=1)),
                                       (3, dict(B=40, T=130, layers=1)), (1, dict(B=1, T=4097))])
def test_layer_rows_are_quantised_exactly(config, kw):
    """v of the int8 layer is engram_project_i8 of engram_quantize_i8 of the
    gathered rows, bit for bit, where the gather writes the codes and where not."""
    log(f"int8 rows {config} {kw}")
    w, lay, L, w8 = _layer_case(config, "bf16", **kw)
    tok = torch.from_numpy(np.ascontiguousarray(w.tokens)).to(DEV)
    B, T = tok.shape
    e = torch.empty((B * T, L.d_mem), dtype=torch.bfloat16, device=DEV)
    eg.retrieve(tok, L, e)
    q, s = eg.quantize_i8(e)
    want = eg.project_i8(q, w8.q[:lay.d], w8.scale[:lay.d], e_scale=s, out_dtype="f32")
    draft = eg.Draft(B, T, L, DEV)
    st = eg.DecodeState(B, 3, lay.branches, 9, lay.d, DEV)
    eg.forward_draft(tok, eg.to_device(w.H, "bf16", DEV), L, st, draft, w8=w8)
    assert torch.equal(draft.v[:, :lay.d], want)


@pytest.mark.parametrize("kw", [dict(B=3, T=50), dict(B=2, T=900)])
def test_layer_rows_of_a_hot_tier_and_beside_mxfp8(kw):
    """Rows from an Engram-Nine hot tier leave the gather as exact codes too, and
    a layer that also has MXFP8 weights gives the same int8 results."""
    log(f"int8 rows, hot tier {kw}")
    from test_gpu_hot import hot_sets
    w = inputs.make_config(1, rows_per_table=997, **kw)
    lay = w.layers[0]
    L = eg.Layer(lay, "bf16", DEV, mxfp8=True)
    w8 = eg.Int8Weights(L)
    tok = torch.from_numpy(np.ascontiguousarray(w.tokens)).to(DEV)
    B, T = tok.shape
    plain = eg.Layer(lay, "bf16", DEV)
    outs = []
    for layer in (L, plain):
        H = eg.to_device(w.H, "bf16", DEV)
        eg.forward_i8(tok, H, layer, w8)
        outs.append(H)
    assert torch.equal(outs[0], outs[1])

    _, hot = hot_sets(w, lay, 40, seed=3)
    plain.set_hot(hot)
    e = torch.empty((B * T, L.d_mem), dtype=torch.bfloat16, device=DEV)
    eg.retrieve(tok, plain, e)
    q, s = eg.quantize_i8(e)
    draft = eg.Draft(B, T, plain, DEV)
    st = eg.DecodeState(B, 3, lay.branches, 9, lay.d, DEV)
    H = eg.to_device(w.H, "bf16", DEV)
    eg.forward_draft(tok, H, plain, st, draft, w8=w8)
    assert torch.equal(draft.v[:, :lay.d], eg.project_i8(q, w8.q[:lay.d], w8.scale[:lay.d], e_scale=s, out_dtype="f32"))
    assert not torch.equal(H, outs[1])          # the tier's rows differ from the tables'


@pytest.mark.parametrize("table", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("B,T", [(3, 50), (2, 900)])
def test_layer_rows_through_a_cache_are_quantised_exactly(table, B, T):
    """Tables of every type behind an HBM row cache, accesses counted: the codes
    are those of the rows that the bf16 gather gives, the counts those of it."""
    log(f"int8 rows, cache, {table} {B}x{T}")
    w = inputs.make_config(1, B=B, T=T, rows_per_table=997)
    lay = w.layers[0]
    hp, rng = lay.hash, np.random.default_rng(4)
    shape = (lay.tables.total_rows, lay.tables.dim)
    rows = {"f32": lambda: rng.standard_normal(shape).astype(np.float32), "bf16": lambda: lay.tables.rows,
            "i8": lambda: rng.integers(-127, 128, shape, dtype=np.int8)}[table]()
    scale = np.exp2(rng.uniform(-9, 0, shape[0])).astype(np.float32) if table == "i8" else None
    lay = dataclasses.replace(lay, tables=dataclasses.replace(lay.tables, rows=rows, scale=scale, dtype=table))
    L = eg.Layer(lay, "bf16", DEV)
    w8 = eg.Int8Weights(L)
    tok = torch.from_numpy(np.ascontiguousarray(w.tokens)).to(DEV)
    L.set_cache(*eg.cache_build(tok[:, ::3].contiguous(), L, shape[0] // 20))
    counts = [torch.zeros(shape[0], dtype=torch.int32, device=DEV) for _ in range(2)]
    e = torch.empty((B * T, L.d_mem), dtype=torch.bfloat16, device=DEV)
    L.set_access_counts(counts[0])
    eg.retrieve(tok, L, e)
    L.set_access_counts(counts[1])
    draft = eg.Draft(B, T, L, DEV)
    eg.forward_draft(tok, eg.to_device(w.H, "bf16", DEV), L, eg.DecodeState(B, hp.max_n, 1, 9, lay.d, DEV), draft, w8=w8)
    q, s = eg.quantize_i8(e)
    assert torch.equal(draft.v[:, :lay.d], eg.project_i8(q, w8.q[:lay.d], w8.scale[:lay.d], e_scale=s, out_dtype="f32"))
    assert torch.equal(*counts) and int(counts[0].sum()) == B * T * hp.n_tables


def test_layer_decode_state():
    """A prefill and single-token steps with the int8 layer against the oracle run over the same chunks."""
    log("forward_i8 decode")
    w = inputs.make_config(3, B=8, T=3, layers=1, context_len=12, rows_per_table=997)
    lay = w.layers[0]
    L = eg.Layer(lay, "bf16", DEV)
    w8 = eg.Int8Weights(L)
    st = eg.DecodeState(8, 3, 1, 9, lay.d, DEV)
    ref = orc.new_state(8, 3, 1, 9, lay.d)
    chunks = [(w.context, w.H_context)] + [(w.tokens[:, t:t + 1], w.H[:, t:t + 1]) for t in range(3)]
    for i, (tk, Hn) in enumerate(chunks):
        H = eg.to_device(Hn, "bf16", DEV)
        alpha, y = eg.forward_i8(torch.from_numpy(np.ascontiguousarray(tk)).to(DEV), H, L, w8, state=st,
                                 want_alpha=True, want_y=True)
        r = orc.forward(tk, Hn, lay, "bf16", state=ref, gemm="int8")
        ref = r["state"]
        check_bf16_layer(to_f64(alpha), r["alpha"], to_f64(y), r["Y"], to_f64(H), orc.bf16_to_f64(Hn), tag=f"chunk {i}")
    assert np.array_equal(st.ids.cpu().numpy(), ref["ids"]) and np.array_equal(st.pos.cpu().numpy(), ref["pos"])


def test_product_in_a_graph_and_on_another_stream():
    """Captured and replayed between eager calls; then on a stream of its own."""
    log("project_i8 graph")
    for n in (1, 24, 300):
        x = torch.randn(n, 1000, device=DEV).to(torch.bfloat16)
        w = torch.randint(-127, 128, (515, 1000), dtype=torch.int8, device=DEV)
        s = torch.rand(515, device=DEV)
        out = torch.empty((n, 515), device=DEV)
        ws = torch.empty(max(eg.lib().engram_project_i8_workspace(n, 1000, 515, eg.BF16), 256), dtype=torch.uint8, device=DEV)
        call = lambda: eg.project_i8(x, w, s, out_dtype="f32", out=out, ws=ws)   # noqa: E731
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        for i in range(3):
            x.copy_(torch.randn(n, 1000, device=DEV))
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, eg.project_i8(x, w, s, out_dtype="f32")), i
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = eg.project_i8(x, w, s, out_dtype="f32", stream=side)
        side.synchronize()
        assert torch.equal(got, out)
