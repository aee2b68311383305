"""GPU: Step 5 with each request's low-rank adapter against float64.

Tolerances: a float32 sum of K products in any order is off by at most K
roundings of its running sum, which the terms' magnitudes bound; a matrix
instruction may round a running sum by a whole unit (2^-23).  So W e: K 2^-23
of |W||e|; the adapter: (K + rank + 2) 2^-23 of |B||s||A||e|, and in bf16 h is
carried as two bf16 numbers (2^-17 of it).  bf16 output adds 2^-8 of the value."""
import numpy as np
import pytest
import torch

import plain_around as plain
from hashed_gram_embedding_amd import engram as eg
from hashed_gram_embedding_amd import inputs
from oracle import engram_oracle as orc
from parity import check_bf16_layer, check_f32_layer, log

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
UNIT = 2.0 ** -23


def _f64(t):
    return t.double().cpu().numpy()


def _inputs(n, K, out, rank, adapters, per, dtype, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + n)

    def normal(*s):
        return torch.randn(*s, generator=g, device=DEV)

    dt = TYPES[dtype]
    e, w = normal(n, K).to(dt), (normal(out, K) / K ** 0.5).to(dt)
    ad = eg.Adapters((normal(adapters, rank, K) / K ** 0.5).to(dt), normal(adapters, out, rank).to(dt),
                     0.5 + torch.rand(adapters, generator=g, device=DEV))
    which = torch.randint(-1, adapters, (-(-n // per),), generator=g, device=DEV, dtype=torch.int32)
    return e, w, ad, which


def _check(out, e, w, ad, which, per, dtype, out_t, rows=None):
    n, K = e.shape
    rows = np.arange(n) if rows is None else np.asarray(rows)
    owner = which.cpu().numpy()[rows // per]
    scale = None if ad.scale is None else _f64(ad.scale)
    ref, size, carried = plain.project_adapted(_f64(e)[rows], _f64(w), _f64(ad.a), _f64(ad.b), scale, owner)
    tol = (K + ad.rank + 2) * UNIT * size + (2.0 ** -17 * carried if dtype == "bf16" else 0.0) + \
        (2.0 ** -8 * np.abs(ref) if out_t == "bf16" else 0.0)
    err = np.abs(_f64(out)[rows] - ref)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dtype,out_t", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("n,K,out,rank,adapters,per", [
    (1, 64, 64, 8, 1, 1), (1, 1024, 2048, 16, 4, 1), (2, 128, 192, 24, 2, 1), (31, 192, 64, 8, 40, 1), (32, 64, 128, 32, 3, 5),
    (33, 320, 64, 16, 3, 7), (65, 256, 320, 40, 64, 1), (250, 128, 64, 128, 5, 64), (300, 64, 192, 8, 300, 1)])
def test_project_adapted(dtype, out_t, n, K, out, rank, adapters, per):
    log(f"project_adapted {dtype} {out_t} {n} {K} {out} {rank} {adapters} {per}")
    e, w, ad, which = _inputs(n, K, out, rank, adapters, per, dtype)
    which[0] = adapters - 1
    got = eg.project_adapted(e, w, ad, which, per=per, out_dtype=out_t)
    assert got.dtype == TYPES[out_t]
    _check(got, e, w, ad, which, per, dtype, out_t)
    assert torch.equal(got, eg.project_adapted(e, w, ad, which, per=per, out_dtype=out_t))


@pytest.mark.parametrize("out_t", ["f32", "bf16"])
@pytest.mark.parametrize("n,K,out,rank,adapters,per", [
    (513, 64, 320, 8, 7, 1), (700, 128, 192, 24, 3, 100), (1000, 192, 128, 16, 20, 3), (5000, 128, 5120, 16, 5, 1024),
    (4100, 64, 4160, 40, 100, 1)])
def test_tiles(out_t, n, K, out, rank, adapters, per):
    """Both tile sizes, ragged in tokens and outputs."""
    log(f"project_adapted tiles {out_t} {n} {K} {out} {rank} {adapters} {per}")
    e, w, ad, which = _inputs(n, K, out, rank, adapters, per, "bf16")
    whole = torch.full((n + 2, out), 7.0, device=DEV, dtype=TYPES[out_t])
    got = eg.project_adapted(e, w, ad, which, per=per, out_dtype=out_t, out=whole[1:n + 1])
    rows = np.unique(np.concatenate([np.arange(0, n, 97), np.arange(max(0, n - 40), n), np.arange(250, 262)]))
    _check(got, e, w, ad, which, per, "bf16", out_t, rows)
    assert (whole[0] == 7).all() and (whole[-1] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 40, 600])
def test_ids_without_an_adapter(dtype, n):
    """Ids outside the adapters, and no adapters at all, leave the plain product."""
    log(f"project_adapted without adapters {dtype} {n}")
    e, w, ad, which = _inputs(n, 128, 128, 8, 3, 1, dtype)
    which.copy_(torch.tensor([-1, 3, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).repeat(n)[:n])
    got = eg.project_adapted(e, w, ad, which)
    _check(got, e, w, ad, which, 1, dtype, "f32")
    none = eg.Adapters(ad.a[:0], ad.b[:0])
    assert torch.equal(got, eg.project_adapted(e, w, none, torch.zeros_like(which)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [40, 600])
def test_bad_adapters_stay_with_their_requests(dtype, n):
    """Infinities and NaN in one adapter, or in one token, reach no other token's outputs."""
    log(f"project_adapted isolation {dtype} {n}")
    e, w, ad, which = _inputs(n, 64, 128, 24, 6, 1, dtype)
    which.copy_(torch.arange(n, device=DEV) % 7 - 1)
    good = eg.project_adapted(e, w, ad, which)
    ad.a[2, 3, 5] = float("nan")
    ad.b[3] = float("inf")
    ad.scale[4] = float("nan")
    e[8] = float("inf")
    got = eg.project_adapted(e, w, ad, which)
    same = (which != 2) & (which != 3) & (which != 4)
    same[8] = False
    assert torch.equal(got[same], good[same]) and torch.isfinite(good).all()
    assert torch.isnan(got[which == 2]).all() and torch.isnan(got[which == 4]).all()
    assert not torch.isfinite(got[which == 3]).any()


# The smallest calls, ragged in tokens and outputs, that each kernel takes with few adapters or many.
KERNELS = [("bf16", 257, 256, 100), ("bf16", 1001, 320, 200), ("bf16", 1701, 320, 1), ("bf16", 3001, 1088, 700), ("bf16", 4097, 1088, 1),
           ("bf16", 3001, 5184, 1024), ("f32", 257, 256, 100), ("f32", 1001, 320, 1), ("f32", 1003, 320, 300), ("f32", 5001, 2112, 1),
           ("f32", 5001, 2112, 900)]


@pytest.mark.parametrize("K,rank", [(64, 8), (192, 24), (320, 128)])
@pytest.mark.parametrize("dtype,n,out,per", KERNELS)
def test_every_kernel(dtype, n, out, per, K, rank):
    log(f"project_adapted kernels {dtype} {n} {out} {per} {K} {rank}")
    e, w, ad, which = _inputs(n, K, out, rank, 30, per, dtype)
    rows = np.unique(np.concatenate([np.arange(0, n, 61), np.arange(n - 40, n), np.arange(125, 135)]))
    for out_t in ("f32", "bf16") if dtype == "bf16" else ("f32",):
        whole = torch.full((n + 2, out), 7.0, device=DEV, dtype=TYPES[out_t])
        got = eg.project_adapted(e, w, ad, which, per=per, out_dtype=out_t, out=whole[1:n + 1])
        _check(got, e, w, ad, which, per, dtype, out_t, rows)
        assert (whole[0] == 7).all() and (whole[-1] == 7).all()


@pytest.mark.parametrize("adapters", [6, 40])
@pytest.mark.parametrize("dtype,n,out", sorted({k[:3] for k in KERNELS}))
def test_bad_adapters_in_every_kernel(dtype, n, out, adapters):
    log(f"project_adapted isolation {dtype} {n} {out} {adapters}")
    e, w, ad, which = _inputs(n, 128, out, 24, adapters, 1, dtype)
    which.copy_(torch.arange(n, device=DEV) % (adapters + 1) - 1)
    good = eg.project_adapted(e, w, ad, which)
    ad.a[2, 3, 5] = float("nan")
    ad.b[3] = float("inf")
    ad.b[5, 7, 23] = float("nan")
    ad.scale[4] = float("nan")
    e[8] = float("inf")
    got = eg.project_adapted(e, w, ad, which)
    same = (which < 2) | (which > 5)
    same[8] = False
    assert torch.equal(got[same], good[same]) and torch.isfinite(good).all()
    assert torch.isnan(got[which == 2]).all() and torch.isnan(got[which == 4]).all()
    assert not torch.isfinite(got[which == 3]).any()
    one = which == 5
    one[8] = False
    assert torch.isnan(got[one][:, 7]).all()
    others = torch.arange(out, device=DEV) != 7
    assert torch.equal(got[one][:, others], good[one][:, others])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 40, 600, 3001])
def test_inner_products_past_the_largest_bf16(dtype, n):
    """h = s A e between bf16's largest number and float32's: finite, and so is B h."""
    log(f"project_adapted large h {dtype} {n}")
    e, w, ad, which = _inputs(n, 64, 128, 8, 2, 1, dtype)
    which.copy_(torch.arange(n, device=DEV) % 3 % 2)
    e[:, 0], ad.a[:] = 1.0, 0.0
    most = torch.finfo(torch.bfloat16).max
    ad.a[0, 0, 0], ad.a[0, 7, 0], ad.a[1, 3, 0] = most, -most, -most
    ad.b[:] = 0.0
    ad.b[0, :, 0], ad.b[0, ::2, 7], ad.b[1, 1::2, 3] = 2.0 ** -120, 2.0 ** -121, 2.0 ** -120
    ad.scale.copy_(torch.tensor([1.003, 1.0039]))   # bf16's halfway point to infinity is 1.00195 of its largest, float32's end 1.0039
    got = eg.project_adapted(e, w, ad, which)
    assert torch.isfinite(got).all()
    _check(got, e, w, ad, which, 1, dtype, "f32")


def test_scale_defaults_to_one():
    log("project_adapted scale")
    e, w, ad, which = _inputs(50, 64, 64, 8, 3, 1, "bf16")
    ones = eg.Adapters(ad.a, ad.b, torch.ones(3, device=DEV))
    assert torch.equal(eg.project_adapted(e, w, eg.Adapters(ad.a, ad.b), which), eg.project_adapted(e, w, ones, which))


def _layer(config, hdtype, B, T):
    w = inputs.make_config(config, B=B, T=T, **({} if config == 0 else dict(rows_per_table=499)))
    lay = w.layers[0]
    L = eg.Layer(lay, hdtype, DEV)
    n_out, d_mem = L.w.shape
    g = torch.Generator(device=DEV).manual_seed(5)
    a = (torch.randn(3, 8, d_mem, generator=g, device=DEV) / d_mem ** 0.5).to(TYPES[hdtype])
    b = (0.02 * torch.randn(3, n_out, 8, generator=g, device=DEV)).to(TYPES[hdtype])
    return w, lay, L, eg.Adapters(a, b, torch.tensor([1.0, 0.5, 2.0], device=DEV))


def _reference(tokens, H, lay, hdtype, ad, which, state=None):
    """orc.forward with each sequence's adapter in Step 5."""
    base = orc.forward(tokens, H, lay, hdtype, state=state)
    B, T = tokens.shape
    w64 = orc.storage_to_f64(lay.w, hdtype)
    kv = plain.project_adapted(base["e"].reshape(B * T, -1), w64, _f64(ad.a), _f64(ad.b), _f64(ad.scale), np.repeat(which, T))[0]
    out = orc.gate_conv(orc.storage_to_f64(H, hdtype), kv.reshape(B, T, -1), lay.conv_w, lay.dilation, lay.eps,
                        None if state is None else state["u"])
    if state is not None:
        span = (lay.kernel_w - 1) * lay.dilation
        uu = np.concatenate([state["u"], np.transpose(out["u"], (0, 2, 1, 3))], axis=2)[:, :, -span:]
        out["state"] = dict(base["state"], u=uu)
    return base, out


@pytest.mark.parametrize("config,hdtype", [(1, "bf16"), (2, "bf16"), (0, "f32")])
@pytest.mark.parametrize("T", [1, 9, 150])
def test_layer_with_adapters(config, hdtype, T):
    log(f"forward_adapted {config} {hdtype} {T}")
    which = np.array([1, -1, 0, 2], dtype=np.int32)
    w, lay, L, ad = _layer(config, hdtype, 4, T)
    H = eg.to_device(w.H, hdtype, DEV)
    alpha, y = eg.forward_adapted(torch.from_numpy(w.tokens).to(DEV), H, L, ad, torch.from_numpy(which).to(DEV),
                                  want_alpha=True, want_y=True)
    base, ref = _reference(w.tokens, w.H, lay, hdtype, ad, which)
    check = check_bf16_layer if hdtype == "bf16" else check_f32_layer
    check(_f64(alpha), ref["alpha"], _f64(y), ref["Y"], _f64(H), orc.storage_to_f64(w.H, hdtype), tag=f"adapted {config} T={T}")
    assert np.abs(ref["Y"][0] - base["Y"][0]).max() > 10 * np.abs(_f64(y)[0] - ref["Y"][0]).max()   # the adapter does something


def test_layer_with_adapters_decodes():
    """A context, then token after token, through the decode state."""
    log("forward_adapted decode")
    which = np.array([2, 0, -1, 1], dtype=np.int32)
    w, lay, L, ad = _layer(1, "bf16", 4, 14)
    span = (lay.kernel_w - 1) * lay.dilation
    st = eg.DecodeState(4, lay.hash.max_n, lay.branches, span, lay.d, DEV)
    state = orc.new_state(4, lay.hash.max_n, lay.branches, span, lay.d)
    ids = torch.from_numpy(which).to(DEV)
    for t0, t1 in [(0, 11), (11, 12), (12, 13), (13, 14)]:
        tk, Hn = np.ascontiguousarray(w.tokens[:, t0:t1]), np.ascontiguousarray(w.H[:, t0:t1])
        H = eg.to_device(Hn, "bf16", DEV)
        alpha, y = eg.forward_adapted(torch.from_numpy(tk).to(DEV), H, L, ad, ids, state=st, want_alpha=True, want_y=True)
        _, ref = _reference(tk, Hn, lay, "bf16", ad, which, state)
        state = ref["state"]
        check_bf16_layer(_f64(alpha), ref["alpha"], _f64(y), ref["Y"], _f64(H), orc.bf16_to_f64(Hn), tag=f"tokens {t0}..{t1 - 1}")
    assert np.array_equal(st.ids.cpu().numpy(), state["ids"]) and (st.pos == 14).all()
