"""The operators around the layer on the CPU: refusals of the C ABI (fake
pointers that never reach a GPU), workspace sizes, refusals of the binding, and
pins of the tests' own plain forms."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import plain_around as plain
from hashed_gram_embedding_amd import engram as eg
from test_speculative_host import _expect, _layer

pytestmark = pytest.mark.skipif(not os.path.exists(eg.LIB_PATH), reason="libengram.so not built")

P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)
OFF8 = ctypes.c_void_p(0x10008)


def test_embed_refusals():
    f = eg.lib().engram_embed

    def call(status, text, ids=P, n=4, table=P, dtype=eg.F32, V=10, dim=16, scale=1.0, branches=2, odt=eg.BF16, out=P):
        _expect(status, text, f, ids, n, table, dtype, V, dim, scale, branches, odt, out, None)

    call(eg.OK, "", n=0, ids=None, table=None, out=None)
    call(eg.EUNSUPPORTED, "dtypes", dtype=eg.I8)
    call(eg.EUNSUPPORTED, "dtypes", odt=eg.I8)
    for name in ("n", "V", "dim", "branches"):
        call(eg.EINVAL, "need n", **{name: -1})
    for name in ("V", "dim", "branches"):
        call(eg.EINVAL, "need n", **{name: 0})
    call(eg.EUNSUPPORTED, "n above", n=1 << 31)
    call(eg.EUNSUPPORTED, "2^31", V=1 << 31)
    call(eg.EUNSUPPORTED, "multiple of 8", dim=12)
    call(eg.EUNSUPPORTED, "multiple of 8", dim=65544)
    call(eg.EUNSUPPORTED, "branches", branches=65)
    for name in ("ids", "table", "out"):
        call(eg.EINVAL, "non-NULL", **{name: None})
        call(eg.EINVAL, "aligned", **{name: ODD})
    call(eg.EINVAL, "aligned", table=OFF8)


def test_embed_backward_refusals():
    f, size = eg.lib().engram_embed_backward, eg.lib().engram_embed_backward_workspace
    need = size(40, 16)
    assert need >= 40 * 8 + 5 * 2 * 16 * 4 and size(0, 16) == 0 and size(-1, 16) == 0 and size(40, 0) == 0
    assert size((1 << 28) + 1, 16) == 0 and size(1 << 28, 65536) > 0 and size(40, 65537) == 0

    def call(status, text, ids=P, n=40, dout=P, dtype=eg.F32, V=10, dim=16, scale=1.0, branches=2, acc=0, odt=eg.F32, dtable=P, ws=P,
             wsb=need):
        _expect(status, text, f, ids, n, dout, dtype, V, dim, scale, branches, acc, odt, dtable, ws, wsb, None)

    call(eg.EUNSUPPORTED, "dtypes", dtype=eg.I8)
    call(eg.EUNSUPPORTED, "dtypes", odt=eg.I8)
    for name in ("n", "V", "dim", "branches"):
        call(eg.EINVAL, "need n", **{name: -1})
    call(eg.EUNSUPPORTED, "n above", n=(1 << 28) + 1)
    call(eg.EUNSUPPORTED, "2^31", V=1 << 31)
    call(eg.EUNSUPPORTED, "multiple of 8", dim=20)
    call(eg.EUNSUPPORTED, "branches", branches=65)
    for name in ("ids", "dout", "dtable"):
        call(eg.EINVAL, "non-NULL", **{name: None})
        call(eg.EINVAL, "aligned", **{name: ODD})
    call(eg.EINVAL, "dtable", n=0, dtable=None)
    call(eg.OK, "", n=0, ids=None, dout=None, acc=1, ws=None, wsb=0)
    call(eg.EINVAL, "workspace", ws=None)
    call(eg.EINVAL, "workspace", wsb=need - 1)
    call(eg.EINVAL, "workspace", ws=OFF8)


def test_project_adapted_refusals():
    f, size = eg.lib().engram_project_adapted, eg.lib().engram_project_adapted_workspace
    need = size(40, eg.BF16, 24)
    assert need == 40 * 2 * 32 * 2 and size(40, eg.F32, 24) == 40 * 24 * 4 and size(0, eg.F32, 8) == 0
    assert size(40, eg.I8, 8) == 0 and size(40, eg.F32, 0) == 0 and size(40, eg.F32, 136) == 0 and size(1 << 31, eg.F32, 8) == 0

    def call(status, text, e=P, w=P, n=40, k=64, o=128, dtype=eg.BF16, which=P, per=1, odt=eg.F32, out=P, ws=P, wsb=need, null=False,
             ad_n=3, rank=24, a=0x10000, b=0x10000, scale=None):
        ad = eg.AdaptersStruct(ad_n, rank, a, b, scale)
        _expect(status, text, f, e, w, n, k, o, dtype, None if null else ctypes.byref(ad), which, per, odt, out, ws, wsb, None)

    call(eg.OK, "", n=0, e=None, null=True)
    call(eg.EUNSUPPORTED, "dtype", dtype=eg.I8)
    call(eg.EUNSUPPORTED, "out_dtype", odt=eg.I8)
    call(eg.EUNSUPPORTED, "out_dtype", dtype=eg.F32, odt=eg.BF16)
    for name in ("k", "o", "per"):
        call(eg.EINVAL, "need n_tok", **{name: 0})
    call(eg.EINVAL, "need n_tok", n=-1)
    call(eg.EUNSUPPORTED, "2^31", n=1 << 31)
    call(eg.EUNSUPPORTED, "2^31", o=1 << 31)
    for bad in (dict(k=96), dict(o=96), dict(k=65600)):
        call(eg.EUNSUPPORTED, "multiples of 64", **bad)
    call(eg.EINVAL, "adapters are NULL", null=True)
    call(eg.EINVAL, "n >= 0", ad_n=-1)
    call(eg.EUNSUPPORTED, "more than", ad_n=(1 << 20) + 1)
    for rank in (0, 4, 12, 136, -8):
        call(eg.EUNSUPPORTED, "rank", rank=rank)
    call(eg.EINVAL, "a and b", a=None)
    call(eg.EINVAL, "a and b", b=None)
    call(eg.EINVAL, "16-byte", a=0x10008)
    call(eg.EINVAL, "scale", scale=0x10002)
    call(eg.EINVAL, "which", which=None)
    call(eg.EINVAL, "which", which=ODD)
    for name in ("e", "w", "out"):
        call(eg.EINVAL, "non-NULL", **{name: None})
        call(eg.EINVAL, "16-byte", **{name: OFF8})
    call(eg.EINVAL, "workspace", ws=None)
    call(eg.EINVAL, "workspace", wsb=need - 1)
    call(eg.EINVAL, "workspace", ws=OFF8)


def test_forward_adapted_refusals():
    L, keep = _layer()
    lib, lp = eg.lib(), ctypes.byref(L)
    ad = eg.AdaptersStruct(3, 8, 0x20000, 0x30000, None)
    size = lib.engram_forward_adapted_workspace
    need = size(2, 4, lp, ctypes.byref(ad))
    assert need > 0 and size(2, 4, None, ctypes.byref(ad)) == 0 and size(2, 4, lp, None) == 0
    assert size(-1, 4, lp, ctypes.byref(ad)) == 0 and size(65536, 4, lp, ctypes.byref(ad)) == 0
    assert size(65535, (1 << 31) - 1, lp, ctypes.byref(ad)) == 0

    def call(status, text, tok=P, H=P, B=2, T=4, layer=lp, adapters=ctypes.byref(ad), which=P, st=None, y=None, ws=P, wsb=need):
        _expect(status, text, lib.engram_forward_adapted, tok, H, B, T, layer, adapters, which, st, None, y, ws, wsb, None)

    call(eg.OK, "", B=0, tok=None, H=None)
    call(eg.EINVAL, "layer", layer=None)
    call(eg.EINVAL, "adapters are NULL", adapters=None)
    call(eg.EINVAL, "which", which=None)
    call(eg.EINVAL, "tokens and H", tok=None)
    call(eg.EINVAL, "tokens and H", H=None)
    call(eg.EINVAL, "H must be", H=OFF8)
    call(eg.EINVAL, "y_out", y=OFF8)
    call(eg.EINVAL, "B and T", T=-1)
    call(eg.EUNSUPPORTED, "65535", B=65536)
    call(eg.EUNSUPPORTED, "2^31-1", B=65535, T=(1 << 31) - 1)
    call(eg.EINVAL, "workspace", wsb=need - 1)
    call(eg.EINVAL, "workspace", ws=OFF8)
    st = eg.DecodeStateStruct(None, 0x50000, 0x60000)
    call(eg.EINVAL, "decode state", st=ctypes.byref(st))
    L.tables.dim = 8                        # d_mem = 32
    call(eg.EUNSUPPORTED, "multiple of 64")


def test_sample_tokens_refusals():
    f = eg.lib().engram_sample_tokens

    def call(status, text, logits=P, dtype=eg.F32, rows=4, V=10, ld=10, t=P, k=P, p=P, m=P, per=2, u=P, tok=P, lp=P):
        _expect(status, text, f, logits, dtype, rows, V, ld, t, k, p, m, per, u, tok, lp, None)

    call(eg.OK, "", rows=0, logits=None, u=None, tok=None)
    call(eg.EUNSUPPORTED, "dtype", dtype=eg.I8)
    call(eg.EINVAL, "rows", rows=-1)
    call(eg.EINVAL, "V", V=0)
    call(eg.EINVAL, "ld", ld=9)
    call(eg.EINVAL, "per", per=0)
    call(eg.EUNSUPPORTED, "2^31", rows=1 << 31)
    call(eg.EUNSUPPORTED, "2^31", V=1 << 31, ld=1 << 31)
    for name in ("logits", "u", "tok"):
        call(eg.EINVAL, "non-NULL", **{name: None})
    for name in ("logits", "t", "k", "p", "m", "u", "tok", "lp"):
        call(eg.EINVAL, "aligned", **{name: ODD})


def test_binding_refusals():
    """Host tensors, wrong types, shapes and strides never reach the library."""
    ids, table = torch.zeros(3, dtype=torch.int32), torch.zeros(5, 16)
    with pytest.raises(ValueError, match="on a GPU"):
        eg.embed(ids, table)
    with pytest.raises(ValueError, match="ids has dtype"):
        eg.embed(ids.long(), table)
    with pytest.raises(ValueError, match="table must be"):
        eg.embed(ids, table[None])
    with pytest.raises(ValueError, match="contiguous"):
        eg.embed(ids, table.t())
    with pytest.raises(ValueError, match="table has dtype"):
        eg.embed(ids, table.half())
    with pytest.raises(ValueError, match="out has shape"):
        eg.embed(ids, table, out=torch.zeros(3, 16))
    dout = torch.zeros(3, 2, 16)
    with pytest.raises(ValueError, match="on a GPU"):
        eg.embed_backward(ids, dout, 5)
    with pytest.raises(ValueError, match="dout must be"):
        eg.embed_backward(ids, dout[:, 0], 5)
    with pytest.raises(ValueError, match="dout has shape"):
        eg.embed_backward(ids, torch.zeros(4, 2, 16), 5)
    with pytest.raises(ValueError, match="accumulate"):
        eg.embed_backward(ids, dout, 5, accumulate=True)
    with pytest.raises(ValueError, match="dtable has shape"):
        eg.embed_backward(ids, dout, 5, dtable=torch.zeros(6, 16))
    with pytest.raises(ValueError, match="ws must be"):
        eg.embed_backward(ids, dout, 5, ws=torch.zeros(9))
    a, b = torch.zeros(2, 8, 64), torch.zeros(2, 128, 8)
    e, w, which = torch.zeros(3, 64), torch.zeros(128, 64), torch.zeros(3, dtype=torch.int32)
    ad = eg.Adapters(a, b)
    with pytest.raises(ValueError, match="on a GPU"):
        eg.project_adapted(e, w, ad, which)
    with pytest.raises(ValueError, match="which has shape"):
        eg.project_adapted(e, w, ad, which, per=2)
    with pytest.raises(ValueError, match="per must"):
        eg.project_adapted(e, w, ad, which, per=0)
    with pytest.raises(ValueError, match="the adapters are"):
        eg.project_adapted(e, torch.zeros(64, 64), ad, which)
    with pytest.raises(ValueError, match="the adapters are"):
        eg.project_adapted(e.bfloat16(), w.bfloat16(), ad, which)
    with pytest.raises(ValueError, match="w has dtype"):
        eg.project_adapted(e, w.bfloat16(), ad, which)
    with pytest.raises(ValueError, match="b has shape"):
        eg.Adapters(a, torch.zeros(2, 128, 16))
    with pytest.raises(ValueError, match="b has dtype"):
        eg.Adapters(a, b.bfloat16())
    with pytest.raises(ValueError, match="scale has shape"):
        eg.Adapters(a, b, torch.zeros(3))
    with pytest.raises(ValueError, match="a must be"):
        eg.Adapters(a[0], b)
    x, u = torch.zeros(2, 3, 10), torch.zeros(2, 3)
    with pytest.raises(ValueError, match="on a GPU"):
        eg.sample_tokens(x, u)
    with pytest.raises(ValueError, match="u has shape"):
        eg.sample_tokens(x, u[0])
    with pytest.raises(ValueError, match="top_k has dtype"):
        eg.sample_tokens(x, u, top_k=torch.zeros(2))
    with pytest.raises(ValueError, match="top_p has shape"):
        eg.sample_tokens(x, u, top_p=torch.zeros(2, 3))
    with pytest.raises(ValueError, match="row stride"):
        eg.sample_tokens(torch.zeros(4, 3, 10)[::2], u)


def test_plain_sampling_by_hand():
    x = np.log(np.array([1.0, 4.0, 2.0, 1.0, 8.0]))                       # weights over 16: 1 4 2 1 8
    assert plain.sample(x, 1.0, 0, 1.0, 0.0, 0.0)[0] == 0
    assert plain.sample(x, 1.0, 0, 1.0, 0.0, 0.07)[0] == 1                # 1/16 = 0.0625
    assert plain.sample(x, 1.0, 0, 1.0, 0.0, 0.49)[0] == 3 and plain.sample(x, 1.0, 0, 1.0, 0.0, 0.51)[0] == 4
    assert plain.sample(x, 1.0, 2, 1.0, 0.0, 0.3)[0] == 1                 # of 4 and 8
    tok, lp, _ = plain.sample(x, 1.0, 2, 1.0, 0.0, 0.4)
    assert tok == 4 and abs(lp - np.log(8 / 12)) < 1e-12
    assert plain.sample(x, 1.0, 0, 0.7, 0.0, 0.3)[0] == 1                 # 8 + 4 reach 0.7 of 16
    assert plain.sample(x, 1.0, 0, 0.8, 0.0, 0.3)[0] == 2                 # 8 + 4 + 2 are needed: 4 | 2 | 8 of 14
    assert plain.sample(x, 1.0, 4, 1.0, 0.0, 0.01)[0] == 0                # of the two ones the first stays
    assert plain.sample(x, 1.0, 0, 1.0, 0.3, 0.2)[0] == 1                 # 4 / 8 reaches min_p, 2 / 8 does not
    assert plain.sample(x, 0.0, 0, 1.0, 0.0, 0.9)[:2] == (4, 0.0)
    assert plain.sample(x, 0.5, 0, 1.0, 0.0, 0.19)[0] == 1                # squares: 1 16 4 1 64 of 86
    assert plain.sample(np.full(3, -np.inf), 1.0, 0, 1.0, 0.0, 0.5)[0] == -1
    assert plain.sample(np.array([0.0, np.nan]), 1.0, 0, 1.0, 0.0, 0.5)[0] == -1


def test_plain_gradient_and_adapters_by_hand():
    d = np.arange(12.0).reshape(3, 2, 2)
    g, size, terms = plain.embed_backward([1, -1, 1], d, 2, 2.0)
    assert g.tolist() == [[0, 0], [2 * (0 + 2 + 8 + 10), 2 * (1 + 3 + 9 + 11)]] and terms.tolist() == [0, 4]
    e = plain.embed(np.array([1, 2, -1]), np.array([[1.0], [3.0]]), 2.0, 2)
    assert e.tolist() == [[[6.0], [6.0]], [[0.0], [0.0]], [[0.0], [0.0]]]
    out, _, _ = plain.project_adapted(np.array([[1.0, 2.0], [1.0, 2.0]]), np.array([[1.0, 1.0]]), np.array([[[3.0, 0.0]]]),
                                      np.array([[[5.0]]]), [2.0], [0, -1])
    assert out.tolist() == [[3.0 + 2 * 5 * 3], [3.0]]


def test_values_of_a_row_on_the_host(tmp_path):
    """Which bf16 values a row's table of weights holds, for every exponent of its largest logit."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    here = os.path.dirname(os.path.abspath(__file__))
    exe = tmp_path / "sample_values_host"
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(os.path.dirname(here), "hashed_gram_embedding_amd", "csrc"),
                    os.path.join(here, "native", "sample_values_host.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "all passed" in r.stdout, r.stdout + r.stderr
