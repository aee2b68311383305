"""The entry points of the speculative decode step on the CPU: refusals of the
C ABI (fake pointers that never reach a GPU), workspace sizes, refusals of the
binding, and the oracle's own pins."""
import ctypes
import os

import numpy as np
import pytest
import torch

from hashed_gram_embedding_amd import engram as eg
from oracle import engram_oracle as orc

pytestmark = pytest.mark.skipif(not os.path.exists(eg.LIB_PATH), reason="libengram.so not built")

P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)


def _layer():
    """A layer descriptor on fake device pointers (the fields that the host checks)."""
    proj = 0x10000
    mult, prime = np.ones((2, 2, 3), dtype=np.uint64), np.array([1009, 1013, 1019, 1021], dtype=np.uint32)
    off, n = np.array([0, 1009, 2022, 3041], dtype=np.int64), prime.astype(np.int64)
    L = eg.LayerStruct()
    L.hash = eg.HashParams(proj, 1000, 3, 2, mult.ctypes.data, prime.ctypes.data)
    L.tables = eg.Tables(4, 16, eg.F32, 0x10000, off.ctypes.data, n.ctypes.data, 4062, None, None, None, None, 0)
    L.w = 0x30000
    L.gc = eg.GateConvParams(64, 1, 4, 3, 1e-6, eg.F32, 0x20000)
    return L, (mult, prime, off, n)


def _expect(status, text, fn, *args):
    assert fn(*args) == status, eg.last_error()
    if text:
        assert text in eg.last_error(), eg.last_error()


def test_quantize_i8_refusals():
    f = eg.lib().engram_quantize_i8
    _expect(eg.OK, "", f, None, eg.F32, 0, 8, None, None, None)
    _expect(eg.EUNSUPPORTED, "dtype", f, P, eg.I8, 4, 8, P, P, None)
    _expect(eg.EINVAL, "rows", f, P, eg.F32, -1, 8, P, P, None)
    _expect(eg.EINVAL, "cols", f, P, eg.F32, 4, 0, P, P, None)
    _expect(eg.EUNSUPPORTED, "2^31", f, P, eg.F32, 1 << 31, 8, P, P, None)
    for args in ((None, P, P), (P, None, P), (P, P, None)):
        _expect(eg.EINVAL, "non-NULL", f, args[0], eg.F32, 4, 8, args[1], args[2], None)
    _expect(eg.EINVAL, "aligned", f, ODD, eg.BF16, 4, 8, P, P, None)
    _expect(eg.EINVAL, "aligned", f, P, eg.BF16, 4, 8, P, ODD, None)


def test_project_i8_refusals():
    f = eg.lib().engram_project_i8

    def call(status, text, e=P, e_dtype=eg.I8, e_scale=P, w=P, w_scale=P, n=4, k=64, o=8, odt=eg.F32, out=P, ws=None, wsb=0):
        _expect(status, text, f, e, e_dtype, e_scale, w, w_scale, n, k, o, odt, out, ws, wsb, None)

    call(eg.OK, "", n=0, e=None, w=None, out=None)
    call(eg.EUNSUPPORTED, "e_dtype", e_dtype=7)
    call(eg.EUNSUPPORTED, "out_dtype", odt=eg.I8)
    call(eg.EINVAL, "n_tok", n=-1)
    call(eg.EINVAL, "d_mem", k=0)
    call(eg.EINVAL, "n_out", o=0)
    call(eg.EUNSUPPORTED, "131071", k=131072)
    call(eg.EUNSUPPORTED, "2^31", n=1 << 31)
    call(eg.EUNSUPPORTED, "2^31", o=1 << 31)
    for name in ("e", "w", "w_scale", "out"):
        call(eg.EINVAL, "non-NULL", **{name: None})
    call(eg.EINVAL, "e_scale", e_scale=None)
    call(eg.EINVAL, "e_scale", e_dtype=eg.BF16)                              # codes' scale with float rows
    call(eg.EINVAL, "aligned", e_scale=ODD)
    call(eg.EINVAL, "aligned", out=ODD)
    call(eg.EINVAL, "aligned", w_scale=ODD)
    call(eg.EINVAL, "16-byte", e=ctypes.c_void_p(0x10008))
    call(eg.EINVAL, "16-byte", w=ctypes.c_void_p(0x10008))
    need = eg.lib().engram_project_i8_workspace(400, 64, 8, eg.BF16)
    assert need >= 400 * 64 + 1600 and eg.lib().engram_project_i8_workspace(400, 64, 8, eg.I8) == 0
    assert eg.lib().engram_project_i8_workspace(400, 70, 8, eg.I8) >= 400 * 80 + 8 * 80
    call(eg.EINVAL, "workspace", n=400, e_dtype=eg.BF16, e_scale=None)
    call(eg.EINVAL, "workspace", n=400, e_dtype=eg.BF16, e_scale=None, ws=P, wsb=need - 1)
    call(eg.EINVAL, "workspace", n=400, e_dtype=eg.BF16, e_scale=None, ws=ctypes.c_void_p(0x10010), wsb=need)


def test_token_probs_refusals():
    f = eg.lib().engram_token_probs

    def call(status, text, logits=P, dtype=eg.F32, rows=4, V=10, ld=10, t=P, per=2, probs=P, ws=P, wsb=1 << 40):
        _expect(status, text, f, logits, dtype, rows, V, ld, t, per, probs, ws, wsb, None)

    call(eg.OK, "", rows=0, logits=None, probs=None)
    call(eg.EUNSUPPORTED, "dtype", dtype=eg.I8)
    call(eg.EINVAL, "rows", rows=-1)
    call(eg.EINVAL, "V", V=0)
    call(eg.EINVAL, "ld", ld=9)
    call(eg.EINVAL, "per", per=0)
    call(eg.EUNSUPPORTED, "2^31", rows=1 << 31)
    call(eg.EUNSUPPORTED, "2^31", V=1 << 31, ld=1 << 31)
    call(eg.EINVAL, "non-NULL", logits=None)
    call(eg.EINVAL, "non-NULL", probs=None)
    call(eg.EINVAL, "aligned", logits=ODD)
    call(eg.EINVAL, "aligned", probs=ODD)
    call(eg.EINVAL, "aligned", t=ODD)


def test_verify_drafts_refusals():
    f = eg.lib().engram_verify_drafts
    need = eg.lib().engram_verify_drafts_workspace(4, 100000)
    assert need > 0 and eg.lib().engram_verify_drafts_workspace(0, 100000) == 0

    def call(status, text, target=P, draft=P, dtype=eg.F32, drafted=P, n=None, ua=P, us=P, S=4, G=2, V=100000, tok=P, acc=P,
             ws=P, wsb=need):
        _expect(status, text, f, target, draft, dtype, drafted, n, ua, us, S, G, V, tok, acc, ws, wsb, None)

    call(eg.OK, "", S=0, target=None)
    call(eg.EUNSUPPORTED, "dtype", dtype=eg.I8)
    call(eg.EINVAL, "S >= 0", S=-1)
    call(eg.EINVAL, "G >= 0", G=-1)
    call(eg.EINVAL, "V >= 1", V=0)
    call(eg.EUNSUPPORTED, "65535", S=65536)
    call(eg.EUNSUPPORTED, "G above", G=eg.MAX_DRAFTS + 1)
    call(eg.EUNSUPPORTED, "V above", V=1 << 31)
    for name in ("target", "us", "tok", "acc"):
        call(eg.EINVAL, "non-NULL", **{name: None})
    for name in ("drafted", "ua"):
        call(eg.EINVAL, "G > 0", **{name: None})
    for name in ("target", "draft", "drafted", "n", "ua", "us", "tok", "acc"):
        call(eg.EINVAL, "aligned", **{name: ODD})
    call(eg.EINVAL, "workspace", ws=None)
    call(eg.EINVAL, "workspace", wsb=need - 1)
    call(eg.EINVAL, "workspace", ws=ctypes.c_void_p(0x10010))


def test_layer_calls_refusals():
    L, keep = _layer()
    lib, lp = eg.lib(), ctypes.byref(L)
    w8 = eg.I8WeightsStruct(0x20000, 0x30000)
    st = eg.DecodeStateStruct(0x40000, 0x50000, 0x60000)
    d, M = L.gc.d, L.gc.branches
    need = lib.engram_forward_i8_workspace(2, 4, lp)
    assert need > 0 and lib.engram_forward_i8_workspace(2, 4, None) == 0
    big = 1 << 40

    def i8(status, text, tok=P, H=P, B=2, T=4, layer=lp, w=ctypes.byref(w8), state=None, ws=P, wsb=big):
        _expect(status, text, lib.engram_forward_i8, tok, H, B, T, layer, w, state, None, None, ws, wsb, None)

    i8(eg.OK, "", B=0)
    i8(eg.EINVAL, "int8 weights", w=None)
    i8(eg.EINVAL, "int8 w", w=ctypes.byref(eg.I8WeightsStruct(None, 0x30000)))
    i8(eg.EINVAL, "int8 w", w=ctypes.byref(eg.I8WeightsStruct(0x20000, None)))
    i8(eg.EINVAL, "aligned", w=ctypes.byref(eg.I8WeightsStruct(0x20000, 0x30002)))
    i8(eg.EINVAL, "layer", layer=None)
    i8(eg.EINVAL, "tokens", tok=None)
    i8(eg.EINVAL, "H", H=None)
    i8(eg.EINVAL, "workspace", wsb=need - 1)
    i8(eg.EINVAL, "decode state", state=ctypes.byref(eg.DecodeStateStruct(None, 0x50000, 0x60000)))

    stride = lib.engram_draft_stride(lp)
    assert stride in (d, (1 + M) * d) and lib.engram_draft_stride(None) == 0
    dr = eg.DraftStruct(0x70000, stride, 0x80000)

    def fwd(status, text, state=ctypes.byref(st), draft=ctypes.byref(dr), layer=lp, w=None, wsb=big, tok=P):
        _expect(status, text, lib.engram_forward_draft, tok, P, 2, 4, layer, w, state, draft, None, None, P, wsb, None)

    fwd(eg.EINVAL, "decode state", state=None)
    fwd(eg.EINVAL, "draft", draft=None)
    fwd(eg.EINVAL, "draft", draft=ctypes.byref(eg.DraftStruct(None, stride, 0x80000)))
    fwd(eg.EINVAL, "aligned", draft=ctypes.byref(eg.DraftStruct(0x70004, stride, 0x80000)))
    fwd(eg.EINVAL, "v_stride", draft=ctypes.byref(eg.DraftStruct(0x70000, stride + 4, 0x80000)))
    fwd(eg.EINVAL, "layer", layer=None)
    fwd(eg.EINVAL, "tokens", tok=None)
    fwd(eg.EINVAL, "workspace", wsb=lib.engram_forward_draft_workspace(2, 4, lp, None) - 1)

    def commit(status, text, tok=P, B=2, T=4, layer=lp, draft=ctypes.byref(dr), acc=P, state=ctypes.byref(st)):
        _expect(status, text, lib.engram_commit_draft, tok, B, T, layer, draft, acc, state, None)

    commit(eg.OK, "", T=0)
    commit(eg.EINVAL, "decode state", state=None)
    commit(eg.EINVAL, "draft", draft=None)
    commit(eg.EINVAL, "n_accepted", acc=None)
    commit(eg.EINVAL, "tokens", tok=None)
    commit(eg.EINVAL, "layer", layer=None)
    commit(eg.EINVAL, "v_stride", draft=ctypes.byref(eg.DraftStruct(0x70000, d - 4, 0x80000)))
    commit(eg.EINVAL, "v_stride", draft=ctypes.byref(eg.DraftStruct(0x70000, d + 2, 0x80000)))


def test_binding_refuses_what_it_would_misread():
    """The binding names the argument: host tensors, other dtypes and shapes, rows that are not contiguous."""
    x, w, s = torch.zeros(4, 32), torch.zeros((8, 32), dtype=torch.int8), torch.zeros(8)
    with pytest.raises(ValueError, match="on a GPU"):
        eg.project_i8(x, w, s)
    with pytest.raises(ValueError, match="w has shape"):
        eg.project_i8(x, w[:, :16].contiguous(), s)
    with pytest.raises(ValueError, match="w must be contiguous"):
        eg.project_i8(x, torch.zeros((32, 8), dtype=torch.int8).t(), s)
    with pytest.raises(ValueError, match="e has dtype"):
        eg.project_i8(x.half(), w, s)
    with pytest.raises(ValueError, match="e has dtype"):
        eg.project_i8(x, w, s, e_scale=torch.zeros(4))
    with pytest.raises(ValueError, match="w_scale has shape"):
        eg.project_i8(x, w, s[:5])
    with pytest.raises(ValueError, match="out has dtype"):
        eg.project_i8(x, w, s, out_dtype="bf16", out=torch.zeros(4, 8))
    with pytest.raises(ValueError, match="x has dtype"):
        eg.quantize_i8(w)
    l3 = torch.zeros(2, 3, 10)
    with pytest.raises(ValueError, match="row stride"):
        eg.token_probs(l3.transpose(0, 1))
    with pytest.raises(ValueError, match="temperature has shape"):
        eg.token_probs(l3, torch.zeros(3))
    with pytest.raises(ValueError, match="uint8 tensor on cpu, not torch.float32"):
        eg.token_probs(torch.zeros(1, 40000), ws=torch.zeros(4096))
    with pytest.raises(ValueError, match="uint8 tensor on cpu, not torch.uint8 on meta"):
        eg.token_probs(torch.zeros(1, 40000), ws=torch.zeros(4096, dtype=torch.uint8, device="meta"))
    with pytest.raises(ValueError, match=r"\[S, R, V\]"):
        eg.token_probs(l3[0, 0])
    p, q, d, ua, us = torch.zeros(2, 4, 9), torch.zeros(2, 3, 9), torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, 3), torch.zeros(2)
    with pytest.raises(ValueError, match="draft has dtype"):
        eg.verify_drafts(p, q.bfloat16(), d, ua, us)
    with pytest.raises(ValueError, match="target has shape"):
        eg.verify_drafts(p[:, :3].contiguous(), q, d, ua, us)
    with pytest.raises(ValueError, match="drafted has dtype"):
        eg.verify_drafts(p, q, d.long(), ua, us)
    with pytest.raises(ValueError, match="n_draft has shape"):
        eg.verify_drafts(p, q, d, ua, us, n_draft=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="on a GPU"):
        eg.verify_drafts(p, q, d, ua, us)


def test_binding_refuses_drafts_and_weights_of_another_layer():
    """A draft's gamma and int8 weights are sized by the layer they were made
    for: with another layer's sizes the kernels would leave them.  (With d the
    same, a fused layer's v rows are as long whatever its branches.)"""
    from hashed_gram_embedding_amd import inputs
    B, T, d = 2, 3, 128
    layers = [inputs.make_shape(B, T, heads=2, dim=32, d=n, branches=m).layers[0] for n, m in ((d, 1), (d, 4), (2 * d, 1), (2 * d, 4))]
    one, four, wide, wide4 = (eg.Layer(lay, "bf16", "cpu", bf16_packed=False) for lay in layers)
    tok, acc = torch.zeros((B, T), dtype=torch.int32), torch.zeros(B, dtype=torch.int32)

    def state(L):
        return eg.DecodeState(B, 3, L.M, 9, L.d, "cpu")

    def hidden(L):
        return torch.zeros((B, T, L.M, L.d), dtype=torch.bfloat16)

    def weights(L):
        return eg.Int8Weights(L, torch.zeros(L.w.shape, dtype=torch.int8), torch.zeros(L.w.shape[0]))

    for L, other in ((four, one), (one, four), (wide, one), (wide4, four)):
        for draft in (eg.Draft(B, T, other, "cpu"), eg.Draft(B, T, other, "cpu", v=torch.zeros(B * T, d))):
            with pytest.raises(ValueError, match="the draft is for a layer of"):
                eg.forward_draft(tok, hidden(L), L, state(L), draft)
            with pytest.raises(ValueError, match="the draft is for a layer of"):
                eg.commit_draft(tok, L, draft, acc, state(L))
        own = eg.Draft(B, T, L, "cpu")
        with pytest.raises(ValueError, match="the int8 weights are"):
            eg.forward_draft(tok, hidden(L), L, state(L), own, w8=weights(other))
        with pytest.raises(ValueError, match="the int8 weights are"):
            eg.forward_i8(tok, hidden(L), L, weights(other))
        elsewhere = weights(L)
        elsewhere.q = elsewhere.q.to("meta")
        with pytest.raises(ValueError, match="the int8 weights are on meta"):
            eg.forward_i8(tok, hidden(L), L, elsewhere)
        # those of the layer itself pass these checks (and stop at the host tensors)
        for call in (lambda: eg.forward_draft(tok, hidden(L), L, state(L), own, w8=weights(L)),
                     lambda: eg.forward_i8(tok, hidden(L), L, weights(L)), lambda: eg.commit_draft(tok, L, own, acc, state(L))):
            with pytest.raises(ValueError, match="on a GPU"):
                call()


def test_oracle_quantize_i8_by_hand():
    q, s = orc.quantize_i8(np.array([[254.0, 127.0, 1.0, -3.0, 0.5], [0.0] * 5, [np.inf, 1, 2, 3, 4]]))
    assert q[0].tolist() == [127, 64, 0, -2, 0]      # 63.5, 0.5, -1.5 to even, 0.25
    assert s[0] == 2.0 and s[1] == 0 and np.isnan(s[2]) and not q[1:].any()


def test_oracle_verification_by_hand():
    p = np.array([[0.5, 0.25, 0.25], [0.0, 0.5, 0.5], [1.0, 0.0, 0.0]])
    q = np.array([[0.25, 0.5, 0.25], [0.0, 0.0, 1.0]])
    # draft 0 (token 1) has p/q = 1/2; draft 1 (token 2) has 1/2
    assert orc.verify_drafts(p, q, [1, 2], [0.4, 0.4], 0.9, 2)[0].tolist() == [1, 2, 0]
    out, a = orc.verify_drafts(p, q, [1, 2], [0.5, 0.4], 0.9, 2)      # refused at the border; p - q leaves token 0
    assert a == 0 and out.tolist() == [0, -1, -1]
    out, a = orc.verify_drafts(p, q, [1, 2], [0.4, 0.5], 0.0, 2)
    assert a == 1 and out.tolist() == [1, 1, -1]
    out, a = orc.verify_drafts(p, None, [0, 1], [0.4, 0.4], 0.0, 1)   # one draft of two
    assert a == 1 and out.tolist() == [0, 1, -1]
    out, a = orc.verify_drafts(p, None, [0, 1], [0.5, 0.4], 0.5, 2)   # 1/4 and 1/4 without token 0: the border is token 2's
    assert a == 0 and out.tolist() == [2, -1, -1]
    assert orc.verify_drafts(0 * p, q, [1, 2], [0.0, 0.0], 0.5, 2)[0].tolist() == [-1, -1, -1]


def test_oracle_verification_keeps_the_target():
    """Exact check over a grid of random numbers: the first token's distribution is p whatever q is."""
    rng = np.random.default_rng(0)
    n = 64
    p, q = rng.multinomial(n, np.ones(4) / 4) / n, rng.multinomial(n, np.ones(4) / 4) / n
    share = np.zeros(4)
    for x in range(4):
        take = min(1.0, p[x] / q[x]) if q[x] > 0 else 0.0
        share[x] += q[x] * take
        rest = np.maximum(p - q, 0)
        if rest.sum() > 0:
            share += q[x] * (1 - take) * rest / rest.sum()
            for u in (np.arange(n) + 0.5) / n:
                if u * q[x] >= p[x] and q[x] > 0:
                    out, a = orc.verify_drafts(np.array([p, p]), q[None], [x], [u], u, 1)
                    assert a == 0 and rest[out[0]] > 0
    assert np.allclose(share, p, atol=1e-12)


def test_oracle_commit_by_hand():
    proj = np.arange(10, 20)
    st = orc.new_state(1, 3, 1, 3, 1)
    st["u"][0, 0, :, 0] = [7, 8, 9]
    st["ids"][0] = [4, 5]
    u = np.array([1.0, 2.0, 3.0, 4.0]).reshape(1, 4, 1, 1)
    for kept, ids, ring in ((0, [4, 5], [7, 8, 9]), (1, [5, 13], [8, 9, 1]), (4, [11, 10], [2, 3, 4])):
        r = orc.commit_draft(st, np.array([[3, 2, 1, 0]]), proj, u, np.array([kept]))
        assert r["ids"][0].tolist() == ids and r["u"][0, 0, :, 0].tolist() == ring and r["pos"][0] == kept
