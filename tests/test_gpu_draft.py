"""GPU: the layer over a drafted chunk with the state only read, the commit of
the kept tokens, and a speculative decode loop of all the operators together
against decoding token by token."""
import concurrent.futures
import ctypes
import dataclasses

import numpy as np
import pytest
import torch

from hashed_gram_embedding_amd import engram as eg
from hashed_gram_embedding_amd import inputs
from oracle import engram_oracle as orc

from parity import log

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.int32 if a.element_size() == 4 else torch.int16),
                       b.contiguous().view(torch.int32 if b.element_size() == 4 else torch.int16))


def _state_like(st, S, max_n, M, span, d):
    c = eg.DecodeState(S, max_n, M, span, d, DEV)
    c.ids.copy_(st.ids)
    c.conv.copy_(st.conv)
    c.pos.copy_(st.pos)
    return c


def _chunk_inputs(config, S, T, M=1):
    w = inputs.make_config(config, B=S, T=T + 12, rows_per_table=997)
    lay = w.layers[0]
    return w, lay


CASES = [(1, "bf16", 3, 1), (1, "bf16", 2, 5), (1, "bf16", 3, 9), (1, "bf16", 2, 14), (2, "bf16", 2, 4), (0, "f32", 1, 6)]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("config,hdtype,S,T", CASES)
def test_draft_then_commit_equals_forward(config, hdtype, S, T, int8):
    """forward_draft gives forward's H, alpha and Y bit for bit and leaves the
    state alone; committing every token leaves forward's state bit for bit, and
    committing k tokens the state of the oracle after k tokens."""
    log(f"draft config {config} S={S} T={T} int8={int8}")
    kw = {} if config == 0 else dict(rows_per_table=997)
    w = inputs.make_config(config, B=S, T=T + 12, **kw)
    lay = w.layers[0]
    L = eg.Layer(lay, hdtype, DEV)
    w8 = eg.Int8Weights(L) if int8 else None
    span, max_n = (lay.kernel_w - 1) * lay.dilation, lay.hash.max_n
    tok = torch.from_numpy(w.tokens).to(DEV)
    H = eg.to_device(w.H, hdtype, DEV)
    run = (lambda t, h, st, **k: eg.forward_i8(t, h, L, w8, state=st, **k)) if int8 else \
        (lambda t, h, st, **k: eg.forward(t, h, L, state=st, **k))
    st = eg.DecodeState(S, max_n, lay.branches, span, lay.d, DEV)
    run(tok[:, :12].contiguous(), H[:, :12].contiguous(), st)
    before = _state_like(st, S, max_n, lay.branches, span, lay.d)
    chunk = tok[:, 12:].contiguous()
    ref_st = _state_like(st, S, max_n, lay.branches, span, lay.d)
    h_ref = H[:, 12:].clone(memory_format=torch.contiguous_format)
    a_ref, y_ref = run(chunk, h_ref, ref_st, want_alpha=True, want_y=True)

    draft = eg.Draft(S, T, L, DEV)
    h = H[:, 12:].clone(memory_format=torch.contiguous_format)
    a, y = eg.forward_draft(chunk, h, L, st, draft, w8=w8, want_alpha=True, want_y=True)
    assert _same(h, h_ref) and _same(a, a_ref) and _same(y, y_ref)
    assert torch.equal(st.ids, before.ids) and torch.equal(st.pos, before.pos) and _same(st.conv, before.conv)

    full = _state_like(st, S, max_n, lay.branches, span, lay.d)
    eg.commit_draft(chunk, L, draft, torch.full((S,), T - 1, dtype=torch.int32, device=DEV), full)
    assert torch.equal(full.ids, ref_st.ids) and torch.equal(full.pos, ref_st.pos) and _same(full.conv, ref_st.conv)

    u = (draft.v[:, :lay.d].double().view(S, T, 1, lay.d) * draft.gamma.double().view(S, T, lay.branches, 1)).cpu().numpy()
    state = {"ids": before.ids.cpu().numpy(), "pos": before.pos.cpu().numpy(),
             "u": np.zeros((S, lay.branches, span, lay.d))}
    for r in range(span):                    # the ring as the last `span` inputs, oldest first
        state["u"][:, :, r] = before.conv[:, :, (12 + r) % span].double().cpu().numpy()
    for k in range(-1, T + 1):
        part = _state_like(st, S, max_n, lay.branches, span, lay.d)
        acc = torch.full((S,), k, dtype=torch.int32, device=DEV)
        acc[0] = T - 1 - max(k, 0)
        eg.commit_draft(chunk, L, draft, acc, part)
        kept = np.clip(acc.cpu().numpy() + 1, 0, T)
        ref = orc.commit_draft(state, chunk.cpu().numpy(), lay.hash.proj, u, kept)
        assert np.array_equal(part.ids.cpu().numpy(), ref["ids"]) and np.array_equal(part.pos.cpu().numpy(), ref["pos"])
        for s in range(S):
            at = [(int(ref["pos"][s]) + r) % span for r in range(span)]
            got = part.conv[s][:, at].double().cpu().numpy()
            assert np.all(np.abs(got - ref["u"][s]) <= 2.0 ** -24 * np.abs(ref["u"][s]) + 2.0 ** -149), (k, s)


def _odd_layer(w, kernel_w, dilation):
    """The workload's layer with another short conv."""
    lay = w.layers[0]
    rng = np.random.default_rng(kernel_w * 10 + dilation)
    conv = (0.1 * rng.standard_normal((lay.branches, lay.d, kernel_w))).astype(np.float32)
    return dataclasses.replace(lay, conv_w=conv, kernel_w=kernel_w, dilation=dilation)


SHAPES = [(dict(), 300, 8, (4, 3)), (dict(branches=4, d=256), 40, 60, (4, 3)), (dict(d=256), 3, 1, (4, 3)),
          (dict(branches=2, d=384), 5, 7, (2, 1)), (dict(d=128), 4, 30, (8, 3)), (dict(max_n=4, heads=4, dim=32, d=256), 6, 5, (3, 5)),
          (dict(max_n=2, heads=4, d=256), 6, 5, (4, 2)), (dict(d=4096), 3, 4, (4, 3)), (dict(branches=4, d=1024), 260, 5, (4, 3)),
          (dict(d=192, heads=4), 5, 9, (4, 3))]


# (MXFP8 layers have d a multiple of 128)
@pytest.mark.parametrize("shape,S,T,conv,form", [(*c, f) for c in SHAPES for f in ("bf16", "mxfp8", "int8")
                                                 if f != "mxfp8" or c[0].get("d", 1024) % 128 == 0])
def test_draft_of_other_layers(shape, S, T, conv, form):
    """Other branch counts, widths, orders, convs and forms of Step 5, over
    chunks of one token to many: forward_draft and a commit of all tokens equal
    the forward call bit for bit, and a commit of some the first of them."""
    log(f"draft {shape} S={S} T={T} conv={conv} {form}")
    pre = 5
    w = inputs.make_shape(S, T + pre, **shape)
    lay = _odd_layer(w, *conv)
    L = eg.Layer(lay, "bf16", DEV, mxfp8=form == "mxfp8")
    w8 = eg.Int8Weights(L) if form == "int8" else None
    span, max_n, M = (lay.kernel_w - 1) * lay.dilation, lay.hash.max_n, lay.branches
    tok = torch.from_numpy(np.ascontiguousarray(w.tokens)).to(DEV)
    H = eg.to_device(w.H, "bf16", DEV)
    run = (lambda t, h, st, **k: eg.forward_i8(t, h, L, w8, state=st, **k)) if w8 is not None else \
        (lambda t, h, st, **k: eg.forward(t, h, L, state=st, **k))
    st = eg.DecodeState(S, max_n, M, span, lay.d, DEV)
    run(tok[:, :pre].contiguous(), H[:, :pre].contiguous(), st)
    before, ref = (_state_like(st, S, max_n, M, span, lay.d) for _ in range(2))
    chunk = tok[:, pre:].contiguous()
    hr, h = (H[:, pre:].clone(memory_format=torch.contiguous_format) for _ in range(2))
    ar, yr = run(chunk, hr, ref, want_alpha=True, want_y=True)
    draft = eg.Draft(S, T, L, DEV)
    a, y = eg.forward_draft(chunk, h, L, st, draft, w8=w8, want_alpha=True, want_y=True)
    assert _same(h, hr) and _same(a, ar) and _same(y, yr)
    assert torch.equal(st.ids, before.ids) and torch.equal(st.pos, before.pos) and _same(st.conv, before.conv)
    full = _state_like(st, S, max_n, M, span, lay.d)
    eg.commit_draft(chunk, L, draft, torch.full((S,), T + 3, dtype=torch.int32, device=DEV), full)
    assert torch.equal(full.ids, ref.ids) and torch.equal(full.pos, ref.pos) and _same(full.conv, ref.conv)

    u = (draft.v[:, :lay.d].view(S, T, 1, lay.d) * draft.gamma.view(S, T, M, 1)).permute(0, 2, 1, 3)
    acc = torch.arange(S, dtype=torch.int32, device=DEV) % (T + 1) - 1
    eg.commit_draft(chunk, L, draft, acc, st)
    k = acc.long() + 1
    assert torch.equal(st.pos, before.pos + k.int())
    ids = torch.cat([before.ids, torch.from_numpy(lay.hash.proj).to(DEV)[chunk.long()]], 1)
    assert torch.equal(st.ids, ids.gather(1, k[:, None] + torch.arange(max_n - 1, device=DEV)))
    for s in range(S):
        want = before.conv[s].clone()
        for t in range(int(k[s])):
            want[:, (pre + t) % span] = u[s, :, t]
        assert torch.equal(st.conv[s], want), s


def test_speculative_calls_of_the_debug_build():
    """Raw ids outside the vocabulary are clamped and reported by the debug
    build's draft, commit and int8 calls; clean ones set no bit and give the
    release build's results."""
    log("debug build: speculative calls")
    from hashed_gram_embedding_amd import build as bld
    release = eg.lib()
    S, T = 7, 4
    w = inputs.make_config(3, B=S, T=T, layers=1, rows_per_table=997)
    lay = w.layers[0]
    V = lay.hash.vocab
    bad = np.ascontiguousarray(w.tokens).copy()
    bad[0, 1], bad[3, 3], bad[6, 0] = -5, V, V + 100
    L = eg.Layer(lay, "bf16", DEV)
    w8 = eg.Int8Weights(L)
    h0 = eg.to_device(w.H, "bf16", DEV)
    acc = torch.full((S,), T - 1, dtype=torch.int32, device=DEV)

    def chunk(tokens, read):
        tok = torch.from_numpy(tokens).to(DEV)
        st, h, draft, bits = eg.DecodeState(S, 3, 1, 9, lay.d, DEV), h0.clone(), eg.Draft(S, T, L, DEV), []
        eg.forward_draft(tok, h, L, st, draft, w8=w8)
        bits.append(read())
        eg.commit_draft(tok, L, draft, acc, st)
        bits.append(read())
        one = h0[:, :1].clone(memory_format=torch.contiguous_format)
        eg.forward_i8(tok[:, :1].contiguous(), one, L, w8, state=st)
        bits.append(read())
        return [h, one, st.ids, st.pos, st.conv], bits

    clamped = np.clip(bad, 0, V - 1)
    want, _ = chunk(clamped, lambda: 0)
    got, _ = chunk(bad, lambda: 0)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dbg = eg.load_library(bld.LIB_DEBUG)
    eg._lib = dbg
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    try:
        eg.debug_set_error_word(word)
        clean, bits = chunk(clamped, eg.debug_read_errors)
        assert bits == [0, 0, 0] and all(torch.equal(a, b) for a, b in zip(clean, want))
        got, bits = chunk(bad, eg.debug_read_errors)
        assert bits == [eg.ERR_TOKEN] * 3 and all(torch.equal(a, b) for a, b in zip(got, want))
    finally:
        torch.cuda.synchronize()
        dbg.engram_debug_set_error_word(None)
        eg._lib = release


def test_commit_in_a_graph():
    log("commit graph")
    S, T = 6, 5
    w = inputs.make_config(3, B=S, T=T, layers=1, rows_per_table=997)
    lay = w.layers[0]
    L = eg.Layer(lay, "bf16", DEV)
    tok = torch.from_numpy(np.ascontiguousarray(w.tokens)).to(DEV)
    h0 = eg.to_device(w.H, "bf16", DEV)
    h = h0.clone()
    st, ref = (eg.DecodeState(S, 3, 1, 9, lay.d, DEV) for _ in range(2))
    draft, dr = eg.Draft(S, T, L, DEV), eg.Draft(S, T, L, DEV)
    acc = torch.tensor([-1, 0, 1, 2, 3, 4], dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    eg.forward_draft(tok, h, L, st, draft)   # loads the code; the state is only read
    with torch.cuda.graph(g):
        eg.forward_draft(tok, h, L, st, draft)
        eg.commit_draft(tok, L, draft, acc, st)
    for i in range(4):
        acc.copy_(acc.roll(1))
        h.copy_(h0)
        g.replay()
        torch.cuda.synchronize()
        hr = h0.clone()
        eg.forward_draft(tok, hr, L, ref, dr)
        eg.commit_draft(tok, L, dr, acc, ref)
        assert _same(h, hr) and torch.equal(st.ids, ref.ids) and torch.equal(st.pos, ref.pos) and _same(st.conv, ref.conv), i


def test_operands_elsewhere_are_refused():
    """Buffers in host memory, or for another batch, never reach a kernel."""
    log("draft refusals")
    w = inputs.make_config(3, B=2, T=4, layers=1, rows_per_table=997)
    lay = w.layers[0]
    L = eg.Layer(lay, "bf16", DEV)
    w8 = eg.Int8Weights(L)
    tok = torch.from_numpy(np.ascontiguousarray(w.tokens)).to(DEV)
    H = eg.to_device(w.H, "bf16", DEV)
    st = eg.DecodeState(2, 3, lay.branches, 9, lay.d, DEV)
    acc = torch.zeros(2, dtype=torch.int32, device=DEV)
    draft = eg.Draft(2, 4, L, DEV)
    with pytest.raises(ValueError, match="draft is on cpu"):
        eg.forward_draft(tok, H, L, st, eg.Draft(2, 4, L, "cpu"))
    with pytest.raises(ValueError, match="draft is on cpu"):
        eg.commit_draft(tok, L, eg.Draft(2, 4, L, "cpu"), acc, st)
    with pytest.raises(ValueError, match="layer is on cuda"):
        eg.forward_draft(tok.cpu(), H, L, st, draft)
    with pytest.raises(ValueError, match="n_accepted is on cpu"):
        eg.commit_draft(tok, L, draft, acc.cpu(), st)
    with pytest.raises(ValueError, match="the draft is for"):
        eg.commit_draft(tok[:, :3].contiguous(), L, draft, acc, st)
    with pytest.raises(ValueError, match="ws must be"):
        eg.forward_i8(tok, H, L, w8, ws=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="state.conv has shape"):
        eg.forward_i8(tok, H, L, w8, state=eg.DecodeState(1, 3, lay.branches, 9, lay.d, DEV))
    with pytest.raises(eg.EngramError, match="workspace"):
        eg.forward_i8(tok, H, L, w8, ws=torch.empty(256, dtype=torch.uint8, device=DEV))


def test_int8_decode_in_a_graph():
    """Single-token steps of the int8 layer, whose state advances in the
    projection's launch: captured, replayed between eager work, against eager steps."""
    log("int8 decode graph")
    S = 5
    w = inputs.make_config(3, B=S, T=6, layers=1, rows_per_table=997)
    lay = w.layers[0]
    L = eg.Layer(lay, "bf16", DEV)
    w8 = eg.Int8Weights(L)
    tok = torch.from_numpy(np.ascontiguousarray(w.tokens)).to(DEV)
    h_all = eg.to_device(w.H, "bf16", DEV).view(S, 6, lay.branches, lay.d)
    st, ref = (eg.DecodeState(S, 3, lay.branches, 9, lay.d, DEV) for _ in range(2))
    one, h = tok[:, :1].contiguous(), h_all[:, :1].clone(memory_format=torch.contiguous_format)
    ws = torch.empty(eg.lib().engram_forward_i8_workspace(S, 1, ctypes.byref(L.s)), dtype=torch.uint8, device=DEV)
    eg.forward_i8(one, h.clone(), L, w8, state=_state_like(ref, S, 3, lay.branches, 9, lay.d), ws=ws)   # loads the code
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        eg.forward_i8(one, h, L, w8, state=st, ws=ws)
    for t in range(6):
        one.copy_(tok[:, t:t + 1])
        h.copy_(h_all[:, t:t + 1])
        g.replay()
        torch.cuda.synchronize()
        hr = h_all[:, t:t + 1].clone(memory_format=torch.contiguous_format)
        eg.forward_i8(tok[:, t:t + 1].contiguous(), hr, L, w8, state=ref)
        assert _same(h, hr) and torch.equal(st.ids, ref.ids) and torch.equal(st.pos, ref.pos) and _same(st.conv, ref.conv), t
    assert (st.pos == 6).all()


class _Decoder:
    """A stand-in model: a token embedding, two Engram layers and the product
    with the vocabulary, all products in 8-bit integers."""

    def __init__(self, S, vocab=1500):
        w = inputs.make_config(3, B=S, T=1, rows_per_table=997)
        self.S, self.vocab, self.d = S, vocab, w.layers[0].d
        self.layers = [eg.Layer(lay, "bf16", DEV) for lay in w.layers]
        self.w8 = [eg.Int8Weights(L) for L in self.layers]
        g = torch.Generator(device=DEV).manual_seed(5)
        self.emb = torch.randn(vocab, self.d, generator=g, device=DEV).to(torch.bfloat16)
        self.head = eg.quantize_i8(torch.randn(vocab, self.d, generator=g, device=DEV))

    def states(self):
        return [eg.DecodeState(self.S, 3, 1, 9, self.d, DEV) for _ in self.layers]

    def logits(self, H):
        return eg.project_i8(H.view(self.S, -1, self.d), *self.head, out_dtype="f32")

    def step(self, tok, states):
        H = self.emb[tok.long()].view(self.S, tok.shape[1], 1, self.d).contiguous()
        for L, w8, st in zip(self.layers, self.w8, states):
            eg.forward_i8(tok, H, L, w8, state=st)
        return self.logits(H)

    def chunk(self, tok, states):
        H = self.emb[tok.long()].view(self.S, tok.shape[1], 1, self.d).contiguous()
        drafts = []
        for L, w8, st in zip(self.layers, self.w8, states):
            drafts.append(eg.Draft(self.S, tok.shape[1], L, DEV))
            eg.forward_draft(tok, H, L, st, drafts[-1], w8=w8)
        return self.logits(H), drafts


def test_speculative_decode_loop():
    """Greedy decoding in chunks of drafts of mixed quality, verified and
    committed, gives the tokens and states of decoding token by token."""
    log("speculative loop")
    S, G, new = 5, 4, 16
    m = _Decoder(S)
    greedy = torch.zeros(S, device=DEV)
    rng = torch.Generator(device=DEV).manual_seed(1)
    start = torch.randint(0, m.vocab, (S, 1), generator=rng, device=DEV, dtype=torch.int32)
    no_draft, no_u, half = torch.empty((S, 0), dtype=torch.int32, device=DEV), torch.empty((S, 0), device=DEV), \
        torch.full((S,), 0.5, device=DEV)
    plain, st = [start], m.states()
    for _ in range(new + G + 1):             # without drafts the next token comes from the one row there is
        tok, _ = eg.verify_drafts(eg.token_probs(m.step(plain[-1], st), greedy), None, no_draft, no_u, half)
        plain.append(tok)
    plain = torch.cat(plain, 1)

    st = m.states()
    seqs = [[int(t)] for t in start[:, 0]]
    accepted = steps = 0
    while max(len(s) for s in seqs) < new:
        known = torch.tensor([len(s) for s in seqs], device=DEV)
        d = plain.gather(1, known[:, None] + torch.arange(G, device=DEV))
        good = (torch.arange(S, device=DEV) + steps) % (G + 1)          # right for so many tokens, then not
        d = torch.where(torch.arange(G, device=DEV) < good[:, None], d, (d + 1) % m.vocab).to(torch.int32)
        last = torch.tensor([[s[-1]] for s in seqs], dtype=torch.int32, device=DEV)
        chunk = torch.cat([last, d], 1)
        logits, drafts = m.chunk(chunk, st)
        tok, acc = eg.verify_drafts(eg.token_probs(logits, greedy), None, d, torch.rand(S, G, device=DEV), half)
        assert torch.equal(acc.long(), good)
        for L, s_, dr in zip(m.layers, st, drafts):
            eg.commit_draft(chunk, L, dr, acc, s_)
        for s in range(S):
            seqs[s] += tok[s, :int(acc[s]) + 1].tolist()
        accepted += int(acc.sum())
        steps += 1
    assert accepted > 0
    for s in range(S):
        assert seqs[s] == plain[s, :len(seqs[s])].tolist(), s

    # each state has consumed all but the last known token of its sequence
    ref = m.states()
    for i in range(max(len(s) for s in seqs) - 1):
        m.step(plain[:, i:i + 1].contiguous(), ref)
        for s in range(S):
            if len(seqs[s]) == i + 2:
                for a, b in zip(st, ref):
                    assert int(a.pos[s]) == int(b.pos[s]) == i + 1 and torch.equal(a.ids[s], b.ids[s])
                # layer 0 sees the same hidden states: v is exact, gamma's sums over d = 1024 run in another
                # order in a one-token launch (up to 4 * 1024 roundings through the gate and the norm)
                a, b = st[0].conv[s], ref[0].conv[s]
                assert torch.all((a - b).abs() <= 4096 * 2.0 ** -24 * b.abs() + 2.0 ** -126), s


def _guarded(shape, dtype, fill):
    """A tensor in the middle of a larger allocation: (tensor, check that its surroundings still hold `fill`)."""
    n = int(np.prod(shape))
    buf = torch.full((n + 128,), fill, dtype=dtype, device=DEV)
    return buf[64:64 + n].view(shape), lambda: bool((buf[:64] == fill).all() and (buf[64 + n:] == fill).all())


@pytest.mark.parametrize("S,T,V", [(3, 4, 515), (2, 5, 40001), (70, 1, 40001), (5, 3, 100003), (1, 1, 3)])
def test_nothing_beside_the_outputs_is_written(S, T, V):
    """Outputs in the middle of larger buffers: what lies around them, states of
    other sequences among it, stays."""
    log(f"guarded outputs {S} x {T} x {V}")
    lib, s = eg.lib(), torch.cuda.current_stream().cuda_stream
    x = torch.randn(S, T, V, device=DEV)
    for dtype in (torch.float32, torch.bfloat16):
        p, whole = _guarded((S, T, V), torch.float32, 7.0)
        eg.token_probs(x.to(dtype), probs=p)
        assert whole() and torch.allclose(p.sum(-1), torch.ones(S, T, device=DEV), atol=1e-4)
        xq = x.to(dtype).view(S * T, V)
        q, q_whole = _guarded((S * T, V), torch.int8, 99)
        sc, sc_whole = _guarded((S * T,), torch.float32, 7.0)
        assert lib.engram_quantize_i8(xq.data_ptr(), eg._DT_OF[dtype], S * T, V, q.data_ptr(), sc.data_ptr(), s) == eg.OK
        want = eg.quantize_i8(xq)
        assert q_whole() and sc_whole() and torch.equal(q, want[0]) and torch.equal(sc, want[1])
    G = T - 1
    d = torch.randint(0, V, (S, G), dtype=torch.int32, device=DEV)
    ua, us = torch.rand(S, G, device=DEV), torch.rand(S, device=DEV)
    want = eg.verify_drafts(p, None, d, ua, us)
    tok, tok_whole = _guarded((S, T), torch.int32, -77)
    acc, acc_whole = _guarded((S,), torch.int32, -77)
    need = lib.engram_verify_drafts_workspace(S, V)
    ws, ws_whole = _guarded((need + 256,), torch.uint8, 5)
    base = (ws.data_ptr() + 255) // 256 * 256
    assert lib.engram_verify_drafts(p.data_ptr(), None, eg.F32, d.data_ptr(), None, ua.data_ptr(), us.data_ptr(), S, G, V, tok.data_ptr(),
                                    acc.data_ptr(), base if need else None, need, s) == eg.OK
    assert tok_whole() and acc_whole() and ws_whole() and torch.equal(tok, want[0]) and torch.equal(acc, want[1])

    w = inputs.make_shape(S, T, d=128, branches=2, heads=4)
    lay = w.layers[0]
    L = eg.Layer(lay, "bf16", DEV)
    w8 = eg.Int8Weights(L)
    tk, h0 = torch.from_numpy(np.ascontiguousarray(w.tokens)).to(DEV), eg.to_device(w.H, "bf16", DEV)
    v, v_whole = _guarded((S * T, 128), torch.float32, 7.0)
    gm, gm_whole = _guarded((S * T, 2), torch.float32, 7.0)
    h, h_whole = _guarded(tuple(h0.shape), torch.bfloat16, 7.0)
    h.copy_(h0)
    draft = eg.Draft(S, T, L, DEV, v=v, gamma=gm)
    big = eg.DecodeState(S + 2, 3, 2, 9, 128, DEV)           # the calls' sequences lie between two others
    big.ids.random_(0, 90000)
    big.conv.normal_()
    big.pos.fill_(11)
    was = _state_like(big, S + 2, 3, 2, 9, 128)
    part = eg.DecodeStateStruct(big.ids[1:].data_ptr(), big.conv[1:].data_ptr(), big.pos[1:].data_ptr())
    need = lib.engram_forward_draft_workspace(S, T, ctypes.byref(L.s), ctypes.byref(w8.s))
    ws, ws_whole = _guarded((need + 256,), torch.uint8, 5)
    base = (ws.data_ptr() + 255) // 256 * 256
    assert lib.engram_forward_draft(tk.data_ptr(), h.data_ptr(), S, T, ctypes.byref(L.s), ctypes.byref(w8.s), ctypes.byref(part),
                                    ctypes.byref(draft.s), None, None, base, need, s) == eg.OK
    assert v_whole() and gm_whole() and h_whole() and ws_whole() and not torch.equal(h, h0)
    assert torch.equal(big.ids, was.ids) and torch.equal(big.pos, was.pos) and torch.equal(big.conv, was.conv)
    n = torch.arange(S, dtype=torch.int32, device=DEV) % T
    assert lib.engram_commit_draft(tk.data_ptr(), S, T, ctypes.byref(L.s), ctypes.byref(draft.s), n.data_ptr(), ctypes.byref(part), s) == eg.OK
    for i in (0, S + 1):
        assert torch.equal(big.ids[i], was.ids[i]) and torch.equal(big.conv[i], was.conv[i]) and int(big.pos[i]) == 11
    assert torch.equal(big.pos[1:S + 1], 12 + n)


def test_two_threads_on_two_streams():
    """The operators called from two host threads at once, each with its own
    stream, state and buffers, give what they give one after the other."""
    log("two threads")
    S, T, V = 6, 5, 40000
    w = inputs.make_config(3, B=2 * S, T=T, layers=1, rows_per_table=997)
    lay = w.layers[0]
    L = eg.Layer(lay, "bf16", DEV)
    w8 = eg.Int8Weights(L)
    head = eg.quantize_i8(torch.randn(V, lay.d, device=DEV))
    tok = torch.from_numpy(np.ascontiguousarray(w.tokens)).to(DEV).view(2, S, T)
    h0 = eg.to_device(w.H, "bf16", DEV).view(2, S, T, 1, lay.d)
    ua, us = torch.rand(2, S, T - 1, device=DEV), torch.rand(2, S, device=DEV)

    def steps(i, stream):
        out, st = [], states[i]
        for _ in range(25):
            with torch.cuda.stream(stream):
                h, draft = h0[i].clone(), eg.Draft(S, T, L, DEV)
            eg.forward_draft(tok[i], h, L, st, draft, w8=w8, stream=stream)
            p = eg.token_probs(eg.project_i8(h.view(S, T, lay.d), *head, stream=stream), stream=stream)
            t, a = eg.verify_drafts(p, None, drafted[i], ua[i], us[i], stream=stream)
            eg.commit_draft(tok[i], L, draft, a, st, stream=stream)
            out += [t, a, h]
        stream.synchronize()
        return out + [st.ids, st.conv, st.pos]

    drafted = torch.randint(0, V, (2, S, T - 1), dtype=torch.int32, device=DEV)
    streams = [torch.cuda.Stream() for _ in range(2)]
    results = []
    for parallel in (False, True):
        states = [eg.DecodeState(S, 3, 1, 9, lay.d, DEV) for _ in range(2)]
        torch.cuda.synchronize()
        if parallel:
            with concurrent.futures.ThreadPoolExecutor(2) as ex:
                results.append([f.result() for f in [ex.submit(steps, i, streams[i]) for i in range(2)]])
        else:
            results.append([steps(i, streams[i]) for i in range(2)])
    for a, b in zip(*results):
        assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))
