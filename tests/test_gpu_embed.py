"""GPU: token embeddings and their gradient against float64.

Tolerances: an embedding is one float32 product (half a step, 2^-24), rounded
once more (2^-8) for bf16.  A gradient of c terms is c - 1 float32 additions in
some order, each off by at most 2^-24 of the running sum, which the terms'
magnitudes bound; the scaling and (accumulating) the last addition add one
each, bf16 output 2^-8 of the value."""
import numpy as np
import pytest
import torch

import plain_around as plain
from hashed_gram_embedding_amd import engram as eg
from parity import log

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 2.0 ** -24
TINY = 2.0 ** -126


def _f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("in_t,out_t", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("n,V,dim,branches", [(1, 1, 8, 1), (3, 5, 24, 2), (257, 100, 1000, 1), (70, 999, 1024, 4), (33, 50, 4104, 3)])
def test_embed(in_t, out_t, n, V, dim, branches):
    log(f"embed {in_t} {out_t} {n} {V} {dim} {branches}")
    g = torch.Generator(device=DEV).manual_seed(n)
    table = torch.randn(V, dim, generator=g, device=DEV).to(TYPES[in_t])
    ids = torch.randint(-2, V + 2, (n,), generator=g, device=DEV, dtype=torch.int32)
    ids[0] = V - 1
    scale = float(np.float32(dim ** 0.5))
    out = eg.embed(ids, table, scale=scale, branches=branches, out_dtype=out_t)
    assert out.shape == (n, branches, dim) and out.dtype == TYPES[out_t]
    ref = plain.embed(ids.cpu().numpy(), _f64(table), scale, branches)
    tol = (EPS * (1 + 2.0 ** -7) + (2.0 ** -8 if out_t == "bf16" else 0.0)) * np.abs(ref) + TINY
    assert (np.abs(_f64(out) - ref) <= tol).all()


def test_embed_extremes():
    """Ids far outside, rows of infinities and NaN, a batch of shape [B, T], the output's surroundings."""
    log("embed extremes")
    table = torch.randn(6, 16, device=DEV)
    table[1] = float("inf")
    table[2] = float("nan")
    ids = torch.tensor([[0, 1, 2], [-2 ** 31, 2 ** 31 - 1, 6]], dtype=torch.int32, device=DEV)
    whole = torch.full((8, 2, 16), 7.0, device=DEV)
    out = eg.embed(ids, table, scale=2.0, branches=2, out=whole[1:7].view(2, 3, 2, 16))
    assert torch.equal(out[0, 0, 1], 2 * table[0]) and torch.isinf(out[0, 1]).all() and torch.isnan(out[0, 2]).all()
    assert (out[1] == 0).all() and (whole[0] == 7).all() and (whole[7] == 7).all()
    assert eg.embed(ids[:0], table).shape == (0, 3, 1, 16)


def test_embed_past_32_bits():
    """A table of more than 2^32 bytes and rows at its far end; outputs of more than 2^31 elements."""
    log("embed past 32 bits")
    V, dim = (1 << 22) + 3, 1032
    table = torch.zeros(V, dim, dtype=torch.bfloat16, device=DEV)
    table[V - 1] = 3.0
    ids = torch.full((300000,), V - 2, dtype=torch.int32, device=DEV)
    ids[-1] = V - 1
    out = eg.embed(ids, table, scale=0.5, branches=8)
    assert out.numel() > 1 << 31
    assert (out[-1] == 1.5).all() and (out[-2] == 0).all()
    d = eg.embed_backward(ids, out, V, dtable=table.zero_(), accumulate=True)
    assert (d[V - 1] == 12.0).all() and (d[V - 2] == 0).all()


def _grad_case(n, V, dim, branches, in_t, ids, scale, out_t, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dout = (torch.randn(n, branches, dim, generator=g, device=DEV) *
            torch.exp2(torch.randint(-6, 6, (n, 1, 1), generator=g, device=DEV).float())).to(TYPES[in_t])
    got = eg.embed_backward(ids, dout, V, scale=scale, out_dtype=out_t)
    ref, size, terms = plain.embed_backward(ids.cpu().numpy(), _f64(dout), V, scale)
    tol = EPS * (terms[:, None] + 2) * size + (2.0 ** -8 if out_t == "bf16" else 0.0) * np.abs(ref) + TINY
    assert (np.abs(_f64(got) - ref) <= tol).all()
    assert torch.equal(got, eg.embed_backward(ids, dout, V, scale=scale, out_dtype=out_t))   # the same bits
    return dout, got


@pytest.mark.parametrize("in_t,out_t", [("bf16", "f32"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("n,V,dim,branches", [(1, 1, 8, 1), (2, 3, 24, 4), (63, 40, 64, 1), (64, 5, 1000, 2), (65, 700, 2056, 1),
                                              (1000, 90, 64, 3), (4097, 300, 40, 1)])
def test_gradient(in_t, out_t, n, V, dim, branches):
    log(f"embed_backward {in_t} {out_t} {n} {V} {dim} {branches}")
    g = torch.Generator(device=DEV).manual_seed(n + 1)
    ids = torch.randint(-2, V + 2, (n,), generator=g, device=DEV, dtype=torch.int32)
    _grad_case(n, V, dim, branches, in_t, ids, float(np.float32(1.7)), out_t, n)


@pytest.mark.parametrize("n", [31, 32, 33, 4096, 16384, 16385, 20481])
@pytest.mark.parametrize("kind", ["one", "two", "ascending", "descending", "padding", "heavy"])
def test_gradient_orders(n, kind):
    """One id throughout, runs that end at and inside tiles, sorted and reversed ids, nothing but padding; both sorts."""
    log(f"embed_backward orders {n} {kind}")
    V = 70000
    i = torch.arange(n, device=DEV)
    ids = {"one": torch.full_like(i, 69999), "two": torch.where(i % 3 == 0, 5, 65536), "ascending": i * 3 % V,
           "descending": (n - 1 - i) * 3 % V, "padding": torch.full_like(i, -1),
           "heavy": torch.where(i % 5 < 3, 256, (i * 7919) % V)}[kind].to(torch.int32)
    dout, got = _grad_case(n, V, 8, 1, "f32", ids, 1.0, "f32", n)
    if kind == "padding":
        assert (got == 0).all()


@pytest.mark.parametrize("V", [1, 255, 256, 65535, 65536, 70001, (1 << 24) - 1, 1 << 24])
def test_gradient_digits(V):
    """Tables around the ends of the sort's digits, first and last rows among the ids."""
    log(f"embed_backward V={V}")
    n = 17000
    g = torch.Generator(device=DEV).manual_seed(V)
    ids = torch.randint(0, V, (n,), generator=g, device=DEV, dtype=torch.int32)
    ids[:4] = torch.tensor([V - 1, 0, V, -1], dtype=torch.int32)
    dout = torch.randint(-8, 9, (n, 1, 8), generator=g, device=DEV).float()   # whole numbers: sums are exact
    ref = torch.zeros(V + 1, 8, device=DEV, dtype=torch.float64)
    at = torch.where((ids >= 0) & (ids < V), ids, V).long()
    ref.index_add_(0, at, dout[:, 0].double())
    assert torch.equal(eg.embed_backward(ids, dout, V).double(), ref[:V])


@pytest.mark.parametrize("out_t", ["f32", "bf16"])
@pytest.mark.parametrize("n", [0, 50, 17000])
def test_gradient_accumulates(n, out_t):
    """Rows without an id keep their bits (an infinity and a NaN among them), the others get the sum added."""
    log(f"embed_backward accumulate {n} {out_t}")
    V, dim = 500, 64
    g = torch.Generator(device=DEV).manual_seed(3)
    ids = (torch.randint(0, V // 2, (n,), generator=g, device=DEV) * 2).to(torch.int32)
    dout = torch.randint(-4, 5, (n, 2, dim), generator=g, device=DEV).to(torch.bfloat16)
    old = torch.randint(-4, 5, (V, dim), generator=g, device=DEV).to(TYPES[out_t])
    old[1] = float("inf")
    old[3] = float("nan")
    ref = old.double().index_add_(0, ids.long(), dout.double().sum(1) * 0.5).to(TYPES[out_t])
    got = old.clone()
    assert eg.embed_backward(ids, dout, V, scale=0.5, dtable=got, accumulate=True) is got
    assert torch.equal(got.nan_to_num(9.0), ref.nan_to_num(9.0))


def test_gradient_with_nothing():
    log("embed_backward n=0")
    ids = torch.zeros(0, dtype=torch.int32, device=DEV)
    whole = torch.full((7, 8), 5.0, device=DEV)
    eg.embed_backward(ids, torch.zeros(0, 1, 8, device=DEV), 5, dtable=whole[1:6])
    assert (whole[1:6] == 0).all() and (whole[0] == 5).all() and (whole[6] == 5).all()


def test_gradient_is_the_derivative():
    """Against differences of the lookup itself: L = sum(c * embed(E)) is linear in E, so a difference over a step of
    any size is exact up to the roundings of the lookup's float32 outputs."""
    log("embed_backward against differences")
    g = torch.Generator(device=DEV).manual_seed(8)
    V, dim, n, M = 13, 16, 50, 2
    table = torch.randn(V, dim, generator=g, device=DEV)
    ids = torch.randint(-1, V, (n,), generator=g, device=DEV, dtype=torch.int32)
    c = torch.randn(n, M, dim, generator=g, device=DEV)
    grad = eg.embed_backward(ids, c, V, scale=1.5)
    step = 0.25
    for v, k in [(0, 0), (5, 7), (12, 15), (3, 2)]:
        up, down = table.clone(), table.clone()
        up[v, k] += step
        down[v, k] -= step
        a, b = eg.embed(ids, up, scale=1.5, branches=M), eg.embed(ids, down, scale=1.5, branches=M)
        diff = float((c.double() * (a.double() - b.double())).sum()) / float(up[v, k].double() - down[v, k].double())
        uses = int((ids == v).sum()) * M
        tol = EPS * float(c.abs().max()) * uses * (2 * float(a.abs().max()) / step + 8 * uses)
        assert abs(diff - float(grad[v, k])) <= tol


def test_hashed_table_gradient():
    """Rows of a layer's hashed tables: the gradient of the gather, on the indices that the gather used."""
    log("embed_backward of hashed tables")
    from hashed_gram_embedding_amd import inputs
    lay = inputs.make_config(1, B=2, T=40, rows_per_table=97).layers[0]
    w = inputs.make_config(1, B=2, T=40, rows_per_table=97)
    L = eg.Layer(lay, "bf16", DEV)
    tokens = torch.from_numpy(w.tokens).to(DEV)
    z = eg.hash_indices(tokens, L)
    rows = (z.long() + torch.from_numpy(L.row_offset).to(DEV)).to(torch.int32)
    nt, dim = z.shape[-1], L.li.tables.dim
    g = torch.Generator(device=DEV).manual_seed(1)
    de = torch.randint(-4, 5, (*z.shape, 1, dim), generator=g, device=DEV).to(torch.bfloat16)   # [B, T, nt * dim] as rows
    total = int(L.s.tables.total_rows)
    got = eg.embed_backward(rows, de, total)
    ref = torch.zeros(total, dim, dtype=torch.float64, device=DEV).index_add_(0, rows.flatten().long(), de.double().view(-1, dim))
    assert torch.equal(got.double(), ref)
    table = L.rows.view(total, dim)
    e = eg.gather(z, L).view(*z.shape, 1, dim)
    assert torch.equal(eg.embed(rows, table), e)


@pytest.mark.parametrize("n", [17000, 70001])
@pytest.mark.parametrize("V", [511, 512, (1 << 18) - 1, 1 << 18, (1 << 27) - 1, 1 << 27])
def test_gradient_ends_of_digits(V, n):
    """Tables at the ends of the sort's 9-bit digits, where the padding's key takes one more, for both lengths of its
    workgroups' shares: every row, in whole numbers."""
    log(f"embed_backward ends of digits V={V} n={n}")
    g = torch.Generator(device=DEV).manual_seed(V + n)
    ids = torch.randint(0, V, (n,), generator=g, device=DEV, dtype=torch.int32)
    ids[::5] = V - 1 - ids[::5] % 3
    ids[:6] = torch.tensor([V - 1, 0, V, -1, 2 ** 31 - 1, V - 1], dtype=torch.int32)
    ids[-2:] = torch.tensor([V, V - 1], dtype=torch.int32)
    dout = torch.randint(-8, 9, (n, 1, 8), generator=g, device=DEV).float()
    at = torch.where((ids >= 0) & (ids < V), ids, V).long()
    ref = torch.zeros(V + 1, 8, device=DEV).index_add_(0, at, dout[:, 0])
    assert torch.equal(eg.embed_backward(ids, dout, V), ref[:V])


@pytest.mark.parametrize("n", [12284, 12288, 12292, 65536, 65540, 131076])
@pytest.mark.parametrize("V", [40000, 1 << 18, 1 << 27])
def test_gradient_adds_in_the_order_of_positions(n, V):
    """Every id four times, anywhere: the bits of their sum in the order of their positions, on both sides of the numbers
    of ids at which the sort changes."""
    log(f"embed_backward order n={n} V={V}")
    g = torch.Generator(device=DEV).manual_seed(n)
    different = n // 4
    rows = torch.arange(different, device=DEV) * (V // different)
    ids = rows.repeat_interleave(4)[torch.randperm(n, generator=g, device=DEV)]
    dout = torch.randn(n, 1, 8, generator=g, device=DEV) * torch.exp2(torch.randint(-12, 13, (n, 1, 1), generator=g, device=DEV).float())
    d = dout[torch.argsort(ids, stable=True), 0].view(different, 4, 8)
    ref = torch.zeros(V, 8, device=DEV)
    ref[rows] = ((d[:, 0] + d[:, 1]) + d[:, 2]) + d[:, 3]
    other = torch.zeros(V, 8, device=DEV)
    other[rows] = ((d[:, 3] + d[:, 2]) + d[:, 1]) + d[:, 0]
    assert not torch.equal(ref, other)
    assert torch.equal(eg.embed_backward(ids.int(), dout, V), ref)
