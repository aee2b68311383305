"""The operators around the layer in float64 numpy, written from their
definitions (tests only)."""
import numpy as np


def embed(ids, table, scale, branches):
    ids = np.asarray(ids)
    ok = (ids >= 0) & (ids < table.shape[0])
    rows = np.where(ok[..., None], table[np.where(ok, ids, 0)] * scale, 0.0)
    return np.repeat(rows[..., None, :], branches, axis=-2)


def embed_backward(ids, dout, vocab, scale):
    """The gradient, and the sums of magnitudes and the numbers of terms behind it."""
    n, m, dim = dout.shape
    grad, size, terms = np.zeros((vocab, dim)), np.zeros((vocab, dim)), np.zeros(vocab)
    for i in range(n):
        v = int(ids[i])
        if 0 <= v < vocab:
            grad[v] += dout[i].sum(0)
            size[v] += np.abs(dout[i]).sum(0)
            terms[v] += m
    return grad * scale, size * abs(scale), terms


def project_adapted(e, w, a, b, scale, owner):
    """out = W e + s B (A e), and the size of the terms that a float32
    evaluation rounds: of the sums, and of h as it is carried on."""
    out, size, carried = e @ w.T, np.abs(e) @ np.abs(w).T, np.zeros((e.shape[0], w.shape[0]))
    for t, i in enumerate(owner):
        if 0 <= i < a.shape[0]:
            s = 1.0 if scale is None else float(scale[i])
            h = s * (a[i] @ e[t])
            out[t] += b[i] @ h
            size[t] += np.abs(b[i]) @ (abs(s) * (np.abs(a[i]) @ np.abs(e[t])))
            carried[t] += np.abs(b[i]) @ np.abs(h)
    return out, size, carried


def sample(logits, t, k, p, m, u):
    """(token, logprob, distance of u from the nearest border it could have
    crossed, in shares of the total) of one row."""
    x = np.asarray(logits, dtype=np.float64)
    v = x.shape[0]
    top = x.max() if not np.isnan(x).any() else np.nan
    if np.isnan(top) or top == -np.inf or (top == np.inf and t > 0):
        return -1, -np.inf, 1.0
    if not t > 0:
        return int(np.argmax(x == top)), 0.0, 1.0
    with np.errstate(over="ignore", invalid="ignore"):
        w = np.where(x == -np.inf, 0.0, np.exp((x - top) / t))
    order = np.lexsort((np.arange(v), -x))
    stay = order if not 0 < k < v else order[:k]
    near = 1.0
    if p < 1:
        c = np.cumsum(w[stay])
        before = np.concatenate([[0.0], c[:-1]])
        edge = np.abs(before[1:] - p * c[-1])
        if edge.size and p > 0:
            near = min(near, float(edge.min()) / c[-1])
        keep = before < p * c[-1]
        keep[0] = True
        stay = stay[keep]
    if m > 0:
        stay = stay[w[stay] >= min(m, 1.0)]
    stay = np.sort(stay)
    c = np.cumsum(w[stay])
    u = min(max(0.0 if np.isnan(u) else float(u), 0.0), 1.0)
    at = int((c <= u * c[-1]).sum())
    if at >= len(stay) or w[stay[at]] == 0:
        at = int(np.nonzero(w[stay])[0][-1])
    inner = c[:-1]
    if inner.size:
        near = min(near, float(np.abs(inner - u * c[-1]).min()) / c[-1])
    return int(stay[at]), float(np.log(w[stay[at]] / c[-1])), near
