"""Plain 64-bit oracle of the recurrent layers and the norms between products
(test infrastructure), with the bounds that tolerances are made of. Written
from include/w12.h; shares no code with the HIP path."""
import numpy as np

U = 2.0 ** -24  # half a step of fp32
BF16 = 2.0 ** -8  # half a step of bf16


def chain(n: int) -> np.ndarray:
    return np.arange(-1, n - 1, dtype=np.int32)


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def sigmoid(x):
    return np.exp(-softplus(-x))


def append(x, window, parent, weight, bias, heads, dim):
    """x [n, channels] (bf16 values), window [w - 1, channels], weight
    [channels, w]. Returns the values [n, channels] (2 * heads heads of dim
    normalised) and the error that fp32 arithmetic may make in them."""
    n, c = x.shape
    w = weight.shape[1]
    path = []
    for i in range(n):
        above = path[parent[i]] if i else list(window)
        path.append((above + [x[i]])[-w:])
    taps = np.stack([np.stack(p) for p in path]).astype(np.float64)  # n, w, channels
    prod = taps * weight.T.astype(np.float64)[None]
    y, size = prod.sum(1), np.abs(prod).sum(1)
    if bias is not None:
        y, size = y + bias, size + np.abs(bias)
    s = y * sigmoid(y)
    # w + 1 products and sums; |d silu| <= 1.1; e^-y off by (|y| + 8) 2^-23 of itself, the quotient by as much
    err = 1.1 * (w + 2) * U * size + np.abs(s) * (np.abs(y) + 8) * 2 * U
    for h in range(2 * heads):
        at = slice(h * dim, (h + 1) * dim)
        r = np.sqrt((s[:, at] ** 2).sum(1, keepdims=True) + 1e-6)
        dr = (np.abs(s[:, at]) * err[:, at]).sum(1, keepdims=True) / r ** 2 + (dim + 8) * U
        s[:, at], err[:, at] = s[:, at] / r, err[:, at] / r + np.abs(s[:, at]) / r * dr
    return s, err


def gates(b, a, a_log, dt_bias):
    """g and beta [n, heads], and the errors of fp32 arithmetic (exponentials
    and logarithms within 4 half steps; softplus turns an error of its argument
    into at most 1.45 times as much, relative to itself)."""
    b, a, a_log, dt_bias = (t.astype(np.float64) for t in (b, a, a_log, dt_bias))
    g, beta = -np.exp(a_log) * softplus(a + dt_bias), sigmoid(b)
    return g, beta, np.abs(g) * U * (1.45 * np.abs(a + dt_bias) + np.abs(a_log) + 24), beta * U * (np.abs(b) + 24)


def rule(S0, k, v, q, g, beta, parent, scale):
    """One head: rows one after another, each from the state behind its parent.
    Returns out, delta, the states behind every row, and the error bounds of out, delta and
    the states. All roundings of a dot product with the state are at most c U of
    the sum of its terms' sizes (3 (dim + rows) of them: a factor may enter in three
    pieces; 100 for exponents up to 90 and the rest); errors of earlier deltas come back
    through k_j . k_i."""
    n, kd = k.shape
    c = (3 * (kd + n) + 100) * U
    S, A, E = [None] * n, [None] * n, [None] * n  # state, its terms' sizes, its error from earlier deltas as (rows, weights)
    out, delta, eo, ed, es = np.zeros((n, S0.shape[1])), np.zeros((n, S0.shape[1])), [], [], []
    for i in range(n):
        f = np.exp(g[i])
        s, a = (S[parent[i]], A[parent[i]]) if i else (S0, np.abs(S0))
        e = E[parent[i]] if i else np.zeros(S0.shape)
        s, a, e = f * s, f * a, f * e
        d = beta[i] * (v[i] - s.T @ k[i])
        # what earlier errors (their own sizes, sign unknown) do to this delta, and its own roundings
        err = np.abs(beta[i]) * (np.abs(e.T) @ np.abs(k[i]) + c * (a.T @ np.abs(k[i])) + 4 * U * np.abs(v[i]))
        S[i] = s + np.outer(k[i], d)
        A[i] = a + np.outer(np.abs(k[i]), np.abs(d))
        E[i] = e + np.outer(np.abs(k[i]), err)
        out[i], delta[i] = scale * (S[i].T @ q[i]), d
        eo.append(abs(scale) * (E[i].T @ np.abs(q[i]) + c * (A[i].T @ np.abs(q[i]))))
        ed.append(err)
        es.append(E[i] + c * A[i])
    return out, delta, S, np.array(eo).reshape(out.shape), np.array(ed).reshape(out.shape), es


def commit(S0, k, delta, g, rows):
    """The state behind the accepted rows, and the fp32 error bound."""
    S, A = S0.astype(np.float64), np.abs(S0).astype(np.float64)
    for r in rows:
        f = np.exp(g[r])
        S, A = f * S + np.outer(k[r], delta[r]), f * A + np.abs(np.outer(k[r], delta[r]))
    return S, (3 * len(rows) + 100) * U * A


def window(old, raw, rows):
    return np.concatenate([old, raw[rows]])[-len(old):]


def rms(x, weight, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight


def norm_before(y, post, gate, eps):
    """t of one call: [rows, groups, width] in 64 bits, and its fp32 error (a
    mean of width squares, a few products, an exponential)."""
    t, width = y.astype(np.float64), y.shape[-1]
    rel = np.zeros(1)
    if post is not None:
        t, rel = rms(t, post.astype(np.float64), eps), rel + (width + 12) * U
    if gate is not None:
        z = gate.astype(np.float64)
        t, rel = t * z * sigmoid(z), rel + (np.abs(z) + 12) * 2 * U
    return t, np.abs(t) * rel
