"""Plain 64-bit oracle of sampled tree acceptance (test infrastructure): the
walk as it is defined, residuals stored and normalised at every rejection.
Shares no code with the HIP path."""
import numpy as np


def softmax(x: np.ndarray) -> np.ndarray:
    p = np.exp(x - x.max())
    return p / p.sum()


def draw(p: np.ndarray, u: float) -> int:
    """The lowest t whose cumulative sum exceeds u times the whole."""
    c = np.cumsum(p)
    over = np.flatnonzero((c > u * c[-1]) & (p > 0))
    return int(over[0]) if len(over) else int(np.flatnonzero(p > 0)[-1])


def walk(parent, token, logits, temperature, draft, u_accept, u_bonus):
    """One tree: (accept_len, path of nodes, bonus). logits, draft [n, vocab]."""
    n, vocab = logits.shape
    bad = n < 1 or parent[0] != -1 or any(not 0 <= parent[i] < i for i in range(1, n))
    bad = bad or not (np.isfinite(temperature) and temperature > 0)
    bad = bad or any(not 0 <= token[i] < vocab for i in range(1, n))
    if bad:
        return -1, [], -1
    node, path = 0, []
    while True:
        path.append(node)
        x = logits[node].astype(np.float64) / np.float64(temperature)
        if np.isnan(x).any() or x.max() == np.inf or x.max() == -np.inf:
            return -1, [], -1
        p, step = softmax(x), None
        for c in (i for i in range(1, n) if parent[i] == node):
            q = draft[node].astype(np.float64) if draft is not None else np.eye(1, vocab, token[c])[0]
            if np.float64(u_accept[c]) * q[token[c]] < p[token[c]]:
                step = c
                break
            left = np.maximum(p - q, 0)
            if left.sum() > 0:
                p = left / left.sum()
        if step is None:
            return len(path) - 1, path, draw(p, np.float64(u_bonus))
        node = step


def forest(node_off, parent, token, logits, temperature, draft, u_accept, u_bonus):
    """All trees, in the outputs' layout."""
    trees, total = len(node_off) - 1, len(parent)
    acc, bonus = np.full(trees, -1, np.int32), np.full(trees, -1, np.int32)
    path = np.full(total, -1, np.int32)
    for t in range(trees):
        r = slice(node_off[t], node_off[t + 1])
        temp = 1.0 if temperature is None else temperature[t]
        acc[t], way, bonus[t] = walk(parent[r], token[r], logits[r], temp, None if draft is None else draft[r],
                                     u_accept[r], u_bonus[t])
        path[node_off[t]:node_off[t] + len(way)] = way
    return acc, path, bonus
