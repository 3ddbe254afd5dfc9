"""The recurrent layers' oracle against closed forms and definitions written
another way (CPU)."""
import numpy as np
import pytest

from oracle import delta as D


def rows(n, kd=8, vd=6, seed=0):
    r = np.random.RandomState(seed)
    k = r.randn(n, kd)
    k /= np.linalg.norm(k, axis=1, keepdims=True)
    return k, r.randn(n, vd), r.randn(n, kd), -r.rand(n), r.rand(n), r.randn(kd, vd)


def parents(n, seed):
    r = np.random.RandomState(seed)
    return np.array([-1] + [r.randint(0, i) for i in range(1, n)], np.int32)


@pytest.mark.parametrize("n", [1, 2, 7, 20])
@pytest.mark.parametrize("tree", [False, True])
def test_rule_is_the_triangular_system(n, tree):
    k, v, q, g, beta, S0 = rows(n, seed=n)
    parent = parents(n, n) if tree else D.chain(n)
    out, delta, S, *_ = D.rule(S0, k, v, q, g, beta, parent, 0.5)
    see = np.eye(n, dtype=bool)
    for i in range(1, n):
        see[i] |= see[parent[i]]
    G = see @ g
    decay = np.where(see, np.exp(np.where(see, G[:, None] - G[None], 0)), 0)
    low = beta[:, None] * decay * (k @ k.T) * ~np.eye(n, dtype=bool)
    d = np.linalg.solve(np.eye(n) + low, beta[:, None] * (v - np.exp(G)[:, None] * (k @ S0)))
    assert np.allclose(d, delta, rtol=0, atol=1e-12)
    o = 0.5 * (np.exp(G)[:, None] * (q @ S0) + (decay * (q @ k.T)) @ d)
    assert np.allclose(o, out, rtol=0, atol=1e-12)


def test_commit_is_the_state_behind_the_path():
    n = 12
    k, v, q, g, beta, S0 = rows(n, seed=3)
    parent = parents(n, 4)
    _, delta, S, *_ = D.rule(S0, k, v, q, g, beta, parent, 1.0)
    for leaf in range(n):
        path, i = [], leaf
        while i >= 0:
            path.append(i)
            i = parent[i]
        got, _ = D.commit(S0, k, delta, g, path[::-1])
        assert np.allclose(got, S[leaf], rtol=0, atol=1e-12)


def test_a_full_strength_row_is_read_back():
    """beta 1, no decay: the state answers the row's key with its value."""
    k, v, q, _, _, S0 = rows(3, seed=5)
    out, _, S, *_ = D.rule(S0, k, v, k, np.zeros(3), np.ones(3), D.chain(3), 1.0)
    assert np.allclose(out, v, atol=1e-12)


def test_rule_does_not_depend_on_its_bounds():
    """Errors of fp32 arithmetic stay within the bounds."""
    n = 24
    k, v, q, g, beta, S0 = rows(n, seed=6)
    f = lambda t: t.astype(np.float32)  # noqa: E731
    k, v, q, g, beta, S0 = (f(t) for t in (k, v, q, g, beta, S0))
    out, delta, S, eo, ed, es = D.rule(*(t.astype(np.float64) for t in (S0, k, v, q, g, beta)), D.chain(n), 0.5)
    s = S0
    for i in range(n):
        s = f(s * np.exp(g[i]))
        d = f(beta[i] * f(v[i] - f(s.T @ k[i])))
        s = f(s + np.outer(k[i], d))
        assert (np.abs(d - delta[i]) <= ed[i]).all() and (np.abs(s - S[i]) <= es[i]).all()
        assert (np.abs(np.float32(0.5) * f(s.T @ q[i]) - out[i]) <= eo[i]).all()


@pytest.mark.parametrize("w", [2, 3, 4])
def test_append_is_the_convolution_of_the_sequence(w):
    """Chain rows: what a convolution over window and rows gives."""
    r = np.random.RandomState(w)
    heads, dim, n = 2, 8, 5
    c = 2 * heads * dim + 10
    x, win, weight, bias = r.randn(n, c), r.randn(w - 1, c), r.randn(c, w), r.randn(c)
    got, _ = D.append(x, win, D.chain(n), weight, bias, heads, dim)
    both = np.concatenate([win, x])
    y = np.stack([(both[i:i + w] * weight.T).sum(0) + bias for i in range(n)])
    s = y / (1 + np.exp(-y))
    z = s[:, :2 * heads * dim].reshape(n, 2 * heads, dim)
    s[:, :2 * heads * dim] = (z / np.sqrt((z ** 2).sum(2, keepdims=True) + 1e-6)).reshape(n, -1)
    assert np.allclose(got, s, atol=1e-13)
    again, _ = D.append(x[2:], both[2:w + 1], D.chain(n - 2), weight, bias, heads, dim)
    assert np.allclose(again, got[2:], atol=1e-13)
    assert np.array_equal(D.window(win, x, [0, 1, 2]), both[3:w + 2])


def test_gates():
    a = np.array([[-60.0, 0.0, 60.0]])
    g, beta, eg, eb = D.gates(a, a, np.log([2.0, 2.0, 2.0]), np.zeros(3))
    assert np.allclose(g[0], [-2 * np.exp(-60), -2 * np.log(2), -120], rtol=1e-14)
    assert np.allclose(beta[0], [np.exp(-60), 0.5, 1], rtol=1e-14) and (eg >= 0).all() and (eb >= 0).all()
