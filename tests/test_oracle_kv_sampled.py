"""The oracles of the KV cache and the sampled tree acceptance against
something other than themselves."""
import numpy as np
import pytest

from oracle import kv_cache as KV
from oracle import tree_sampled as TS


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("v", [0, 1])
def test_places_are_a_bijection_in_1kb_fragments(v, dim):
    p = KV.places(v, 96, dim)
    assert np.array_equal(np.sort(p.ravel()), np.arange(96 * dim))
    for t in (0, 31, 32, 95):
        for d in (0, 31, 32, dim - 1):
            assert p[t, d] // 1024 == t // 32 * (dim // 32) + d // 32


def test_places_by_hand():
    k, v = KV.key_places(32, 64), KV.value_places(32, 64)
    assert (k[0, 0], k[1, 0], k[0, 15], k[0, 16], k[5, 33]) == (0, 16, 15, 512, 1024 + 5 * 16 + 1)
    assert (v[0, 0], v[3, 0], v[4, 0], v[8, 0], v[0, 1], v[29, 2]) == (0, 3, 512, 4, 16, 512 + 2 * 16 + 13)


def test_e4m3_values_and_rounding():
    t = KV.e4m3_values()
    assert t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6 and t[126] == 448 and (np.diff(t) > 0).all()
    c, s = KV.quantise(np.array([448.0, 17.0, 17.5, 19.0, -21.0, 2.0 ** -10, 0.0]), False)
    assert s == 1 and c.tolist() == [448, 16, 18, 20, -20, 0, 0]  # 17 and 19, 21 lie half way: the even code


@pytest.mark.parametrize("amax,scale", [(448, 1), (449, 2), (0.875, 2.0 ** -9), (1, 2.0 ** -8), (0, 1), (2.0 ** -133, 2.0 ** -90)])
def test_e4m3_scale_is_the_smallest_power(amax, scale):
    assert KV.quantise(np.array([amax, 0.0]), False)[1] == scale


def test_int8_codes():
    c, s = KV.quantise(np.array([2.0, -2.0, 0.0, 1.0]), True)
    assert c.tolist() == [127, -127, 0, 64] and s == np.float32(2) / np.float32(127)
    assert np.isnan(KV.quantise(np.array([1.0, np.inf]), True)[1])


def test_rotation_keeps_lengths_and_turns_by_the_angle():
    r = np.random.RandomState(0)
    x, pos = r.randn(5, 3, 64), np.array([0, 1, 7, 100, 31])
    ang = np.arange(128)[:, None] * 10000.0 ** (-np.arange(0, 32, 2) / 32)
    rope = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    for inter in (False, True):
        y, _ = KV.rotate(x, pos, rope, inter)
        assert np.allclose(np.linalg.norm(y, axis=2), np.linalg.norm(x, axis=2))
        assert np.array_equal(y[..., 32:], x[..., 32:]) and np.allclose(y[0], x[0])
    # scores of rotated vectors depend on the distance alone
    q, k = r.randn(2, 1, 1, 32)
    s = [float((KV.rotate(q, np.array([a]), rope, False)[0] * KV.rotate(k, np.array([b]), rope, False)[0]).sum())
         for a, b in ((5, 2), (103, 100))]
    assert abs(s[0] - s[1]) < 1e-9


def test_attention_by_hand():
    q = np.array([[[1.0, 0.0]]])
    k, v = np.array([[0.0, 0], [np.log(3), 0], [50, 0]]), np.array([[4.0, 0], [8, 0], [99, 9]])
    out, av, _ = KV.attention(q, k, v, np.array([[True, True, False]]), 1.0)
    assert np.allclose(out[0, 0], [7, 0]) and np.allclose(av[0, 0], [7, 0])


def test_commit_closes_blocks_whatever_the_grouping():
    r = np.random.RandomState(1)
    x, y = r.randn(2, 70, 64)
    a, b = KV.Sequence(32, False, 64), KV.Sequence(32, False, 64)
    a.commit(x, y)
    for i in range(70):
        b.commit(x[i:i + 1], y[i:i + 1])
    assert len(a.blocks) == 2 and np.array_equal(a.k, b.k) and np.array_equal(a.v, b.v)
    assert np.array_equal(a.k[64:], x[64:]) and not np.array_equal(a.k[:64], x[:64])


def test_sampled_walk_by_hand():
    # p = (1/2, 1/4, 1/4); drafts chosen: token 0 is rejected at u >= 1/2, then token 1 has half of what is left
    lg = np.tile(np.log([0.5, 0.25, 0.25]), (3, 1))
    go = lambda u1, u2, ub, draft=None: TS.walk([-1, 0, 0], [9, 0, 1], lg, 1.0, draft, [0, u1, u2], ub)
    assert go(0.49, 0.9, 0.0) == (1, [0, 1], 0)
    assert go(0.51, 0.49, 0.99) == (1, [0, 2], 2)
    assert go(0.51, 0.51, 0.5) == (0, [0], 2)
    # drawn from q = (1/4, 1/2, 1/4): token 1 is accepted below 1/2, and max(p - q, 0) leaves token 0 alone
    q = np.tile([0.25, 0.5, 0.25], (3, 1))
    two = lambda u, ub: TS.walk([-1, 0], [9, 1], lg[:2], 1.0, q[:2], [0, u], ub)
    assert two(0.49, 0.1) == (1, [0, 1], 0)
    assert two(0.51, 0.999) == (0, [0], 0)
    assert TS.walk([-1, 0], [9, 3], lg[:2], 1.0, None, [0, 0.1], 0.1)[0] == -1
    assert TS.walk([-1, 0], [9, 1], lg[:2], 0.0, None, [0, 0.1], 0.1)[0] == -1


def test_sampled_tokens_follow_the_target():
    """Over a grid of random numbers and all drafts by their probability, the
    first token that comes out has the target's distribution."""
    p, q = np.array([0.5, 0.2, 0.3]), np.array([0.2, 0.5, 0.3])
    lg, n = np.tile(np.log(p), (3, 1)), 60
    grid = (np.arange(n) + 0.5) / n
    got = np.zeros(3)
    for x in range(3):
        for y in range(3):
            w = q[x] * q[y] / n ** 3
            for u1 in grid:
                for u2 in grid:
                    a, path, bonus = TS.walk([-1, 0, 0], [0, x, y], lg, 1.0, np.tile(q, (3, 1)), [0, u1, u2], 0.5)
                    if a == 1:
                        got[[x, y][path[1] - 1]] += w * n
                    else:
                        for ub in (0.25, 0.75):  # the residual after two rejections holds few tokens
                            got[TS.walk([-1, 0, 0], [0, x, y], lg, 1.0, np.tile(q, (3, 1)), [0, u1, u2], ub)[2]] += w * n / 2
    assert np.abs(got - p).max() < 0.03  # two grids of 60 cells and a residual split in two
