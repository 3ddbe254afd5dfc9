"""What an infinity or NaN in a staged row of the delta rule reaches (through
the C ABI): everything on the paths behind it, in every form of the kernel, and
nothing else."""
import numpy as np
import pytest

from test_gpu_delta import DEV, Step, w12  # noqa: F401

pytestmark = pytest.mark.gpu


def paths(st, tree):
    """see[i, j]: row j is on row i's path."""
    see = np.eye(st.total, dtype=bool)
    for s in range(len(st.rows)):
        a = int(st.off[s])
        for i in range(a + 1, int(st.off[s + 1])):
            see[i] |= see[i - 1 if tree is None else a + int(st.parent[i])]
    return see


def spoil(st, where, at, value):
    """Puts value into row `at`; returns the value heads and, of their dims, those that it enters."""
    every = list(range(st.vd))
    if where == "k":  # of key head 0
        st.c.kv[0, at, 3] = value
        return list(range(st.hv // st.hk)), every
    if where == "v":
        st.c.kv[0, at, st.hk * st.kd + 9] = value
        return [0], [9]
    if where == "q":
        st.q[at, 0, 17] = value
        return list(range(st.hv // st.hk)), every
    st.c.gates[0, at, 0 if where == "g" else 1, st.hv - 1] = value
    return [st.hv - 1], every


def check(w12, rows, tree, where, value, at, keep, hk=1, hv=2, kd=128, vd=128):
    import torch
    clean, st = (Step(w12, rows, hk, hv, kd, vd, tree=tree, seed=61) for _ in range(2))
    heads, dims = spoil(st, where, at, value)
    a, b = clean.rule(keep=keep).view(-1, hv, vd), st.rule(keep=keep).view(-1, hv, vd)
    d0, d1 = clean.c.delta[0, :st.total], st.c.delta[0, :st.total]
    bits = {torch.bfloat16: torch.int16, torch.float32: torch.int32}

    def compare(x, y, rows_hit, what):
        """[rows, heads, dims]: what is hit holds no number, the rest of those heads' rows none or the same, all else the same."""
        same, number = x.view(bits[x.dtype]) == y.view(bits[y.dtype]), torch.isfinite(y)
        must = torch.zeros(x.shape, dtype=torch.bool, device=DEV)
        may = must.clone()
        for h in heads:
            may[rows_hit, h] = True
            for d in dims:
                must[rows_hit, h, d] = True
        assert not number[must].any(), (what, "a number")
        assert (same | (may & ~number)).all(), (what, "of others")

    behind = torch.tensor(paths(st, tree)[:, at], device=DEV)
    own = torch.arange(st.total, device=DEV) == at
    compare(a, b, own if where == "q" else behind, "out")
    if not keep:
        compare(d0, d1, torch.zeros_like(own) if where == "q" else behind, "delta")
        return
    s = next(i for i in range(len(rows)) if st.off[i] <= at < st.off[i + 1])
    x, y = (c.state[0].transpose(1, 2).reshape(-1, hv, vd) for c in (clean.c, st.c))  # [slots * key dims, heads, dims]
    hit = torch.zeros(st.slots, kd, dtype=torch.bool, device=DEV)
    hit[int(st.slot[s])] = where != "q"
    compare(x, y, hit.flatten(), "state")


BAD = [(w, v) for w in ("k", "v", "g", "beta", "q") for v in (float("nan"), float("inf"))]


@pytest.mark.parametrize("rows,tree,at", [([12], "star", 0), ([16], "random", 5), ([40, 6], "random", 5), ([40, 6], "line", 20), ([33], "star", 0),
                                          ([90], "random", 5), ([90], "line", 70), ([200, 3], "random", 2), ([150], "line", 1),
                                          ([50] + [2] * 9, "random", 5), ([100] + [1] * 20, "line", 18), ([100] + [1] * 20, "star", 0),
                                          ([1, 1, 9], "random", 2)], ids=str)
@pytest.mark.parametrize("where,value", BAD)
def test_trees(w12, rows, tree, at, where, value):  # noqa: F811
    check(w12, rows, tree, where, value, at, False)


@pytest.mark.parametrize("rows,at", [([1], 0), ([1] * 5, 2), ([4, 0, 0, 0], 1), ([8, 1, 1], 3), ([16], 0), ([17], 5), ([40], 33), ([90], 5),
                                     ([300, 2], 100), ([30] + [1] * 5, 5), ([50] + [2] * 9, 17)], ids=str)
@pytest.mark.parametrize("where,value", BAD)
@pytest.mark.parametrize("keep", [False, True])
def test_chains(w12, rows, at, where, value, keep):  # noqa: F811
    check(w12, rows, None, where, value, at, keep)


@pytest.mark.parametrize("kd,vd", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("rows,tree", [([1] * 12, None), ([70] * 9, None), ([20] * 9, None), ([40] * 9, "random"), ([9] * 9, "random")], ids=str)
@pytest.mark.parametrize("where", ["k", "v", "g"])
def test_many_heads(w12, kd, vd, rows, tree, where):  # noqa: F811
    """The forms of a full card, and every head size."""
    rows = rows[:512 // rows[0]]
    check(w12, rows, tree, where, float("nan"), rows[0] + min(5, rows[0] - 1), tree is None, 4, 16, kd, vd)
