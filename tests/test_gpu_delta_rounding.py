"""A row that joins a state rounds it once: with no decay and a delta that fp32
holds, every entry is the nearest fp32 value of S + k delta, whichever kernel
moves the state on. No tolerance: S + k delta is one sum of two fp32 values."""
import numpy as np
import pytest

from test_gpu_delta import DEV, Step, i32, w12  # noqa: F401

pytestmark = pytest.mark.gpu


def nearest(state, add):
    """fp32 sums of fp32 values, rounded once (64 bits hold any sum of two whose exponents are this near)."""
    return (state.astype(np.float64) + add.astype(np.float64)).astype(np.float32)


@pytest.mark.parametrize("kd,vd", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("row", [0, 3, 31])
def test_commit(w12, kd, vd, row):  # noqa: F811
    """One row of a path has keys (of ones), at several places of a turn."""
    import torch
    st = Step(w12, [40], 1, 3, kd, vd, layers=2, seed=71)
    c = st.c
    c.gates[:, :, 0] = 0
    c.kv.zero_()
    c.kv[:, row, :kd] = 1
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    c.state.mul_(4 * torch.rand(c.state.shape, generator=g, device=DEV))
    before, delta = c.state.cpu().numpy(), c.delta[:, row].cpu().numpy()  # [layers, heads, dims]
    kept = w12.w12_delta_commit(c, i32(st.off), i32([row]), slot=i32(st.slot), rows=st.total)
    assert kept.tolist() == [row + 1]
    s = int(st.slot[0])
    want = nearest(before[:, s], delta[:, :, None, :])
    assert np.array_equal(c.state[:, s].cpu().numpy(), want)


@pytest.mark.parametrize("kd,vd", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("rows", [[1], [1] * 5, [3], [9, 2], [16], [17], [40], [100, 7], [5, 0, 0, 0], [20] * 9], ids=str)
def test_kept_rows(w12, rows, kd, vd):  # noqa: F811
    """Each sequence's first row has two keys, of ones, whose rows of the state
    are x and -x: the state answers 0, delta is beta (all its 24 bits), and x
    and -x take it. The other rows have no keys."""
    import torch
    hv = 6
    st = Step(w12, rows, 2, hv, kd, vd, seed=72)
    c = st.c
    c.gates[:, :, 0] = 0
    c.kv[:, :, :2 * kd] = 0
    c.kv[:, :, 2 * kd:] = 1
    live = [s for s, n in enumerate(rows) if n]
    first = [int(st.off[s]) for s in live]
    for head in range(2):
        for at in (3, 7):
            c.kv[0, first, head * kd + at] = 1
    c.state[0, :, :, 7] = -c.state[0, :, :, 3]
    before = c.state[0].cpu().numpy()
    beta = c.gates[0, :, 1].cpu().numpy()
    st.rule(keep=True)
    torch.cuda.synchronize()
    got = c.state[0].cpu().numpy()
    for s, row in zip(live, first):
        slot = int(st.slot[s])
        want = before[slot].copy()
        for at in (3, 7):
            want[:, at] = nearest(before[slot][:, at], beta[row][:, None])
        assert np.array_equal(got[slot], want), s
