"""A step of short and long sequences in two calls, the short ones' rows first:
each call answers its own rows and leaves the other's, and both together are the
step, within the bounds of the 64-bit oracle."""
import numpy as np
import pytest

from oracle import delta as D
from test_gpu_delta import DEV, Step, f64, i32, w12  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("short,long", [([1] * 20, [100]), ([1] * 33, [70, 64]), ([2, 1, 3], [40])], ids=str)
@pytest.mark.parametrize("tree,keep", [(None, True), (None, False), ("random", False)])
def test_two_calls(w12, short, long, tree, keep):  # noqa: F811
    import torch
    st = Step(w12, short + long, 2, 4, tree=tree, seed=91)
    want = {(s, h): st.want(s, h) for s in range(len(st.rows)) for h in range(st.hv)}
    state, conv = st.c.state.clone(), st.c.conv.clone()
    cut, seqs = sum(short), len(short)
    out = torch.full((st.total, st.hv * st.vd), 7.0, dtype=torch.bfloat16, device=DEV)
    off, slot, parent = i32(st.off), i32(st.slot), i32(st.parent)
    w12.w12_delta_rule(st.c, 0, st.q[:cut], off[:seqs + 1], slot=slot[:seqs], parent=None if tree is None else parent[:cut], keep=keep, out=out[:cut])
    assert (out[cut:] == 7).all()
    late = [int(s) for s in st.slot[seqs:]]
    assert torch.equal(state[0, late], st.c.state[0, late]) and torch.equal(conv[0, late], st.c.conv[0, late])
    first = out[:cut].clone()
    w12.w12_delta_rule(st.c, 0, st.q, off[seqs:].clone(), slot=slot[seqs:].clone(), parent=parent, keep=keep, out=out)
    assert torch.equal(first, out[:cut])
    got, delta, after = f64(out).reshape(st.total, st.hv, st.vd), f64(st.c.delta[0]), f64(st.c.state[0])
    for (s, h), (o, d, S, eo, ed, es) in want.items():
        a, b = int(st.off[s]), int(st.off[s + 1])
        assert (np.abs(got[a:b, h] - o) <= D.BF16 * np.abs(o) * 1.01 + eo * 1.01).all(), ("out", s, h)
        if keep:
            assert (np.abs(after[int(st.slot[s]), h] - S[-1]) <= es[-1] + D.U * np.abs(S[-1])).all(), ("state", s, h)
        else:
            assert (np.abs(delta[a:b, h] - d) <= ed + D.U * np.abs(d)).all(), ("delta", s, h)
