"""The binding of the recurrent layers and norms refuses what is no tensor of
the kind that a call takes, with the error that says so, before it calls the
library; and the library arrays that lie over each other, on memory that a call
may otherwise have."""
import ctypes

import pytest

from test_gpu_delta import DEV, Inputs, Step, i32, w12  # noqa: F401

pytestmark = pytest.mark.gpu
NONE = [None, 3, [1.0], "x"]


@pytest.mark.parametrize("bad", NONE, ids=str)
def test_no_tensors(w12, bad):  # noqa: F811
    import torch
    st = Step(w12, [4, 2], 1, 2, seed=81)
    x = Inputs(st)
    for name in ("qkv", "ba", "weight", "a_log", "dt"):
        keep = getattr(x, name)
        setattr(x, name, bad)
        with pytest.raises(TypeError):
            x.go(st)
        setattr(x, name, keep)
    y = torch.zeros(4, 64, device=DEV)
    calls = [lambda: w12.w12_delta_rule(st.c, 0, bad, i32(st.off)), lambda: w12.w12_delta_rule(st.c, 0, st.q, bad),
             lambda: w12.w12_delta_commit(st.c, bad, i32([0, 0])), lambda: w12.w12_delta_commit(st.c, i32(st.off), bad)]
    if bad is not None:
        calls += [lambda: x.go(st, out=bad), lambda: x.go(st, conv_bias=bad), lambda: x.go(st, slot=bad), lambda: x.go(st, parent=bad),
                  lambda: st.rule(out=bad), lambda: st.rule(slot=bad), lambda: st.rule(parent=bad),
                  lambda: w12.w12_delta_commit(st.c, i32(st.off), i32([0, 0]), path=bad),
                  lambda: w12.w12_delta_commit(st.c, i32(st.off), i32([0, 0]), slot=bad)]
        calls += [lambda k=k: w12.w12_norm(**{**dict(y=y), k: bad}) for k in ("y", "weight", "post_weight", "gate", "h", "out")]
    for i, call in enumerate(calls):
        with pytest.raises(TypeError):
            call()
            raise AssertionError(i)


def test_arrays_over_each_other(w12):  # noqa: F811
    """A good call is taken, and the same call with one output over one input is not."""
    import torch
    st = Step(w12, [4, 2], 1, 2, seed=82)
    L, d = w12.lib(), st.c.desc()
    off, slot, acc = i32(st.off), i32(st.slot), i32([1, 0])
    kept = torch.zeros(8, dtype=torch.int32, device=DEV)

    def commit(kept_at):
        status = L.w12_delta_commit(ctypes.byref(d), 2, slot.data_ptr(), off.data_ptr(), 6, acc.data_ptr(), None, kept_at,
                                    torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        return status

    state = st.c.state.clone()
    for t in (off, slot, acc):
        assert commit(t.data_ptr()) == w12.W12_EINVAL
    assert torch.equal(state, st.c.state) and off.tolist() == st.off.tolist() and slot.tolist() == st.slot.tolist()
    assert commit(kept.data_ptr()) == w12.W12_OK and kept.tolist() == [2, 1, 0, 0, 0, 0, 0, 0]
    out = torch.empty(6, 256, dtype=torch.bfloat16, device=DEV)
    assert torch.isfinite(st.rule(out=out)).all()
    with pytest.raises(w12.W12Error):
        st.rule(out=out, parent=out.view(torch.int32).flatten()[:6])
    x = Inputs(st)
    q = torch.empty(6, 1, 128, dtype=torch.bfloat16, device=DEV)
    assert torch.isfinite(x.go(st, out=q)).all()
    with pytest.raises(w12.W12Error):
        x.go(st, out=q, slot=q.view(torch.int32).flatten()[:2])
