"""The recurrent layers at the ends of what w12.h allows: the most heads,
staged rows and inputs past 32 bits, states moved on by replays of captured
prompts and single tokens."""
import numpy as np
import pytest

from oracle import delta as D
from test_gpu_delta import DEV, Inputs, Step, check_append, check_commit, check_rule, f64, i32, w12  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hk,rows,tree", [(256, [3, 20], "random"), (1, [40, 2], "line"), (256, [1, 1], None), (64, [70, 5], None)], ids=str)
def test_most_heads(w12, hk, rows, tree):  # noqa: F811
    st = Step(w12, rows, hk, 256, tree=tree, seed=95)
    check_rule(st, heads=(0, 101, 255))
    if tree is None:
        check_rule(Step(w12, rows, hk, 256, seed=96), keep=True, heads=(0, 255))


def test_append_most_heads(w12):  # noqa: F811
    st = Step(w12, [5, 2], 256, 256, tree="random", seed=97)
    check_append(st, Inputs(st, "bf16"))


def test_staged_rows_past_32_bits(w12):  # noqa: F811
    """Layers whose staged rows begin past 2^31 values, in every array of the step."""
    import torch
    layers, steps, hk, hv = 5, 65536, 6, 66
    small = Step(w12, [9, 4], hk, hv, tree="random", seed=98)
    c = w12.DeltaCache(torch.zeros(layers, small.slots, hv, 128, 128, device=DEV), torch.zeros(layers, small.slots, 3, small.c.channels, dtype=torch.bfloat16, device=DEV),
                       torch.zeros(layers, steps, small.c.channels, dtype=torch.bfloat16, device=DEV),
                       torch.zeros(layers, steps, small.c.kv.shape[2], dtype=torch.bfloat16, device=DEV),
                       torch.zeros(layers, steps, 2, hv, device=DEV), torch.zeros(layers, steps, hv, 128, device=DEV), key_heads=hk)
    assert (layers - 1) * steps * hv * 128 > 2 ** 31 and (layers - 1) * steps * c.kv.shape[2] > 2 ** 31
    last = layers - 1
    c.state[last], c.conv[last] = small.c.state[0], small.c.conv[0]
    x = Inputs(small, "bf16")
    big = Step.__new__(Step)
    big.__dict__.update(small.__dict__)
    big.c = c
    a, b = x.go(small), x.go(big, last)
    assert torch.equal(a, b)
    small.q = big.q = a
    assert torch.equal(small.rule(), big.rule(last))
    n = small.total
    for p, o in ((small.c.raw, c.raw), (small.c.kv, c.kv), (small.c.gates, c.gates), (small.c.delta, c.delta)):
        assert torch.equal(p[0, :n], o[last, :n]) and not o[:last].any() and not o[last, n:].any()
    path = np.full(n, -1)
    path[0], path[9:11] = 0, [0, 1]
    for st in (small, big):
        assert w12.w12_delta_commit(st.c, i32(st.off), i32([0, 1]), path=i32(path), slot=i32(st.slot)).tolist() == [1, 2]
    assert torch.equal(small.c.state[0], c.state[last]) and torch.equal(small.c.conv[0], c.conv[last])
    assert not c.state[:last].any()


def test_append_inputs_past_32_bits(w12):  # noqa: F811
    """Rows 2^23 values apart: the last begins past 2^32 bytes' worth of values."""
    import torch
    st = Step(w12, [300], 1, 2, tree="random", seed=99)
    x = Inputs(st, "bf16")
    want, kv, gates = x.go(st).clone(), st.c.kv.clone(), st.c.gates.clone()
    wide = torch.empty(300, 1 << 23, dtype=torch.bfloat16, device=DEV)
    c, hv = st.c.channels, st.hv
    at = (1 << 23) - 8 - 2 * hv
    wide[:, 64:64 + c], wide[:, at:at + 2 * hv] = x.qkv, x.ba
    x.qkv, x.ba = wide[:, 64:64 + c], wide[:, at:at + 2 * hv]
    st.c.kv.zero_(), st.c.gates.zero_()
    assert torch.equal(want, x.go(st))
    assert torch.equal(kv[0, :300], st.c.kv[0, :300]) and torch.equal(gates[0, :300], st.c.gates[0, :300])


@pytest.mark.parametrize("rows", [[100, 70], [1] * 6, [12, 3], [20] * 9], ids=str)
def test_kept_steps_in_graphs(w12, rows):  # noqa: F811
    """Captured prompts and single tokens: every replay goes on from the state and window the one before left."""
    import torch
    make = lambda: Step(w12, rows, 4, 16, seed=100, rate=0.5)  # noqa: E731
    eager, st = make(), make()
    x = Inputs(eager, "bf16")
    off, slot = i32(st.off), i32(st.slot)
    bufs = [(torch.zeros_like(st.q), torch.zeros(st.total, 16 * 128, dtype=torch.bfloat16, device=DEV)) for _ in range(2)]

    def step(e, q, out):
        w12.w12_delta_append(e.c, 0, x.qkv, x.ba, off, x.weight, x.a_log, x.dt, conv_bias=x.bias, slot=slot, out=q)
        w12.w12_delta_rule(e.c, 0, q, off, slot=slot, keep=True, out=out)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(st, *bufs[1])
    for i in range(4):
        step(eager, *bufs[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs[0][1], bufs[1][1]) and torch.isfinite(bufs[1][1]).all(), i
        assert torch.equal(eager.c.state, st.c.state) and torch.equal(eager.c.conv, st.c.conv), i
        x.qkv.mul_(-0.9)
        eager.c.state.square().sum().item()


def test_commit_of_the_longest_path_of_many_heads(w12):  # noqa: F811
    st = Step(w12, [512], 2, 16, seed=101, rate=0.5)
    check_commit(st, [list(range(512))], use_path=False)
