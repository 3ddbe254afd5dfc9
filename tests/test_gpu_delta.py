"""GPU parity of the recurrent layers (w12_delta_append, w12_delta_rule,
w12_delta_commit, through the C ABI) against the 64-bit oracle, within the
roundings that the tolerances count."""
import numpy as np
import pytest

from oracle import delta as D

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def say(*a):
    print("[delta]", *a, flush=True)


@pytest.fixture(scope="module")
def w12():
    import torch
    import w12_weight_streaming_amd as w
    assert torch.cuda.is_available()
    w.lib()
    return w


def i32(a):
    import torch
    return None if a is None else torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def f32(a):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.float32, device=DEV)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def parents(r, n, kind):
    if kind == "star":
        return np.array([-1] + [0] * (n - 1), np.int32)
    if kind == "line":
        return D.chain(n)
    return np.array([-1] + [int(r.randint(max(0, i - 6), i)) for i in range(1, n)], np.int32)


class Step:
    """A step's staged rows and states on the GPU, and their values in 64 bits."""

    def __init__(self, w12, rows, hk=2, hv=4, kd=128, vd=128, layers=1, width=4, tree=None, seed=0, rate=0.05, extra=3, slots=None):
        import torch
        self.w12, self.rows, self.hk, self.hv, self.kd, self.vd, self.layers, self.tree = w12, rows, hk, hv, kd, vd, layers, tree
        g = torch.Generator(device=DEV)
        g.manual_seed(seed + 1)
        r = self.r = np.random.RandomState(seed)
        n = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        self.total = sum(rows)
        self.slots = len(rows) + 2 if slots is None else slots
        self.off = np.concatenate([[0], np.cumsum(rows)])
        self.slot = r.permutation(self.slots)[:len(rows)]
        c = w12.delta_cache(layers, self.slots, hk, hv, kd, vd, width, self.total + extra, device=DEV)
        c.state.copy_(n(*c.state.shape))
        c.conv.copy_(n(*c.conv.shape))
        c.raw.copy_(n(*c.raw.shape))
        k = n(layers, self.total + extra, hk, kd)
        c.kv.copy_(torch.cat([(k / k.norm(dim=3, keepdim=True)).flatten(2), n(layers, self.total + extra, hv * vd)], 2))
        c.gates[:, :, 0] = -rate * 2 * torch.rand(c.gates[:, :, 0].shape, generator=g, device=DEV)
        c.gates[:, :, 1] = torch.rand(c.gates[:, :, 1].shape, generator=g, device=DEV)
        c.delta.copy_(n(*c.delta.shape))
        self.c = c
        q = n(self.total, hk, kd)
        self.q = (q / q.norm(dim=2, keepdim=True)).bfloat16()
        self.parent = None if tree is None else np.concatenate([parents(r, m, tree) if m else np.zeros(0, np.int32) for m in rows])

    def rule(self, layer=0, keep=False, **kw):
        a = dict(slot=i32(self.slot), parent=i32(self.parent), keep=keep)
        a.update(kw)
        return self.w12.w12_delta_rule(self.c, layer, self.q, i32(self.off), **a)

    def want(self, s, h, layer=0, scale=None):
        """The oracle's answer for sequence s, value head h."""
        a, b = int(self.off[s]), int(self.off[s + 1])
        key = h // (self.hv // self.hk)
        kv = f64(self.c.kv[layer, a:b])
        k = kv[:, key * self.kd:(key + 1) * self.kd]
        v = kv[:, self.hk * self.kd + h * self.vd:][:, :self.vd]
        gates = f64(self.c.gates[layer, a:b])
        parent = D.chain(b - a) if self.parent is None else self.parent[a:b]
        return D.rule(f64(self.c.state[layer, int(self.slot[s]), h]), k, v, f64(self.q[a:b, key]), gates[:, 0, h], gates[:, 1, h],
                      parent, self.kd ** -0.5 if scale is None else scale)


def check_rule(st, layer=0, keep=False, heads=None, **kw):
    """Runs the rule and compares every output (of these heads); what it must leave stays bit for bit."""
    import torch
    heads = range(st.hv) if heads is None else heads
    live = [s for s, n in enumerate(st.rows) if n]
    want = {(s, h): st.want(s, h, layer) for s in live for h in heads}
    before = [t.clone() for t in (st.c.state, st.c.conv, st.c.raw, st.c.kv, st.c.gates, st.c.delta)]
    out = st.rule(layer, keep, **kw)
    torch.cuda.synchronize()
    got = f64(out).reshape(st.total, st.hv, st.vd)
    delta, state = f64(st.c.delta[layer]), f64(st.c.state[layer])
    for (s, h), (o, d, S, eo, ed, es) in want.items():
        a, b = int(st.off[s]), int(st.off[s + 1])
        assert (np.abs(got[a:b, h] - o) <= D.BF16 * np.abs(o) * 1.01 + eo * 1.01).all(), ("out", s, h)
        if keep:
            assert (np.abs(state[int(st.slot[s]), h] - S[-1]) <= es[-1] + D.U * np.abs(S[-1])).all(), ("state", s, h)
        else:
            assert (np.abs(delta[a:b, h] - d) <= ed + D.U * np.abs(d)).all(), ("delta", s, h)
    after = [st.c.state, st.c.conv, st.c.raw, st.c.kv, st.c.gates, st.c.delta]
    same = lambda x, y: torch.equal(x.view(torch.uint8), y.view(torch.uint8))  # noqa: E731
    assert all(same(x, y) for x, y in zip(before[2:5], after[2:5]))
    if keep:
        others = [i for i in range(st.slots) if i not in [int(st.slot[s]) for s in live]]
        assert same(before[0][layer, others], after[0][layer, others]) and same(before[1][layer, others], after[1][layer, others])
        assert same(before[5], after[5])
        for s in live:
            a, b, slot = int(st.off[s]), int(st.off[s + 1]), int(st.slot[s])
            assert torch.equal(after[1][layer, slot], torch.cat([before[1][layer, slot], before[2][layer, a:b]])[-before[1].shape[2]:])
    else:
        assert same(before[0], after[0]) and same(before[1], after[1]) and same(before[5][layer, st.total:], after[5][layer, st.total:])
    for lay in range(st.layers):
        if lay != layer:
            assert all(same(x[lay], y[lay]) for x, y in zip(before, after))
    return out


ROWS = [[1], [1, 1, 1], [2], [5, 1, 3], [8] * 6, [15], [16], [17], [31, 0, 5], [33], [1, 47, 2], [64], [65], [100, 7], [130]]


@pytest.mark.parametrize("rows", ROWS, ids=str)
@pytest.mark.parametrize("keep", [False, True])
def test_rule_chains(w12, rows, keep):
    check_rule(Step(w12, rows, seed=len(rows) + rows[0]), keep=keep)


@pytest.mark.parametrize("rows", [r for r in ROWS if max(r) > 1], ids=str)
@pytest.mark.parametrize("tree", ["random", "star", "line"])
def test_rule_trees(w12, rows, tree):
    check_rule(Step(w12, rows, tree=tree, seed=rows[0]))


RAGGED = [[70] + [2] * 9, [1] * 5 + [100] + [3] * 20, [60, 10, 20], [1, 40, 1, 90, 1], [2] * 80, [1] * 70 + [33], [0, 2, 1, 1], [0, 0, 4, 0]]


@pytest.mark.parametrize("rows", RAGGED, ids=str)
@pytest.mark.parametrize("tree", [None, "random", "line"])
def test_rule_ragged(w12, rows, tree):
    """Few long sequences among short ones, more than 64 of them, empty ones."""
    check_rule(Step(w12, rows, 1, 2, tree=tree, seed=len(rows)), heads=(1,))
    if tree is None:
        check_rule(Step(w12, rows, 1, 2, seed=len(rows)), keep=True, heads=(0,))


@pytest.mark.parametrize("rows", [[1] * 33, [0, 2] + [1] * 31, [20] * 9, [33, 3, 40, 17, 16, 31, 20, 18, 50], [20] * 20, [40, 60, 3, 70, 50, 65, 33, 66, 40]], ids=str)
@pytest.mark.parametrize("kd,vd", [(128, 128), (64, 128), (128, 64)])
def test_rule_many_heads(w12, rows, kd, vd):
    """Enough sequences and heads for the forms that a full card takes."""
    for keep in (False, True):
        check_rule(Step(w12, rows, 4, 16, kd, vd, seed=kd + vd), keep=keep, heads=(0, 15))
    check_rule(Step(w12, rows, 4, 16, kd, vd, tree="random", seed=kd + vd), heads=(7,))


@pytest.mark.parametrize("hk,hv", [(1, 1), (1, 3), (3, 3), (2, 6), (4, 4)])
@pytest.mark.parametrize("kd,vd", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("tree", [None, "random"])
def test_rule_heads(w12, hk, hv, kd, vd, tree):
    check_rule(Step(w12, [19, 4], hk, hv, kd, vd, tree=tree, seed=hv), keep=False)
    if tree is None:
        check_rule(Step(w12, [1, 35], hk, hv, kd, vd, layers=2, width=3, seed=hv), layer=1, keep=True)


@pytest.mark.parametrize("rows,tree,keep", [([512], None, True), ([300, 211, 1], None, False), ([512], "random", False),
                                            ([257, 40], "line", False)], ids=str)
def test_rule_long(w12, rows, tree, keep):
    """Decays of about 0.5 a row: errors of early rows fade, and the bounds stay small."""
    check_rule(Step(w12, rows, 1, 3, tree=tree, seed=7, rate=0.5), keep=keep, heads=(0, 2))


@pytest.mark.parametrize("tree", [None, "random"])
@pytest.mark.parametrize("rate", [0.0, 5.0, 400.0])
def test_rule_decays(w12, tree, rate):
    """No decay at all; decays that leave a few rows; decays beyond every exponent."""
    check_rule(Step(w12, [40, 9], 1, 2, tree=tree, seed=11, rate=rate))


@pytest.mark.parametrize("rows,tree", [([64], None), ([200, 5], None), ([14], None), ([32], "line"), ([130], "line"), ([60], "random")], ids=str)
def test_rule_the_same_key_again(w12, rows, tree):
    """Every row the same key at full strength and no decay: a row reads its own
    value back, and its delta is its value less its parent's. L is all ones on
    the path, so a tile's inverse is exact, where powers of L reach 3432; left are the
    roundings of a sum of at most `rows` deltas."""
    st = Step(w12, rows, 1, 2, tree=tree, seed=51)
    st.c.kv[0, :, :128] = 0
    st.c.kv[0, :, 3] = 1
    st.q.zero_()
    st.q[:, 0, 3] = 1
    st.c.gates[0, :, 0], st.c.gates[0, :, 1] = 0, 1
    out, delta = f64(st.rule(scale=0.5)).reshape(-1, 2, 128), f64(st.c.delta[0])
    v = f64(st.c.kv[0, :, 128:]).reshape(-1, 2, 128)
    for s, n in enumerate(rows):
        a = int(st.off[s])
        first = f64(st.c.state[0, int(st.slot[s]), :, 3])
        size = 4 * max(np.abs(v[a:a + n]).max(), np.abs(first).max())
        tol = (3 * n + 100) * D.U * size
        for i in range(n):
            p = i - 1 if tree is None else int(st.parent[a + i])
            before = v[a + p] if i else first
            assert (np.abs(delta[a + i] - (v[a + i] - before)) <= tol).all(), (s, i)
            assert (np.abs(out[a + i] - 0.5 * v[a + i]) <= D.BF16 * np.abs(0.5 * v[a + i]) + tol).all(), (s, i)


def test_rule_decay_of_minus_infinity(w12):
    """The state is forgotten, and what follows is as from a state of zeros."""
    import torch
    st = Step(w12, [20], 1, 2, seed=12)
    st.c.gates[0, 7, 0] = float("-inf")
    out = check_rule(st, keep=False)
    assert torch.isfinite(out).all()
    late = Step(w12, [20], 1, 2, seed=12)
    late.c.gates[0, 7, 0] = float("-inf")
    late.c.state.zero_()
    assert torch.equal(out[7:], late.rule()[7:])


@pytest.mark.parametrize("rows,tree", [([12], "star"), ([40, 6], "random"), ([20], None), ([90], "random"), ([90], None),
                                       ([50] + [2] * 9, "random"), ([50] + [2] * 9, None), ([8, 1, 1], None)], ids=str)
@pytest.mark.parametrize("where", ["k", "v", "g", "beta", "q"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_rule_rows_that_are_no_numbers(w12, rows, tree, where, value):
    """They reach the rows behind them, and no other row's bits."""
    import torch
    make = lambda: Step(w12, rows, 1, 2, tree=tree, seed=13)  # noqa: E731
    clean, st = make(), make()
    at = 5
    if where == "k":
        st.c.kv[0, at, 3] = value
    elif where == "v":
        st.c.kv[0, at, 128 + 9] = value  # of head 0
    elif where == "q":
        st.q[at, 0, 17] = value
    else:
        st.c.gates[0, at, 0 if where == "g" else 1, 1] = value
    a, b = clean.rule().view(torch.int16), st.rule()
    see = np.eye(st.total, dtype=bool)
    for s, n in enumerate(rows):
        for i in range(int(st.off[s]), int(st.off[s + 1])):
            p = i - 1 if tree is None else int(st.off[s]) + int(st.parent[i])
            if i > st.off[s]:
                see[i] |= see[p]
    behind = torch.tensor(see[:, at], device=DEV) & (torch.arange(st.total, device=DEV) != at if where == "q" else True)
    hit = torch.tensor([i == at if where == "q" else bool(x) for i, x in enumerate(see[:, at])], device=DEV)
    assert torch.equal(a[~hit], b.view(torch.int16)[~hit])
    d0, d1 = clean.c.delta[0, :st.total].view(torch.int32), st.c.delta[0, :st.total].view(torch.int32)
    assert torch.equal(d0[~behind], d1[~behind]) if where != "q" else torch.equal(d0, d1)
    bad = ~torch.isfinite(b[at].view(2, -1))
    assert bad.any()


@pytest.mark.parametrize("rows", [[8, 1, 1], [40], [30] + [1] * 5], ids=str)
def test_rule_kept_rows_that_are_no_numbers(w12, rows):
    """They stay with their sequence's state, and their head."""
    import torch
    clean, st = Step(w12, rows, 2, 2, seed=43), Step(w12, rows, 2, 2, seed=43)
    st.c.kv[0, 4, 2 * 128 + 5] = float("nan")  # a value of head 0
    a, b = clean.rule(keep=True).view(-1, 2, 128), st.rule(keep=True).view(-1, 2, 128)
    assert torch.equal(a[:4], b[:4]) and torch.equal(a[:, 1], b[:, 1]) and torch.isnan(b[4:rows[0], 0, 5]).all()
    assert torch.equal(a[rows[0]:], b[rows[0]:])
    s0 = int(st.slot[0])
    assert torch.isnan(st.c.state[0, s0, 0, :, 5]).all() and torch.equal(st.c.state[0, s0, 1], clean.c.state[0, s0, 1])
    rest = [i for i in range(st.slots) if i != s0]
    assert torch.equal(st.c.state[0, rest], clean.c.state[0, rest]) and torch.equal(st.c.conv, clean.c.conv)


@pytest.mark.parametrize("rows", [[1] * 5, [9, 2], [40], [30] + [1] * 5], ids=str)
def test_rule_queries_that_are_no_numbers_leave_the_state(w12, rows):
    import torch
    clean, st = Step(w12, rows, 1, 2, seed=48), Step(w12, rows, 1, 2, seed=48)
    st.q[0, 0, 7] = float("inf")
    a, b = clean.rule(keep=True), st.rule(keep=True)
    assert torch.equal(a[1:], b[1:]) and not torch.isfinite(b[0]).any() and torch.equal(clean.c.state, st.c.state)


def test_two_steps_in_flight(w12):
    """Two descriptions over the same state and window, each with its step's arrays and its own stream."""
    import torch
    one, two = Step(w12, [20, 7, 1], 2, 4, seed=49, slots=8), Step(w12, [5, 40], 2, 4, seed=50, slots=8)
    one.slot, two.slot = np.array([0, 3, 6]), np.array([5, 1])
    c = two.c
    two.c = w12.DeltaCache(state=one.c.state, conv=one.c.conv, raw=c.raw, kv=c.kv, gates=c.gates, delta=c.delta, key_heads=2)
    state, conv = one.c.state.clone(), one.c.conv.clone()
    xs = [Inputs(one, seed=1), Inputs(two, seed=2)]
    fixed = [dict(off=i32(s.off), slot=i32(s.slot), acc=i32([n - 1 for n in s.rows])) for s in (one, two)]

    def step(st, x, f):
        q = w12.w12_delta_append(st.c, 0, x.qkv, x.ba, f["off"], x.weight, x.a_log, x.dt, slot=f["slot"])
        out = w12.w12_delta_rule(st.c, 0, q, f["off"], slot=f["slot"])
        w12.w12_delta_commit(st.c, f["off"], f["acc"], slot=f["slot"], rows=st.total)
        return out

    want = [step(st, x, f) for st, x, f in zip((one, two), xs, fixed)]
    after = one.c.state.clone(), one.c.conv.clone()
    for _ in range(3):
        one.c.state.copy_(state)
        one.c.conv.copy_(conv)
        torch.cuda.synchronize()
        streams, got = [torch.cuda.Stream() for _ in range(2)], []
        for s, st, x, f in zip(streams, (one, two), xs, fixed):
            with torch.cuda.stream(s):
                got.append(step(st, x, f))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert torch.equal(after[0], one.c.state) and torch.equal(after[1], one.c.conv)


def test_rule_refuses_on_the_device(w12):
    """Trees and slots that are none: NaN for that sequence, nothing else written."""
    import torch
    for kind in ("parent", "root", "slot", "negative"):
        make = lambda: Step(w12, [9, 20, 6], 1, 2, tree="random", seed=14)  # noqa: E731
        clean, st = make(), make()
        if kind == "parent":
            st.parent[9 + 4] = 4
        elif kind == "root":
            st.parent[9] = 0
        else:
            st.slot[1] = st.slots if kind == "slot" else -1
        before = st.c.delta.clone()
        a, b = clean.rule(), st.rule()
        rest = torch.tensor([i for i in range(35) if not 9 <= i < 29], device=DEV)
        assert torch.isnan(b[9:29]).all() and torch.equal(a[rest], b[rest]), kind
        assert torch.equal(before[0, 9:29], st.c.delta[0, 9:29]) and torch.equal(before[0, 35:], st.c.delta[0, 35:])


def test_rule_refuses_far_sequences(w12):
    """Sequences past the 64th, and rows past the 64th of a tree."""
    import torch
    make = lambda: Step(w12, [1] * 70 + [100], 1, 2, tree="random", seed=44)  # noqa: E731
    clean, st, bad = make(), make(), make()
    a = clean.rule()
    bad.parent[70 + 90] = 90
    b = bad.rule()
    assert torch.isnan(b[70:]).all() and torch.equal(a[:70], b[:70])
    st.slot[68] = -1
    b = st.rule()
    assert torch.isnan(b[68]).all() and torch.equal(a[:68], b[:68]) and torch.equal(a[69:], b[69:])
    keep = Step(w12, [1] * 70, 1, 2, seed=45)
    keep.slot[69] = keep.slot[66]
    b = keep.rule(keep=True)
    assert torch.isnan(b[69]).all() and torch.isfinite(b[:69]).all()


def test_rule_keeps_a_slot_once(w12):
    import torch
    st = Step(w12, [3, 4, 2], 1, 2, seed=15)
    st.slot[2] = st.slot[0]
    alone = Step(w12, [3, 4, 2], 1, 2, seed=15)
    out, a = st.rule(keep=True), alone.rule(keep=True)
    assert torch.isnan(out[7:]).all() and torch.equal(out[:7], a[:7])
    s0 = int(st.slot[0])
    assert torch.equal(st.c.state[0, s0], alone.c.state[0, s0]) and torch.equal(st.c.conv[0, s0], alone.c.conv[0, s0])


def test_rule_a_slot_read_twice(w12):
    st = Step(w12, [6, 4, 6], 1, 2, tree="random", seed=16)
    st.slot[2] = st.slot[0]
    check_rule(st)


def test_rule_slot_is_the_sequence(w12):
    st = Step(w12, [6, 4], 1, 2, seed=17)
    st.slot = np.arange(2)
    check_rule(st, slot=None, keep=True)


@pytest.mark.parametrize("tree", [None, "random"])
def test_rule_ranges_that_are_none(w12, tree):
    """Offsets that run backwards, leave the step or meet: no rows; rows of no sequence stay."""
    import torch
    st = Step(w12, [6, 8, 5], 1, 2, tree=tree, seed=18)
    whole = Step(w12, [6, 8, 5], 1, 2, tree=tree, seed=18)
    a = whole.rule()
    out = torch.full_like(a, 7.0)
    before = st.c.delta.clone()
    st.off = np.array([0, 6, 2, 5])  # the second runs backwards, the third meets the first
    st.rule(out=out)
    assert torch.equal(out[:6], a[:6]) and (out[6:] == 7).all() and torch.equal(st.c.delta[0, 6:], before[0, 6:])
    st.off = np.array([0, 6, 30, 19])  # past the step
    out.fill_(7.0)
    st.rule(out=out)
    assert torch.equal(out[:6], a[:6]) and (out[6:] == 7).all() and torch.equal(st.c.delta[0, 6:], before[0, 6:])


def test_rule_is_reproducible_on_any_stream_and_in_graphs(w12):
    import torch
    st = Step(w12, [33, 8], 2, 4, tree="random", seed=19)
    a = st.rule().clone()
    d = st.c.delta.clone()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        b = st.rule()
    s.synchronize()
    assert torch.equal(a, b) and torch.equal(d, st.c.delta)
    out = torch.zeros_like(a)
    args = dict(slot=i32(st.slot), parent=i32(st.parent), out=out)
    off = i32(st.off)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w12.w12_delta_rule(st.c, 0, st.q, off, **args)
    for i in range(4):
        out.zero_()
        st.c.delta.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, out) and torch.equal(d[0, :st.total], st.c.delta[0, :st.total]), i
        (st.q.float() @ st.q.float().transpose(1, 2)).sum().item()


def test_rule_states_past_32_bits(w12):
    """The last slots of a state of more than 2^31 values, and the first."""
    import torch
    slots = 2 ** 31 // (8 * 128 * 128) + 40
    st = Step.__new__(Step)
    small = Step(w12, [5, 18], 2, 8, seed=20)
    st.__dict__.update(small.__dict__)
    c = w12.delta_cache(1, slots, 2, 8, 128, 128, 4, small.total, device=DEV)
    st.slots, st.slot = slots, np.array([slots - 1, 0])
    for s in range(2):
        c.state[0, int(st.slot[s])] = small.c.state[0, int(small.slot[s])]
        c.conv[0, int(st.slot[s])] = small.c.conv[0, int(small.slot[s])]
    for x, y in ((c.raw, small.c.raw), (c.kv, small.c.kv), (c.gates, small.c.gates), (c.delta, small.c.delta)):
        x.copy_(y[:, :small.total])
    st.c = c
    a, b = small.rule(keep=True), st.rule(keep=True)
    assert torch.equal(a, b)
    for s in range(2):
        assert torch.equal(c.state[0, int(st.slot[s])], small.c.state[0, int(small.slot[s])])
        assert torch.equal(c.conv[0, int(st.slot[s])], small.c.conv[0, int(small.slot[s])])
    assert not c.state[0, 1:slots - 1].any()


# ---------------------------------------------------------------------------------------------- append

class Inputs:
    def __init__(self, st, kind="f32", seed=0, layer=0, bias=True, wide=True):
        import torch
        g = torch.Generator(device=DEV)
        g.manual_seed(seed + 99)
        n = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        c, hv = st.c.channels, st.hv
        pad = hv * st.vd if wide else 0  # the output gate's columns lie between
        proj = n(st.total, -(-(c + pad + 2 * hv) // 32) * 32 if wide else c)
        proj = proj if kind == "f32" else proj.bfloat16()
        ba = proj[:, c + pad:c + pad + 2 * hv] if wide else (2 * n(st.total, 2 * hv)).to(proj.dtype)
        self.qkv, self.ba = (proj[:, :c], ba) if wide else (proj, ba)
        self.weight, self.bias = n(c, st.c.conv_width), n(c) if bias else None
        self.a_log, self.dt = torch.rand(hv, generator=g, device=DEV) * 2.7, n(hv) - 3

    def go(self, st, layer=0, **kw):
        a = dict(conv_bias=self.bias, slot=i32(st.slot), parent=i32(st.parent))
        a.update(kw)
        return st.w12.w12_delta_append(st.c, layer, self.qkv, self.ba, i32(st.off), self.weight, self.a_log, self.dt, **a)


def check_append(st, x, layer=0, **kw):
    import torch
    before = [t.clone() for t in (st.c.state, st.c.conv, st.c.raw, st.c.kv, st.c.gates, st.c.delta)]
    q = x.go(st, layer, **kw)
    torch.cuda.synchronize()
    raw = x.qkv.bfloat16()
    c = st.c
    same = lambda p, o: torch.equal(p.contiguous().view(torch.uint8), o.contiguous().view(torch.uint8))  # noqa: E731
    assert same(c.raw[layer, :st.total], raw)
    for i, t in enumerate((c.state, c.conv, c.raw, c.kv, c.gates, c.delta)):
        assert same(before[i][layer, st.total:], t[layer, st.total:]) if 2 <= i < 5 else same(before[i], t)
        for lay in range(st.layers):
            assert lay == layer or same(before[i][lay], t[lay])
    bias = None if x.bias is None else f64(x.bias)
    got = np.concatenate([f64(q).reshape(st.total, -1), f64(c.kv[layer, :st.total])], 1)
    for s in range(len(st.rows)):
        a, b = int(st.off[s]), int(st.off[s + 1])
        if a == b:
            continue
        parent = D.chain(b - a) if st.parent is None else st.parent[a:b]
        want, err = D.append(f64(raw[a:b]), f64(c.conv[layer, int(st.slot[s])]), parent, f64(x.weight), bias, st.hk, st.kd)
        assert (np.abs(got[a:b] - want) <= D.BF16 * np.abs(want) + 1.02 * err + 1e-38).all(), s
    ba = f64(x.ba)
    g, beta, eg, eb = D.gates(ba[:, :st.hv], ba[:, st.hv:], f64(x.a_log), f64(x.dt))
    gates = f64(c.gates[layer, :st.total])
    assert (np.abs(gates[:, 0] - g) <= eg + 1e-44).all() and (np.abs(gates[:, 1] - beta) <= eb + 1e-44).all()
    return q


@pytest.mark.parametrize("rows", [[1], [1, 1, 2], [3, 7], [33, 0, 1], [130], [1] * 70 + [5, 0, 2], [66, 1, 70, 3]], ids=str)
@pytest.mark.parametrize("tree", [None, "random", "star", "line"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_append(w12, rows, tree, kind):
    st = Step(w12, rows, tree=tree, seed=21)
    check_append(st, Inputs(st, kind))


@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("hk,hv,kd,vd", [(1, 1, 64, 64), (3, 6, 64, 128), (1, 3, 128, 64), (5, 5, 128, 128)])
def test_append_sizes(w12, width, hk, hv, kd, vd):
    st = Step(w12, [9, 2], hk, hv, kd, vd, layers=2, width=width, tree="random", seed=22)
    check_append(st, Inputs(st, "bf16" if width == 3 else "f32", bias=width != 3, wide=hk != 3), layer=1)


def test_append_gates_at_their_ends(w12):
    import torch
    st = Step(w12, [8], 1, 2, seed=23)
    x = Inputs(st)
    x.ba.copy_(torch.tensor([-300.0, -90.0, -20.0, -1.0, 0.0, 20.0, 100.0, 1000.0], device=DEV)[:, None].expand(8, 4))
    check_append(st, x)
    x.ba[3, 1] = float("nan")
    x.ba[4, 2] = float("nan")
    x.go(st)
    bad = torch.isnan(st.c.gates[0, :8])
    assert bad.sum() == 2 and bad[3, 1, 1] and bad[4, 0, 0]


def test_append_zero_rows_have_zero_heads(w12):
    st = Step(w12, [6], 1, 2, seed=24)
    x = Inputs(st, bias=False)
    x.qkv.zero_()
    st.c.conv.zero_()
    assert not check_append(st, x).any()


def test_append_large_inputs(w12):
    """SiLU's exponential beyond its range on both sides."""
    st = Step(w12, [6], 1, 2, seed=25)
    x = Inputs(st)
    x.qkv.mul_(1e4)
    check_append(st, x)


def test_append_refuses_on_the_device(w12):
    import torch
    for kind in ("parent", "root", "slot"):
        st = Step(w12, [4, 7, 3], 1, 2, tree="random", seed=26)
        x = Inputs(st)
        a = x.go(st).clone()
        keep = [t.clone() for t in (st.c.raw, st.c.kv, st.c.gates)]
        if kind == "slot":
            st.slot[1] = st.slots
        else:
            st.parent[4 + (3 if kind == "parent" else 0)] = 3
        for t in (st.c.raw, st.c.kv, st.c.gates):
            t[0, 4:11] = 5
        b = x.go(st)
        rest = torch.tensor([0, 1, 2, 3, 11, 12, 13], device=DEV)
        assert torch.isnan(b[4:11]).all() and torch.equal(a[rest], b[rest]), kind
        for t, o in zip((st.c.raw, st.c.kv, st.c.gates), keep):
            assert (t[0, 4:11] == 5).all() and torch.equal(t[0, rest], o[0, rest])


def test_append_rows_of_no_sequence(w12):
    import torch
    st = Step(w12, [4, 7], 1, 2, seed=27)
    x = Inputs(st)
    a = x.go(st).clone()
    q = torch.full_like(a, 7.0)
    st.off = np.array([0, 4, 2])
    st.c.raw.fill_(5)
    x.go(st, out=q)
    assert torch.equal(q[:4], a[:4]) and (q[4:] == 7).all() and (st.c.raw[0, 4:] == 5).all()


def test_append_strides(w12):
    """Columns of a wider product and a copy of them; rows that overlap or are not contiguous are refused."""
    import torch
    st = Step(w12, [5, 6], 1, 2, tree="random", seed=28)
    x = Inputs(st, "bf16")
    a = x.go(st).clone()
    kv = st.c.kv.clone()
    x.qkv, x.ba = x.qkv.contiguous(), x.ba.contiguous()
    assert torch.equal(a, x.go(st)) and torch.equal(kv, st.c.kv)
    keep = x.qkv
    x.qkv = keep[:1].expand(11, -1)
    with pytest.raises(ValueError):
        x.go(st)
    x.qkv = keep.t().contiguous().t()
    with pytest.raises(ValueError):
        x.go(st)
    wide = torch.zeros(11, keep.shape[1] + 3, dtype=keep.dtype, device=DEV)
    x.qkv = wide[:, :keep.shape[1]]  # rows that begin off 16 bytes
    with pytest.raises(w12.W12Error):
        x.go(st)


# ---------------------------------------------------------------------------------------------- commit

def root_path(r, parent):
    node, path = int(r.randint(len(parent))), []
    while node >= 0:
        path.append(node)
        node = int(parent[node])
    return path[::-1]


def check_commit(st, paths, use_path=True, refused=()):
    """paths: the rows kept of each sequence (tree-local)."""
    import torch
    c = st.c
    before = [t.clone() for t in (c.state, c.conv, c.raw, c.kv, c.gates, c.delta)]
    acc = [len(p) - 1 for p in paths]
    full = np.full(st.total, -1)
    for s, p in enumerate(paths):
        full[int(st.off[s]):int(st.off[s]) + len(p)] = p
    kept = st.w12.w12_delta_commit(c, i32(st.off), i32(acc), path=i32(full) if use_path else None, slot=i32(st.slot), rows=st.total)
    torch.cuda.synchronize()
    assert kept.tolist() == [-1 if s in refused else len(p) for s, p in enumerate(paths)]
    same = lambda x, y: torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))  # noqa: E731
    assert all(same(x, y) for x, y in zip(before[2:], (c.raw, c.kv, c.gates, c.delta)))
    touched = {int(st.slot[s]) for s, p in enumerate(paths) if p and s not in refused}
    others = [i for i in range(st.slots) if i not in touched]
    assert same(before[0][:, others], c.state[:, others]) and same(before[1][:, others], c.conv[:, others])
    for s, p in enumerate(paths):
        if not p or s in refused:
            continue
        rows, slot = [int(st.off[s]) + i for i in p], int(st.slot[s])
        assert torch.equal(c.conv[:, slot], torch.cat([before[1][:, slot], c.raw[:, rows]], 1)[:, -c.conv.shape[2]:])
        for lay in range(st.layers):
            kv, gates, delta = f64(c.kv[lay]), f64(c.gates[lay]), f64(c.delta[lay])
            for h in range(st.hv):
                key = h // (st.hv // st.hk)
                want, err = D.commit(f64(before[0][lay, slot, h]), kv[:, key * st.kd:(key + 1) * st.kd], delta[:, h], gates[:, 0, h], rows)
                got = f64(c.state[lay, slot, h])
                assert (np.abs(got - want) <= err + D.U * np.abs(want)).all(), (s, lay, h)


@pytest.mark.parametrize("rows", [[1], [2, 1, 9], [32], [17, 40], [150]], ids=str)
@pytest.mark.parametrize("hk,hv,kd,vd,width", [(1, 2, 128, 128, 4), (2, 2, 64, 128, 2), (1, 3, 128, 64, 3), (2, 4, 64, 64, 4)])
def test_commit_trees(w12, rows, hk, hv, kd, vd, width):
    st = Step(w12, rows, hk, hv, kd, vd, layers=2, width=width, tree="random", seed=31)
    check_commit(st, [root_path(st.r, st.parent[int(a):int(b)]) for a, b in zip(st.off[:-1], st.off[1:])])


@pytest.mark.parametrize("took", [[1], [5, 0, 3], [15], [16], [17], [31, 33], [64], [65], [512], [200, 100]], ids=str)
def test_commit_chains(w12, took):
    st = Step(w12, [max(t, 2) if t < 512 else t for t in took], 1, 2, layers=1, seed=32)
    check_commit(st, [list(range(t)) for t in took], use_path=False)


def test_commit_decays(w12):
    for rate in (0.0, 30.0, 400.0):
        st = Step(w12, [40], 1, 2, tree="random", seed=33, rate=rate)
        check_commit(st, [root_path(st.r, st.parent)])
    st = Step(w12, [9], 1, 2, seed=34)
    st.c.gates[0, 4, 0, 1] = float("-inf")
    check_commit(st, [list(range(9))], use_path=False)


def test_commit_refuses_on_the_device(w12):
    make = lambda: Step(w12, [6, 8, 5], 1, 2, layers=2, seed=35)  # noqa: E731
    check_commit(make(), [[0, 2], [1, 3], [0]], refused=(1,))            # not from the root
    check_commit(make(), [[0, 2], [0, 3, 3], [0]], refused=(1,))         # not ascending
    check_commit(make(), [[0, 2], [0, 3, 8], [0, 1]], refused=(1,))      # past its rows
    check_commit(make(), [[0, 2], list(range(8)), []])                   # a refused tree keeps nothing
    st = make()
    st.slot[2] = st.slot[0]
    check_commit(st, [[0, 2], [0, 3], [0]], refused=(2,))
    for bad in (st.slots, -1):
        st = make()
        st.slot[1] = bad
        check_commit(st, [[0], [0, 3], [0, 4]], refused=(1,))


def test_commit_accept_len_outside(w12):
    import torch
    for acc in (-2, 8, 1 << 30):
        st = Step(w12, [6, 8, 5], 1, 2, seed=36)
        before = st.c.state.clone()
        kept = w12.w12_delta_commit(st.c, i32(st.off), i32([0, acc, 1]), slot=i32(st.slot), rows=st.total)
        assert kept.tolist() == [1, -1, 2]
        s1 = int(st.slot[1])
        assert torch.equal(before[0, s1], st.c.state[0, s1])


def test_commit_values_that_are_no_numbers(w12):
    """Of rows that are not accepted: they reach nothing."""
    import torch
    st, clean = Step(w12, [12], 1, 2, seed=37), Step(w12, [12], 1, 2, seed=37)
    for c in (st.c,):
        c.kv[0, 3] = float("nan")
        c.delta[0, 3] = float("inf")
        c.gates[0, 3] = float("nan")
        c.raw[0, 3] = float("nan")
    path = np.concatenate([[0, 1, 2, 4, 9], np.full(7, -1)])
    for x in (st, clean):
        w12.w12_delta_commit(x.c, i32(x.off), i32([4]), path=i32(path), slot=i32(x.slot))
    assert torch.equal(st.c.state, clean.c.state) and torch.equal(st.c.conv, clean.c.conv)


def test_commit_a_batch(w12):
    """More than 64 sequences, one of them refused, one empty."""
    st = Step(w12, [3] * 70 + [0, 2], 1, 1, 64, 64, tree="line", seed=46)
    st.slot[69] = st.slots + 3
    check_commit(st, [[0, 1]] * 35 + [[0]] * 35 + [[], [0, 1]], refused=(69,))


def test_commit_and_append_in_graphs(w12):
    """A captured step, replayed: every replay goes on from the state the one before left."""
    import torch
    eager, st = Step(w12, [9, 4], 2, 4, tree="random", seed=47), Step(w12, [9, 4], 2, 4, tree="random", seed=47)
    x = Inputs(st, "bf16")
    path = np.full(13, -1)
    path[0], path[9:11] = 0, [0, 1]
    fixed = [(i32(e.off), i32(e.slot), i32(e.parent), i32([0, 1]), i32(path)) for e in (eager, st)]

    def step(e, off, slot, parent, acc, p, q, out):
        w12.w12_delta_append(e.c, 0, x.qkv, x.ba, off, x.weight, x.a_log, x.dt, conv_bias=x.bias, slot=slot, parent=parent, out=q)
        w12.w12_delta_rule(e.c, 0, q, off, slot=slot, parent=parent, out=out)
        return w12.w12_delta_commit(e.c, off, acc, path=p, slot=slot)

    bufs = [(torch.zeros(13, 2, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(13, 512, dtype=torch.bfloat16, device=DEV)) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kept = step(st, *fixed[1], *bufs[1])
    for i in range(4):
        want = step(eager, *fixed[0], *bufs[0])
        graph.replay()
        torch.cuda.synchronize()
        assert want.tolist() == kept.tolist() == [1, 2]
        assert torch.equal(bufs[0][1], bufs[1][1]) and torch.equal(eager.c.state, st.c.state) and torch.equal(eager.c.conv, st.c.conv), i
        eager.c.state.square().sum().item()


# ---------------------------------------------------------------------------------------------- together

def test_a_committed_path_is_the_chain_of_its_rows(w12):
    """Tree, acceptance, commit, and then: the states that a chain of the same rows leaves."""
    import torch
    tree = Step(w12, [24, 10], 2, 4, tree="random", seed=41)
    x = Inputs(tree, "bf16", seed=5)
    paths = [root_path(tree.r, tree.parent[:24]), root_path(tree.r, tree.parent[24:])]
    rows = [len(p) for p in paths]
    line = Step(w12, rows, 2, 4, seed=41)
    line.slot, line.slots = tree.slot, tree.slots
    for a, b in ((line.c.state, tree.c.state), (line.c.conv, tree.c.conv)):
        a.copy_(b)
    y = Inputs(line, "bf16", seed=5)
    at = torch.tensor(paths[0] + [24 + i for i in paths[1]], device=DEV)
    y.qkv, y.ba, y.weight, y.bias, y.a_log, y.dt = x.qkv[at], x.ba[at], x.weight, x.bias, x.a_log, x.dt
    tree.q, line.q = x.go(tree), y.go(line)
    assert torch.equal(tree.q[at], line.q) and torch.equal(tree.c.kv[0, at], line.c.kv[0, :len(at)])
    a, b = tree.rule(), line.rule(keep=True)
    full = np.full(34, -1)
    full[:rows[0]], full[24:24 + rows[1]] = paths[0], paths[1]
    kept = w12.w12_delta_commit(tree.c, i32(tree.off), i32([r - 1 for r in rows]), path=i32(full), slot=i32(tree.slot))
    assert kept.tolist() == rows
    assert torch.equal(tree.c.conv, line.c.conv)
    # both within their bounds of the same 64-bit states
    got, other = f64(tree.c.state), f64(line.c.state)
    assert np.abs(got - other).max() <= 2e-5 * max(1, np.abs(other).max())
    assert np.abs(f64(a[at]) - f64(b)).max() <= 2.5 * D.BF16 * np.abs(f64(b)).max()
