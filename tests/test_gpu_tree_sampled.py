"""GPU parity of tree_accept_sampled (through the C ABI) against the 64-bit
oracle: accepted lengths, paths and bonus tokens are equal."""
import numpy as np
import pytest

from oracle import tree_sampled as TS

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def say(*a):
    print("[sampled]", *a, flush=True)


@pytest.fixture(scope="module")
def w12():
    import torch
    import w12_weight_streaming_amd as w
    assert torch.cuda.is_available()
    w.lib()
    return w


def forest(seed, sizes, vocab, drafted, chain=False, f32=True, spread=3.0, clash=0.2):
    """Trees whose drafts are drawn from (or are the likely tokens of) a
    noisy copy of the target's rows; some siblings share a token."""
    import torch
    r = np.random.RandomState(seed)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    total = int(off[-1])
    logits = torch.tensor(r.randn(total, vocab) * spread, dtype=torch.float32)
    logits = logits if f32 else logits.bfloat16()
    lg = logits.float().numpy()
    guess = lg + r.randn(total, vocab).astype(np.float32)
    draft = np.exp(guess - guess.max(1, keepdims=True))
    draft = (draft / draft.sum(1, keepdims=True)).astype(np.float32)
    parent, token = [], []
    for s, n in enumerate(sizes):
        seen = {}
        for i in range(n):
            p = -1 if i == 0 else (i - 1 if chain else int(r.randint(max(0, i - 5), i)))
            parent.append(p)
            row = draft[off[s] + max(p, 0)].astype(np.float64)
            k = seen.get(p, 0)
            seen[p] = k + (0 if r.rand() < clash else 1)
            token.append(int(r.choice(vocab, p=row / row.sum())) if drafted else int(np.argsort(-row)[k % vocab]))
    temp = r.uniform(0.5, 1.3, len(sizes)).astype(np.float32)
    u, ub = r.rand(total).astype(np.float32), r.rand(len(sizes)).astype(np.float32)
    return dict(off=off, parent=np.array(parent, np.int32), token=np.array(token, np.int32), logits=logits, lg=lg, temp=temp,
                draft=draft if drafted else None, u=u, ub=ub)


def call(w12, f, **kw):
    import torch
    t = lambda a: None if a is None else torch.tensor(np.asarray(a), device=DEV)
    out = w12.tree_accept_sampled(t(f["off"]), t(f["parent"]), t(f["token"]), f["logits"].to(DEV), t(f["u"]), t(f["ub"]),
                                  temperature=t(f["temp"]), draft=t(f["draft"]), **kw)
    return [o.cpu().numpy() for o in out]


def both(w12, f):
    got = call(w12, f)
    ref = TS.forest(f["off"], f["parent"], f["token"], f["lg"], f["temp"], f["draft"], f["u"], f["ub"])
    for g, r, nm in zip(got, ref, ("accept_len", "path", "bonus")):
        assert np.array_equal(g, r), (nm, g, r)
    return got


@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("vocab", [1, 2, 37, 1000, 4096, 4097, 20001])
def test_forests(w12, vocab, chain, drafted):
    say("forest", vocab, chain, drafted)
    lens = []
    for seed in range(3):
        f = forest(100 * vocab + seed, [1, 9, 8, 17, 3, 32], vocab, drafted, chain, f32=seed != 1)
        lens += both(w12, f)[0].tolist()
    if vocab <= 1000:  # at more tokens these flat rows accept few drafts, by the oracle too
        assert max(lens) >= 1


@pytest.mark.parametrize("drafted", [False, True])
def test_full_vocabulary(w12, drafted):
    say("152064", drafted)
    both(w12, forest(7, [9, 32], 152064, drafted, f32=True, spread=4.0))
    both(w12, forest(8, [8] * 3, 152064, drafted, chain=True, f32=False, spread=4.0))


def test_wide_and_large_trees(w12):
    say("wide")
    f = forest(9, [40], 300, True, spread=0.5)
    f["parent"][1:] = 0  # one row of 39 children
    both(w12, f)
    f["draft"] = None
    both(w12, f)
    both(w12, forest(10, [1024, 700], 64, False, spread=1.0))


def test_random_numbers_at_their_ends(w12):
    say("ends")
    for u, ub in ((0.0, 0.0), (1.0, 1.0), (np.float32(1) - np.float32(2.0 ** -24), np.float32(1) - np.float32(2.0 ** -24))):
        for drafted in (False, True):
            f = forest(11, [9, 8, 12], 501, drafted)
            f["u"][:], f["ub"][:] = u, ub
            both(w12, f)


def test_masked_vocabularies_and_refused_rows(w12):
    import torch
    say("masks")
    f = forest(12, [8, 8, 8, 8, 8, 8], 5000, False)
    lg = f["lg"].copy()
    lg[:, 100:4900] = -np.inf               # a constrained vocabulary
    f["token"] = (f["token"] % 100).astype(np.int32)
    lg[8] = -np.inf                          # tree 1's root: nothing to draw
    lg[16, 4999] = np.nan                    # tree 2's root
    lg[24, 0] = np.inf                       # tree 3's root
    f["lg"], f["logits"] = lg, torch.tensor(lg)
    f["u"][32:] = 1.0                        # trees 4, 5 stop at their roots: other rows do not matter
    lg[33:40] = np.nan
    f["logits"] = torch.tensor(lg)
    got = both(w12, f)
    assert got[0][1:4].tolist() == [-1, -1, -1] and got[2][4] >= 0


def test_refused_trees(w12):
    say("refused")
    f = forest(13, [6] * 8, 100, False)
    f["parent"][6] = 0
    f["parent"][12 + 3] = 3
    f["parent"][18 + 2] = -1
    f["token"][24 + 1] = 100
    f["token"][30 + 5] = -1
    f["temp"][6] = 0.0
    f["temp"][7] = np.nan
    got = both(w12, f)
    assert got[0][1:].tolist() == [-1] * 7 and got[0][0] >= 0
    assert (got[1][6:] == -1).all()
    f = forest(14, [6] * 4, 100, False)
    f["off"][1:4] = [30, 12, 12]  # a range past the end, one that runs backwards, an empty one
    got = call(w12, f)
    assert got[0][:3].tolist() == [-1, -1, -1] and got[2][:3].tolist() == [-1, -1, -1]


def test_without_temperature_on_a_stream_and_replayed(w12):
    import torch
    say("streams")
    f = forest(15, [9, 9], 30000, True)
    f["temp"] = None
    want = both(w12, f)
    t = lambda a: torch.tensor(np.asarray(a), device=DEV)
    args = [t(f["off"]), t(f["parent"]), t(f["token"]), f["logits"].to(DEV), t(f["u"]), t(f["ub"])]
    draft = t(f["draft"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = w12.tree_accept_sampled(*args, draft=draft)
    s.synchronize()
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = w12.tree_accept_sampled(*args, draft=draft)
    for _ in range(3):
        for o in out:
            o.fill_(77)
        g.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(out, want))
        w12.tree_accept_sampled(*args, draft=draft)


def test_chosen_drafts_agree_with_tree_accept_at_low_temperature(w12):
    """As the temperature falls the walk becomes greedy acceptance."""
    import torch
    say("greedy limit")
    f = forest(16, [12, 8, 9], 4000, False, clash=0.0)
    f["temp"][:] = 1e-3
    acc, path, bonus = call(w12, f)
    t = lambda a: torch.tensor(np.asarray(a, np.int32), device=DEV)
    am = f["lg"].argmax(1)
    ref = [x.cpu().numpy() for x in w12.tree_accept(t(f["off"]), t(f["parent"]), t(f["token"]), t(am))]
    assert np.array_equal(acc, ref[0]) and np.array_equal(path, ref[1]) and np.array_equal(bonus, ref[2])


@pytest.mark.parametrize("drafted", [False, True])
def test_temperatures_of_every_size(w12, drafted):
    """Down to a denormal one (only the row's maxima are left) and up to where
    a mask of the type's lowest value still has weight; ties at the maximum,
    lowest values and -inf among the logits."""
    import torch
    say("temperatures", drafted)
    temps = np.array([1e-40, 1e-30, 1e-12, 1e-6, 1e-2, 1e3, 1e20, 3e38], np.float32)
    f = forest(17, [7] * len(temps), 2200, drafted, spread=30.0)
    lg = f["lg"].copy()
    lg[:, 300:900] = np.finfo(np.float32).min
    lg[:, 1500:1600] = -np.inf
    top = lg.max(1)
    lg[:, 40] = lg[:, 2100] = top            # three at the maximum, in two chunks
    lg[::3, 41] = np.nextafter(top[::3], np.float32(-np.inf), dtype=np.float32)
    f["token"][1::2] = np.where(np.arange(len(f["token"][1::2])) % 2, 40, 2100)
    f["lg"], f["logits"], f["temp"] = lg, torch.tensor(lg), temps
    if drafted:
        f["draft"][:, [40, 2100]] += np.float32(0.25)
    got = both(w12, f)
    assert (got[0] >= 0).all()


def test_offsets_that_are_no_ranges(w12):
    """A tree whose range leaves the nodes or meets an earlier tree's is
    refused, and takes no row from the others."""
    say("offsets")
    f = forest(18, [6] * 4, 1500, False)
    want = both(w12, f)
    f["off"] = np.array([0, 30, 6, 12, 18, 24, 6, 9], np.int32)  # out of range, backwards, trees 1 .. 3, backwards, rows of tree 1
    f["temp"] = np.array([9.0, 9.0, *f["temp"][1:], 9.0, 9.0], np.float32)
    f["ub"] = np.array([0.5, 0.5, *f["ub"][1:], 0.5, 0.5], np.float32)
    got = call(w12, f)
    assert got[0].tolist() == [-1, -1, *want[0][1:], -1, -1]
    assert got[2].tolist() == [-1, -1, *want[2][1:], -1, -1]
    assert np.array_equal(got[1][6:], want[1][6:])


@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("vocab", [262144, 262145, 600001])
def test_vocabularies_of_more_chunks_than_threads(w12, vocab, drafted):
    """A search for the drawn token that takes several turns, found in each
    of them and at their ends."""
    say("long rows", vocab, drafted)
    f = forest(19, [3] * 6, vocab, drafted, f32=not drafted, spread=1.0)
    f["ub"][:] = [0.0, 0.3, 0.4369, 0.6, 0.9, np.float32(1) - np.float32(2.0 ** -24)]
    f["temp"][:] = 5.0
    both(w12, f)


def test_draft_rows_of_nodes_without_children_are_not_read(w12):
    """Whatever such a row holds (here zeros, NaN, infinities, the largest
    value), the walk that ends at its node draws from the target's row."""
    say("drafts of leaves")
    f = forest(20, [1] * 12 + [6] * 4, 3000, True, chain=True, spread=1.0)
    f["u"][:] = 0.0  # every draft that the target allows is accepted: each walk ends at its leaf
    leaves = np.append(np.arange(12), f["off"][13:] - 1)
    want = call(w12, f)
    draft, odd = f["draft"].copy(), np.random.RandomState(20)
    for i in leaves:
        draft[i] = odd.choice(np.array([0, np.nan, np.inf, -np.inf, np.finfo(np.float32).max], np.float32), 3000)
    f["draft"] = draft
    got = both(w12, f)
    assert got[0].tolist() == [0] * 12 + [5] * 4
    assert all(np.array_equal(a, b) for a, b in zip(got, want))


def test_rows_past_32_bits(w12):
    """Logits of more than 2^32 bytes and 2^31 values: trees at both ends draw
    what they draw alone."""
    import torch
    say("32 bits")
    vocab, trees = 152064, 15000
    gen = torch.Generator(device=DEV).manual_seed(21)
    logits = torch.randn((trees, vocab), generator=gen, device=DEV, dtype=torch.bfloat16)  # 4.6 GB
    logits *= 3
    # the last tree: a root and four children
    sizes = [1] * (trees - 5) + [5]
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    parent = np.full(trees, -1, np.int32)
    parent[-4:] = 0
    r = np.random.RandomState(22)
    token = np.zeros(trees, np.int32)
    token[-4:] = logits[-5].float().topk(4).indices.cpu().numpy()
    u, ub = r.rand(trees).astype(np.float32), r.rand(len(sizes)).astype(np.float32)
    t = lambda a: torch.tensor(a, device=DEV)
    got = [x.cpu().numpy() for x in w12.tree_accept_sampled(t(off), t(parent), t(token), logits, t(u), t(ub))]
    for tree in (0, 1, 7000, 14123, 14124, trees - 6, trees - 5):
        a, b = off[tree], off[tree + 1]
        lg = logits[a:b].float().cpu().numpy()
        acc, way, bonus = TS.walk(parent[a:b], token[a:b], lg, 1.0, None, u[a:b], ub[tree])
        assert got[0][tree] == acc and got[1][a:a + len(way)].tolist() == way and got[2][tree] == bonus, tree


def test_no_trees_and_many_empty_ones(w12):
    """Trees without nodes are refused one by one; the others stand."""
    say("empty")
    f = forest(23, [4, 3], 500, False)
    want = both(w12, f)
    f["off"] = np.array([0] * 70 + [4] * 70 + [7] * 3, np.int32)
    n = len(f["off"]) - 1
    temp, ub = np.ones(n, np.float32), np.zeros(n, np.float32)
    temp[[69, 139]], ub[[69, 139]] = f["temp"], f["ub"]
    f["temp"], f["ub"] = temp, ub
    got = call(w12, f)
    keep = np.isin(np.arange(n), [69, 139])
    assert got[0][keep].tolist() == want[0].tolist() and got[2][keep].tolist() == want[2].tolist()
    assert (got[0][~keep] == -1).all() and (got[2][~keep] == -1).all() and np.array_equal(got[1], want[1])


@pytest.mark.parametrize("vocab,kids", [(5000, 1023), (300, 1023), (70000, 200)])
def test_many_siblings_that_share_tokens(w12, vocab, kids):
    """A node of as many children as a tree can have, most of them with a
    token that an earlier sibling had, several in a chunk of the vocabulary:
    accepted early, late and not at all."""
    say("siblings", vocab, kids)
    r = np.random.RandomState(24)
    for u in (0.0, 0.9, 0.995, np.float32(1) - np.float32(2.0 ** -20)):
        f = forest(25, [kids + 1, 3], vocab, False, spread=1.0)
        f["parent"][1:kids + 1] = 0
        f["token"][1:kids + 1] = r.choice(r.permutation(vocab)[:vocab // 20], kids)
        f["u"][:] = u
        f["temp"][:] = 1.0
        got = both(w12, f)
    assert got[0][0] == 0  # the last of them
