"""GPU parity of the KV cache (w12_kv_append, w12_kv_attention, w12_kv_commit,
through the C ABI) against the 64-bit oracle. Committed bytes and scales match
exactly; rotated rows and attention outputs within the roundings that the
tolerances count."""
import numpy as np
import pytest

import synth
from oracle import kv_cache as KV

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def say(*a):
    print("[kv]", *a, flush=True)


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


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def bf16(a):
    """numpy -> bf16 tensor on the GPU, and the values it holds."""
    import torch
    t = torch.tensor(np.asarray(a), dtype=torch.float32).bfloat16()
    return t.to(DEV), f64(t)


def rope_table(positions, rot):
    ang = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def random_parents(rng, n):
    return np.array([-1] + [int(rng.randint(max(0, i - 6), i)) for i in range(1, n)], np.int32)


class Serving:
    """A cache on the GPU and the oracle's state of it, driven step by step."""

    def __init__(self, w12, seqs, kv, group, dim, page, int8=False, layers=1, step_rows=64, blocks=24, seed=0,
                 rot=None, interleaved=False, positions=4096):
        import torch
        self.w12, self.seqs, self.kv, self.group, self.dim, self.page, self.layers = w12, seqs, kv, group, dim, page, layers
        self.rng = np.random.RandomState(seed)
        self.slots = seqs + 2
        self.slot = self.rng.permutation(self.slots)[:seqs].astype(np.int32)
        pages = seqs * blocks + 3
        self.cache = w12.kv_cache(layers, kv, dim, pages, self.slots, blocks, page, step_rows, int8, DEV)
        ids = self.rng.permutation(pages)[:seqs * blocks].reshape(seqs, blocks)
        table = np.full((self.slots, blocks), -7, np.int32)
        table[self.slot] = ids
        self.table = table
        self.cache.page_table.copy_(i32(table))
        # what no token wrote yet must never matter
        self.cache.recent.fill_(float("nan"))
        self.cache.scales.fill_(float("nan"))
        self.int8, self.rot, self.interleaved = int8, rot or dim, interleaved
        self.rope = rope_table(positions, self.rot)
        self.rope_t = torch.tensor(self.rope, device=DEV)
        self.state = [[[KV.Sequence(page, int8, dim) for _ in range(kv)] for _ in range(seqs)] for _ in range(layers)]

    def step(self, rows, parents=None, f32=False, check=True, commit=None, paths=None, qkv=None):
        """Append and attend in every layer, then commit. rows: rows of each
        sequence; parents: per sequence or None (chains); commit: accept_len
        of each (default: all rows of a chain, a root path of a tree)."""
        import torch
        w12, off = self.w12, np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        total, heads = int(off[-1]), self.kv * self.group
        par = None if parents is None else i32(np.concatenate(parents))
        each = parents if parents is not None else [KV.chain(n) for n in rows]
        width = (heads + 2 * self.kv) * self.dim
        drafted = []
        for layer in range(self.layers):
            x = self.rng.randn(total, width).astype(np.float32) if qkv is None else qkv
            xt = torch.tensor(x, device=DEV)
            xt = xt if f32 else xt.bfloat16()
            xv = f64(xt).reshape(total, -1, self.dim)
            q = w12.w12_kv_append(self.cache, layer, xt, i32(off), self.rope_t, heads, slot=i32(self.slot), parent=par,
                                  interleaved=self.interleaved)
            out = w12.w12_kv_attention(self.cache, layer, q, i32(off), slot=i32(self.slot), parent=par)
            torch.cuda.synchronize()
            got_q, got = f64(q), f64(out).reshape(total, heads, self.dim)
            rec = f64(self.cache.recent[layer])
            per_seq = []
            for s in range(self.seqs):
                a, b = off[s], off[s + 1]
                if a == b:
                    per_seq.append(None)
                    continue
                length = self.state[layer][s][0].length
                pos = length + KV.depths(each[s])
                turned, size = KV.rotate(xv[a:b, :heads + self.kv], pos, self.rope, self.interleaved)
                # one rounding to bf16, and three in fp32 of |x cos| + |y sin|
                tol = 2.0 ** -8 * np.abs(turned) + 4 * 2.0 ** -24 * size
                tail = length % self.page
                at = np.arange(tail, tail + b - a)
                k = np.stack([rec[self.slot[s], h, 0][KV.key_places(tail + b - a, self.dim)[at]] for h in range(self.kv)], 1)
                v = np.stack([rec[self.slot[s], h, 1][KV.value_places(tail + b - a, self.dim)[at]] for h in range(self.kv)], 1)
                if check:
                    assert (np.abs(got_q[a:b] - turned[:, :heads]) <= tol[:, :heads]).all(), ("q", layer, s)
                    assert (np.abs(k - turned[:, heads:]) <= tol[:, heads:]).all(), ("k", layer, s)
                    want_v = xv[a:b, heads + self.kv:]
                    assert (np.abs(v - want_v) <= 2.0 ** -8 * np.abs(want_v)).all(), ("v", layer, s)
                    for h in range(self.kv):
                        seq = self.state[layer][s][h]
                        see = np.concatenate([np.ones((b - a, length), bool), KV.ancestors(each[s])], 1)
                        ref, av, sz = KV.attention(got_q[a:b, h * self.group:(h + 1) * self.group],
                                                   np.concatenate([seq.k, k[:, h]]), np.concatenate([seq.v, v[:, h]]), see,
                                                   self.dim ** -0.5)
                        lim = KV.attention_tolerance(ref, av, sz, length + b - a, self.dim)
                        err = np.abs(got[a:b, h * self.group:(h + 1) * self.group] - ref)
                        assert (err <= lim).all(), ("attention", layer, s, h, float((err / lim).max()))
                per_seq.append((k, v))
            drafted.append(per_seq)
        acc, path = [], []
        for s in range(self.seqs):
            n = rows[s]
            if parents is None:
                a = n - 1 if commit is None else commit[s]
                way = np.arange(n)
            else:
                node = int(self.rng.randint(n))
                way = [node]
                while each[s][way[0]] >= 0:
                    way.insert(0, int(each[s][way[0]]))
                a = len(way) - 1
                if commit is not None:
                    a = min(a, commit[s])
            acc.append(a)
            path.append(np.concatenate([np.asarray(way, np.int32)[:a + 1], np.full(n - min(a + 1, n), -1, np.int32)]))
        w12.w12_kv_commit(self.cache, i32(off), i32(acc), path=None if parents is None else i32(np.concatenate(path)),
                          slot=i32(self.slot))
        for layer in range(self.layers):
            for s in range(self.seqs):
                if acc[s] >= 0:
                    k, v = drafted[layer][s]
                    for h in range(self.kv):
                        self.state[layer][s][h].commit(k[path[s][:acc[s] + 1], h], v[path[s][:acc[s] + 1], h])
        if check:
            self.check()
        return acc

    def check(self):
        """Lengths, pages, scales and the recent tail are the oracle's, bit for bit."""
        length = self.cache.length.cpu().numpy()
        codes = self.cache.pages.float().cpu().numpy()
        scales = self.cache.scales.cpu().numpy()
        for layer in range(self.layers):
            rec = f64(self.cache.recent[layer])
            for s in range(self.seqs):
                assert length[self.slot[s]] == self.state[layer][s][0].length
                for h in range(self.kv):
                    seq = self.state[layer][s][h]
                    for b, blk in enumerate(seq.blocks):
                        pid = self.table[self.slot[s], b]
                        for v in (0, 1):
                            assert np.array_equal(scales[layer, pid, h, v], blk[2 * v + 1], equal_nan=True), (layer, s, h, b, v)
                            if blk[2 * v] is not None:
                                got = codes[layer, pid, h, v][KV.places(v, self.page, self.dim)]
                                assert np.array_equal(got, blk[2 * v]), ("codes", layer, s, h, b, v)
                    tail = seq.length % self.page
                    if tail:
                        for v, x in ((0, seq.k), (1, seq.v)):
                            got = rec[self.slot[s], h, v][KV.places(v, tail, self.dim)]
                            assert np.array_equal(got, x[seq.length - tail:], equal_nan=True), ("tail", layer, s, h, v)


# (seqs, kv heads, group, dim, page, int8, rows of the steps)
CASES = [
    (1, 1, 1, 64, 32, False, [1, 1, 31, 1, 64, 3]),
    (3, 2, 6, 128, 64, False, [40, 24, 1, 64, 63, 2]),
    (2, 4, 6, 256, 64, False, [64, 33, 30, 1, 1]),
    (2, 3, 5, 64, 96, True, [64, 31, 1, 1, 64]),
    (4, 1, 8, 128, 128, True, [64, 63, 1, 5, 64, 60]),
    (2, 2, 12, 256, 32, True, [17, 47, 32, 1]),
    (5, 8, 1, 128, 64, False, [3, 60, 1, 1]),
]


@pytest.mark.parametrize("seqs,kv,group,dim,page,int8,steps", CASES)
def test_chains(w12, seqs, kv, group, dim, page, int8, steps):
    say("chains", seqs, kv, group, dim, page, int8)
    sv = Serving(w12, seqs, kv, group, dim, page, int8, seed=dim + page)
    for i, n in enumerate(steps):
        rows = [max(1, n - 5 * s) for s in range(seqs)]
        sv.step(rows, f32=i % 2 == 1)


@pytest.mark.parametrize("seqs,kv,group,dim,page,int8,steps", CASES)
def test_trees_keep_one_path(w12, seqs, kv, group, dim, page, int8, steps):
    say("trees", seqs, kv, group, dim, page, int8)
    sv = Serving(w12, seqs, kv, group, dim, page, int8, seed=dim + page + 1, layers=2 if dim < 256 else 1)
    sv.step([page - 3 if page < 65 else 61] * seqs)
    for i in range(6):
        rows = [int(sv.rng.randint(1, 33)) for _ in range(seqs)]
        sv.step(rows, parents=[random_parents(sv.rng, n) for n in rows])


@pytest.mark.parametrize("rot,interleaved", [(128, False), (64, False), (32, True), (2, False), (2, True), (30, False), (126, True)])
def test_rotations(w12, rot, interleaved):
    say("rotation", rot, interleaved)
    sv = Serving(w12, 2, 2, 3, 128, 32, seed=rot, rot=rot, interleaved=interleaved)
    sv.step([40, 7])
    rows = [9, 20]
    sv.step(rows, parents=[random_parents(sv.rng, n) for n in rows], f32=True)


@pytest.mark.parametrize("dim,group", [(64, 6), (128, 2)])
def test_prompt_of_512_rows(w12, dim, group):
    say("prompt 512", dim)
    sv = Serving(w12, 1, 1, group, dim, 64, step_rows=512, seed=dim)
    sv.step([45])
    sv.step([512])
    sv.step([1])


def test_long_context_is_split_and_joined(w12):
    """A sequence long enough that many workgroups share an item, next to
    short and empty ones."""
    say("long")
    sv = Serving(w12, 3, 2, 4, 64, 32, step_rows=512, blocks=200, seed=4, positions=8192)
    for n in range(10):
        sv.step([490, 20, 1], check=n in (0, 9), commit=[489, -1, 0])  # 511 rows: a step holds 512
    rows = [32, 5, 1]
    sv.step(rows, parents=[random_parents(sv.rng, n) for n in rows])


def test_512_sequences_of_one_row(w12):
    say("512 sequences")
    sv = Serving(w12, 512, 1, 2, 64, 32, step_rows=8, blocks=2, seed=5)
    for _ in range(2):
        sv.step([1] * 512)


def test_pages_do_not_depend_on_grouping(w12):
    """The same tokens in one prompt, or one by one behind rejected drafts,
    leave the same pages and tail."""
    import torch
    say("grouping")
    rng = np.random.RandomState(6)
    kv, dim, n = 2, 128, 70
    x = rng.randn(n, 4 * dim).astype(np.float32)
    junk = rng.randn(n, 4 * dim).astype(np.float32)
    rope = torch.tensor(rope_table(200, dim), device=DEV)
    caches = []
    for one_by_one in (False, True):
        c = w12.kv_cache(1, 1, dim, 4, 1, 4, 32, 96, False, DEV)
        c.page_table.copy_(i32([[0, 1, 2, 3]]))
        if not one_by_one:
            w12.w12_kv_append(c, 0, torch.tensor(x, device=DEV), i32([0, n]), rope, 2)
            w12.w12_kv_commit(c, i32([0, n]), i32([n - 1]))
        else:
            for i in range(n):  # a row, with two drafts behind it that are dropped
                rows = np.stack([x[i], junk[i], junk[i] * 100])
                w12.w12_kv_append(c, 0, torch.tensor(rows, device=DEV), i32([0, 3]), rope, 2, parent=i32([-1, 0, 0]))
                w12.w12_kv_commit(c, i32([0, 3]), i32([0]), path=i32([0, -1, -1]))
        assert c.length.item() == n
        caches.append(c)
    a, b = caches
    assert torch.equal(a.pages.view(torch.uint8)[:, :2], b.pages.view(torch.uint8)[:, :2])
    assert torch.equal(a.scales[:, :2], b.scales[:, :2])
    for v in (0, 1):
        at = torch.tensor(KV.places(v, n % 32, dim).ravel(), device=DEV)
        assert torch.equal(a.recent[0, 0, 0, v][at], b.recent[0, 0, 0, v][at])


def test_special_values_close_blocks(w12):
    """Zeros, one large value, tiny values, an infinity and a NaN in a block."""
    import torch
    say("special blocks")
    for int8 in (False, True):
        dim, page = 64, 32
        sv = Serving(w12, 1, 1, 1, dim, page, int8, seed=8, step_rows=256)
        x = np.zeros((6 * page, 3 * dim), np.float32)
        r = np.random.RandomState(9)
        x[page:2 * page] = r.randn(page, 3 * dim) * 2.0 ** -120
        x[2 * page:3 * page] = r.randn(page, 3 * dim)
        x[2 * page + 5, dim + 3] = 3e38
        x[3 * page:4 * page] = r.randn(page, 3 * dim)
        x[3 * page + 1, 2 * dim + 7] = np.inf
        x[4 * page:5 * page] = r.randn(page, 3 * dim)
        x[4 * page + 1, 2 * dim + 9] = np.nan
        x[5 * page:] = 448 * r.choice([-1, 1], (page, 3 * dim))
        # each block in one step from row 0, so that rotation leaves its first row alone
        off, q = i32([0, 6 * page]), None
        rope = torch.tensor(np.concatenate([np.ones((256, dim // 2)), np.zeros((256, dim // 2))], 1), dtype=torch.float32, device=DEV)
        w12.w12_kv_append(sv.cache, 0, torch.tensor(x, device=DEV), off, rope, 1, slot=i32(sv.slot))
        w12.w12_kv_commit(sv.cache, off, i32([6 * page - 1]), slot=i32(sv.slot))
        _, vals = bf16(x)
        with np.errstate(invalid="ignore"):
            sv.state[0][0][0].commit(vals[:, dim:2 * dim], vals[:, 2 * dim:])
        sv.check()


def test_nan_and_inf_reach_only_rows_that_see_them(w12):
    """Siblings' infinities and NaN, in keys and values, and garbage behind
    the rows, stay out of a row's output; its own ancestors' come through."""
    import torch
    say("nan")
    kv, group, dim, page, n = 1, 3, 128, 32, 40
    sv = Serving(w12, 1, kv, group, dim, page, seed=10)
    sv.step([29])
    parent = np.array([-1] + [0] * 10 + list(range(10, 39)), np.int32)  # ten leaves, then a chain from the tenth
    rng = np.random.RandomState(11)
    x = rng.randn(n, (kv * group + 2 * kv) * dim).astype(np.float32)
    outs = []
    for dirty in (False, True):
        y = x.copy()
        if dirty:
            y[1, group * dim + 5] = np.inf                # leaf 1's key
            y[2, (group + 1) * dim:] = np.nan             # leaf 2's value
            y[3, (group + 1) * dim + 7] = -np.inf         # leaf 3's value
            y[39, (group + 1) * dim + 100] = np.inf       # the chain's last row
        q = w12.w12_kv_append(sv.cache, 0, torch.tensor(y, device=DEV), i32([0, n]), sv.rope_t, group, slot=i32(sv.slot),
                              parent=i32(parent))
        outs.append(f64(w12.w12_kv_attention(sv.cache, 0, q, i32([0, n]), slot=i32(sv.slot), parent=i32(parent))))
    clean, dirty = outs
    same = [i for i in range(n) if i not in (1, 2, 3, 39)]
    assert np.array_equal(clean[same], dirty[same])
    d = dirty.reshape(n, group, dim)
    assert np.isnan(d[1]).all() and np.isnan(d[2]).all()
    assert (d[3, :, 7] == -np.inf).all() and np.isfinite(np.delete(d[3], 7, axis=1)).all()
    assert (d[39, :, 100] == np.inf).all() and np.array_equal(np.delete(d[39], 100, axis=1), np.delete(clean.reshape(n, group, dim)[39], 100, axis=1))


def attend(w12, sv, q, off, **kw):
    import torch
    out = torch.full((q.shape[0] + 2, q.shape[1] * q.shape[2]), 7.0, dtype=torch.bfloat16, device=DEV)
    w12.w12_kv_attention(sv.cache, 0, q, i32(off), out=out, **kw)
    torch.cuda.synchronize()
    return f64(out)


def test_device_detected_errors_poison_only_their_sequence(w12):
    import torch
    say("refused sequences")
    sv = Serving(w12, 4, 2, 2, 64, 32, seed=12)
    sv.step([40, 40, 40, 40])
    off = [0, 3, 6, 9, 12]
    q, _ = bf16(sv.rng.randn(12, 4, 64))
    good = attend(w12, sv, q, off, slot=i32(sv.slot))
    assert np.isfinite(good).all() and (good[12:] == 7).all()

    def only(seq, got, where):
        rows = np.arange(off[seq], off[seq + 1])
        rest = np.setdiff1d(np.arange(14), rows)
        assert np.isnan(got[rows]).all(), where
        assert np.array_equal(got[rest], good[rest]), where
    par = [np.array([-1, 0, 1]) for _ in range(4)]
    assert np.array_equal(attend(w12, sv, q, off, slot=i32(sv.slot), parent=i32(np.concatenate(par))), good)
    for bad in ([0, 0, 1], [-1, 1, 1], [-1, 0, 2], [-1, -1, 0], [-1, 0, 9999], [-2, 0, 1]):
        p = [x.copy() for x in par]
        p[2] = np.array(bad)
        only(2, attend(w12, sv, q, off, slot=i32(sv.slot), parent=i32(np.concatenate(p))), bad)
    for bad_slot in (-1, sv.slots, 1 << 30):
        sl = sv.slot.copy()
        sl[1] = bad_slot
        only(1, attend(w12, sv, q, off, slot=i32(sl)), bad_slot)
    for bad_len in (-1, 24 * 32 + 1, 1 << 30):
        keep = sv.cache.length.clone()
        sv.cache.length[int(sv.slot[3])] = bad_len
        only(3, attend(w12, sv, q, off, slot=i32(sv.slot)), bad_len)
        sv.cache.length.copy_(keep)
    for bad_page in (-1, sv.cache.pages.shape[1], -(1 << 31), (1 << 31) - 1):
        keep = sv.cache.page_table.clone()
        sv.cache.page_table[int(sv.slot[0]), 0] = bad_page
        only(0, attend(w12, sv, q, off, slot=i32(sv.slot)), bad_page)
        sv.cache.page_table.copy_(keep)
    # offsets: sequences whose rows are no range have no rows; the others' stand
    got = attend(w12, sv, q, [0, 3, 99, 9, 12], slot=i32(sv.slot))
    assert np.array_equal(got[:3], good[:3]) and (got[3:9] == 7).all() and np.array_equal(got[9:], good[9:])
    # more rows than the recent rows hold: 40 % 32 + 96 > 96
    big, _ = bf16(np.ones((96, 4, 64)))
    assert np.isnan(attend(w12, sv, big, [0, 96], slot=i32(sv.slot[:1]))[:96]).all()


def test_append_and_commit_refuse_on_the_device(w12):
    import torch
    say("append, commit refused")
    sv = Serving(w12, 3, 1, 1, 64, 32, seed=13, positions=64)
    sv.step([30, 30, 30])
    before = [t.clone() for t in (sv.cache.pages.view(torch.uint8), sv.cache.scales, sv.cache.recent)]
    off = i32([0, 4, 8, 12])
    x = torch.ones(12, 3 * 64, device=DEV)

    def untouched():
        return all(torch.equal(a.view(torch.uint8) if a.dtype != torch.uint8 else a, b.contiguous().view(torch.uint8))
                   for a, b in zip(before, (sv.cache.pages.view(torch.uint8), sv.cache.scales, sv.cache.recent)))
    # a slot named twice, one outside, a broken tree: only that sequence is refused
    sl = np.array([sv.slot[0], sv.slot[0], sv.slots], np.int32)
    q = w12.w12_kv_append(sv.cache, 0, x, off, sv.rope_t, 1, slot=i32(sl), parent=i32([-1, 0, 1, 2] * 3))
    assert torch.isfinite(q[:4]).all() and torch.isnan(q[4:]).all()
    sv.cache.recent.copy_(before[2])
    q = w12.w12_kv_append(sv.cache, 0, x, off, sv.rope_t, 1, slot=i32(sv.slot), parent=i32([0, 0, 1, 2] + [-1, 0, 1, 4] + [-1, 0, 0, 3 - 4]))
    assert torch.isnan(q).all() and untouched()
    # positions past the table: the rows beyond it
    sv.cache.length[int(sv.slot[0])] = 62
    q = w12.w12_kv_append(sv.cache, 0, x[:4], i32([0, 4]), sv.rope_t, 1, slot=i32(sv.slot[:1]))
    assert torch.isfinite(q[:2]).all() and torch.isnan(q[2:]).all()
    sv.cache.length[int(sv.slot[0])] = 30
    sv.cache.recent.copy_(before[2])
    # commits
    for acc, path in (([4, 0, 0], None), ([-2, 0, 0], None), ([2, 0, 0], [0, 2, 1, -1]), ([1, 0, 0], [1, 2, -1, -1]),
                      ([2, 0, 0], [0, 1, 4, -1]), ([1, 0, 0], [0, 0, -1, -1])):
        p = None if path is None else i32(path + [0, -1, -1, -1] * 2)
        got = w12.w12_kv_commit(sv.cache, off, i32(acc), path=p, slot=i32(sv.slot), length_out=sv.cache.length.clone())
        assert got[sv.slot].tolist() == [-1, 31, 31], (acc, path)
        assert untouched()
    # no room in the page table, a page that is none
    keep = sv.cache.page_table.clone()
    for bad in (-1, sv.cache.pages.shape[1]):
        sv.cache.page_table[int(sv.slot[1]), 0] = bad
        got = w12.w12_kv_commit(sv.cache, off, i32([0, 3, 0]), slot=i32(sv.slot), length_out=sv.cache.length.clone())
        assert got[sv.slot].tolist() == [31, -1, 31] and untouched()
    sv.cache.page_table.copy_(keep)
    # a refused tree (accept_len -1) keeps nothing and is no error; a slot named twice is committed once
    got = w12.w12_kv_commit(sv.cache, off, i32([-1, 0, 0]), slot=i32(sv.slot), length_out=sv.cache.length.clone())
    assert got[sv.slot].tolist() == [30, 31, 31]
    got = w12.w12_kv_commit(sv.cache, off, i32([0, 1, 0]), slot=i32([sv.slot[0], sv.slot[0], sv.slot[2]]),
                            length_out=sv.cache.length.clone())
    assert got[sv.slot].tolist() == [31, 30, 31]


def test_repeats_are_bitwise_and_shapes_share_a_workspace(w12):
    import torch
    say("determinism")
    first = {}
    for rep in range(3):
        for seqs, kv, group, dim, rows in ((1, 2, 6, 128, 3), (3, 1, 4, 64, 20), (2, 4, 6, 256, 9)):
            sv = Serving(w12, seqs, kv, group, dim, 32, seed=14, step_rows=512, blocks=60)
            for _ in range(2):
                sv.step([400] * seqs if seqs == 1 else [150] * seqs, check=False)
            q, _ = bf16(sv.rng.randn(rows * seqs, kv * group, dim))
            off = np.arange(seqs + 1) * rows
            for _ in range(3):
                got = attend(w12, sv, q, off, slot=i32(sv.slot))
                key = (seqs, dim)
                assert np.array_equal(first.setdefault(key, got), got)


def test_graph_replays_and_other_streams(w12):
    """One step captured with its append, attention and commit; replayed with
    eager calls of the same shapes in between, and calls on another stream."""
    import torch
    say("graphs")
    sv = Serving(w12, 2, 2, 6, 128, 64, seed=15, step_rows=64, blocks=40)
    sv.step([50, 64])
    sv.step([64, 64])
    rows, heads = 16, 12
    off = i32([0, 8, 16])
    x = torch.randn(rows, (heads + 4) * 128, device=DEV)
    slot = i32(sv.slot)
    length = sv.cache.length.clone()

    def step():
        q = w12.w12_kv_append(sv.cache, 0, x, off, sv.rope_t, heads, slot=slot)
        out = w12.w12_kv_attention(sv.cache, 0, q, off, slot=slot)
        w12.w12_kv_commit(sv.cache, off, i7, slot=slot, length_out=length)
        return out
    i7 = i32([3, 7])
    want = []
    inputs = [torch.randn_like(x) for _ in range(4)]
    for y in inputs:
        x.copy_(y)
        want.append((step().clone(), length.clone()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                out = step()
            graphs.append((g, out))
    torch.cuda.synchronize()
    for i, y in enumerate(inputs):
        for g, out in graphs:
            x.copy_(y)
            out.zero_()
            length.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[i][0]) and torch.equal(length, want[i][1]), i
            assert torch.equal(step(), want[i][0])  # eager, between replays
    other = torch.cuda.Stream()
    x.copy_(inputs[2])
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        got = step()
    other.synchronize()
    assert torch.equal(got, want[2][0])


def test_binding_refusals(w12):
    import torch
    say("binding")
    c = w12.kv_cache(1, 2, 64, 4, 2, 2, 32, 16, False, DEV)
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16, device=DEV)
    off = i32([0, 4])
    with pytest.raises(TypeError):
        w12.w12_kv_attention(c, 0, q.float(), off)
    with pytest.raises(ValueError):
        w12.w12_kv_attention(c, 0, q[..., :32].contiguous(), off)
    with pytest.raises(ValueError):
        w12.w12_kv_attention(c, 0, q, off, parent=i32([-1, 0, 1]))
    with pytest.raises(ValueError):
        w12.w12_kv_attention(c, 0, q, off, slot=i32([0, 1]))
    with pytest.raises(w12.W12Error):
        w12.w12_kv_attention(c, 1, q, off)  # no such layer
    with pytest.raises(w12.W12Error):
        w12.w12_kv_attention(c, 0, q[:, :3].contiguous(), off)  # 3 query heads on 2 kv heads
    with pytest.raises(w12.W12Error):
        w12.w12_kv_attention(c, 0, q, off, ws=torch.zeros(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        w12.w12_kv_attention(c, 0, q, off, out=torch.zeros(3, 256, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        w12.w12_kv_append(c, 0, torch.zeros(4, 64, device=DEV), off, torch.zeros(8, 64, device=DEV), 4)
    with pytest.raises(ValueError):
        w12.w12_kv_commit(c, off, i32([0, 0]))
    with pytest.raises(ValueError):
        w12.KvCache(c.pages, c.scales[:, :3].contiguous(), c.recent, c.page_table, c.length, 64)
    with pytest.raises(TypeError):
        w12.KvCache(c.pages.view(torch.uint8), c.scales, c.recent, c.page_table, c.length, 64)


def test_offsets_that_are_no_ranges(w12):
    """Sequences whose range runs backwards, leaves the rows or meets an
    earlier one's have no rows; the others stand, in every call."""
    import torch
    say("offsets")
    sv = Serving(w12, 4, 1, 2, 64, 32, seed=21)
    sv.step([20, 20, 20, 20])
    x = torch.tensor(sv.rng.randn(12, 4 * 64), dtype=torch.float32, device=DEV)
    slot, acc = i32(sv.slot), i32([2, 2, 2, 2])

    def run(off):
        start = [t.clone() for t in (sv.cache.recent, sv.cache.length)]
        q = torch.full((12, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        w12.w12_kv_append(sv.cache, 0, x, i32(off), sv.rope_t, 2, slot=slot, out=q)
        out = torch.full((12, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        w12.w12_kv_attention(sv.cache, 0, q, i32(off), slot=slot, out=out)
        length = w12.w12_kv_commit(sv.cache, i32(off), acc, slot=slot, length_out=sv.cache.length.clone(), rows=12)[slot.long()]
        recent = sv.cache.recent.clone()
        for t, b in zip((sv.cache.recent, sv.cache.length), start):
            t.copy_(b)
        return q, out, length.tolist(), recent
    good = run([0, 3, 6, 9, 12])
    assert good[2] == [23] * 4
    # (offsets, rows of sequences that stand, lengths after)
    for off, kept, length in (([0, 3, 99, 9, 12], [0, 1, 2, 9, 10, 11], [23, -1, -1, 23]),
                              ([0, 3, -5, 9, 12], [0, 1, 2, 9, 10, 11], [23, -1, -1, 23]),
                              ([0, 3, 1, 9, 12], [0, 1, 2, 9, 10, 11], [23, -1, -1, 23]),
                              ([6, 9, 0, 6, 12], [], [23, -1, 23, -1])):
        q, out, got, _ = run(off)
        assert got == length, off
        if kept:
            rest = np.setdiff1d(np.arange(12), kept)
            assert torch.equal(q[kept], good[0][kept]) and torch.equal(out[kept], good[1][kept]), off
            assert (q[rest] == 7).all() and (out[rest] == 7).all(), off
        else:  # rows 6 .. 9 are sequence 0's now, 0 .. 6 sequence 2's
            assert torch.isfinite(out[:9].float()).all() and (out[:9] != 7).any(1).all() and (out[9:] == 7).all()


def test_output_over_an_input_is_refused(w12):
    import torch
    say("overlap")
    c = w12.kv_cache(1, 2, 64, 4, 1, 2, 32, 16, False, DEV)
    off, rope = i32([0, 4]), torch.zeros(8, 64, device=DEV)
    buf = torch.zeros(4, 8 * 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(w12.W12Error):
        w12.w12_kv_append(c, 0, buf, off, rope, 4, out=buf)
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(w12.W12Error):
        w12.w12_kv_attention(c, 0, q, off, out=q)


def test_a_cache_keeps_its_arrays(w12):
    """The description holds addresses: another tensor in place of one of the
    arrays would be passed by."""
    c = w12.kv_cache(1, 2, 64, 4, 1, 2, 32, 16, False, DEV)
    for name in ("pages", "scales", "recent", "page_table", "length", "head_dim"):
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(c, name))


@pytest.mark.parametrize("size", [2.0 ** -80, 2.0 ** -95, 2.0 ** -119, 2.0 ** -130])
def test_tiny_blocks(w12, size):
    """A block of tiny values next to an ordinary one: its tokens keep their
    share of the softmax, whatever its scale."""
    import torch
    say("tiny", size)
    for int8 in (False, True):
        dim, page = 64, 32
        sv = Serving(w12, 1, 1, 1, dim, page, int8, seed=22)
        x = sv.rng.randn(2 * page, 3 * dim)
        x[:page, 2 * dim:] *= size
        rope = torch.tensor(np.concatenate([np.ones((256, dim // 2)), np.zeros((256, dim // 2))], 1), dtype=torch.float32, device=DEV)
        xt, vals = bf16(x)
        w12.w12_kv_append(sv.cache, 0, xt, i32([0, 2 * page]), rope, 1, slot=i32(sv.slot))
        w12.w12_kv_commit(sv.cache, i32([0, 2 * page]), i32([2 * page - 1]), slot=i32(sv.slot))
        sv.state[0][0][0].commit(vals[:, dim:2 * dim], vals[:, 2 * dim:])
        sv.check()
        # a last row with a zero query and value: every score is zero
        q = w12.w12_kv_append(sv.cache, 0, bf16(np.zeros((1, 3 * dim)))[0], i32([0, 1]), rope, 1, slot=i32(sv.slot))
        got = f64(w12.w12_kv_attention(sv.cache, 0, q, i32([0, 1]), slot=i32(sv.slot)))
        seq, n = sv.state[0][0][0], 2 * page + 1
        ref, av = seq.v.sum(0) / n, np.abs(seq.v).sum(0) / n
        # scores of zero: no rounding but the probabilities', the sums' and the output's
        lim = KV.attention_tolerance(ref, av[None], np.zeros(1), n, dim)[0]
        assert (np.abs(got[0] - ref) <= lim).all()


@pytest.mark.parametrize("dim,kv,group", [(64, 8, 6), (64, 16, 1), (128, 4, 6), (128, 8, 3), (256, 4, 5)])
@pytest.mark.parametrize("int8", [False, True])
def test_blocks_of_several_tiles(w12, dim, kv, group, int8):
    """Enough query rows that waves share a block's tiles, full, in part and
    not at all (sequences of unlike sizes in one call), over pages, tails and
    the step's own rows."""
    say("blocks", dim, kv, group, int8)
    sv = Serving(w12, 3, kv, group, dim, 64, int8, seed=23, step_rows=256)
    sv.step([200, 67, 130])
    sv.step([170, 9, 250])
    rng = np.random.RandomState(24)
    sizes = [100, 256, 41]
    sv.step(sizes, parents=[random_parents(rng, n) for n in sizes])
    sv.step([255, 1, 256])


def test_commit_keeps_no_more_than_the_page_table_holds(w12):
    """A length past the page table's pages is refused by every call, so the
    commit that would lead to one is: the last token that has a page is kept,
    the next one is not."""
    import torch
    say("full page table")
    page, blocks = 32, 2
    sv = Serving(w12, 2, 1, 2, 64, page, seed=25, blocks=blocks)
    sv.step([60, 50])
    before = [t.clone() for t in (sv.cache.pages.view(torch.uint8), sv.cache.scales, sv.cache.recent)]
    off, x = i32([0, 6, 12]), torch.ones(12, 4 * 64, device=DEV)
    w12.w12_kv_append(sv.cache, 0, x, off, sv.rope_t, 2, slot=i32(sv.slot))
    recent = sv.cache.recent.clone()
    for acc, want in (([4, 0], [-1, 51]), ([5, -1], [-1, 50])):  # 65 and 66 tokens of 64
        got = w12.w12_kv_commit(sv.cache, off, i32(acc), slot=i32(sv.slot), length_out=sv.cache.length.clone())
        assert got[sv.slot].tolist() == want, acc
        assert torch.equal(sv.cache.pages.view(torch.uint8), before[0])
        assert torch.equal(sv.cache.scales.view(torch.uint8), before[1].view(torch.uint8))
        assert torch.equal(sv.cache.recent.view(torch.int16), recent.view(torch.int16))
    sv.cache.recent.copy_(before[2])
    sv.step([4, 5])  # 64 of 64, 55 of 64
    # a full sequence is still read: its last row is the step's own
    q, _ = bf16(np.ones((1, 2, 64)))
    assert np.isfinite(attend(w12, sv, q, [0, 1], slot=i32(sv.slot[:1]))[:1]).all()


def test_two_host_threads_on_one_stream(w12):
    """Calls of unlike shapes, long enough to be split among workgroups, made
    by two threads at once on the default stream: each gets its own results,
    the same bits as alone, and leaves the rows behind its own."""
    import threading

    import torch
    say("two threads")
    sv = Serving(w12, 2, 2, 4, 64, 32, seed=26, step_rows=256, blocks=40, positions=2048)
    for _ in range(4):
        sv.step([250, 120], check=False)
    slot = i32(sv.slot)
    shapes = [(slot[:1], [0, 5]), (slot, [0, 100, 131])]
    args = []
    for sl, off in shapes:
        q, _ = bf16(sv.rng.randn(off[-1], 8, 64))
        args.append((q, off, sl))
    want = [attend(w12, sv, q, off, slot=sl) for q, off, sl in args]
    bad = []

    def go(i):
        try:
            q, off, sl = args[i]
            off_t = i32(off)
            outs = [torch.full((q.shape[0] + 2, 512), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(200)]
            for out in outs:
                w12.w12_kv_attention(sv.cache, 0, q, off_t, slot=sl, out=out)
            torch.cuda.synchronize()
            bad.extend((i, k) for k, out in enumerate(outs) if not np.array_equal(f64(out), want[i]))
        except Exception as e:  # noqa: BLE001 - told by the assertion below
            bad.append((i, repr(e)))
    threads = [threading.Thread(target=go, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(100)
    assert not bad


def filled(w12, lengths, tail_rows, kv, dim, page, int8, seed):
    """A cache with random codes and scales for these lengths (one a slot),
    random recent rows up to tail_rows behind the tail, NaN wherever nothing
    was written; and its keys and values [slot][head] as the codes stand for
    them, in 64 bits."""
    import torch
    rng, gen = np.random.RandomState(seed), torch.Generator(device=DEV).manual_seed(seed)
    blocks = max(lengths) // page + 2
    pages = len(lengths) * blocks + 1
    c = w12.kv_cache(1, kv, dim, pages, len(lengths), blocks, page, 256, int8, DEV)
    ids = rng.permutation(pages)[:len(lengths) * blocks].reshape(len(lengths), blocks)
    c.page_table.copy_(i32(ids))
    c.length.copy_(i32(lengths))
    c.scales.fill_(float("nan"))
    c.recent.fill_(float("nan"))
    kv_of = []
    for s, n in enumerate(lengths):
        full = n // page
        own = torch.tensor(ids[s, :full], device=DEV)
        x = torch.randn((full, kv, 2, page * dim), generator=gen, device=DEV)
        codes = (x * 40).round().clamp(-127, 127).to(torch.int8) if int8 else (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
        scale = torch.exp(0.4 * torch.randn((full, kv, 2), generator=gen, device=DEV)) / (40 if int8 else 100)
        c.pages.view(torch.uint8)[0, own] = codes.view(torch.uint8)
        c.scales[0, own] = scale
        tail = n % page + tail_rows
        rec = torch.randn((kv, 2, tail, dim), generator=gen, device=DEV).bfloat16()
        got, sc, rc = codes.float().cpu().numpy().astype(np.float64), f64(scale), f64(rec)
        heads = []
        for h in range(kv):
            both = []
            for v in (0, 1):
                at = torch.tensor(KV.places(v, tail, dim), device=DEV)
                c.recent[0, s, h, v].view(-1)[at] = rec[h, v]
                paged = got[:, h, v][:, KV.places(v, page, dim)] * sc[:, h, v][:, None, None]
                both.append(np.concatenate([paged.reshape(-1, dim), rc[h, v]]))
            heads.append(both)
        kv_of.append(heads)
    return c, kv_of


# (lengths of the slots, sequences, rows of each, query heads, kv heads, dim, page, int8, scale); what
# makes the run of one wave's pages longer than the 64 whose ids it holds at a time is beside each
LONG = [
    ((17100,), 512, 1, 1, 1, 64, 32, False, None),      # a tile a block: eight waves share 534 groups of tokens, 67 each or 66
    ((4322,), 256, 2, 64, 1, 64, 64, True, 0.07),       # four tiles: two waves share 134
    ((8650,), 256, 2, 32, 1, 128, 96, True, None),      # two tiles: four waves share 270, 68 each or 67
    ((8700, 9001), 256, 2, 32, 1, 128, 64, False, 0.2),  # 272 and 280, at two lengths: runs end inside a sequence
    ((8577,), 256, 2, 32, 1, 256, 128, False, 0.02),    # 268 among four, 67 each
    ((17170,), 512, 1, 4, 1, 256, 96, True, None),      # 534 among eight
    ((33000,), 128, 1, 12, 2, 128, 64, False, None),    # 1030 among eight, 129 each or 128: three turns
]


@pytest.mark.parametrize("lengths,seqs,rows,q_heads,kv,dim,page,int8,scale", LONG)
def test_runs_of_many_pages(w12, lengths, seqs, rows, q_heads, kv, dim, page, int8, scale):
    """Contexts so long, for so many sequences, that a wave walks more pages
    than it holds the ids of. The sequences share the slots in turn (which
    attention allows), so the oracle's keys and values are few. Every query
    points at one token, two thirds of them near the pages' end, which takes
    most of its weight: a page left out or read twice shows."""
    say("long runs", lengths, seqs, dim, page, int8)
    c, kv_of = filled(w12, lengths, rows, kv, dim, page, int8, seed=dim + page)
    rng = np.random.RandomState(27)
    slot = np.arange(seqs) % len(lengths)
    off = np.arange(seqs + 1) * rows
    group = q_heads // kv
    scale_of = dim ** -0.5 if scale is None else scale
    x = np.zeros((seqs * rows, q_heads, dim))
    for i in range(seqs * rows):
        n = lengths[slot[i // rows]] // page * page
        for h in range(q_heads):
            k = kv_of[slot[i // rows]][h // group][0][rng.randint(n - int(n * rng.choice([1, 0.04, 0.005])), n)]
            x[i, h] = k * (2 / scale_of / np.linalg.norm(k))  # a score of 2 |k|, others' of spread 2
    q, qv = bf16(x)
    got = f64(w12.w12_kv_attention(c, 0, q, i32(off), slot=i32(slot), scale=scale)).reshape(seqs * rows, q_heads, dim)
    assert np.isfinite(got).all()
    for s in sorted({0, 1, seqs // 2, seqs - 2, seqs - 1, *rng.randint(0, seqs, 6).tolist()}):
        n, r = lengths[slot[s]], slice(off[s], off[s + 1])
        see = np.concatenate([np.ones((rows, n), bool), KV.ancestors(KV.chain(rows))], 1)
        for h in range(kv):
            heads = slice(h * group, (h + 1) * group)
            k, v = kv_of[slot[s]][h]
            ref, av, sz = KV.attention(qv[r, heads], k, v, see, scale_of)
            err = np.abs(got[r, heads] - ref) / KV.attention_tolerance(ref, av, sz, n + rows, dim)
            assert (err <= 1).all(), (s, h, float(err.max()))


@pytest.mark.parametrize("page", [96, 128])
@pytest.mark.parametrize("int8", [False, True])
def test_large_pages_of_256_dims(w12, page, int8):
    """The largest blocks: closed several at a time as they lie (chains, a
    prompt of 512 rows), and gathered from a tree's path."""
    say("256 dims", page, int8)
    sv = Serving(w12, 2, 2, 3, 256, page, int8, seed=28, step_rows=256, layers=2)
    sv.step([page - 5, 256])
    sv.step([250, 1])
    for _ in range(4):
        rows = [40, 40]
        sv.step(rows, parents=[np.array([-1] + [max(0, i - 1 - int(sv.rng.rand() < 0.2)) for i in range(1, n)], np.int32) for n in rows])
    sv = Serving(w12, 1, 1, 2, 256, page, int8, seed=29, step_rows=512)
    sv.step([45])
    sv.step([512])
    sv.step([3])


def test_one_kv_head_for_256_query_heads(w12):
    say("256 query heads")
    sv = Serving(w12, 2, 1, 256, 64, 32, seed=30)
    sv.step([40, 3])
    sv.step([3, 1], parents=[np.array([-1, 0, 0]), np.array([-1])])


def test_offsets_past_32_bits(w12):
    """Pages and recent rows more than 2^32 bytes (and 2^31 values) into their
    arrays: the same bits as in a small cache."""
    import torch
    say("32 bits")
    dim, page, kv, heads = 256, 128, 1, 3
    rng = np.random.RandomState(31)
    big = w12.kv_cache(2, kv, dim, 40000, 30000, 4, page, 32, False, DEV)  # 5 GB of pages, 10 GB of recent rows
    small = w12.kv_cache(1, kv, dim, 8, 2, 4, page, 32, False, DEV)
    assert big.pages.numel() > 1 << 32 and big.recent.numel() > 1 << 32
    at, slots = np.array([[39999, 39990, 39001, 39000], [3, 39998, 5, 39997]]), [29999, 29998]
    big.page_table[slots] = i32(at)
    small.page_table.copy_(i32([[0, 1, 2, 3], [4, 5, 6, 7]]))
    rope = torch.tensor(rope_table(600, dim), device=DEV)
    for n in (32, 32, 32, 32, 32, 1, 32, 32, 32, 32, 7):
        off = i32([0, n, 2 * n])
        x = torch.tensor(rng.randn(2 * n, (heads + 2 * kv) * dim), dtype=torch.float32, device=DEV)
        res = []
        for c, layer, slot in ((big, 1, i32(slots)), (small, 0, None)):
            q = w12.w12_kv_append(c, layer, x, off, rope, heads, slot=slot)
            res.append(w12.w12_kv_attention(c, layer, q, off, slot=slot))
            w12.w12_kv_commit(c, off, i32([n - 1, n - 1]), slot=slot)
        assert torch.isfinite(res[0].float()).all() and torch.equal(res[0], res[1])
    assert big.length[slots].tolist() == small.length.tolist() == [296, 296]
    for s in (0, 1):
        for b in (0, 1):
            assert torch.equal(big.pages[1, at[s, b]].view(torch.uint8), small.pages[0, 4 * s + b].view(torch.uint8))
            assert torch.equal(big.scales[1, at[s, b]], small.scales[0, 4 * s + b])


def test_workspace_over_queries_or_output_is_refused(w12):
    import torch
    say("workspace overlap")
    c = w12.kv_cache(1, 2, 64, 4, 1, 2, 32, 16, False, DEV)
    off, n = i32([0, 4]), 4 * 4 * 64 * 2
    free = torch.zeros(96 << 20, dtype=torch.uint8, device=DEV)
    ws = free[1 << 20:65 << 20]
    q = torch.ones(4, 4, 64, dtype=torch.bfloat16, device=DEV)
    c.recent.zero_()
    w12.w12_kv_attention(c, 0, q, off, ws=ws)
    for at in ((1 << 20) - 256, 1 << 20, 8 << 20):
        over = free[at:at + n].view(torch.bfloat16)
        with pytest.raises(w12.W12Error, match="EINVAL"):
            w12.w12_kv_attention(c, 0, q, off, ws=ws, out=over)
        over.copy_(q.view(-1))
        with pytest.raises(w12.W12Error, match="EINVAL"):
            w12.w12_kv_attention(c, 0, over.view(4, 4, 64), off, ws=ws)
    w12.w12_kv_attention(c, 0, q, off, ws=ws, out=free[(1 << 20) - n:1 << 20].view(torch.bfloat16))


def test_commit_of_512_sequences_that_share_slots(w12):
    """The first sequence of a slot stands, refused or not, however far the
    others are behind it; slots of none are left as they are."""
    say("shared slots")
    slots, seqs = 400, 512
    c = w12.kv_cache(1, 1, 64, 8, slots, 1, 32, 16, False, DEV)
    rng = np.random.RandomState(32)
    slot = rng.randint(-3, slots + 3, seqs)
    acc = rng.choice([-1, 0, 0, 0, 1], seqs)  # of one row each: 1 is refused
    length = rng.randint(0, 20, slots)
    c.length.copy_(i32(length))
    want = np.full(slots, 77)
    for s in reversed(range(seqs)):
        if 0 <= slot[s] < slots:
            want[slot[s]] = -1 if acc[s] == 1 else length[slot[s]] + acc[s] + 1
    out = w12.w12_kv_commit(c, i32(np.arange(seqs + 1)), i32(acc), slot=i32(slot), length_out=i32(np.full(slots, 77)), rows=seqs)
    assert out.tolist() == want.tolist()
