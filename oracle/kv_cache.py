"""Plain 64-bit oracle of the KV cache (test infrastructure): the fragment
order, the position rotation, block quantisation, attention of tree rows and
the bookkeeping of appended and committed rows. Written from include/w12.h;
shares no code with the HIP path."""
import numpy as np


def key_places(rows: int, dim: int) -> np.ndarray:
    """[rows, dim] places of keys in fragment order."""
    t, d = np.meshgrid(np.arange(rows), np.arange(dim), indexing="ij")
    fragment = (t // 32) * (dim // 32) + d // 32
    return fragment * 1024 + (d % 32 // 16) * 512 + (t % 32) * 16 + d % 16


def value_places(rows: int, dim: int) -> np.ndarray:
    """[rows, dim] places of values: half h of a fragment holds the tokens 8 i + 4 h + j at 4 i + j."""
    t, d = np.meshgrid(np.arange(rows), np.arange(dim), indexing="ij")
    fragment = (t // 32) * (dim // 32) + d // 32
    i, h, j = t % 32 // 8, t % 8 // 4, t % 4
    return fragment * 1024 + h * 512 + (d % 32) * 16 + 4 * i + j


def places(v: int, rows: int, dim: int) -> np.ndarray:
    return value_places(rows, dim) if v else key_places(rows, dim)


def depths(parent) -> np.ndarray:
    out = []
    for i, p in enumerate(parent):
        out.append(0 if i == 0 else out[p] + 1)
    return np.array(out, np.int64)


def chain(n: int) -> np.ndarray:
    return np.arange(-1, n - 1, dtype=np.int32)


def ancestors(parent) -> np.ndarray:
    """[n, n] truth: row j is row i or above it."""
    n = len(parent)
    a = np.zeros((n, n), bool)
    for i in range(n):
        if i:
            a[i] = a[parent[i]]
        a[i, i] = True
    return a


def rotate(x: np.ndarray, pos: np.ndarray, rope: np.ndarray, interleaved: bool):
    """x [rows, heads, dim] turned by rope[pos] (fp32 table [positions, rot]);
    returns the values in 64 bits and the size |x cos| + |y sin| that bounds
    the rounding of each."""
    x = x.astype(np.float64)
    rot = rope.shape[1]
    cs = rope.astype(np.float64)[pos][:, None, :]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    out, size = x.copy(), np.abs(x)
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    u, v = x[..., a], x[..., b]
    out[..., a], out[..., b] = u * c - v * s, v * c + u * s
    size[..., a] = np.abs(u * c) + np.abs(v * s)
    size[..., b] = np.abs(v * c) + np.abs(u * s)
    return out, size


def e4m3_values() -> np.ndarray:
    """The 127 values of e4m3 codes 0 .. 126 (code 127 is NaN)."""
    code = np.arange(127)
    e, m = code >> 3, code & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def quantise(x: np.ndarray, int8: bool):
    """One block (any shape, bf16 values): codes as values in 64 bits, and
    the fp32 scale. A block with an infinity or NaN: scale NaN, no codes."""
    if not np.isfinite(x).all():
        return None, np.float32(np.nan)
    amax = float(np.abs(x).max())
    if amax == 0:
        return np.zeros_like(x, np.float64), np.float32(1)
    if int8:
        scale = max(np.float32(np.float32(amax) / np.float32(127)), np.float32(2.0 ** -90))
        # one fp32 division, then round half to even
        q = np.rint((x.astype(np.float32) / scale).astype(np.float64))
        return np.clip(q, -127, 127), scale
    e = -90
    while amax > 448 * 2.0 ** e:
        e += 1
    scale = 2.0 ** e
    table = e4m3_values()
    y = np.abs(x.astype(np.float64)) / scale
    hi = np.clip(np.searchsorted(table, y), 1, 126)
    lo = hi - 1
    up = (y - table[lo] > table[hi] - y) | ((y - table[lo] == table[hi] - y) & (hi % 2 == 0))
    return np.copysign(table[np.where(up, hi, lo)], x), np.float32(scale)


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, see: np.ndarray, scale: float):
    """q [rows, group, dim], k, v [tokens, dim], see [rows, tokens]: outputs
    [rows, group, dim] in 64 bits, and what a tolerance is made of:
    sum p |v| / sum p and the largest sum |q k| scale over the seen tokens."""
    q, k, v = (t.astype(np.float64) for t in (q, k, v))
    out, av, sz = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2])
    for i in range(q.shape[0]):
        kk, vv = k[see[i]], v[see[i]]
        s = q[i] @ kk.T * scale
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        out[i], av[i] = p @ vv, p @ np.abs(vv)
        sz[i] = (np.abs(q[i]) @ np.abs(kk).T * scale).max(1)
    return out, av, sz


def attention_tolerance(out, av, sz, tokens: int, dim: int):
    """|got - out| of the device's attention, from its roundings: the
    probabilities (times their value's scale) and the output are rounded to
    bf16 (2^-8 each; the sum is taken over the rounded ones); a score is
    an fp32 sum of dim exact products, so off by dim 2^-24 sum |q k|, and
    scaled in fp32 (3 roundings of |score| <= sum |q k|); an exponent off by x
    changes a probability by e^x - 1, in the sums above and below (twice); the
    device's exp2 adds 2^-21; fp32 sums over the tokens add tokens 2^-24 of
    sum p |v| above and of sum p below, and the joins of partial sums a few
    2^-22 more."""
    s = (dim + 3) * 2.0 ** -24 * sz[..., None] * 1.01 + 2.0 ** -21
    return 2.0 ** -8 * np.abs(out) * 1.01 + (2.0 ** -8 + 2 * s + 2 * tokens * 2.0 ** -24 + 2.0 ** -18) * av * 1.01


class Sequence:
    """One sequence of one (layer, kv head): committed tokens as attention sees
    them (blocks quantised when they fill), then the step's rows."""

    def __init__(self, page: int, int8: bool, dim: int):
        self.page, self.int8, self.dim = page, int8, dim
        self.k, self.v = np.zeros((0, dim)), np.zeros((0, dim))  # committed, values
        self.blocks = []                                          # (k codes, k scale, v codes, v scale)

    @property
    def length(self):
        return len(self.k)

    def commit(self, k: np.ndarray, v: np.ndarray):
        """k, v [n, dim] bf16 values of the accepted rows, in order."""
        self.k, self.v = np.concatenate([self.k, k]), np.concatenate([self.v, v])
        while len(self.k) // self.page > len(self.blocks):
            at = slice(len(self.blocks) * self.page, (len(self.blocks) + 1) * self.page)
            got = []
            for x in (self.k, self.v):
                c, s = quantise(x[at], self.int8)
                x[at] = np.nan if c is None else c * np.float64(s)
                got += [c, s]
            self.blocks.append(tuple(got))
