"""Measured cases of the verify pass's cache, attention and sampling operators.

A pass through one of four operators, each in its plain form (elementary torch
operations in 32 or 64 bits) and as a user calls it from the framework:

  append     rotates the queries and keys of a step's rows by their positions
             and stages keys and values behind the committed tokens
  attention  rows of draft trees (or prompt chunks) attend to the committed
             tokens, held in 8-bit pages, and to their own ancestors
  commit     keeps the accepted rows of every layer; full blocks become 8-bit
             pages with one scale for each block, head and K or V
  sampled    accepts drafted tokens against the target's probabilities from
             given random numbers

The cache's arrays have the layout that include/w12.h documents: keys of 32
tokens x 32 dims are 1 KB fragments [2 halves of 16 dims][32 tokens][16 dims],
values [2][32 dims][16 tokens], a half holding the tokens 4h..4h+3 of each 8.
"""
import math

import numpy as np
import torch

own = False

E4M3, INT8 = 0, 1
DEV = "cuda:0"
VOCAB = 152064


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a single token of one short conversation: latency
        dict(name="attention_one_token", op="attention", seqs=1, rows=1, length=700, kv_heads=8, group=6, dim=128, page=64, kind=E4M3, tree=False),
        # plain decoding of a ragged batch over long contexts: the cache's bytes
        dict(name="attention_batch_decode", op="attention", seqs=32, rows=1, length=16384, kv_heads=8, group=6, dim=128, page=64, kind=E4M3, tree=False),
        # the headline's 32-node tree on one long context
        dict(name="attention_tree_32", op="attention", seqs=1, rows=32, length=32000, kv_heads=4, group=6, dim=256, page=64, kind=E4M3, tree=True),
        # 24 requests sharing 192 rows, as the batched verify pass runs them, int8 pages
        dict(name="attention_24x8_int8", op="attention", seqs=24, rows=8, length=8191, kv_heads=8, group=6, dim=128, page=64, kind=INT8, tree=True),
        # a prompt chunk of the most rows that one step takes, small heads
        dict(name="attention_prompt_512", op="attention", seqs=1, rows=512, length=4100, kv_heads=16, group=6, dim=64, page=128, kind=E4M3, tree=False),
        # one decoded token's keys and values: latency
        dict(name="append_one_token", op="append", seqs=1, rows=1, length=700, kv_heads=8, group=6, dim=128, page=64, rot=128, pairs=False, f32=False, tree=False),
        # the same for 24 drafted trees of 8 rows, a quarter of the dims rotated
        dict(name="append_24x8", op="append", seqs=24, rows=8, length=8191, kv_heads=4, group=6, dim=256, page=64, rot=64, pairs=False, f32=False, tree=True),
        # a prompt chunk, fp32 from the projection, neighbouring dims rotated
        dict(name="append_prompt_512", op="append", seqs=1, rows=512, length=1000, kv_heads=8, group=6, dim=128, page=64, rot=128, pairs=True, f32=True, tree=False),
        # the accepted path of one 32-node tree, all 64 layers
        dict(name="commit_tree_32", op="commit", layers=64, seqs=1, rows=32, length=1022, kv_heads=4, dim=256, page=64, kind=E4M3, tree=True),
        # a prompt chunk over all layers: eight blocks and more become pages
        dict(name="commit_prompt_512", op="commit", layers=64, seqs=1, rows=512, length=45, kv_heads=8, dim=128, page=64, kind=E4M3, tree=False),
        # a chain of 8 drafts against the drafter's own probabilities
        dict(name="sampled_chain_8", op="sampled", trees=1, nodes=9, vocab=VOCAB, drafted=True, f32=True, tree=False),
        # 24 best-first trees of 8 rows, as the batched verify pass runs them
        dict(name="sampled_24x8", op="sampled", trees=24, nodes=8, vocab=VOCAB, drafted=False, f32=False, tree=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attention", "attention", "append", "commit", "sampled"))
    if op == "sampled":
        trees = _log(rng, 1, 32)
        vocab = _log(rng, 300, VOCAB)
        nodes = _log(rng, 1, max(1, min(64, 192 // trees)))
        return dict(op=op, trees=trees, nodes=nodes, vocab=vocab, drafted=rng.random() < 0.5, f32=rng.random() < 0.5, tree=rng.random() < 0.6)
    dim = rng.choice((64, 128, 256))
    kv_heads = rng.choice((1, 2, 3, 4, 8))
    page = rng.choice((32, 64, 96, 128))
    tree = rng.random() < 0.6
    seqs = _log(rng, 1, 32)
    rows = _log(rng, 1, max(1, (64 if tree else 512) // seqs))
    if op == "commit":
        layers = max(1, min(rng.choice((1, 4, 17, 64)), (1 << 25) // (seqs * (rows + page) * kv_heads * dim)))
        return dict(op=op, layers=layers, seqs=seqs, rows=rows, length=_log(rng, 1, 20000), kv_heads=kv_heads, dim=dim, page=page, kind=rng.choice((E4M3, INT8)), tree=tree)
    group = rng.choice((1, 2, 4, 5, 6, 8, 12))
    if op == "append":
        return dict(op=op, seqs=seqs, rows=rows, length=_log(rng, 1, 30000), kv_heads=kv_heads, group=group, dim=dim, page=page,
                    rot=rng.choice((dim, dim // 2, dim // 4)), pairs=rng.random() < 0.5, f32=rng.random() < 0.5, tree=tree)
    most = min(32000, 2 ** 27 // (seqs * kv_heads * dim), 2 ** 33 // (rows * seqs * kv_heads * group * dim))
    return dict(op=op, seqs=seqs, rows=rows, length=_log(rng, 1, max(2, most)), kv_heads=kv_heads, group=group, dim=dim, page=page,
                kind=rng.choice((E4M3, INT8)), tree=tree)


def lengths_of(case):
    """Committed tokens of each sequence: the case's for the first, ragged below it (a fresh sequence among them)."""
    r = np.random.RandomState(case["length"] * 31 + case["seqs"])
    n = r.randint(max(1, case["length"] // 8), case["length"] + 1, case["seqs"])
    n[0] = case["length"]
    if case["seqs"] > 4:
        n[3] = 0
    return n.astype(np.int32)


def rows_of(case):
    """Rows of each sequence: the case's, and fewer for some where it has many sequences of several."""
    r = np.random.RandomState(case["rows"] * 17 + case["seqs"])
    n = np.full(case["seqs"], case["rows"])
    if case["seqs"] > 2:
        n[1::3] = r.randint(1, case["rows"] + 1, len(n[1::3]))
    return n


def work(case):
    if case["op"] == "sampled":
        rows, v = case["trees"] * case["nodes"], case["vocab"]
        # every row's logits; the drafter's probabilities of the rows with children
        inner = case["trees"] * (max(1, case["nodes"] // 2) if case["tree"] else max(1, case["nodes"] - 1))
        return {"bytes": rows * v * (4 if case["f32"] else 2) + (4 * inner * v if case["drafted"] else 0), "flops": 4 * rows * v}
    lens, rows = lengths_of(case).astype(np.int64), rows_of(case).astype(np.int64)
    width = case["kv_heads"] * case["dim"]
    if case["op"] == "append":
        q = width * case["group"]
        n = int(rows.sum())
        return {"bytes": n * (q + 2 * width) * (4 if case["f32"] else 2) + n * 4 * case["rot"] + n * (q + 2 * width) * 2, "flops": 3 * n * (q + width)}
    full = lens // case["page"]
    tail = lens - full * case["page"]
    if case["op"] == "commit":
        took = _accepted(case, rows)[0] + 1
        new = (tail + took) // case["page"]
        kept = np.where(new > 0, (tail + took) % case["page"], 0) + np.where(new > 0, 0, took if case["tree"] else 0)
        per = 2 * case["layers"] * width
        return {"bytes": int(per * (3 * case["page"] * new.sum() + 4 * kept.sum()) + 24 * case["seqs"]), "flops": int(per * 3 * case["page"] * new.sum())}
    q = width * case["group"]
    seen = lens * rows + (rows * (rows + 1) // 2 if not case["tree"] else rows * 4)
    return {"bytes": int(2 * width * (full * case["page"]).sum() + 4 * width * (tail + rows).sum() + 4 * q * rows.sum()), "flops": int(4 * q * seen.sum())}


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _trees(r, sizes, most_depth=16, chain=False):
    """Parents of trees of these sizes: any earlier node of less depth, or the row before (a chain)."""
    out = []
    for n in sizes:
        depth = [0] * n
        parent = [-1] * n
        for i in range(1, n):
            parent[i] = i - 1 if chain else int(r.choice([j for j in range(i) if depth[j] < most_depth]))
            depth[i] = depth[parent[i]] + 1
        out.append(np.array(parent, np.int32))
    return out


def _accepted(case, rows, seed=0):
    """Accepted drafts and their paths, as tree acceptance gives them: prompts keep every row, trees a root path."""
    if not case["tree"]:
        return rows - 1, [np.arange(n, dtype=np.int32) for n in rows]
    r = np.random.RandomState(97 + case["rows"])
    got = []
    for parent in _trees(r, rows):
        node, path = int(r.randint(len(parent))), []
        while node >= 0:
            path.append(node)
            node = int(parent[node])
        got.append(np.concatenate([path[::-1], np.full(len(parent) - len(path), -1)]).astype(np.int32))
    return np.array([int((p >= 0).sum()) - 1 for p in got]), got


def _dev(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), dtype=dtype, device=DEV)


def _cache(case, seed, layers, only_new=False):
    """A cache as it stands in the middle of serving: pages in no order, values of unit spread with a scale of their own for each head."""
    g, r = _gen(seed), np.random.RandomState(seed % (1 << 31))
    lens, rows = lengths_of(case), rows_of(case)
    seqs, page, heads, dim = case["seqs"], case["page"], case["kv_heads"], case["dim"]
    slots = seqs + 2
    slot = r.permutation(slots)[:seqs].astype(np.int32)
    have = lens // page + (case["rows"] + page - 1) // page + 1
    table = np.zeros((slots, int(have.max())), np.int32)
    first = lens // page if only_new else np.zeros_like(lens)  # the commit touches no older page: those share page 0
    pages = int((have - first).sum()) + 1
    order, at = r.permutation(pages - 1) + 1, 0
    for s in range(seqs):
        n = int(have[s] - first[s])
        table[slot[s], first[s]:have[s]] = order[at:at + n]
        at += n
    recent_rows = -(-(page - 1 + case["rows"]) // 32) * 32
    length = np.zeros(slots, np.int32)
    length[slot] = lens
    codes = torch.empty((layers, pages, heads, 2, page * dim), dtype=torch.float8_e4m3fn if case.get("kind", E4M3) == E4M3 else torch.int8, device=DEV)
    scales = torch.empty((layers, pages, heads, 2), dtype=torch.float32, device=DEV)
    for lay in range(layers):
        for p0 in range(0, pages, 2048):
            x = torch.randn((min(2048, pages - p0), heads, 2, page * dim), generator=g, device=DEV)
            x *= torch.exp(0.5 * torch.randn((1, heads, 2, 1), generator=g, device=DEV))
            c, s = _quantise(x.bfloat16().float(), case.get("kind", E4M3))
            codes[lay, p0:p0 + 2048], scales[lay, p0:p0 + 2048] = c, s
    recent = torch.randn((layers, slots, heads, 2, recent_rows * dim), generator=g, device=DEV, dtype=torch.float32).bfloat16()
    off = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    return dict(case=case, codes=codes, scales=scales, recent=recent, table=_dev(table), length=_dev(length), slot=_dev(slot), row_off=_dev(off),
                total=int(off[-1]), recent_rows=recent_rows, slots=slots, pages=pages, most_pages=int(have.max()), rows=rows)


def prepare(case, seed):
    op = case["op"]
    g, r = _gen(seed * 7 + 3), np.random.RandomState((seed * 13 + 5) % (1 << 31))
    if op == "sampled":
        return _prepare_sampled(case, g, r)
    if op == "commit":
        s = _cache(case, seed, case["layers"], only_new=True)
        took, path = _accepted(case, s["rows"], seed)
        s["accept_len"], s["path"] = _dev(took), _dev(np.concatenate(path)) if case["tree"] else None
        s["length_out"] = s["length"].clone()
        return s
    s = _cache(case, seed, 1, only_new=op == "append")
    s["parent"] = _dev(np.concatenate(_trees(r, s["rows"]))) if case["tree"] else None
    heads, dim = case["kv_heads"] * case["group"], case["dim"]
    if op == "attention":
        s["q"] = (1.5 * torch.randn((s["total"], heads, dim), generator=g, device=DEV)).bfloat16()
        s["out"] = torch.zeros((s["total"] + 1, heads * dim), dtype=torch.bfloat16, device=DEV)
        return s
    x = torch.randn((s["total"], (heads + 2 * case["kv_heads"]) * dim), generator=g, device=DEV)
    s["qkv"] = x if case["f32"] else x.bfloat16()
    s["q"] = torch.zeros((s["total"], heads, dim), dtype=torch.bfloat16, device=DEV)
    s["rope"] = _rope_table(case["length"] + case["rows"], case["rot"])
    return s


def _rope_table(positions, rot):
    """[positions, rot]: cosines, then sines, of position x 10000^(-2i/rot); angles of far positions in 64 bits."""
    f = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=DEV), -torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _prepare_sampled(case, g, r):
    trees, nodes, v = case["trees"], case["nodes"], case["vocab"]
    total = trees * nodes
    parent = np.concatenate(_trees(r, [nodes] * trees, chain=not case["tree"]))
    off = np.arange(trees + 1, dtype=np.int32) * nodes
    # peaked rows, as a language model's: a flat part and a few likely tokens
    logits = torch.randn((total, v), generator=g, device=DEV) * 2
    logits.scatter_add_(1, torch.randint(0, v, (total, 12), generator=g, device=DEV), 4 + 4 * torch.rand((total, 12), generator=g, device=DEV))
    logits = logits if case["f32"] else logits.bfloat16()
    temp = 0.6 + 0.6 * torch.rand(trees, generator=g, device=DEV)
    guess = logits.float() + torch.randn((total, v), generator=g, device=DEV)
    base = torch.arange(total, device=DEV) // nodes * nodes
    up = base + torch.tensor(parent, device=DEV).clamp(min=0)
    if case["drafted"]:
        draft = torch.softmax(guess, 1)
        token = torch.multinomial(draft[up], 1, generator=g)[:, 0]
    else:  # each node's children take its likely tokens in turn
        draft = None
        best = torch.topk(guess, min(16, v), 1).indices
        rank, seen = np.zeros(total, np.int64), {}
        for i in range(total):
            key = (i // nodes, int(parent[i]))
            rank[i] = seen.get(key, 0) % min(16, v)
            seen[key] = rank[i] + 1
        token = best[up, torch.tensor(rank, device=DEV)]
    return dict(case=case, row_off=_dev(off), parent=_dev(parent), token=token.int(), logits=logits, temp=temp, draft=draft,
                u=torch.rand(total, generator=g, device=DEV), u_bonus=torch.rand(trees, generator=g, device=DEV))


# ---------------------------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        import w12_weight_streaming_amd as w12

        if op == "sampled":
            return w12.tree_accept_sampled(s["row_off"], s["parent"], s["token"], s["logits"], s["u"], s["u_bonus"], temperature=s["temp"], draft=s["draft"])
        cache = w12.KvCache(pages=s["codes"], scales=s["scales"], recent=s["recent"], page_table=s["table"], length=s["length"], head_dim=s["case"]["dim"])
        if op == "append":
            w12.w12_kv_append(cache, 0, s["qkv"], s["row_off"], s["rope"], s["case"]["kv_heads"] * s["case"]["group"], slot=s["slot"], parent=s["parent"],
                              interleaved=s["case"]["pairs"], out=s["q"])
            return s["q"], s["recent"]
        if op == "attention":
            return w12.w12_kv_attention(cache, 0, s["q"], s["row_off"], slot=s["slot"], parent=s["parent"], out=s["out"])
        w12.w12_kv_commit(cache, s["row_off"], s["accept_len"], path=s["path"], slot=s["slot"], length_out=s["length_out"])
        return s["codes"], s["scales"], s["recent"], s["length_out"]
    return {"append": _append, "attention": _attention, "commit": _commit, "sampled": _sampled}[op](s)


def _rows_index(s):
    """Each sequence's rows, padded to the longest: their places, and which there are."""
    off = s["row_off"].long()
    i = torch.arange(s["case"]["rows"], device=DEV)
    at = off[:-1, None] + i
    ok = at < off[1:, None]
    return torch.where(ok, at, 0), ok


def _ancestors(s, at, ok):
    """[seqs, rows, rows]: whether row j is row i or one of its ancestors."""
    n = at.shape[1]
    i = torch.arange(n, device=DEV)
    if s["parent"] is None:
        return (i[:, None] >= i[None, :])[None] & ok[:, None, :]
    up = torch.where(ok, s["parent"].long()[at], -1)
    a = torch.eye(n, device=DEV)[None] + (up[:, :, None] == i).float()
    for _ in range(max(1, (n - 1).bit_length())):
        a = (a @ a).clamp(max=1)
    return a > 0


def _order(x, *last):
    """`x` with its last dims in this order."""
    lead = x.dim() - len(last)
    return x.permute(*range(lead), *(lead + i for i in last))


def _of_keys(x, dim):
    """Fragments [..., n * dim] as keys [..., n, dim]."""
    return _order(x.unflatten(-1, (-1, dim // 32, 2, 32, 16)), 0, 3, 1, 2, 4).flatten(-3).flatten(-3, -2)


def _of_values(x, dim):
    """Fragments [..., n * dim] as values [..., n, dim]."""
    x = x.unflatten(-1, (-1, dim // 32, 2, 32, 2, 2, 4))  # group, dims, half, dim, 16s, 8s, token
    return _order(x, 0, 4, 5, 2, 6, 1, 3).flatten(-2).flatten(-6, -2)


def _to_keys(x):
    """Keys [..., n, dim] as fragments."""
    return _order(x.unflatten(-1, (-1, 2, 16)).unflatten(-4, (-1, 32)), 0, 2, 3, 1, 4).flatten(-5)


def _to_values(x):
    """Values [..., n, dim] as fragments."""
    x = x.unflatten(-1, (-1, 32)).unflatten(-3, (-1, 2, 2, 2, 4))  # group, 16s, 8s, half, token, dims, dim
    return _order(x, 0, 5, 3, 6, 1, 2, 4).flatten(-7)


def _quantise(x, kind):
    """Blocks [..., n] as 8-bit codes and scales [...]: a power of two that brings the largest to 448 or below, or the largest / 127."""
    most = x.abs().amax(-1)
    if kind == INT8:
        scale = torch.where(most > 0, most / 127, 1.0)
        return torch.round(x / scale[..., None]).clamp(-127, 127).to(torch.int8), scale
    f, e = torch.frexp(most)
    scale = torch.ldexp(torch.ones_like(most), torch.where(most > 0, e - 9 + (f > 0.875).int(), 0).clamp(min=-126))
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def _append(s):
    case = s["case"]
    heads, kv, dim, rot = case["kv_heads"] * case["group"], case["kv_heads"], case["dim"], case["rot"]
    at, ok = _rows_index(s)
    held = s["length"].long()[s["slot"].long()]
    if s["parent"] is None:
        depth = torch.arange(at.shape[1], device=DEV).expand_as(at)
    else:
        depth = _ancestors(s, at, ok).sum(2) - 1
    pos = torch.zeros(s["total"], dtype=torch.long, device=DEV)
    pos[at[ok]] = (held[:, None] + depth)[ok]
    cos, sin = s["rope"][pos][:, None].chunk(2, -1)
    x = s["qkv"].float().unflatten(1, (heads + 2 * kv, dim))
    part = x[:, :heads + kv, :rot]
    a, b = (part[..., 0::2], part[..., 1::2]) if case["pairs"] else part.chunk(2, -1)
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([c, d], -1).flatten(-2) if case["pairs"] else torch.cat([c, d], -1)
    x = torch.cat([torch.cat([turned, x[:, :heads + kv, rot:]], 2), x[:, heads + kv:]], 1).bfloat16()
    s["q"].copy_(x[:, :heads])
    rec = s["recent"][0]
    slot = s["slot"].long()[:, None].expand_as(at)[ok]
    to = ((held % case["page"])[:, None] + torch.arange(at.shape[1], device=DEV))[ok]
    keys, values = _of_keys(rec[:, :, 0], dim), _of_values(rec[:, :, 1], dim)
    keys[slot, :, to] = x[at[ok], heads:heads + kv]
    values[slot, :, to] = x[at[ok], heads + kv:]
    rec[:, :, 0], rec[:, :, 1] = _to_keys(keys), _to_values(values)
    return s["q"], s["recent"]


def _attention(s):
    case = s["case"]
    kv, group, dim, page = case["kv_heads"], case["group"], case["dim"], case["page"]
    at, ok = _rows_index(s)
    slot = s["slot"].long()
    held = s["length"].long()[slot]
    full = held // page
    blocks = s["table"].long()[slot][:, :case["length"] // page]
    x = (s["codes"][0][blocks].float() * s["scales"][0][blocks][..., None]).movedim(1, 2)  # seqs, heads, blocks, K or V, values
    rec = s["recent"][0][slot].float()
    k = torch.cat([_of_keys(x[:, :, :, 0], dim).flatten(2, 3), _of_keys(rec[:, :, 0], dim)], 2)
    v = torch.cat([_of_values(x[:, :, :, 1], dim).flatten(2, 3), _of_values(rec[:, :, 1], dim)], 2)
    del x
    n, i = blocks.shape[1] * page, torch.arange(s["recent_rows"], device=DEV)
    old = torch.arange(n, device=DEV)[None] < (full * page)[:, None]
    local = i[None] - (held - full * page)[:, None]  # the row that a recent place holds; below 0: a committed token
    anc = _ancestors(s, at, ok)
    mine = torch.gather(anc, 2, local.clamp(0, at.shape[1] - 1)[:, None].expand(-1, at.shape[1], -1)) & (local < at.shape[1])[:, None]
    see = torch.cat([old[:, None].expand(-1, at.shape[1], -1), (local < 0)[:, None] | mine], 2)
    q = s["q"].float()[at].unflatten(2, (kv, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # seqs, kv, rows x group, dim
    sc = (q @ k.transpose(2, 3).contiguous()) * dim ** -0.5
    sc = sc.masked_fill_(~see.repeat_interleave(group, 1)[:, None], -math.inf)
    p = torch.exp(sc.sub_(sc.amax(3, keepdim=True)))
    o = (p @ v) / p.sum(3, keepdim=True)
    o = o.unflatten(2, (-1, group)).permute(0, 2, 1, 3, 4).flatten(2)
    s["out"][at[ok]] = o[ok].bfloat16()
    return s["out"]


def _commit(s):
    case = s["case"]
    dim, page = case["dim"], case["page"]
    slot = s["slot"].long()
    held = s["length"].long()[slot]
    full, tail = held // page, held % page
    at, ok = _rows_index(s)
    took = s["accept_len"].long() + 1
    step = s["path"].long()[at] if s["path"] is not None else torch.arange(at.shape[1], device=DEV).expand_as(at)
    # the place that each of the logical rows (committed tail, then accepted rows) comes from
    i = torch.arange(s["recent_rows"], device=DEV)[None]
    j = i - tail[:, None]
    src = torch.where(j < 0, i, tail[:, None] + torch.gather(step, 1, j.clamp(0, at.shape[1] - 1)).clamp(min=0))
    src = torch.where(j < took[:, None], src, i)
    n = tail + took
    rec = s["recent"][:, slot]
    keys, values = _of_keys(rec[..., 0, :], dim), _of_values(rec[..., 1, :], dim)  # layers, seqs, heads, rows, dim
    ix = src[None, :, None, :, None].expand(keys.shape[0], -1, keys.shape[2], -1, dim)
    new_k, new_v = torch.gather(keys, 3, ix), torch.gather(values, 3, ix)
    most = s["recent_rows"] // page
    whole = torch.arange(most, device=DEV)[None] < (n // page)[:, None]
    seq, blk = whole.nonzero(as_tuple=True)
    ids = s["table"].long()[slot[seq], full[seq] + blk]
    for part, x, pack in ((0, new_k, _to_keys), (1, new_v, _to_values)):
        blocks = x[:, :, :, :most * page].unflatten(3, (most, page)).movedim(3, 2)[:, seq, blk]  # layers, blocks, heads, page, dim
        c, sc = _quantise(pack(blocks).float(), case["kind"])
        s["codes"][:, ids, :, part], s["scales"][:, ids, :, part] = c, sc
    # what is left moves to the front; rows behind it stay
    shift = torch.where(i < (n % page)[:, None], i + (n // page * page)[:, None], 0).clamp(max=s["recent_rows"] - 1)
    ix = shift[None, :, None, :, None].expand_as(ix)
    keep = (i >= (n % page)[:, None])[None, :, None, :, None]
    s["recent"][:, slot, :, 0] = _to_keys(torch.where(keep, keys, torch.gather(new_k, 3, ix)))
    s["recent"][:, slot, :, 1] = _to_values(torch.where(keep, values, torch.gather(new_v, 3, ix)))
    s["length_out"][slot] = (held + took).int()
    return s["codes"], s["scales"], s["recent"], s["length_out"]


def _sampled(s):
    trees, nodes, v = s["case"]["trees"], s["case"]["nodes"], s["case"]["vocab"]
    x = s["logits"].double() / s["temp"].double().repeat_interleave(nodes)[:, None]
    p = torch.exp(x - x.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    i = torch.arange(trees * nodes, device=DEV)
    base = i // nodes * nodes
    up = torch.where(s["parent"] < 0, -1, base + s["parent"].long())
    token = s["token"].long()
    same = up[:, None] == up[None, :]  # siblings
    rank = (same & (i[None, :] < i[:, None])).sum(1)
    above = up.clamp(min=0)
    px = p[above, token]
    u = s["u"].double()
    if s["draft"] is None:  # a drafted token is rejected for good: its probability leaves the row
        first = same & (token[:, None] == token[None, :]) & (i[None, :] < i[:, None])
        again = first.any(1)
        gone = ((same & (i[None, :] < i[:, None]) & ~again[None, :]).double() * px[None, :]).sum(1)
        passes = (u * (1 - gone) < px) & ~again
    else:  # residual after r rejections: max(p - c q, 0) / n, with c' = c + n
        q = s["draft"].double()
        qx = q[above, token]
        c, n = torch.zeros(trees * nodes, dtype=torch.float64, device=DEV), torch.ones(trees * nodes, dtype=torch.float64, device=DEV)
        passes = torch.zeros(trees * nodes, dtype=torch.bool, device=DEV)
        kids = (up[:, None] == i[None, :]).sum(0)
        cs = []
        for r in range(int(nodes)):
            passes |= (rank == r) & (u * qx * n[above] < px - c[above] * qx)
            cs.append(torch.where(kids >= r, c, cs[-1] if cs else c))
            if not bool((kids > r).any()):
                break
            c = torch.where(kids > r, c + n, c)
            n = torch.where(kids > r, (p - c[:, None] * q).clamp(min=0).sum(1), n)
        c_last = c
    passes &= up >= 0
    # a node's chosen child is the first that passes; the path follows the choices from the root
    choice = torch.full((trees * nodes,), trees * nodes, device=DEV).scatter_reduce(0, above[passes], i[passes], "amin")
    node = torch.arange(trees, device=DEV) * nodes
    path = torch.full((trees, nodes), -1, dtype=torch.int32, device=DEV)
    length = torch.full((trees,), -1, dtype=torch.int32, device=DEV)
    alive, last = torch.ones(trees, dtype=torch.bool, device=DEV), node
    for d in range(nodes):
        path[:, d] = torch.where(alive, node % nodes, -1).int()
        length += alive.int()
        last = torch.where(alive, node, last)
        step = choice[last]
        alive = alive & (step < trees * nodes)
        node = torch.where(alive, step, node)
    # the next token, from what is left at the path's end
    w = p[last]
    if s["draft"] is None:
        out = up[None, :] == last[:, None]
        t, k = out.nonzero(as_tuple=True)
        w[t, token[k]] = 0
    else:
        r = (w - c_last[last][:, None] * s["draft"].double()[last]).clamp(min=0)
        w = torch.where(r.sum(1, keepdim=True) > 0, r, w)
    cum = w.cumsum(1)
    below = cum <= s["u_bonus"].double()[:, None] * cum[:, -1:]
    bonus = torch.minimum(below.sum(1), (w > 0).double().mul(torch.arange(1, v + 1, device=DEV)).amax(1).long() - 1).int()
    return length, path.flatten(), bonus


# ---------------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "commit": _exact_commit, "sampled": _exact_sampled}[case["op"]](s)


def _host_rows(s):
    off = s["row_off"].tolist()
    slot, held = s["slot"].tolist(), s["length"].tolist()
    parent = s["parent"].tolist() if s.get("parent") is not None else None
    for n, (a, b) in enumerate(zip(off[:-1], off[1:])):
        yield n, slot[n], held[slot[n]], a, b, (parent[a:b] if parent else list(range(-1, b - a - 1)))


def _key_place(t, d, dim):
    """Where a fragment array holds dim d of row t's key."""
    return ((t // 32 * (dim // 32) + d // 32) * 64 + d % 32 // 16 * 32 + t % 32) * 16 + d % 16


def _value_place(t, d, dim):
    """Where a fragment array holds dim d of row t's value."""
    return ((t // 32 * (dim // 32) + d // 32) * 64 + t % 8 // 4 * 32 + d % 32) * 16 + t % 32 // 16 * 8 + t % 16 // 8 * 4 + t % 4


def _places(rows, dim):
    t, d = torch.arange(rows, device=DEV)[:, None], torch.arange(dim, device=DEV)[None, :]
    return _key_place(t, d, dim), _value_place(t, d, dim)


def _exact_append(s):
    case = s["case"]
    heads, kv, dim, rot = case["kv_heads"] * case["group"], case["kv_heads"], case["dim"], case["rot"]
    q, rec = s["q"].double(), s["recent"].double()
    pk, pv = _places(s["recent_rows"], dim)
    half = torch.arange(rot // 2, device=DEV)
    lo, hi = (2 * half, 2 * half + 1) if case["pairs"] else (half, half + rot // 2)
    freq = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=DEV), -2.0 * half.double() / rot)
    for n, slot, held, a, b, parent in _host_rows(s):
        depth = []
        for i in range(b - a):
            depth.append(0 if parent[i] < 0 else depth[parent[i]] + 1)
        turn = (held + torch.tensor(depth, dtype=torch.float64, device=DEV))[:, None] * freq
        z = torch.polar(torch.ones_like(turn), turn)[:, None]
        x = s["qkv"][a:b].double().view(b - a, heads + 2 * kv, dim).clone()
        y = torch.complex(x[:, :heads + kv][..., lo], x[:, :heads + kv][..., hi]) * z
        x[:, :heads + kv, lo], x[:, :heads + kv, hi] = y.real, y.imag
        q[a:b] = x[:, :heads]
        at = held % case["page"] + torch.arange(b - a, device=DEV)
        rec[0, slot, :, 0].scatter_(1, pk[at].flatten().expand(kv, -1), x[:, heads:heads + kv].transpose(0, 1).reshape(kv, -1))
        rec[0, slot, :, 1].scatter_(1, pv[at].flatten().expand(kv, -1), x[:, heads + kv:].transpose(0, 1).reshape(kv, -1))
    return q, rec


def _exact_attention(s):
    case = s["case"]
    kv, group, dim, page = case["kv_heads"], case["group"], case["dim"], case["page"]
    out = s["out"].double()
    pk, pv = _places(page, dim)
    rk, rv = _places(s["recent_rows"], dim)
    for n, slot, held, a, b, parent in _host_rows(s):
        full, tail = held // page, held % page
        see = torch.zeros((b - a, tail + b - a), dtype=torch.bool)
        see[:, :tail] = True
        for i in range(b - a):
            if parent[i] >= 0:
                see[i] |= see[parent[i]]
            see[i, tail + i] = True
        see = torch.cat([torch.ones((b - a, full * page), dtype=torch.bool), see], 1).to(DEV).repeat_interleave(group, 0)
        ids = s["table"][slot, :full].long()
        for h in range(kv):
            x = s["codes"][0, ids, h].double() * s["scales"][0, ids, h].double()[..., None]
            k = torch.cat([x[:, 0][:, pk.flatten()].view(-1, dim), s["recent"][0, slot, h, 0].double()[rk[:tail + b - a]]])
            v = torch.cat([x[:, 1][:, pv.flatten()].view(-1, dim), s["recent"][0, slot, h, 1].double()[rv[:tail + b - a]]])
            q = s["q"][a:b, h * group:(h + 1) * group].double().reshape(-1, dim)
            w = torch.where(see, q @ k.t().contiguous() / math.sqrt(dim), -math.inf)
            o = torch.softmax(w, 1) @ v
            out[a:b, h * group * dim:(h + 1) * group * dim] = o.view(b - a, group * dim)
    return out


def _exact_commit(s):
    case = s["case"]
    dim, page = case["dim"], case["page"]
    codes, scales, rec = s["codes"].double(), s["scales"].double(), s["recent"].double()
    length = s["length_out"].clone()
    places = _places(s["recent_rows"], dim)
    into = _places(page, dim)
    took, path = s["accept_len"].tolist(), s["path"].tolist() if s["path"] is not None else None
    for n, slot, held, a, b, _ in _host_rows(s):
        full, tail = held // page, held % page
        rows = list(range(tail)) + [tail + (path[a + j] if path else j) for j in range(took[n] + 1)]
        length[slot] = held + took[n] + 1
        for part in (0, 1):
            x = s["recent"][:, slot, :, part].double()[..., places[part][torch.tensor(rows, device=DEV)]]  # layers, heads, rows, dim
            new = len(rows) // page
            for blk in range(new):
                y = x[:, :, blk * page:(blk + 1) * page]
                most = y.abs().amax((2, 3))
                if case["kind"] == INT8:
                    sc = (most / 127).float().double()
                    c = torch.round(y / sc[..., None, None])
                else:
                    sc = torch.exp2(torch.ceil(torch.log2(most / 448)))
                    z = y / sc[..., None, None]
                    unit = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
                    c = torch.round(z / unit) * unit
                page_id = int(s["table"][slot, full + blk])
                flat = torch.zeros((*c.shape[:2], page * dim), dtype=torch.float64, device=DEV)
                flat[..., into[part].flatten()] = c.flatten(2)
                codes[:, page_id, :, part], scales[:, page_id, :, part] = flat, sc
            left = x[:, :, new * page:]
            rec[:, slot, :, part].scatter_(2, places[part][:left.shape[2]].flatten().expand(*left.shape[:2], -1), left.flatten(2))
    return codes, scales, rec, length


def _exact_sampled(s):
    """The walk itself, row by row, with residuals as they are defined."""
    trees, nodes = s["case"]["trees"], s["case"]["nodes"]
    logits, token = s["logits"].double().cpu().numpy(), s["token"].cpu().numpy()
    parent, temp = s["parent"].cpu().numpy(), s["temp"].double().cpu().numpy()
    draft = None if s["draft"] is None else s["draft"].double().cpu().numpy()
    u, ub = s["u"].double().cpu().numpy(), s["u_bonus"].double().cpu().numpy()
    lens, paths, bonus = [], np.full((trees, nodes), -1, np.int32), []
    for t in range(trees):
        base, node, d = t * nodes, 0, 0
        while True:
            paths[t, d] = node
            row = base + node
            x = logits[row] / temp[t]
            p = np.exp(x - x.max())
            p /= p.sum()
            nxt = None
            for c in [i for i in range(1, nodes) if parent[base + i] == node]:
                tok = token[base + c]
                q = draft[row][tok] if draft is not None else 1.0
                if u[base + c] * q < p[tok]:
                    nxt = c
                    break
                if draft is None:
                    res = p.copy()
                    res[tok] = 0
                else:
                    res = np.maximum(p - draft[row], 0)
                if res.sum() > 0:
                    p = res / res.sum()
            if nxt is None:
                break
            node, d = nxt, d + 1
        cum = np.cumsum(p)
        over = np.flatnonzero(cum > ub[t] * cum[-1])
        lens.append(d)
        bonus.append(int(over[0]) if len(over) else int(np.flatnonzero(p > 0)[-1]))
    return np.array(lens, np.int32), paths.reshape(-1), np.array(bonus, np.int32)
