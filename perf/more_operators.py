"""Measured cases of the recurrent layers' operators and of the norms between products.

A pass through one of four operators, each in its plain form (elementary torch
operations in 32 bits, decays summed in 64) and as a user calls it:

  append  the short causal convolution of a recurrent layer along each row's
          root path, SiLU, normalised query and key heads, decay and strength
          of every value head; stages the step's rows
  rule    the gated delta rule over the rows of draft trees, prompt chunks or
          single tokens, from each sequence's state; prompts and plain
          decoding keep the state behind their last row
  commit  the accepted rows of every layer join the states and the
          convolution's windows
  norm    what stands between two products: norm of a block's output, gate,
          residual with its scale, norm before the next block

The arrays have the layout that include/w12.h documents: states are
[layers, slots, value heads, key dim, value dim] fp32, staged rows are indexed
by the step's row.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
EPS = 1e-6


# ---------------------------------------------------------------------------------------------- cases

def listed():
    big = dict(key_heads=16, value_heads=48, key_dim=128, value_dim=128)
    return [
        # one decoded token of one conversation: latency
        dict(name="rule_one_token", op="rule", seqs=1, rows=1, tree=False, keep=True, **big),
        # plain decoding of a batch: every state read and written once
        dict(name="rule_batch_decode", op="rule", seqs=32, rows=1, tree=False, keep=True, **big),
        # the headline's 32-node tree
        dict(name="rule_tree_32", op="rule", seqs=1, rows=32, tree=True, keep=False, **big),
        # 24 requests sharing 192 rows, as the batched verify pass runs them
        dict(name="rule_24x8", op="rule", seqs=24, rows=8, tree=True, keep=False, **big),
        # a prompt chunk of the most rows that one step takes
        dict(name="rule_prompt_512", op="rule", seqs=1, rows=512, tree=False, keep=True, **big),
        # the inputs of one 32-node tree
        dict(name="append_tree_32", op="append", seqs=1, rows=32, tree=True, width=4, f32=False, **big),
        # a prompt chunk, fp32 from the projection
        dict(name="append_prompt_512", op="append", seqs=1, rows=512, tree=False, width=4, f32=True, **big),
        # the accepted path of one 32-node tree, all 48 recurrent layers
        dict(name="commit_tree_32", op="commit", layers=48, seqs=1, rows=32, tree=True, width=4, **big),
        # 24 requests of 8 rows over a dozen layers
        dict(name="commit_24x8", op="commit", layers=12, seqs=24, rows=8, tree=True, width=4, **big),
        # residual and norm between two products of the headline's 32 rows
        dict(name="norm_block_32", op="norm", rows=32, groups=1, width=5120, y_f32=False, h="bf16", post=False, gate=False, weight=True),
        # the same around a block whose output is normed too, for the most rows of a step, fp32 residual
        dict(name="norm_around_512", op="norm", rows=512, groups=1, width=5120, y_f32=True, h="f32", post=True, gate=False, weight=True),
        # the norm of every value head and its gate, behind the delta rule of 192 rows
        dict(name="norm_heads_192", op="norm", rows=192, groups=48, width=128, y_f32=False, h="", post=True, gate=True, weight=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rule", "rule", "append", "commit", "norm"))
    if op == "norm":
        if rng.random() < 0.4:  # heads
            groups, width = rng.choice((1, 3, 8, 16, 48)), rng.choice((64, 96, 128, 256))
        else:
            groups, width = 1, _log(rng, 500, 5200)
        kind = rng.choice(("residual", "around", "gate", "first"))
        return dict(op=op, rows=_log(rng, 1, 512 if groups < 48 else 384), groups=groups, width=width, y_f32=rng.random() < 0.5,
                    h="" if kind == "gate" else rng.choice(("bf16", "f32")), post=kind == "around" or (kind == "gate" and rng.random() < 0.7),
                    gate=kind == "gate" or (kind == "around" and rng.random() < 0.5), weight=kind != "gate")
    key_heads = rng.choice((1, 2, 4, 8, 16))
    heads = dict(key_heads=key_heads, value_heads=key_heads * rng.choice((1, 2, 3)), key_dim=rng.choice((64, 128)), value_dim=rng.choice((64, 128)))
    tree = rng.random() < 0.6
    seqs = _log(rng, 1, 32)
    rows = _log(rng, 1, max(1, (64 if tree else 512) // seqs))
    if op == "append":
        return dict(op=op, seqs=seqs, rows=rows, tree=tree, width=rng.choice((2, 3, 4)), f32=rng.random() < 0.5, **heads)
    if op == "rule":
        return dict(op=op, seqs=seqs, rows=rows, tree=tree, keep=not tree and rng.random() < 0.7, **heads)
    most = (1 << 27) // (seqs * heads["value_heads"] * heads["key_dim"] * heads["value_dim"])
    return dict(op=op, layers=max(1, min(rng.choice((1, 5, 12, 48)), most)), seqs=seqs, rows=rows, tree=tree, width=rng.choice((2, 3, 4)), **heads)


def channels_of(case):
    return 2 * case["key_heads"] * case["key_dim"] + case["value_heads"] * case["value_dim"]


def rows_of(case):
    """Rows of each sequence: the case's, and fewer for some where it has many sequences of several."""
    r = np.random.RandomState(case["rows"] * 17 + case["seqs"])
    n = np.full(case["seqs"], case["rows"])
    if case["seqs"] > 2:
        n[1::3] = r.randint(1, case["rows"] + 1, len(n[1::3]))
    return n


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["groups"] * case["width"]
        y = 4 if case["y_f32"] else 2
        h = {"": 0, "bf16": 4, "f32": 8}[case["h"]]
        return {"bytes": n * (y + h + 2 + (2 if case["gate"] else 0)), "flops": 8 * n}
    rows = rows_of(case).astype(np.int64)
    n, c = int(rows.sum()), channels_of(case)
    kd, vd, hv = case["key_dim"], case["value_dim"], case["value_heads"]
    if case["op"] == "append":
        return {"bytes": n * (c + 2 * hv) * (4 if case["f32"] else 2) + n * (4 * c + 8 * hv) + case["seqs"] * (case["width"] - 1) * c * 2 + 4 * case["width"] * c,
                "flops": n * c * (2 * case["width"] + 8)}
    state = 4 * hv * kd * vd
    if case["op"] == "rule":
        pairs = int((rows * (rows + 1) // 2).sum()) if not case["tree"] else 4 * n
        return {"bytes": case["seqs"] * state * (2 if case["keep"] else 1) + n * (2 * c + 8 * hv + 2 * hv * vd) + (0 if case["keep"] else 4 * n * hv * vd),
                "flops": n * hv * kd * vd * (6 if case["keep"] else 4) + pairs * hv * 4 * (kd + vd)}
    took = int((_accepted(case, rows)[0] + 1).sum())
    window = 2 * (case["width"] - 1) * c
    per_row = 2 * case["key_heads"] * kd + 4 * hv * vd + 4 * hv
    return {"bytes": case["layers"] * (case["seqs"] * (2 * state + 2 * window) + took * per_row), "flops": case["layers"] * 2 * hv * kd * vd * took}


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) % (1 << 62))
    return g


def _trees(r, sizes, most_depth=16):
    """Parents of trees of these sizes: any earlier node of less depth."""
    out = []
    for n in sizes:
        depth, parent = [0] * n, [-1] * n
        for i in range(1, n):
            parent[i] = int(r.choice([j for j in range(i) if depth[j] < most_depth]))
            depth[i] = depth[parent[i]] + 1
        out.append(np.array(parent, np.int32))
    return out


def _accepted(case, rows):
    """Accepted drafts and their paths, as tree acceptance gives them: chains keep every row, trees a root path."""
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


def _decay(g, layers, rows, heads):
    """Log decays as trained layers have them: a rate in [1, 16) for each head times a step around 0.001 to 0.1 (softplus of a projection)."""
    rate = 1 + 15 * torch.rand((layers, 1, heads), generator=g, device=DEV)
    step = torch.exp(math.log(0.001) + math.log(100) * torch.rand((layers, 1, heads), generator=g, device=DEV))
    return -rate * step * torch.exp(0.5 * torch.randn((layers, rows, heads), generator=g, device=DEV))


def prepare(case, seed):
    g, r = _gen(seed * 7 + 3), np.random.RandomState((seed * 13 + 5) % (1 << 31))

    def normal(*size):
        return torch.randn(size, generator=g, device=DEV)

    if case["op"] == "norm":
        rows, width, wide = case["rows"], case["width"], case["groups"] * case["width"]
        s = dict(case=case, y=normal(rows, wide) * torch.exp(0.5 * normal(rows, 1)), h=None, gate=None, post=None, weight=None, scale=0.8)
        s["y"] = s["y"] if case["y_f32"] else s["y"].bfloat16()
        if case["h"]:
            s["h"] = (3 * normal(rows, wide)).to(torch.float32 if case["h"] == "f32" else torch.bfloat16)
        if case["gate"]:  # columns of a fused projection
            proj = (1.5 * normal(rows, 2 * wide + 64)).bfloat16()
            s["gate"] = proj[:, wide:2 * wide]
        if case["post"]:
            s["post"] = 1 + 0.2 * normal(width)
        if case["weight"]:
            s["weight"] = 1 + 0.2 * normal(width)
        return s
    rows = rows_of(case)
    total, seqs = int(rows.sum()), case["seqs"]
    slots = seqs + 2
    hk, hv, kd, vd, c = case["key_heads"], case["value_heads"], case["key_dim"], case["value_dim"], channels_of(case)
    layers, width = case.get("layers", 1), case.get("width", 4)
    off = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    s = dict(case=case, total=total, width=width, row_off=_dev(off), slot=_dev(r.permutation(slots)[:seqs]), parent=None)
    if case["tree"] and case["op"] != "commit":
        s["parent"] = _dev(np.concatenate(_trees(r, rows)))
    step = total + 3  # the staging holds more rows than this step has
    s["state"] = torch.empty((layers, slots, hv, kd, vd), device=DEV)
    for lay in range(layers):
        s["state"][lay] = 0.5 * normal(slots, hv, kd, vd)
    s["conv"] = normal(layers, slots, width - 1, c).bfloat16()
    s["raw"] = normal(layers, step, c).bfloat16()
    k = normal(layers, step, hk, kd)
    k = k / k.square().sum(3, keepdim=True).sqrt()
    v = normal(layers, step, hv * vd)
    s["kv"] = torch.cat([k.flatten(2), v * torch.sigmoid(v)], 2).bfloat16()
    s["gates"] = torch.stack([_decay(g, layers, step, hv), torch.sigmoid(normal(layers, step, hv))], 2)
    s["delta"] = 0.5 * normal(layers, step, hv, vd)
    if case["op"] == "append":  # the fused projection: q|k|v, the output's gate, strengths, decays, filled up to whole strips
        wide = -(-(c + hv * vd + 2 * hv) // 32) * 32
        proj = normal(total, wide)
        proj = proj if case["f32"] else proj.bfloat16()
        s["qkv"], s["ba"] = proj[:, :c], proj[:, c + hv * vd:c + hv * vd + 2 * hv]
        s["conv_weight"] = normal(c, width) / math.sqrt(width)
        s["a_log"] = torch.log(1 + 15 * torch.rand(hv, generator=g, device=DEV))
        dt = torch.exp(math.log(0.001) + math.log(100) * torch.rand(hv, generator=g, device=DEV))
        s["dt_bias"] = torch.log(torch.expm1(dt))
    if case["op"] == "rule":
        q = normal(total, hk, kd)
        s["q"] = (q / q.square().sum(2, keepdim=True).sqrt()).bfloat16()
        s["out"] = torch.zeros((total, hv * vd), dtype=torch.bfloat16, device=DEV)
    if case["op"] == "commit":
        took, path = _accepted(case, rows)
        s["accept_len"], s["path"] = _dev(took), _dev(np.concatenate(path)) if case["tree"] else None
    return s


# ---------------------------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        import w12_weight_streaming_amd as w12

        if op == "norm":
            out = w12.w12_norm(s["y"], weight=s["weight"], post_weight=s["post"], gate=s["gate"], h=s["h"], scale=s["scale"], groups=s["case"]["groups"], eps=EPS)
            return (out, s["h"]) if s["h"] is not None else (out,)
        cache = w12.DeltaCache(state=s["state"], conv=s["conv"], raw=s["raw"], kv=s["kv"], gates=s["gates"], delta=s["delta"], key_heads=s["case"]["key_heads"])
        if op == "append":
            q = w12.w12_delta_append(cache, 0, s["qkv"], s["ba"], s["row_off"], s["conv_weight"], s["a_log"], s["dt_bias"], slot=s["slot"], parent=s["parent"])
            return q, s["raw"], s["kv"], s["gates"]
        if op == "rule":
            keep = s["case"]["keep"]
            w12.w12_delta_rule(cache, 0, s["q"], s["row_off"], slot=s["slot"], parent=s["parent"], keep=keep, out=s["out"])
            return (s["out"], s["state"], s["conv"]) if keep else (s["out"], s["delta"])
        kept = w12.w12_delta_commit(cache, s["row_off"], s["accept_len"], path=s["path"], slot=s["slot"], rows=s["total"])
        return s["state"], s["conv"], kept
    return {"append": _append, "rule": _rule, "commit": _commit, "norm": _norm}[op](s)


def _rms(x, weight):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight


def _norm(s):
    shape = (s["case"]["rows"], s["case"]["groups"], s["case"]["width"])
    t = s["y"].float().view(shape)
    if s["post"] is not None:
        t = _rms(t, s["post"])
    if s["gate"] is not None:
        z = s["gate"].float().reshape(shape)
        t = t * (z / (1 + torch.exp(-z)))
    if s["h"] is not None:
        s["h"].copy_((s["h"].float().view(shape) + s["scale"] * t).view(s["h"].shape))
        t = s["h"].float().view(shape)
    if s["weight"] is not None:
        t = _rms(t, s["weight"])
    out = t.flatten(1).bfloat16()
    return (out, s["h"]) if s["h"] is not None else (out,)


def _sequence(s):
    """The sequence of each of the step's rows."""
    return (torch.arange(s["total"], device=DEV)[:, None] >= s["row_off"][None, 1:]).sum(1)


def _append(s):
    case = s["case"]
    hk, hv, kd, c, width = case["key_heads"], case["value_heads"], case["key_dim"], channels_of(case), s["width"]
    n, seq = s["total"], _sequence(s)
    first, slot = s["row_off"].long()[seq], s["slot"].long()[seq]
    row = torch.arange(n, device=DEV)
    up = first + s["parent"].long() if s["parent"] is not None else row - 1
    up = torch.where(row == first, -1, up)  # the row above; -1: the window's newest row
    raw = s["qkv"].bfloat16()
    x = raw.float()
    window = s["conv"][0].float()
    y, at = x * s["conv_weight"][:, width - 1], row
    for tap in range(1, width):
        at = torch.where(at >= 0, up[at.clamp(min=0)], at - 1)
        y = y + torch.where((at >= 0)[:, None], x[at.clamp(min=0)], window[slot, (width - 1 + at).clamp(0, width - 2)]) * s["conv_weight"][:, width - 1 - tap]
    y = y / (1 + torch.exp(-y))
    heads = y[:, :2 * hk * kd].unflatten(1, (2 * hk, kd))
    heads = (heads * torch.rsqrt(heads.square().sum(2, keepdim=True) + EPS)).flatten(1)
    q = heads[:, :hk * kd].bfloat16().view(n, hk, kd)
    s["raw"][0, :n] = raw
    s["kv"][0, :n] = torch.cat([heads[:, hk * kd:], y[:, 2 * hk * kd:]], 1).bfloat16()
    b, a = s["ba"].float().split(hv, 1)
    a = a + s["dt_bias"]
    soft = a.clamp(min=0) + torch.log1p(torch.exp(-a.abs()))
    s["gates"][0, :n, 0] = -torch.exp(s["a_log"]) * soft
    s["gates"][0, :n, 1] = 1 / (1 + torch.exp(-b))
    return q, s["raw"], s["kv"], s["gates"]


def _rows_index(s):
    """Each sequence's rows, padded to the longest: their places, and which there are."""
    off = s["row_off"].long()
    at = off[:-1, None] + torch.arange(s["case"]["rows"], device=DEV)
    ok = at < off[1:, None]
    return torch.where(ok, at, 0), ok


def _ancestors(s, at, ok):
    """[seqs, rows, rows]: whether row j is row i or one of its ancestors."""
    n = at.shape[1]
    i = torch.arange(n, device=DEV)
    if s["parent"] is None:
        return (i[:, None] >= i[None, :])[None] & ok[:, None, :] & ok[:, :, None]
    up = torch.where(ok, s["parent"].long()[at], -1)
    a = torch.eye(n, device=DEV)[None] + (up[:, :, None] == i).float()
    for _ in range(max(1, (n - 1).bit_length())):
        a = (a @ a).clamp(max=1)
    return (a > 0) & ok[:, None, :] & ok[:, :, None]


def _rule(s):
    """The rule's closed form: every row's product with the old state, and a triangular system over the rows of its path."""
    case = s["case"]
    hk, hv, kd, vd = case["key_heads"], case["value_heads"], case["key_dim"], case["value_dim"]
    group = hv // hk
    at, ok = _rows_index(s)
    anc = _ancestors(s, at, ok)
    slot = s["slot"].long()
    k = s["kv"][0][at][..., :hk * kd].float().unflatten(2, (hk, kd)).transpose(1, 2).repeat_interleave(group, 1)
    v = s["kv"][0][at][..., hk * kd:].float().unflatten(2, (hv, vd)).transpose(1, 2)
    q = s["q"][at].float().transpose(1, 2).repeat_interleave(group, 1)
    g, beta = s["gates"][0][at].unbind(2)
    g, beta = torch.where(ok[..., None], g, 0).transpose(1, 2).double(), torch.where(ok[..., None], beta, 0).transpose(1, 2)
    sums = (anc[:, None].double() @ g[..., None])[..., 0]  # seqs, heads, rows
    decay = torch.where(anc[:, None], sums[..., :, None] - sums[..., None, :], -math.inf).exp().float()
    old = torch.exp(sums).float()[..., None]
    state = s["state"][0][slot]
    kt = k.transpose(2, 3).contiguous()
    rhs = beta[..., None] * (v - old * (k @ state))
    low = beta[..., None] * decay * (k @ kt)
    n = at.shape[1]
    d = rhs.clone()
    for i in range(1, n):
        d[:, :, i] -= (low[:, :, i:i + 1, :i] @ d[:, :, :i])[:, :, 0]
    o = kd ** -0.5 * (old * (q @ state) + (decay * (q @ kt)) @ d)
    s["out"][at[ok]] = o.transpose(1, 2).flatten(2)[ok].bfloat16()
    if not case["keep"]:
        s["delta"][0, at[ok]] = d.transpose(1, 2)[ok]
        return s["out"], s["delta"]
    last = ok.sum(1) - 1
    end = torch.gather(sums, 2, last[:, None, None].expand(-1, hv, 1))  # seqs, heads, 1
    part = torch.where(ok[:, None], torch.exp(end - sums), 0).float()
    s["state"][0, slot] = torch.exp(end).float()[..., None] * state + kt @ (part[..., None] * d)
    s["conv"][0, slot] = _window(s["conv"][0, slot], s["raw"][0][at], last + 1)
    return s["out"], s["state"], s["conv"]


def _window(old, rows, took):
    """The last rows of (old, the first `took` of rows): [..., seqs, rows, channels] each."""
    both = torch.cat([old, rows], -2)
    ix = took[:, None] + torch.arange(old.shape[-2], device=DEV)
    return torch.gather(both, -2, ix[..., None].expand(*old.shape))


def _commit(s):
    case = s["case"]
    hk, hv, kd = case["key_heads"], case["value_heads"], case["key_dim"]
    slot = s["slot"].long()
    at, ok = _rows_index(s)
    took = s["accept_len"].long() + 1
    if s["path"] is not None:
        at = s["row_off"].long()[:-1, None] + s["path"].long()[at].clamp(min=0)
    on = torch.arange(at.shape[1], device=DEV)[None] < took[:, None]
    at = torch.where(on, at, 0)
    g = torch.where(on[..., None], s["gates"][:, at, 0].double(), 0)  # layers, seqs, rows, heads
    sums = g.cumsum(2)
    end = sums[:, :, -1:]
    part = torch.where(on[..., None], torch.exp(end - sums), 0).float()
    k = s["kv"][:, at, :hk * kd].float().unflatten(3, (hk, kd)).movedim(2, 4).repeat_interleave(hv // hk, 2)  # layers, seqs, heads, dim, rows
    d = (part[..., None] * s["delta"][:, at]).movedim(2, 3)  # layers, seqs, heads, rows, dim
    keep = torch.exp(end[:, :, 0]).float()[..., None, None]
    s["state"][:, slot] = keep * s["state"][:, slot] + k.contiguous() @ d
    s["conv"][:, slot] = _window(s["conv"][:, slot], s["raw"][:, at], took)
    return s["state"], s["conv"], took.int()


# ---------------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "rule": _exact_rule, "commit": _exact_commit, "norm": _exact_norm}[case["op"]](s)


def _exact_norm(s):
    rows, groups, width = s["case"]["rows"], s["case"]["groups"], s["case"]["width"]

    def over(x, weight):
        return x / torch.sqrt((x * x).sum(2, keepdim=True) / width + EPS) * weight.double()

    t = s["y"].double().reshape(rows, groups, width)
    if s["post"] is not None:
        t = over(t, s["post"])
    if s["gate"] is not None:
        z = s["gate"].double().reshape(rows, groups, width)
        t = t * z * torch.sigmoid(z)
    h = None
    if s["h"] is not None:
        h = s["h"].double() + s["scale"] * t.reshape(rows, -1)
        t = h.to(s["h"].dtype).double().reshape(rows, groups, width)  # the norm is of what the residual holds
    if s["weight"] is not None:
        t = over(t, s["weight"])
    return (t.reshape(rows, -1), h) if h is not None else (t.reshape(rows, -1),)


def _host_rows(s):
    off, slot = s["row_off"].tolist(), s["slot"].tolist()
    parent = s["parent"].tolist() if s["parent"] is not None else None
    for n, (a, b) in enumerate(zip(off[:-1], off[1:])):
        yield n, slot[n], a, b, (parent[a:b] if parent else list(range(-1, b - a - 1)))


def _exact_append(s):
    case = s["case"]
    hk, hv, kd, c, width = case["key_heads"], case["value_heads"], case["key_dim"], channels_of(case), s["width"]
    raw, kv, gates = s["raw"].clone(), s["kv"].double(), s["gates"].double()
    q = torch.zeros((s["total"], hk, kd), dtype=torch.float64, device=DEV)
    w = s["conv_weight"].double()
    for _, slot, a, b, parent in _host_rows(s):
        window = [s["conv"][0, slot, i].double() for i in range(width - 1)]
        paths = []  # the last rows up to each row
        for i in range(b - a):
            raw[0, a + i] = s["qkv"][a + i].bfloat16()
            above = paths[parent[i]] if parent[i] >= 0 else window
            paths.append(above[-(width - 1):] + [raw[0, a + i].double()])
        x = torch.stack([torch.stack(p[-width:]) for p in paths])  # rows, width, channels
        y = torch.einsum("nwc,cw->nc", x, w)
        y = y * torch.sigmoid(y)
        for h in range(2 * hk):
            z = y[:, h * kd:(h + 1) * kd]
            y[:, h * kd:(h + 1) * kd] = z / torch.sqrt((z * z).sum(1, keepdim=True) + EPS)
        q[a:b] = y[:, :hk * kd].reshape(b - a, hk, kd)
        kv[0, a:b] = y[:, hk * kd:]
    n = s["total"]
    z = s["ba"][:, hv:].double() + s["dt_bias"].double()
    gates[0, :n, 0] = -torch.exp(s["a_log"].double()) * torch.where(z > 30, z, torch.log1p(torch.exp(z.clamp(max=30))))
    gates[0, :n, 1] = torch.sigmoid(s["ba"][:, :hv].double())
    return q, raw.double(), kv, gates


def _exact_rule(s):
    """Row by row, each from the state of the row above it."""
    case = s["case"]
    hk, hv, kd, vd = case["key_heads"], case["value_heads"], case["key_dim"], case["value_dim"]
    head = torch.arange(hv, device=DEV) // (hv // hk)
    out, delta, state, conv = s["out"].double(), s["delta"].double(), s["state"].double(), s["conv"].double()
    for _, slot, a, b, parent in _host_rows(s):
        first = state[0, slot].clone()
        if s["parent"] is not None and (b - a) * first.numel() * 8 > 6e9:
            return None
        seen, now = [], first
        for i in range(b - a):
            above = now if s["parent"] is None else seen[parent[i]] if parent[i] >= 0 else first
            k = s["kv"][0, a + i, :hk * kd].double().view(hk, kd)[head]
            v = s["kv"][0, a + i, hk * kd:].double().view(hv, vd)
            now = above * torch.exp(s["gates"][0, a + i, 0].double())[:, None, None]
            d = s["gates"][0, a + i, 1].double()[:, None] * (v - (now * k[:, :, None]).sum(1))
            now = now + k[:, :, None] * d[:, None, :]
            out[a + i] = ((now * s["q"][a + i].double()[head][:, :, None]).sum(1) / math.sqrt(kd)).reshape(-1)
            delta[0, a + i] = d
            if s["parent"] is not None:
                seen.append(now)
        if case["keep"]:
            state[0, slot] = now
            rows = torch.cat([s["conv"][0, slot], s["raw"][0, a:b]])
            conv[0, slot] = rows[-(s["width"] - 1):].double()
    return (out, state, conv) if case["keep"] else (out, delta)


def _exact_commit(s):
    case = s["case"]
    hk, hv, kd = case["key_heads"], case["value_heads"], case["key_dim"]
    state, conv = s["state"].double(), s["conv"].double()
    head = torch.arange(hv, device=DEV) // (hv // hk)
    took, path = s["accept_len"].tolist(), s["path"].tolist() if s["path"] is not None else None
    for n, slot, a, b, _ in _host_rows(s):
        rows = [a + (path[a + j] if path else j) for j in range(took[n] + 1)]
        now = state[:, slot]
        for r in rows:
            k = s["kv"][:, r, :hk * kd].double().view(-1, hk, kd)[:, head]
            now = now * torch.exp(s["gates"][:, r, 0].double())[..., None, None] + k[..., None] * s["delta"][:, r].double()[:, :, None, :]
        state[:, slot] = now
        conv[:, slot] = torch.cat([s["conv"][:, slot], s["raw"][:, rows]], 1)[:, -(s["width"] - 1):].double()
    return state, conv, s["accept_len"] + 1
