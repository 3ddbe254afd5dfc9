"""Verify steps of a small model of recurrent layers as a program runs them: W12
products, norms, the delta rule over drafted trees, head argmax, acceptance and
commit, step after step, against a plain 64-bit model that decodes the accepted
tokens one at a time."""
import numpy as np
import pytest

from oracle import delta as D

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HID, VOCAB, LAYERS, HK, HV, KD, VD, W = 256, 512, 2, 2, 4, 64, 64, 4
C = 2 * HK * KD + HV * VD
WIDE = -(-(C + HV * VD + 2 * HV) // 32) * 32  # q|k|v, output gate, strengths and decays, filled up to whole strips


@pytest.fixture(scope="module")
def w12():
    import torch
    import w12_weight_streaming_amd as w
    assert torch.cuda.is_available()
    w.lib()
    return w


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


class Model:
    def __init__(self, w12, seed=0):
        import torch
        self.w12 = w12
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        pack = lambda w: w12.w12_pack(w.to(DEV))  # noqa: E731
        self.layers = []
        for _ in range(LAYERS):
            w_in, w_out = (n(WIDE, HID) / 16).bfloat16(), (n(HID, HV * VD) / 16).bfloat16()
            self.layers.append(dict(
                w_in=w_in, w_out=w_out, p_in=pack(w_in), p_out=pack(w_out), conv=n(C, W) / 2, a_log=torch.rand(HV, generator=g) * 2,
                dt=n(HV) - 2, head=1 + 0.1 * n(VD), norm=1 + 0.1 * n(HID)))
        self.table = n(VOCAB, HID).bfloat16()
        self.w_head = (n(VOCAB, HID) / 16).bfloat16()
        self.p_head, self.final = pack(self.w_head), 1 + 0.1 * n(HID)
        self.dev = [{k: v.to(DEV) for k, v in la.items() if hasattr(v, "to")} for la in self.layers]
        self.dtable, self.dfinal = self.table.to(DEV), self.final.to(DEV)

    def step(self, cache, tokens, off, parent=None, slot=None, keep=False):
        """Rows of tokens through all layers; returns the head's (argmax, hidden rows)."""
        w12 = self.w12
        h = self.dtable[tokens.long()].float()
        x = w12.w12_norm(None, h=h, weight=self.dev[0]["norm"])
        for i, (la, d) in enumerate(zip(self.layers, self.dev)):
            proj = w12.w12_gemm(la["p_in"], x)
            q = w12.w12_delta_append(cache, i, proj[:, :C], proj[:, C + HV * VD:C + HV * VD + 2 * HV], off, d["conv"], d["a_log"], d["dt"],
                                     slot=slot, parent=parent)
            o = w12.w12_delta_rule(cache, i, q, off, slot=slot, parent=parent, keep=keep)
            o = w12.w12_norm(o, post_weight=d["head"], gate=proj[:, C:C + HV * VD], groups=HV)
            y = w12.w12_gemm(la["p_out"], o, out_dtype=__import__("torch").bfloat16)
            x = w12.w12_norm(y, h=h, weight=self.dev[i + 1]["norm"] if i + 1 < LAYERS else self.dfinal)
        return w12.w12_head_argmax(self.p_head, x)[0], x

    def plain(self, tokens):
        """The same model in 64 bits without roundings, one sequence of tokens: hidden rows before the head."""
        f = lambda t: t.float().numpy().astype(np.float64)  # noqa: E731
        h = f(self.table)[tokens]
        x = D.rms(h, f(self.layers[0]["norm"]), 1e-6)
        n = len(tokens)
        for i, la in enumerate(self.layers):
            proj = x @ f(la["w_in"]).T
            z = proj[:, C:C + HV * VD]
            s, _ = D.append(proj[:, :C], np.zeros((W - 1, C)), D.chain(n), f(la["conv"]), None, HK, KD)
            b, a = proj[:, C + HV * VD:C + HV * VD + HV], proj[:, C + HV * VD + HV:C + HV * VD + 2 * HV]
            g, beta, _, _ = D.gates(b, a, f(la["a_log"]), f(la["dt"]))
            o = np.zeros((n, HV, VD))
            for hd in range(HV):
                key = hd // (HV // HK)
                k = s[:, (HK + key) * KD:(HK + key + 1) * KD]
                v = s[:, 2 * HK * KD + hd * VD:][:, :VD]
                o[:, hd] = D.rule(np.zeros((KD, VD)), k, v, s[:, key * KD:(key + 1) * KD], g[:, hd], beta[:, hd], D.chain(n), KD ** -0.5)[0]
            o = D.rms(o, f(la["head"]), 1e-6).reshape(n, -1) * z * D.sigmoid(z)
            h = h + o @ f(la["w_out"]).T
            x = D.rms(h, f(self.layers[i + 1]["norm"]) if i + 1 < LAYERS else f(self.final), 1e-6)
        return x


def test_verify_steps(w12):
    """Prompts (kept at once), then trees of drafts: what is committed is the
    sequence of accepted tokens, for every sequence of a ragged batch."""
    import torch
    m = Model(w12)
    r = np.random.RandomState(3)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
    cache = w12.delta_cache(LAYERS, 5, HK, HV, KD, VD, W, step_rows=128, device=DEV)
    slots = i32([4, 1, 2])
    prompts = [list(r.randint(0, VOCAB, n)) for n in (40, 1, 7)]
    off = np.concatenate([[0], np.cumsum([len(p) for p in prompts])])
    rows = i32(np.concatenate(prompts))
    arg, x = m.step(cache, rows, i32(off), slot=slots, keep=True)
    seqs = [list(p) for p in prompts]
    hidden = [list(f64(x[off[s]:off[s + 1]])) for s in range(3)]
    nxt = [int(arg[off[s + 1] - 1]) for s in range(3)]
    for turn in range(4):
        trees, toks = [], []
        for s in range(3):
            n = int(r.randint(1, 12))
            # the root is the next token; drafts are random, and a chain of what plain decoding would take among them
            parent = np.array([-1] + [int(r.randint(0, i)) for i in range(1, n)], np.int32)
            trees.append(parent)
            toks.append([nxt[s]] + list(r.randint(0, VOCAB, n - 1)))
        off = np.concatenate([[0], np.cumsum([len(p) for p in trees])])
        parent, token = i32(np.concatenate(trees)), i32(np.concatenate(toks))
        arg, x = m.step(cache, token, i32(off), parent=parent, slot=slots)
        # make one draft of each tree right, so that acceptance goes deeper than the root: its own argmax
        host, fixed = arg.cpu().numpy(), token.cpu().numpy().copy()
        for s in range(3):
            kids = [i for i in range(1, len(trees[s])) if trees[s][i] == 0]
            if kids:
                fixed[off[s] + kids[-1]] = host[off[s]]
        token = i32(fixed)
        arg, x = m.step(cache, token, i32(off), parent=parent, slot=slots)  # staging again overwrites the step's rows
        acc, path, bonus = w12.tree_accept(i32(off), parent, token, arg)
        kept = w12.w12_delta_commit(cache, i32(off), acc, path=path, slot=slots)
        assert kept.tolist() == [a + 1 for a in acc.tolist()]
        path = path.cpu().numpy()
        for s in range(3):
            for j in range(int(acc[s]) + 1):
                at = off[s] + path[off[s] + j]
                seqs[s].append(int(fixed[at]))
                hidden[s].append(f64(x[at]))
            nxt[s] = int(bonus[s])
    assert max(len(q) for q in seqs) > 44
    for s in range(3):
        want = m.plain(np.array(seqs[s]))
        got = np.stack(hidden[s])
        # bf16 hidden rows, products' inputs, queries, keys, values and outputs: about a dozen roundings of 2^-8 a
        # layer, most of them averaged over a product's terms; an order of magnitude below any wrong row
        off_by = np.linalg.norm(got - want, axis=1) / np.linalg.norm(want, axis=1)
        assert off_by.max() <= 12 * LAYERS * D.BF16, (s, off_by)


def test_plain_decoding_goes_on_from_a_prompt(w12):
    """One token a step, kept, after a prompt: the rows of the prompt and its continuation in one call."""
    import torch
    m = Model(w12, seed=7)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
    tokens = np.random.RandomState(5).randint(0, VOCAB, 50)
    one, other = (w12.delta_cache(LAYERS, 1, HK, HV, KD, VD, W, step_rows=64, device=DEV) for _ in range(2))
    _, whole = m.step(one, i32(tokens), i32([0, 50]), keep=True)
    _, first = m.step(other, i32(tokens[:33]), i32([0, 33]), keep=True)
    rest = [m.step(other, i32(tokens[i:i + 1]), i32([0, 1]), keep=True)[1] for i in range(33, 50)]
    got = torch.cat([first, *rest])
    want = m.plain(tokens)
    for x in (whole, got):
        off_by = np.linalg.norm(f64(x) - want, axis=1) / np.linalg.norm(want, axis=1)
        assert off_by.max() <= 12 * LAYERS * D.BF16
    assert (one.state - other.state).norm() <= 0.05 * one.state.norm()
