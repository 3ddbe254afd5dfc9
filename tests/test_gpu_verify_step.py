"""A verify step as it is used: Wq|Wk|Wv product, append, attention, Wo
product, head product, sampled and greedy acceptance, commit, over several
steps of a ragged batch (trees, a prompt chunk, plain decoding). Each stage is
checked against its oracle on the inputs that the stage before produced."""
import numpy as np
import pytest

import synth
from oracle import kv_cache as KV
from oracle import tree_sampled as TS
from oracle import verify as V

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HIDDEN, KVH, GROUP, DIM, PAGE, VOCAB, LAYERS = 512, 2, 4, 64, 32, 1056, 2
HEADS = KVH * GROUP


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.fixture(scope="module")
def model():
    import torch
    import w12_weight_streaming_amd as w12
    assert torch.cuda.is_available()
    layers = []
    for li in range(LAYERS):
        qkv = synth.weights_bf16((HEADS + 2 * KVH) * DIM, HIDDEN, seed=700 + li, p_zero=0.01, p_outlier=0.0)
        wo = synth.weights_bf16(HIDDEN, HEADS * DIM, seed=710 + li, p_zero=0.01, p_outlier=0.0)
        layers.append({"qkv": (w12.w12_pack(qkv.to(DEV)), synth.bits_u16(qkv)),
                       "wo": (w12.w12_pack(wo.to(DEV)), synth.bits_u16(wo))})
    head = synth.weights_bf16(VOCAB, HIDDEN, seed=720, p_zero=0.01, p_outlier=0.0)
    return w12, layers, (w12.w12_pack(head.to(DEV)), synth.bits_u16(head))


def product(w12, packed, x):
    """The W12 product, checked, in fp32."""
    pw, bits = packed
    y = w12.w12_gemm(pw, x)
    ref, bound = V.gemm_ref(synth.bits_u16(x.cpu()), bits)
    assert V.within_tolerance(y.cpu().numpy(), ref, bound).all()
    return y


def test_steps_of_a_ragged_batch(model):
    import torch
    w12, layers, head = model
    rng = np.random.RandomState(3)
    seqs, slots, blocks = 4, 5, 8
    cache = w12.kv_cache(LAYERS, KVH, DIM, seqs * blocks, slots, blocks, PAGE, 64, False, DEV)
    slot = np.array([3, 0, 4, 1], np.int32)
    table = np.zeros((slots, blocks), np.int32)
    table[slot] = rng.permutation(seqs * blocks).reshape(seqs, blocks)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)
    cache.page_table.copy_(i32(table))
    ang = np.arange(300)[:, None] * 10000.0 ** (-np.arange(0, DIM, 2) / DIM)
    rope = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    rope_t = torch.tensor(rope, device=DEV)
    embed = (rng.randn(VOCAB, HIDDEN)).astype(np.float32)
    state = [[[KV.Sequence(PAGE, False, DIM) for _ in range(KVH)] for _ in range(seqs)] for _ in range(LAYERS)]
    last = rng.randint(0, VOCAB, seqs)

    def tree(n):
        return np.array([-1] + [int(rng.randint(max(0, i - 4), i)) for i in range(1, n)], np.int32)
    steps = [[KV.chain(40), KV.chain(1), KV.chain(63), KV.chain(31)],          # prompts of other lengths
             [tree(12), KV.chain(1), tree(9), KV.chain(5)],
             [tree(7), KV.chain(2), KV.chain(1), tree(30)],
             [KV.chain(1), KV.chain(60), tree(16), tree(16)]]
    for si, parents in enumerate(steps):
        prompt = si == 0
        rows = [len(p) for p in parents]
        off = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        total = int(off[-1])
        token = rng.randint(0, VOCAB, total).astype(np.int32)
        token[off[:-1]] = last
        parent = np.concatenate(parents).astype(np.int32)
        d_off, d_par, d_slot = i32(off), i32(parent), i32(slot)
        x = torch.tensor(embed[token], device=DEV)
        kept = []
        for li, layer in enumerate(layers):
            h = (x / x.pow(2).mean(1, keepdim=True).sqrt()).bfloat16()
            qkv = product(w12, layer["qkv"], h)
            q = w12.w12_kv_append(cache, li, qkv, d_off, rope_t, HEADS, slot=d_slot, parent=d_par)
            att = w12.w12_kv_attention(cache, li, q, d_off, slot=d_slot, parent=d_par)
            got_q, got, rec = f64(q), f64(att).reshape(total, HEADS, DIM), f64(cache.recent[li])
            raw = f64(qkv).reshape(total, -1, DIM)
            per_seq = []
            for s in range(seqs):
                a, b = off[s], off[s + 1]
                length = state[li][s][0].length
                turned, size = KV.rotate(raw[a:b, :HEADS + KVH], length + KV.depths(parents[s]), rope, False)
                tol = 2.0 ** -8 * np.abs(turned) + 4 * 2.0 ** -24 * size
                at = np.arange(length % PAGE, length % PAGE + b - a)
                k, v = (np.stack([rec[slot[s], g, w][KV.places(w, at[-1] + 1, DIM)[at]] for g in range(KVH)], 1) for w in (0, 1))
                assert (np.abs(got_q[a:b] - turned[:, :HEADS]) <= tol[:, :HEADS]).all()
                assert (np.abs(k - turned[:, HEADS:]) <= tol[:, HEADS:]).all()
                assert (np.abs(v - raw[a:b, HEADS + KVH:]) <= 2.0 ** -8 * np.abs(raw[a:b, HEADS + KVH:])).all()
                see = np.concatenate([np.ones((b - a, length), bool), KV.ancestors(parents[s])], 1)
                for g in range(KVH):
                    seq, hs = state[li][s][g], slice(g * GROUP, (g + 1) * GROUP)
                    ref, av, sz = KV.attention(got_q[a:b, hs], np.concatenate([seq.k, k[:, g]]), np.concatenate([seq.v, v[:, g]]),
                                               see, DIM ** -0.5)
                    assert (np.abs(got[a:b, hs] - ref) <= KV.attention_tolerance(ref, av, sz, length + b - a, DIM)).all()
                per_seq.append((k, v))
            kept.append(per_seq)
            x = x + product(w12, layer["wo"], att)
        h = (x / x.pow(2).mean(1, keepdim=True).sqrt()).bfloat16()
        logits = product(w12, head, h)
        lg = logits.cpu().numpy()
        # give the drafts a chance: some children carry their parent's likely tokens
        for s in range(seqs):
            for i in range(1, rows[s]):
                if not prompt and rng.rand() < 0.7:
                    token[off[s] + i] = int(np.argsort(-lg[off[s] + parents[s][i]])[rng.randint(2)])
        u, ub = rng.rand(total).astype(np.float32), rng.rand(seqs).astype(np.float32)
        temp = rng.uniform(0.05, 0.6, seqs).astype(np.float32)
        f32 = lambda a: torch.tensor(a, device=DEV)
        if prompt:
            acc, path = i32(np.array(rows) - 1), None
            last = lg[off[1:] - 1].argmax(1)
        elif si % 2:
            acc, path, bonus = w12.tree_accept_sampled(d_off, d_par, i32(token), logits, f32(u), f32(ub), temperature=f32(temp))
            ref = TS.forest(off, parent, token, lg, temp, None, u, ub)
            assert all(np.array_equal(g.cpu().numpy(), r) for g, r in zip((acc, path, bonus), ref))
            last = bonus.cpu().numpy()
        else:
            am, _ = w12.w12_head_argmax(head[0], h)
            acc, path, bonus = w12.tree_accept(d_off, d_par, i32(token), am)
            last = bonus.cpu().numpy()
        w12.w12_kv_commit(cache, d_off, acc, path=path, slot=d_slot)
        n_acc = acc.cpu().numpy()
        way = None if path is None else path.cpu().numpy()
        codes, scales = cache.pages.float().cpu().numpy(), cache.scales.cpu().numpy()
        for s in range(seqs):
            take = np.arange(rows[s]) if way is None else way[off[s]:off[s] + n_acc[s] + 1]
            for li in range(LAYERS):
                for g in range(KVH):
                    seq = state[li][s][g]
                    seq.commit(kept[li][s][0][take, g], kept[li][s][1][take, g])
                    for b, blk in enumerate(seq.blocks):
                        for w in (0, 1):
                            pid = table[slot[s], b]
                            assert scales[li, pid, g, w] == blk[2 * w + 1]
                            assert np.array_equal(codes[li, pid, g, w][KV.places(w, PAGE, DIM)], blk[2 * w])
            assert cache.length[int(slot[s])].item() == state[0][s][0].length
        print("[step]", si, "accepted", n_acc.tolist(), "lengths", cache.length.tolist(), flush=True)
