"""The KV cache's and the sampled tree acceptance's entry points reject bad
arguments before launching anything. No compute call is made here."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def w12():
    import w12_weight_streaming_amd as w
    if not os.path.exists(w.LIB_PATH):
        from w12_weight_streaming_amd import build
        build.build()
    w.lib()
    return w


FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x1002)
NULL = ctypes.c_void_p(0)
FAR = ctypes.c_void_p(1 << 40)


def cache(w12, **kw):
    f = dict(kvtype=0, layers=2, num_pages=8, kv_heads=4, page_tokens=64, head_dim=128, slots=4, recent_rows=96,
             max_pages=8, pages=0x1000, scales=0x1000, recent=0x1000, page_table=0x1000, len=0x1000)
    assert set(kw) <= set(f)
    f.update(kw)
    return w12.W12KvCache(*f.values())


BAD_CACHES = [dict(kvtype=2), dict(layers=0), dict(num_pages=0), dict(kv_heads=0), dict(kv_heads=257), dict(page_tokens=16),
              dict(page_tokens=48), dict(page_tokens=256), dict(head_dim=96), dict(head_dim=512), dict(slots=0),
              dict(recent_rows=32), dict(recent_rows=100), dict(recent_rows=2048), dict(max_pages=0), dict(max_pages=1 << 30),
              dict(pages=0), dict(pages=0x1008), dict(scales=0x1004), dict(recent=0x1008), dict(page_table=0), dict(len=0x1001)]


def calls(w12, c):
    """Every call with this cache, good otherwise."""
    L, d = w12.lib(), ctypes.byref(c)
    sz = ctypes.c_size_t(0)
    return {"append": L.w12_kv_append(d, 0, 1, NULL, FAKE, 4, NULL, FAKE, 0, 8, FAKE, 16, 128, 0, FAKE, NULL),
            "attention": L.w12_kv_attention(d, 0, 1, NULL, FAKE, 4, NULL, FAKE, 8, 0.1, FAKE, FAKE, 1 << 40, NULL),
            "workspace": L.w12_kv_attention_workspace(d, 1, 4, 8, ctypes.byref(sz)),
            "commit": L.w12_kv_commit(d, 1, NULL, FAKE, 4, FAKE, NULL, FAKE, NULL)}


@pytest.mark.parametrize("kw", BAD_CACHES, ids=str)
def test_bad_caches(w12, kw):
    assert set(calls(w12, cache(w12, **kw)).values()) == {w12.W12_EINVAL}


def test_no_cache(w12):
    L = w12.lib()
    assert L.w12_kv_commit(None, 1, NULL, FAKE, 4, FAKE, NULL, FAKE, NULL) == w12.W12_EINVAL


def test_append_arguments(w12):
    L, d = w12.lib(), ctypes.byref(cache(w12))

    def go(layer=0, seqs=1, off=FAKE, rows=4, qkv=FAKE, kind=0, heads=8, rope=FAKE, positions=16, rot=128, q=FAR):
        return L.w12_kv_append(d, layer, seqs, NULL, off, rows, NULL, qkv, kind, heads, rope, positions, rot, 0, q, NULL)
    for kw in (dict(layer=-1), dict(layer=2), dict(seqs=0), dict(seqs=513), dict(off=NULL), dict(rows=0), dict(rows=513),
               dict(qkv=NULL), dict(qkv=ODD), dict(kind=2), dict(heads=0), dict(heads=6), dict(heads=260), dict(rope=NULL),
               dict(positions=0), dict(rot=0), dict(rot=3), dict(rot=130), dict(q=NULL), dict(q=ctypes.c_void_p((1 << 40) + 2)),
               dict(q=FAKE), dict(q=ctypes.c_void_p(0x1000 + 16))):  # over qkv
        assert go(**kw) == w12.W12_EINVAL, kw


def test_attention_arguments(w12):
    L, d = w12.lib(), ctypes.byref(cache(w12))

    def go(layer=0, seqs=1, off=FAKE, rows=4, q=FAKE, heads=8, scale=0.1, out=FAR, ws=FAKE):
        return L.w12_kv_attention(d, layer, seqs, NULL, off, rows, NULL, q, heads, scale, out, ws, 0, NULL)
    for kw in (dict(layer=2), dict(seqs=0), dict(seqs=513), dict(off=NULL), dict(rows=0), dict(rows=513), dict(q=NULL),
               dict(q=ODD), dict(heads=0), dict(heads=7), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(out=NULL), dict(out=ctypes.c_void_p((1 << 40) + 2)), dict(out=FAKE), dict(ws=NULL), dict(ws=ctypes.c_void_p(0x1010))):
        assert go(**kw) == w12.W12_EINVAL, kw
    sz = ctypes.c_size_t(0)
    for seqs, rows, heads in ((0, 4, 8), (1, 0, 8), (1, 513, 8), (1, 4, 9)):
        assert L.w12_kv_attention_workspace(d, seqs, rows, heads, ctypes.byref(sz)) == w12.W12_EINVAL
    assert L.w12_kv_attention_workspace(d, 1, 4, 8, None) == w12.W12_EINVAL


def test_commit_arguments(w12):
    L, d = w12.lib(), ctypes.byref(cache(w12))
    for seqs, off, rows, acc, out in ((0, FAKE, 4, FAKE, FAKE), (513, FAKE, 4, FAKE, FAKE), (1, NULL, 4, FAKE, FAKE),
                                      (1, FAKE, 0, FAKE, FAKE), (1, FAKE, 513, FAKE, FAKE), (1, FAKE, 4, NULL, FAKE),
                                      (1, FAKE, 4, FAKE, NULL)):
        assert L.w12_kv_commit(d, seqs, NULL, off, rows, acc, NULL, out, NULL) == w12.W12_EINVAL


def test_sampled_arguments(w12):
    L = w12.lib()
    sz = ctypes.c_size_t(0)
    assert L.tree_accept_sampled_workspace(24, 192, 152064, ctypes.byref(sz)) == w12.W12_OK and sz.value > 0
    for t, n, v in ((0, 4, 8), (1, 0, 8), (1, 4, 0), (65536, 4, 8), (1, 65536, 8), (1, 4, (1 << 28) + 1)):
        assert L.tree_accept_sampled_workspace(t, n, v, ctypes.byref(sz)) == w12.W12_EINVAL

    def go(trees=1, off=FAKE, nodes=4, parent=FAKE, token=FAKE, logits=FAKE, kind=0, vocab=8, temp=NULL, draft=NULL, u=FAKE,
           ub=FAKE, acc=FAKE, path=FAKE, bonus=FAKE, ws=FAKE, nbytes=1 << 30):
        return L.tree_accept_sampled(trees, off, nodes, parent, token, logits, kind, vocab, temp, draft, u, ub, acc, path,
                                     bonus, ws, nbytes, NULL)
    for kw in (dict(trees=0), dict(nodes=0), dict(vocab=0), dict(kind=3), dict(logits=ctypes.c_void_p(0x1001)),
               dict(draft=ODD), dict(ws=ctypes.c_void_p(0x1004)),
               *({k: NULL} for k in ("off", "parent", "token", "logits", "u", "ub", "acc", "path", "bonus", "ws"))):
        assert go(**kw) == w12.W12_EINVAL, kw
    assert go(nbytes=16) == w12.W12_ENOSPC


def test_binding_refuses_cpu_tensors(w12):
    import torch
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)
    with pytest.raises(ValueError):
        w12.kv_cache(1, 1, 64, 2, 1, 1, device="cpu")
    with pytest.raises(TypeError):
        w12.KvCache(None, None, None, None, None, 64)
    with pytest.raises(ValueError):
        w12.tree_accept_sampled(z(2, dt=torch.int32), z(3, dt=torch.int32), z(3, dt=torch.int32), z(3, 8), z(3), z(1))
    with pytest.raises(TypeError):
        w12.tree_accept_sampled(z(2, dt=torch.int32), z(3, dt=torch.int32), z(3, dt=torch.int32), z(3, 8).half(), z(3), z(1))


# Addresses that no two arguments share, so that only the cache can be what a call refuses.
APART = [ctypes.c_void_p((i + 1) << 40) for i in range(4)]


def call_apart(w12, c, ws_bytes=1 << 40):
    L, d = w12.lib(), ctypes.byref(c)
    qkv, q, out, ws = APART
    return (lambda: L.w12_kv_append(d, 0, 1, NULL, FAKE, 4, NULL, qkv, 0, 8, FAKE, 16, 128, 0, q, NULL),
            lambda: L.w12_kv_attention(d, 0, 1, NULL, FAKE, 4, NULL, q, 8, 0.1, out, ws, ws_bytes, NULL))


@pytest.mark.parametrize("kw", BAD_CACHES +
                         [dict(layers=1025), dict(slots=(1 << 20) + 1), dict(scales=0), dict(recent=0), dict(len=0),
                          dict(page_table=0x1002), dict(recent_rows=1056)], ids=str)
def test_bad_caches_with_arguments_that_lie_apart(w12, kw):
    append, attention = call_apart(w12, cache(w12, **kw))
    assert append() == w12.W12_EINVAL
    assert attention() == w12.W12_EINVAL


def test_a_good_cache_passes_the_checks(w12):
    """What the test above refuses is the cache: with a good one the call
    goes on to its workspace's size (to the missing GPU where there is none)."""
    _, attention = call_apart(w12, cache(w12), ws_bytes=0)
    assert attention() in (w12.W12_ENOSPC, w12.W12_EHIP)
