"""The recurrent layers' and the norms' entry points reject bad arguments
before launching anything. No compute call is made here."""
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


P = ctypes.c_void_p
FAKE, ODD, NULL, FAR = P(0x1000), P(0x1002), P(0), P(1 << 40)  # never dereferenced: validation fails first
C = 2 * 4 * 64 + 8 * 128  # channels of the description below


def cache(w12, **kw):
    f = dict(layers=2, slots=4, step_rows=96, key_heads=4, value_heads=8, key_dim=64, value_dim=128, conv_width=4,
             state=0x1000, conv=0x1000, raw=0x1000, kv=0x1000, gates=0x1000, delta=0x1000)
    assert set(kw) <= set(f)
    f.update(kw)
    return w12.W12DeltaCache(*f.values())


def calls(w12, c):
    """Every call with this cache, good otherwise."""
    L, d = w12.lib(), ctypes.byref(c)
    return {"append": L.w12_delta_append(d, 0, 1, NULL, FAKE, 4, NULL, FAKE, C, FAKE, 16, 0, FAKE, NULL, FAKE, FAKE, FAR, NULL),
            "rule": L.w12_delta_rule(d, 0, 1, NULL, FAKE, 4, NULL, FAKE, 0.1, 0, FAR, NULL),
            "commit": L.w12_delta_commit(d, 1, NULL, FAKE, 4, FAKE, NULL, FAR, NULL)}


BAD = [dict(layers=0), dict(layers=1025), dict(slots=0), dict(slots=(1 << 20) + 1), dict(step_rows=0), dict(step_rows=65537),
       dict(key_heads=0), dict(value_heads=0), dict(value_heads=6), dict(value_heads=260), dict(key_dim=32),
       dict(key_dim=96), dict(key_dim=256), dict(value_dim=32), dict(value_dim=256), dict(conv_width=1),
       dict(conv_width=5), dict(step_rows=3), dict(state=0), dict(conv=0), dict(raw=0), dict(kv=0), dict(gates=0), dict(delta=0),
       dict(state=0x1008), dict(conv=0x1008), dict(raw=0x1002), dict(kv=0x1008), dict(gates=0x1004), dict(delta=0x1004)]


@pytest.mark.parametrize("kw", BAD, ids=str)
def test_bad_caches(w12, kw):
    assert set(calls(w12, cache(w12, **kw)).values()) == {w12.W12_EINVAL}


def test_no_cache(w12):
    L = w12.lib()
    assert L.w12_delta_commit(None, 1, NULL, FAKE, 4, FAKE, NULL, FAR, NULL) == w12.W12_EINVAL
    assert L.w12_delta_rule(None, 0, 1, NULL, FAKE, 4, NULL, FAKE, 0.1, 0, FAR, NULL) == w12.W12_EINVAL


def test_append_arguments(w12):
    L, d = w12.lib(), ctypes.byref(cache(w12))

    def go(layer=0, seqs=1, off=FAKE, rows=4, x=FAKE, xs=C, ba=FAKE, bs=16, kind=0, w=FAKE, bias=NULL, a=FAKE, dt=FAKE, q=FAR):
        return L.w12_delta_append(d, layer, seqs, NULL, off, rows, NULL, x, xs, ba, bs, kind, w, bias, a, dt, q, NULL)
    for kw in (dict(layer=-1), dict(layer=2), dict(seqs=0), dict(seqs=513), dict(off=NULL), dict(rows=0), dict(rows=97),
               dict(x=NULL), dict(x=ODD), dict(xs=C - 4), dict(xs=C + 2), dict(xs=C + 4, kind=1), dict(xs=1 << 33), dict(xs=-C),
               dict(ba=NULL), dict(ba=ODD), dict(ba=P(0x1001), kind=1), dict(bs=15), dict(bs=1 << 33), dict(kind=2), dict(w=NULL),
               dict(w=P(0x1008)), dict(bias=P(0x1004)), dict(a=NULL), dict(a=ODD), dict(dt=NULL), dict(dt=ODD), dict(q=NULL),
               dict(q=P((1 << 40) + 2)), dict(q=FAKE), dict(q=P(0x1000 + 16)), dict(x=FAR, q=P(0x1010)),  # the last over ba
               dict(x=FAR, ba=FAR, q=P(0x1000 + 4096))):  # over the state
        assert go(**kw) == w12.W12_EINVAL, kw


def test_rule_arguments(w12):
    L, d = w12.lib(), ctypes.byref(cache(w12))

    def go(layer=0, seqs=1, off=FAKE, rows=4, parent=NULL, q=FAKE, scale=0.1, keep=0, out=FAR):
        return L.w12_delta_rule(d, layer, seqs, NULL, off, rows, parent, q, scale, keep, out, NULL)
    for kw in (dict(layer=2), dict(seqs=0), dict(seqs=513), dict(off=NULL), dict(rows=0), dict(rows=97), dict(q=NULL), dict(q=ODD),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(out=NULL), dict(out=P((1 << 40) + 8)), dict(out=FAKE),
               dict(out=P(0x1000 + 4 * 4 * 64 * 2 - 16)), dict(q=FAR, out=P(0x1000)), dict(q=FAR, out=P(0x1000 + (1 << 20))),
               dict(keep=1, parent=FAKE)):
        assert go(**kw) == w12.W12_EINVAL, kw


def test_commit_arguments(w12):
    L, d = w12.lib(), ctypes.byref(cache(w12))

    def go(seqs=2, off=FAKE, rows=4, acc=FAKE, path=NULL, kept=FAR):
        return L.w12_delta_commit(d, seqs, NULL, off, rows, acc, path, kept, NULL)
    for kw in (dict(seqs=0), dict(seqs=513), dict(off=NULL), dict(rows=0), dict(rows=97), dict(acc=NULL), dict(kept=NULL),
               dict(kept=P(0x1004)), dict(acc=FAR, path=FAKE, kept=P(0x100C)), dict(acc=FAR, kept=P(0x1000 + (1 << 20)))):
        assert go(**kw) == w12.W12_EINVAL, kw


def test_norm_arguments(w12):
    L = w12.lib()

    def go(rows=4, groups=2, width=64, y=FAKE, yt=0, ys=128, post=NULL, gate=NULL, gt=0, gs=128, scale=1.0, h=NULL, ht=0,
           weight=NULL, eps=1e-6, out=FAR):
        return L.w12_norm(rows, groups, width, y, yt, ys, post, gate, gt, gs, scale, h, ht, weight, eps, out, NULL)
    far = P((1 << 40) + (1 << 30))
    for kw in (dict(rows=0), dict(rows=(1 << 24) + 1), dict(groups=0), dict(groups=1025), dict(width=0), dict(width=32769),
               dict(y=NULL), dict(y=NULL, h=far, gate=FAKE), dict(y=NULL, h=far, post=FAKE), dict(y=ODD), dict(y=P(0x1001), yt=1),
               dict(yt=2), dict(ys=127), dict(ys=1 << 33), dict(gate=ODD), dict(gate=far, gt=2), dict(gate=far, gs=100),
               dict(scale=float("inf")), dict(h=P(0x2002)), dict(h=far, ht=3), dict(post=ODD), dict(weight=ODD), dict(eps=0.0),
               dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(out=NULL), dict(out=P((1 << 40) + 1)),
               dict(out=FAKE), dict(out=P(0x1000 + 3 * 512 + 508)), dict(gate=FAR), dict(h=FAR), dict(h=FAKE),
               dict(h=far, gate=P((1 << 40) + (1 << 30) + 256)), dict(post=FAR), dict(weight=P((1 << 40) + 1020)),
               dict(h=far, weight=far), dict(h=far, post=P((1 << 40) + (1 << 30) + 2044))):
        assert go(**kw) == w12.W12_EINVAL, kw


def test_binding_refuses(w12):
    import torch
    y = torch.zeros(2, 8)
    with pytest.raises((TypeError, ValueError)):
        w12.w12_norm(y)  # on the CPU
    with pytest.raises(TypeError):
        w12.w12_norm(None)
    with pytest.raises(ValueError):
        w12.w12_norm(y, groups=3)
    with pytest.raises(ValueError):
        w12.w12_norm(None, h=y, gate=y)
    with pytest.raises((TypeError, ValueError)):
        w12.DeltaCache(*[torch.zeros(1)] * 6, key_heads=1)
