"""The recurrent layers' entry points refuse each bad argument by itself, with
every array of the call apart from the others, so that nothing else is wrong
with it. No compute call is made here."""
import ctypes

import pytest

from test_abi_delta_cpu import BAD
from test_abi_delta_overlap_cpu import AT, C, CACHE, HK, HV, KD, LAYERS, ROWS, SEQS, SLOTS, STEP, VD, w12  # noqa: F401

SIZES = dict(layers=LAYERS, slots=SLOTS, step_rows=STEP, key_heads=HK, value_heads=HV, key_dim=KD, value_dim=VD, conv_width=4)


def cache(w12, **kw):  # noqa: F811
    moved = {k: 0 if v == 0 else AT[k] + (v & 15) for k, v in kw.items() if k in CACHE}
    return w12.W12DeltaCache(*{**SIZES, **{n: AT[n] for n in CACHE}, **kw, **moved}.values())


def calls(w12, cache, **kw):  # noqa: F811
    """The calls with these arguments instead of their good ones."""
    a = {**AT, **dict(layer=0, seqs=SEQS, rows=ROWS, qkv_stride=C, ba_stride=2 * HV, kind=0, scale=0.1, keep=0), **kw}
    L, d = w12.lib(), ctypes.byref(cache)
    step = a["seqs"], a["slot"], a["row_off"], a["rows"]
    return dict(
        append=lambda: L.w12_delta_append(d, a["layer"], *step, a["parent"], a["qkv"], a["qkv_stride"], a["ba"], a["ba_stride"], a["kind"],
                                          a["conv_weight"], a["conv_bias"], a["a_log"], a["dt_bias"], a["q"], None),
        rule=lambda: L.w12_delta_rule(d, a["layer"], *step, a["parent"], a["q"], a["scale"], a["keep"], a["out"], None),
        commit=lambda: L.w12_delta_commit(d, *step, a["accept_len"], a["path"], a["kept"], None))


@pytest.mark.parametrize("kw", BAD, ids=str)
def test_bad_caches(w12, kw):  # noqa: F811
    for name, call in calls(w12, cache(w12, **kw)).items():
        assert call() == w12.W12_EINVAL, name


STEPS = [dict(seqs=0), dict(seqs=513), dict(row_off=0), dict(rows=0), dict(rows=STEP + 1)]
APPEND = [dict(layer=-1), dict(layer=LAYERS), dict(qkv=0), dict(qkv=AT["qkv"] + 8), dict(qkv_stride=C - 4), dict(qkv_stride=C + 2),
          dict(qkv_stride=C + 4, kind=1), dict(qkv_stride=1 << 33), dict(qkv_stride=-C), dict(ba=0), dict(ba=AT["ba"] + 2),
          dict(ba=AT["ba"] + 1, kind=1), dict(ba_stride=2 * HV - 1), dict(ba_stride=1 << 33), dict(kind=2), dict(conv_weight=0),
          dict(conv_weight=AT["conv_weight"] + 8), dict(conv_bias=AT["conv_bias"] + 4), dict(a_log=0), dict(a_log=AT["a_log"] + 2),
          dict(dt_bias=0), dict(dt_bias=AT["dt_bias"] + 2), dict(q=0), dict(q=AT["q"] + 8)]
RULE = [dict(layer=-1), dict(layer=LAYERS), dict(q=0), dict(q=AT["q"] + 8), dict(scale=float("nan")), dict(scale=float("inf")), dict(out=0),
        dict(out=AT["out"] + 8), dict(keep=1)]  # keep with parents
COMMIT = [dict(accept_len=0), dict(kept=0)]


@pytest.mark.parametrize("name,kw", [(n, kw) for n, more in (("append", APPEND), ("rule", RULE), ("commit", COMMIT)) for kw in STEPS + more],
                         ids=str)
def test_bad_arguments(w12, name, kw):  # noqa: F811
    assert calls(w12, cache(w12), **kw)[name]() == w12.W12_EINVAL


@pytest.mark.parametrize("name,out", [("append", "q"), ("rule", "out"), ("commit", "kept")])
@pytest.mark.parametrize("over", list(CACHE))
def test_outputs_over_the_cache(w12, name, out, over):  # noqa: F811
    for at in (AT[over], AT[over] + CACHE[over] - 16):
        assert calls(w12, cache(w12), **{out: at})[name]() == w12.W12_EINVAL
