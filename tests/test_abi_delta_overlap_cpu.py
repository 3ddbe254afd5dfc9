"""The recurrent layers' entry points refuse outputs that lie over anything
the same call reads, to the last byte, before launching anything. Every array
of these calls lies apart but for the two that are named. No compute call is
made here."""
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


HK, HV, KD, VD, ROWS, SEQS = 4, 8, 64, 128, 6, 3
LAYERS, SLOTS, STEP = 2, 4, 96
KV = HK * KD + HV * VD
C = KV + HK * KD
CACHE = dict(state=LAYERS * SLOTS * HV * KD * VD * 4, conv=LAYERS * SLOTS * 3 * C * 2, raw=LAYERS * STEP * C * 2,
             kv=LAYERS * STEP * KV * 2, gates=LAYERS * STEP * 2 * HV * 4, delta=LAYERS * STEP * HV * VD * 4)
AT = {n: (i + 1) << 32 for i, n in enumerate([*CACHE, "slot", "row_off", "parent", "qkv", "ba", "conv_weight", "conv_bias",
                                              "a_log", "dt_bias", "q", "out", "accept_len", "path", "kept"])}  # never dereferenced
STEP_READS = dict(slot=SEQS * 4, row_off=(SEQS + 1) * 4, parent=ROWS * 4)


def meet(written, written_bytes, read, read_bytes):
    """Places of `read` whose first or last 16 bytes (4, if it has no more) lie in `written`, and inside it."""
    step = 16 if min(read_bytes, written_bytes) >= 16 else 4
    return [written + written_bytes - step, written - (read_bytes - step) // 16 * 16, written + (written_bytes - step) // 32 * 16]


def cache(w12):
    return w12.W12DeltaCache(LAYERS, SLOTS, STEP, HK, HV, KD, VD, 4, *(AT[n] for n in CACHE))


def refused(w12, call, base, written, reads):
    """Each array that is read, moved over each that is written."""
    for w, wb in written.items():
        for r, rb in reads.items():
            for at in meet(base[w], wb, base[r], rb):
                assert at + rb > base[w] and at < base[w] + wb
                assert call({**base, r: at}) == w12.W12_EINVAL, (w, r, hex(at))


def append(w12):
    L, d = w12.lib(), cache(w12)

    def call(a):
        return L.w12_delta_append(ctypes.byref(d), 0, SEQS, a["slot"], a["row_off"], ROWS, a["parent"], a["qkv"], C, a["ba"], 2 * HV, 0,
                                  a["conv_weight"], a["conv_bias"], a["a_log"], a["dt_bias"], a["q"], None)
    return call, dict(STEP_READS, qkv=ROWS * C * 4, ba=ROWS * 2 * HV * 4, conv_weight=C * 16, conv_bias=C * 4, a_log=HV * 4, dt_bias=HV * 4)


def test_append_outputs_over_what_it_reads(w12):
    call, reads = append(w12)
    refused(w12, call, AT, dict(q=ROWS * HK * KD * 2), reads)


def test_append_staged_rows_over_what_it_reads(w12):
    call, reads = append(w12)
    refused(w12, call, AT, {n: CACHE[n] for n in ("raw", "kv", "gates")}, reads)


def rule(w12, keep):
    L, d = w12.lib(), cache(w12)

    def call(a):
        return L.w12_delta_rule(ctypes.byref(d), 0, SEQS, a["slot"], a["row_off"], ROWS, 0 if keep else a["parent"], a["q"], 0.1, keep,
                                a["out"], None)
    reads = dict(STEP_READS, q=ROWS * HK * KD * 2)
    if keep:
        del reads["parent"]
    return call, reads


@pytest.mark.parametrize("keep", [0, 1])
def test_rule_outputs_over_what_it_reads(w12, keep):
    call, reads = rule(w12, keep)
    refused(w12, call, AT, dict(out=ROWS * HV * VD * 2), reads)


@pytest.mark.parametrize("keep", [0, 1])
def test_rule_kept_arrays_over_what_it_reads(w12, keep):
    """The deltas, or the state and the window that a call with keep moves on."""
    call, reads = rule(w12, keep)
    refused(w12, call, AT, {n: CACHE[n] for n in (("state", "conv") if keep else ("delta",))}, reads)


def commit(w12):
    L, d = w12.lib(), cache(w12)

    def call(a):
        return L.w12_delta_commit(ctypes.byref(d), SEQS, a["slot"], a["row_off"], ROWS, a["accept_len"], a["path"], a["kept"], None)
    return call, dict(slot=SEQS * 4, row_off=(SEQS + 1) * 4, accept_len=SEQS * 4, path=ROWS * 4)


def test_commit_counts_over_what_it_reads(w12):
    call, reads = commit(w12)
    refused(w12, call, AT, dict(kept=SEQS * 4), reads)


def test_commit_states_over_what_it_reads(w12):
    call, reads = commit(w12)
    refused(w12, call, AT, {n: CACHE[n] for n in ("state", "conv")}, reads)


@pytest.mark.parametrize("off", [1, 2, 3])
def test_misaligned_step_arrays(w12, off):
    """The arrays of 32-bit numbers, as the header's conventions say."""
    for make, names in ((append(w12), STEP_READS), (rule(w12, 0), STEP_READS), (rule(w12, 1), ("slot", "row_off")),
                        (commit(w12), ("slot", "row_off", "accept_len", "path", "kept"))):
        for n in names:
            assert make[0]({**AT, n: AT[n] + off}) == w12.W12_EINVAL, n
