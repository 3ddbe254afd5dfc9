"""Workspaces that the binding takes for its caller: calls of two host threads
on one stream, whose launches may come in any order, never share one. The
library itself is not called: no GPU is needed."""
import threading
from types import SimpleNamespace

import pytest
import torch

import w12_weight_streaming_amd as w12


def in_two_threads(fn):
    """fn(i) in two threads; what they return, or the first exception."""
    got, errors = [None, None], []

    def go(i):
        try:
            got[i] = fn(i)
        except Exception as e:  # noqa: BLE001 - handed to the test
            errors.append(e)
    threads = [threading.Thread(target=go, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    if errors:
        raise errors[0]
    return got


@pytest.fixture
def one_stream(monkeypatch):
    """Tensors of the CPU in place of a GPU's, every thread on stream 0."""
    monkeypatch.setattr(w12, "_get", lambda t, *a, **k: t.data_ptr())
    monkeypatch.setattr(w12, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)


def test_attention_calls_of_two_threads_have_a_workspace_each(one_stream, monkeypatch):
    need, meet = 4096, threading.Barrier(2, timeout=30)
    monkeypatch.setattr(w12, "_attention_workspace_bytes", lambda *a: need)
    used = {}

    def run(index, what, *args):
        assert what == "w12_kv_attention" and args[-1] >= need
        used[threading.get_ident()] = args[-2]
        meet.wait()  # both calls are in progress
    monkeypatch.setattr(w12, "_run", run)
    cache = SimpleNamespace(index=0, head_dim=64, kv_heads=2, _ref=None)
    q, off = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.tensor([0, 3], dtype=torch.int32)
    for _ in range(3):
        used.clear()
        in_two_threads(lambda i: w12.w12_kv_attention(cache, 0, q, off))
        a, b = used.values()
        assert abs(a - b) >= need


@pytest.mark.parametrize("tag", ["gemm", "head", "cert"])
def test_kept_workspaces_belong_to_one_thread(one_stream, tag):
    """The products' workspaces are kept from call to call, for each thread by
    itself; a larger one replaces a smaller one."""
    dev, meet = torch.device("cpu"), threading.Barrier(2, timeout=30)

    def take(i):
        a = w12.workspace(1000, dev, tag)
        assert w12.workspace(500, dev, tag) is a and not a.any()
        meet.wait()
        b = w12.workspace(5000, dev, tag)
        assert b.numel() >= 5000 and w12.workspace(1000, dev, tag) is b
        return a, b
    first, second = in_two_threads(take)
    for a, b in zip(first, second):
        assert abs(a.data_ptr() - b.data_ptr()) >= a.numel()


def test_scratch_is_no_zero_filled_workspace(one_stream, monkeypatch):
    """A workspace that a call leaves dirty must not be one that a later
    product takes for zero-filled; the caller's own memory may be."""
    ran, dev = [], torch.device("cpu")
    monkeypatch.setattr(w12, "_attention_workspace_bytes", lambda *a: 4096)
    monkeypatch.setattr(w12, "_run", lambda index, what, *args: ran.append(args[-2]))
    cache = SimpleNamespace(index=0, head_dim=64, kv_heads=2, _ref=None)
    q, off = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.tensor([0, 3], dtype=torch.int32)
    ints = torch.tensor([-1, 0, 0], dtype=torch.int32)

    def both(ws):
        w12.w12_kv_attention(cache, 0, q, off, ws=ws)
        w12.tree_accept_sampled(off, ints, ints, torch.zeros(3, 8), torch.zeros(3), torch.zeros(1), ws=ws)
    for tag in ("gemm", "head", "cert"):
        kept = w12.workspace(10000, dev, tag)
        for ws in (kept, kept[256:], kept.view(torch.int32)):
            with pytest.raises(ValueError, match="zero-filled"):
                w12.w12_kv_attention(cache, 0, q, off, ws=ws)
            with pytest.raises(ValueError, match="zero-filled"):
                w12.tree_accept_sampled(off, ints, ints, torch.zeros(3, 8), torch.zeros(3), torch.zeros(1), ws=ws)
        w12.workspace(20000, dev, tag)  # replaced: still what its holder may give a product
        with pytest.raises(ValueError, match="zero-filled"):
            w12.w12_kv_attention(cache, 0, q, off, ws=kept)
    assert not ran
    for ws in (torch.empty(10000, dtype=torch.uint8), w12.workspace(10000, dev, "of my own")):
        both(ws)
        assert ran == [ws.data_ptr()] * 2
        ran.clear()
