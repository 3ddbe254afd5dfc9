"""GPU parity of w12_norm (through the C ABI) against the 64-bit oracle."""
import numpy as np
import pytest

from oracle import delta as D

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6


@pytest.fixture(scope="module")
def w12():
    import torch
    import w12_weight_streaming_amd as w
    assert torch.cuda.is_available()
    w.lib()
    return w


def f64(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def make(rows, groups, width, y="f32", gate=None, h=None, post=False, weight=True, seed=0, pad=0):
    import torch
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    wide = groups * width
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}
    a = dict(y=None, gate=None, h=None, post_weight=None, weight=None)
    if y:
        a["y"] = (n(rows, wide + pad) * torch.exp(n(rows, 1))).to(dt[y])[:, :wide]
    if gate:
        a["gate"] = (3 * n(rows, 2 * wide + pad)).to(dt[gate])[:, wide:2 * wide]
    if h:
        a["h"] = (2 * n(rows, wide)).to(dt[h])
    if post:
        a["post_weight"] = n(width)
    if weight:
        a["weight"] = n(width)
    return a


def check(w12, a, groups, scale=0.75, eps=EPS, **kw):
    import torch
    first = a["y"] if a["y"] is not None else a["h"]
    rows, wide = first.shape
    width = wide // groups
    shape = (rows, groups, width)
    h0 = f64(a["h"])
    keep = {k: v.clone() for k, v in a.items() if v is not None and k != "h"}
    out = w12.w12_norm(groups=groups, scale=scale, eps=eps, **a, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(a[k].view(torch.int16 if v.dtype == torch.bfloat16 else torch.int32) if a[k].is_contiguous() else a[k], v.view(torch.int16 if v.dtype == torch.bfloat16 else torch.int32) if v.is_contiguous() and a[k].is_contiguous() else v) for k, v in keep.items())
    if a["y"] is not None:
        t, err = D.norm_before(f64(a["y"]).reshape(shape), f64(a["post_weight"]), None if a["gate"] is None else f64(a["gate"]).reshape(shape), eps)
    if a["h"] is not None:
        got = f64(a["h"]).reshape(shape)
        if a["y"] is None:
            assert np.array_equal(f64(a["h"]), h0)
        else:
            want = h0.reshape(shape) + np.float32(scale).astype(np.float64) * t
            half = D.BF16 if a["h"].dtype == torch.bfloat16 else D.U
            tol = abs(scale) * err + 3 * D.U * (np.abs(h0.reshape(shape)) + abs(scale) * np.abs(t))
            assert (np.abs(got - want) <= tol + half * (np.abs(want) + tol)).all()
        t, err = got, 0  # the norm is of what the residual holds
    if a["weight"] is not None:
        u = D.rms(t, f64(a["weight"]), eps)
        size = np.abs(f64(a["weight"])) / np.sqrt((t * t).mean(-1, keepdims=True) + eps)
        # an error of one value, and what all of them do to the mean
        share = np.sqrt((np.broadcast_to(err, t.shape) ** 2).mean(-1, keepdims=True) / ((t * t).mean(-1, keepdims=True) + eps))
        err = size * err + np.abs(u) * (share + (width + 12) * D.U)
        t = u
    got = f64(out).reshape(shape)
    assert (np.abs(got - t) <= 1.01 * err + D.BF16 * (np.abs(t) + 1.01 * err) + 1e-38).all()
    return out


WIDTHS = [1, 7, 8, 64, 65, 96, 128, 200, 256, 500, 512, 520, 1000, 2048, 2056, 4099, 5120, 8200, 17408, 32768]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("kind", ["first", "residual", "around", "gated", "gate"])
def test_norm_widths(w12, width, kind):
    rows = 5 if width > 2000 else 37
    a = {"first": dict(y=None, h="bf16"), "residual": dict(y="bf16", h="f32"), "around": dict(y="f32", h="bf16", post=True),
         "gated": dict(y="bf16", gate="f32", post=True, weight=False), "gate": dict(y="f32", gate="bf16", weight=False)}[kind]
    check(w12, make(rows, 1, width, seed=width, **a), 1)


@pytest.mark.parametrize("groups,width", [(48, 128), (3, 64), (5, 96), (2, 40), (7, 33), (2, 1024), (3, 5000), (1024, 8)])
@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [0, 3, 32])
def test_norm_groups_and_strides(w12, groups, width, y, pad):
    check(w12, make(9, groups, width, y=y, gate="bf16" if pad else "f32", post=True, weight=False, seed=pad, pad=pad), groups)
    check(w12, make(4, groups, width, y=y, gate="bf16", h=y, post=True, seed=pad + 1, pad=pad), groups)


@pytest.mark.parametrize("rows", [1, 2, 3, 63, 64, 65, 512, 5000])
@pytest.mark.parametrize("width", [128, 1000])
def test_norm_rows(w12, rows, width):
    check(w12, make(rows, 1, width, y="bf16", h="f32", seed=rows), 1)


@pytest.mark.parametrize("h", ["f32", "bf16"])
def test_norm_without_weights(w12, h):
    """h alone rounded to bf16; y alone rounded to bf16."""
    check(w12, make(6, 1, 300, y="f32", h=h, weight=False), 1)
    check(w12, make(6, 1, 300, y="f32", weight=False), 1)
    check(w12, make(6, 1, 304, y=None, h=h, weight=False), 1)


@pytest.mark.parametrize("scale", [0.0, 1.0, -2.5, 1e-3])
def test_norm_scales(w12, scale):
    check(w12, make(6, 1, 640, y="f32", h="f32"), 1, scale=scale)


def test_norm_zero_rows_and_large_gates(w12):
    import torch
    a = make(6, 2, 128, y="f32", gate="f32", post=True, weight=False)
    a["y"][2].zero_()
    a["gate"][3].fill_(-200.0)
    a["gate"][4].fill_(200.0)
    out = check(w12, a, 2)
    assert not out[2].any() and torch.isfinite(out).all()


@pytest.mark.parametrize("width", [128, 5120])
def test_norm_rows_that_are_no_numbers(w12, width):
    """They stay with their own row and group."""
    import torch
    a, b = make(7, 2, width, y="f32", h="f32", post=True, seed=3), make(7, 2, width, y="f32", h="f32", post=True, seed=3)
    b["y"][2, width + 3] = float("nan")
    b["y"][5, 4] = float("inf")
    x, y = (w12.w12_norm(groups=2, **t).view(7, 2, width) for t in (a, b))
    assert torch.isnan(y[2, 1]).all() and not torch.isfinite(y[5, 0]).all()
    y[2, 1], y[5, 0] = x[2, 1], x[5, 0]
    assert torch.equal(x, y)


def test_norm_streams_and_graphs(w12):
    import torch
    a = make(33, 1, 5120, y="bf16", post=True, gate="bf16", weight=False)
    want = w12.w12_norm(**a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.default_stream())
    with torch.cuda.stream(s):
        got = w12.w12_norm(**a)
    s.synchronize()
    assert torch.equal(want, got)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w12.w12_norm(out=out, **a)
    for _ in range(4):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, out)
        out.float().sum().item()


def test_norm_refusals(w12):
    import torch
    a = make(6, 1, 64, y="f32", h="f32")
    for kw in (dict(h=a["h"].t()), dict(h=a["h"][:, :32]), dict(h=a["h"][:3]), dict(h=a["h"].cpu()), dict(h=a["h"].half()),
               dict(y=a["y"].t()), dict(y=a["y"][:1].expand(6, -1)), dict(y=a["y"].double()), dict(weight=a["weight"][:5]),
               dict(weight=a["weight"].bfloat16()), dict(post_weight=a["weight"].cpu()), dict(gate=a["y"][:, :32]), dict(groups=0),
               dict(out=torch.zeros(5, dtype=torch.bfloat16, device=DEV)), dict(out=torch.zeros(6, 64, device=DEV))):
        with pytest.raises((TypeError, ValueError)):
            w12.w12_norm(**{**a, **kw})
    same = torch.zeros(6, 64, dtype=torch.bfloat16, device=DEV)
    for kw in (dict(y=same, out=same), dict(y=same, h=same), dict(h=same, out=same), dict(eps=0.0), dict(scale=float("nan"))):
        with pytest.raises(w12.W12Error):
            w12.w12_norm(**{**a, **kw})


def test_norm_past_32_bits(w12):
    """More than 2^31 values, and bytes past 2^32 in every array."""
    import torch
    rows, wide = 140000, 16384
    y = torch.empty(rows, wide, dtype=torch.bfloat16, device=DEV).fill_(1.5)
    y[-1] = 3.0
    y[-2, ::2] = 0
    out = w12.w12_norm(y, post_weight=torch.full((128,), 2.0, device=DEV), groups=128)
    assert (out[::1000] == 2).all() and (out[-1] == 2).all()
    assert (out[-2, ::2] == 0).all() and (out[-2, 1::2] == 2 * 2 ** 0.5).logical_or((out[-2, 1::2].float() - 2.828).abs() < 0.02).all()
