"""w12_norm over more rows than its grid has workgroups: a workgroup goes on to
further rows. Every row equals, bit for bit, what a call of fewer rows gives
it, and a sample the 64-bit oracle."""
import numpy as np
import pytest

from oracle import delta as D
from test_gpu_norm import DEV, EPS, f64, w12  # noqa: F401

pytestmark = pytest.mark.gpu


def normal(rows, wide, seed):
    """bf16, made a part at a time."""
    import torch
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    out = torch.empty(rows, wide, dtype=torch.bfloat16, device=DEV)
    for part in out.split(max(1, (1 << 28) // wide)):
        part.copy_(torch.randn(part.shape, generator=g, device=DEV))
    return out


@pytest.mark.parametrize("width", [520, 515, 8200], ids=["vector", "scalar", "two pieces"])
def test_wide_groups(w12, width):  # noqa: F811
    """Two sums a row (norm behind and before a block), 2^20 workgroups, rows in the third turn."""
    import torch
    rows = (1 << 21) + 70 if width < 1000 else (1 << 20) + 70
    y = normal(rows, width, 3)
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    post, weight = (torch.randn(width, generator=g, device=DEV) for _ in range(2))
    h = y.roll(1, 0)
    h0 = h[-200:].clone()
    out = w12.w12_norm(y, weight=weight, post_weight=post, h=h, scale=0.5)
    got_h = h[-200:].clone()
    part = (1 << 19) + 3
    for a in range(0, rows, part):
        b = min(a + part, rows)
        again = y[a - 1:b - 1].clone() if a else torch.cat([y[-1:], y[:b - 1]])
        assert torch.equal(out[a:b], w12.w12_norm(y[a:b], weight=weight, post_weight=post, h=again, scale=0.5)), a
        assert torch.equal(again, h[a:b]), a
    t, err = D.norm_before(f64(y[-200:])[:, None], f64(post), None, EPS)
    want = f64(h0)[:, None] + 0.5 * t
    tol = 0.5 * err + 3 * D.U * (np.abs(f64(h0))[:, None] + 0.5 * np.abs(t))
    assert (np.abs(f64(got_h)[:, None] - want) <= tol + D.BF16 * (np.abs(want) + tol)).all()
    u = D.rms(f64(got_h), f64(weight), EPS)
    assert (np.abs(f64(out[-200:]) - u) <= 1.01 * D.BF16 * np.abs(u) + (width + 12) * D.U * np.abs(u)).all()


def test_narrow_groups(w12):  # noqa: F811
    """Groups of one value, 256 a workgroup, 2^22 workgroups: 2^30 groups a turn, and the most rows of a call."""
    import torch
    rows, groups = 1 << 24, 66
    y = normal(rows, groups, 5)
    post = torch.full((1,), 1.5, device=DEV)
    out = w12.w12_norm(y, post_weight=post, groups=groups, eps=0.25)
    for a in range(0, rows, 1 << 22):
        part = slice(a, a + (1 << 22))
        assert torch.equal(out[part], w12.w12_norm(y[part], post_weight=post, groups=groups, eps=0.25)), a
    t, err = D.norm_before(f64(y[-1000:])[:, :, None], f64(post), None, 0.25)
    assert (np.abs(f64(out[-1000:])[:, :, None] - t) <= 1.01 * (err + D.BF16 * np.abs(t))).all()
