"""GPU tests of the projections from 8-bit integers whose sums are split over k: as exact as those that are not."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

# tiles of 64, 128, 192 and 256 columns, with rows of multiples of 4 and not
SHAPES = [(60, 4096, 200), (60, 4096, 201), (840, 16464, 4608), (839, 16464, 4607), (341, 8448, 11536), (8305, 7552, 480), (33, 131072, 24)]


def _codes(rows, k, n):
    """Products of one sign in the first half of k and of the other in the second: large parts, small sums."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(k)
    xq = torch.randint(60, 128, (rows, k), device="cuda", generator=g, dtype=torch.int8)
    half = torch.randint(60, 128, (n, k // 2), device="cuda", generator=g, dtype=torch.int8)
    xq[:, k // 2:] = xq[:, :k // 2]
    wq = torch.cat([half, -half], 1)
    at = torch.randint(0, k, (n, 8), device="cuda", generator=g)
    wq.scatter_(1, at, torch.randint(-127, 128, (n, 8), device="cuda", generator=g, dtype=torch.int8))
    return xq, wq


@pytest.mark.parametrize("rows,k,n", SHAPES)
def test_split_sums_are_exact(ssd, rows, k, n):
    """Scales of 1: the sums themselves, below 2^24, bit for bit. And scales with which a part alone would
    overflow: the sum's value, 3 roundings off at most."""
    import torch
    assert ssd.ssd_linear_int_workspace_bytes(rows, k, n) > 0   # split
    xq, wq = _codes(rows, k, n)
    want = xq.double() @ wq.double().t().contiguous()
    assert float(want.abs().max()) < 2 ** 24
    one = torch.ones(max(rows, n), device="cuda")
    got = ssd.ssd_linear_int(xq, one[:rows], wq, one[:n], dtype=torch.float32)
    big = ssd.ssd_linear_int(xq, one[:rows] * 1e16, wq, one[:n] * 1e16, dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(got.double(), want)
    ref = want * float(torch.tensor(1e16)) ** 2
    assert bool(((big.double() - ref).abs() <= 3 * 2.0 ** -24 * ref.abs()).all())


def test_split_sums_of_one_row_scale_each(ssd):
    """Every row and column with a scale of its own, the bias, activation and residual behind them."""
    import torch
    for rows, k, n in ((60, 4096, 200), (839, 16464, 4607)):
        xq, wq = _codes(rows, k, n)
        xs, ws = 1e-3 * (1 + torch.arange(rows, device="cuda")), 1e-3 * (1 + torch.arange(n, device="cuda") % 7)
        b, r = torch.randn(n, device="cuda"), torch.randn(rows, n, device="cuda")
        y = ssd.ssd_linear_int(xq, xs, wq, ws, bias=b, act="silu", residual=r, dtype=torch.float32)
        torch.cuda.synchronize()
        z = (xq.double() @ wq.double().t().contiguous()) * xs.double()[:, None] * ws.double()
        size, z = z.abs() + b.double().abs(), z + b.double()
        ref = torch.nn.functional.silu(z)
        lim = 1.13 * 2.0 ** -24 * (3 * size + z.abs()) + 2.0 ** -20 * ref.abs() + 2.0 ** -24 * (ref + r.double()).abs()
        assert bool(((y.double() - ref - r.double()).abs() <= lim + 1e-37).all())
