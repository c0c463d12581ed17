"""GPU tests of the projections from 8-bit integers with scales far from 1: y is finite wherever
xscale wscale sum is, in every form of the product.

Tolerance: the sum rounded to fp32 and one rounding for each scale, 3 * 2^-24 of the value; bias and residual one more each
of the values that they are added to."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
# one row, few rows, tiles, rows of no multiple of 4, sums split over k
SHAPES = [(1, 4096, 40), (8, 2048, 130), (40, 512, 200), (200, 256, 301), (300, 2048, 640), (60, 4096, 200), (840, 16464, 72)]


@pytest.mark.parametrize("rows,k,n", SHAPES)
@pytest.mark.parametrize("xs,ws", [(1e35, 1e-10), (1e-10, 1e35), (1e38 / 127, 1e-12), (3e38, 1e-30), (1e-38, 1e3), (1e3, 1e-38)])
@pytest.mark.parametrize("act,extra", [("none", False), ("none", True), ("silu", True)])
def test_wide_scales(ssd, rows, k, n, xs, ws, act, extra):
    import torch
    g = torch.Generator(device="cuda").manual_seed(rows)
    xq = torch.randint(-127, 128, (rows, k), device="cuda", generator=g, dtype=torch.int8)
    wq = torch.randint(-127, 128, (n, k), device="cuda", generator=g, dtype=torch.int8)
    xscale = xs * (0.5 + 0.5 * torch.rand(rows, device="cuda", generator=g))
    wscale = ws * (0.5 + 0.5 * torch.rand(n, device="cuda", generator=g))
    wscale[0] *= -1                  # any sign
    if rows > 2:
        xq[1], xscale[1] = 0, 3e38   # zero stays zero
        xscale[2] *= 1e-20           # rows of other sizes beside it
    sums = xq.double() @ wq.double().t().contiguous()
    z = sums * xscale.double()[:, None] * wscale.double()
    b = torch.randn(n, device="cuda", generator=g) if extra else None
    r = torch.randn(rows, n, device="cuda", generator=g) if extra else None
    got = ssd.ssd_linear_int(xq, xscale, wq, wscale, bias=b, residual=r, act=act, dtype=torch.float32)
    torch.cuda.synchronize()
    size = z.abs()
    if extra:
        z = z + b.double()
        size = size + b.double().abs()
    ref = torch.nn.functional.silu(z) if act == "silu" else z
    lim = 1.13 * U32 * (3 * size + z.abs()) + (2.0 ** -20 * ref.abs() if act == "silu" else 0)
    if extra:
        ref = ref + r.double()
        lim = lim + U32 * ref.abs()
    assert float(ref.abs().max()) < 3e38
    assert bool(torch.isfinite(got).all())
    assert bool(((got.double() - ref).abs() <= lim + 1e-44).all())
