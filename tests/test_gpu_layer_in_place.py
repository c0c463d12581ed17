"""GPU tests of calls whose output is one of the inputs (the residual of a projection, a norm's x), bit for bit against
the same call out of place, and of 8-bit blocks that are not numbers."""
from __future__ import annotations

import math

import pytest

from tests.gpu_util import log
from tests.linear_plans import plan_of
from tests.test_gpu_linear import _draw

pytestmark = pytest.mark.gpu


# up to 16 rows; each tile; split sums; columns in two kernels
@pytest.mark.parametrize("m,k,n", [(5, 72, 33), (16, 2048, 515), (64, 2048, 515), (1000, 64, 1000), (1157, 208, 10024),
                                   (3859, 250, 4867), (8305, 3776, 480)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_projection_onto_its_residual(ssd, m, k, n, dtype):
    import torch
    log(f"[in place] {m}x{k}x{n} {dtype} {plan_of(ssd, 'fwd', dtype, m, k, n) if m > 16 else ''}")
    x, w, b, r, _ = _draw(m, k, n, dtype, 21)
    for act in ("none", "gelu"):
        want, _ = ssd.ssd_linear(x, w, bias=b, act=act, residual=r)
        got = r.clone()
        y, _ = ssd.ssd_linear(x, w, bias=b, act=act, residual=got, y=got)
        torch.cuda.synchronize()
        assert y is got and torch.equal(got, want)


@pytest.mark.parametrize("m,k,n", [(5, 96, 33), (700, 2048, 772), (3859, 256, 4867)])
def test_eight_bit_projection_onto_its_residual(ssd, m, k, n):
    import torch
    x, w, _, r, _ = _draw(m, k, n, "bf16", 22)
    q, s = ssd.ssd_mx_quantize(x)
    wq, ws = ssd.ssd_mx_quantize(w)
    want = ssd.ssd_linear_mx(q, s, wq, ws, residual=r)
    got = r.clone()
    ssd.ssd_linear_mx(q, s, wq, ws, residual=got, y=got)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("rows,dim,groups", [(3, 333, 1), (7, 8192, 1), (2000, 2048, 8), (2, 40000, 1), (1, 65536, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_onto_its_input(ssd, rows, dim, groups, dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(dim)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, r = (torch.randn(rows, dim, device="cuda", generator=g).to(t) for _ in range(2))
    w = torch.rand(dim, device="cuda", generator=g) + 0.5
    want, h, _ = ssd.ssd_rms_norm(x, w, 1e-5, residual=r, groups=groups)
    got, res = x.clone(), r.clone()
    ssd.ssd_rms_norm(got, w, 1e-5, residual=res, residual_out=res, groups=groups, y=got)
    alone, _, _ = ssd.ssd_rms_norm(x, w, 1e-5, groups=groups)
    same = x.clone()
    ssd.ssd_rms_norm(same, w, 1e-5, groups=groups, y=same)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(res, h) and torch.equal(same, alone)


@pytest.mark.parametrize("m,k,n", [(1, 32, 5), (9, 416, 130), (300, 416, 900), (4000, 416, 2100)])
def test_eight_bit_blocks_that_are_not_numbers(ssd, m, k, n):
    """A NaN or an infinity makes its block, and so its row (or column) of the product, NaN, and nothing else."""
    import torch
    x, w, _, _, _ = _draw(m, k, n, "bf16", 24)
    clean = ssd.ssd_linear_mx(*ssd.ssd_mx_quantize(x), *ssd.ssd_mx_quantize(w))
    rows, cols = torch.ones(m, dtype=torch.bool, device="cuda"), torch.ones(n, dtype=torch.bool, device="cuda")
    for i, v in ((m // 2, math.nan), (m - 1, math.inf)):
        x[i, (37 * i) % k] = v
        rows[i] = False
    w[n // 3, k - 1] = -math.inf
    cols[n // 3] = False
    y = ssd.ssd_linear_mx(*ssd.ssd_mx_quantize(x), *ssd.ssd_mx_quantize(w))
    torch.cuda.synchronize()
    assert torch.equal(y[rows][:, cols], clean[rows][:, cols])
    assert bool(torch.isnan(y[~rows]).all()) and bool(torch.isnan(y[:, ~cols]).all())
