"""GPU test of the projections' large tiles on tensors of more than 2^31 values: dense operands, and the rows and columns
at both ends, around 2^31 values and in the middle against the formulas in 64 bits. Tolerances: those of
tests/test_gpu_linear.py, which hold for any size."""
from __future__ import annotations

import pytest

from tests.gpu_util import log
from tests.linear_plans import T64, plan_of
from tests.test_gpu_linear import HALF, U32, _act, _slope, _sum_tol

pytestmark = pytest.mark.gpu

M, K, N = (1 << 17) + 3, 512, 16392


@pytest.fixture(autouse=True)
def _free():
    import torch
    yield
    torch.cuda.empty_cache()


def _near(got, ref, mag, k, extra=0.0):
    lim = 1.13 * _sum_tol(k, "bf16") * mag + HALF["bf16"] * ref.abs() + extra
    assert bool(((got.double() - ref).abs() <= lim).all()), float(((got.double() - ref).abs() / lim).max())


def _operands():
    import torch
    g = torch.Generator(device="cuda").manual_seed(31)
    x = torch.empty(M, K, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    w = (torch.randn(N, K, device="cuda", generator=g) * K ** -0.5).bfloat16()
    r = torch.empty(M, N, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    return x, w, r, 0.5 * torch.randn(N, device="cuda", generator=g), g


ROWS = [0, 1, 65535, (1 << 31) // N, (1 << 31) // N + 1, M - 257, M - 1]


def test_forward(ssd):
    import torch
    assert M * N > 1 << 31 and plan_of(ssd, "fwd", "bf16", M, K, N)[0] != T64
    x, w, r, b, _ = _operands()
    log(f"[large tiles] {M}x{K}x{N} {plan_of(ssd, 'fwd', 'bf16', M, K, N)}")
    y, pre = ssd.ssd_linear(x, w, bias=b, act="silu", residual=r, want_preact=True)
    xd = x[ROWS].double()
    z, mag = xd @ w.double().t() + b.double(), xd.abs() @ w.double().abs().t() + b.double().abs()
    _near(pre[ROWS], z, mag, K)
    _near(y[ROWS], _act(z, "silu") + r[ROWS].double(), mag, K, 16 * U32 * z.abs() + 1e-7 + 4 * U32 * r[ROWS].double().abs())


def test_backward(ssd):
    import torch
    assert plan_of(ssd, "dw", "bf16", M, K, N)[0] != T64 and plan_of(ssd, "dx", "bf16", M, K, N)[0] != T64
    x, w, dy, _, g = _operands()
    pre = torch.empty(M, N, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    log(f"[large tiles] backward dx {plan_of(ssd, 'dx', 'bf16', M, K, N)} dw {plan_of(ssd, 'dw', 'bf16', M, K, N)}")
    dx, dw, db = ssd.ssd_linear_bwd(dy, x, w, act="silu", preact=pre, want_bias=True)
    off = HALF["bf16"] + 32 * U32  # dz is rounded, and its slope is fp32
    dz = dy[ROWS].double() * _slope(pre[ROWS].double(), "silu")
    size = dz.abs() + dy[ROWS].double().abs()
    mag = size @ w.double().abs()
    _near(dx[ROWS], dz @ w.double(), mag, N, off * mag)
    cols = [0, 255, 256, N // 2, N - 9, N - 1]
    dz = dy[:, cols].double() * _slope(pre[:, cols].double(), "silu")
    size = (dz.abs() + dy[:, cols].double().abs()).t().contiguous()
    xd = x.double()
    mag = size @ xd.abs()
    _near(dw[cols], dz.t().contiguous() @ xd, mag, M, off * mag)
    # 32 rows a lane and work-group, 33 of 2049 shares, and a few more: under 512 additions
    assert bool(((db[cols].double() - dz.sum(0)).abs() <= (512 + 32) * U32 * size.sum(1)).all())
