"""GPU tests of the projections at the sizes that take the larger tiles (tests/linear_plans.py), dense, against the
formulas in 64 bits, and of dz and the bias's gradient at the sizes that take each of their kernels. Tolerances: those
of tests/test_gpu_linear.py, which hold for any size."""
from __future__ import annotations

import math

import pytest

from tests.gpu_util import log
from tests.linear_plans import BACKWARD, EIGHT_BITS, FORWARD, plan_of
from tests.test_gpu_linear import HALF, U32, _backward, _behind, _draw, _forward, _slope, _t, test_linear_mx as _mx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,m,k,n,tile,split,rest", FORWARD)
def test_forward(ssd, dtype, m, k, n, tile, split, rest):
    assert plan_of(ssd, "fwd", dtype, m, k, n) == (tile, split, rest)
    log(f"[tiles] {m}x{k}x{n} {dtype} {tile} split {split} rest {rest}")
    _forward(ssd, m, k, n, dtype, "none", False, True, seed=11)
    _forward(ssd, m, k, n, dtype, "gelu", True, True, seed=12)
    _forward(ssd, m, k, n, dtype, "silu", True, False, seed=13)


@pytest.mark.parametrize("m,k,n,tile,split,rest", EIGHT_BITS)
def test_eight_bits(ssd, m, k, n, tile, split, rest):
    assert plan_of(ssd, "mx", "bf16", m, k, n) == (tile, split, rest)
    _mx(ssd, m, k, n)


@pytest.mark.parametrize("dtype,m,k,n,dx,dw", BACKWARD)
def test_backward(ssd, dtype, m, k, n, dx, dw):
    assert dx is None or plan_of(ssd, "dx", dtype, m, k, n) == dx
    assert dw is None or plan_of(ssd, "dw", dtype, m, k, n) == dw
    log(f"[tiles] backward {m}x{k}x{n} {dtype} dx {dx} dw {dw}")
    _backward(ssd, m, k, n, dtype, "silu", seed=14)
    _backward(ssd, m, k, n, dtype, "none", seed=15)


# shares of 64 rows, from 16 wavefronts (fewer than 1024 work-groups of 512 columns) and from 4
@pytest.mark.parametrize("m,n", [(16400, 200), (16400, 203), (16400, 2000), (16400, 1999), (70001, 8), (70001, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_dz_and_the_bias_of_many_rows(ssd, m, n, dtype, act):
    import torch
    log(f"[dz] {m}x{n} {dtype} {act}")
    assert ssd.load()._ZN3ssd7dz_rowsEll(m, n) == 64
    dx, _, db, (dy, _, _, pre) = _backward(ssd, m, 24, n, dtype, act, seed=16)
    # each row of dz by itself: a product with w = 1 at (j, 0) gives dz's column j
    j = n - 1
    w = torch.zeros(n, 24, device="cuda", dtype=_t(dtype))
    w[j, 0] = 1.0
    got, _, _ = ssd.ssd_linear_bwd(dy, _draw(m, 24, 1, dtype, 1)[0], w, act=act, preact=pre, want_w=False)
    ref = dy[:, j].double() * (_slope(pre[:, j].double(), act) if act != "none" else 1.0)
    lim = 2 * HALF[dtype] * ref.abs() + 64 * U32 * dy[:, j].double().abs()  # dz and dx are rounded
    assert bool(((got[:, 0].double() - ref).abs() <= lim).all())
    assert float(got[:, 1:].abs().max()) == 0


@pytest.mark.parametrize("m", [17, 300, 9000])
def test_fp32_infinities_stay_in_their_rows(ssd, m):
    """Beyond 16 rows an infinite fp32 operand gives NaN or infinity in its own row (or column) and nothing elsewhere."""
    import torch
    x, w, _, _, _ = _draw(m, 256, 900, "f32", 4)
    clean, _ = ssd.ssd_linear(x, w, act="silu")
    x[3, 17] = math.nan
    x[5, 200] = math.inf
    x[m - 1, 255] = -math.inf
    w[7, 0] = math.inf
    y, _ = ssd.ssd_linear(x, w)
    s, _ = ssd.ssd_linear(x, w, act="silu")
    torch.cuda.synchronize()
    rows, cols = torch.ones(m, dtype=torch.bool, device="cuda"), torch.ones(900, dtype=torch.bool, device="cuda")
    rows[[3, 5, m - 1]] = False
    cols[7] = False
    assert torch.equal(s[rows][:, cols], clean[rows][:, cols])
    assert bool(torch.isnan(y[3]).all()) and not bool(torch.isfinite(y[~rows]).any())
    assert not bool(torch.isfinite(y[:, 7]).any())


@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** 60])
def test_fp32_far_from_one(ssd, scale):
    """The three parts of an fp32 operand keep its 24 bits, but for what lies below 2^-126."""
    import torch
    m, k, n = 300, 264, 200
    x, w, _, _, g = _draw(m, k, n, "f32", 17)
    x = _behind(x * scale, math.nan)
    y, _ = ssd.ssd_linear(x, w)
    z, mag = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
    lost = 2.0 ** -126 * w.double().abs().sum(1)  # of x; w's values lie far above
    assert bool(((y.double() - z).abs() <= (k / 2 + 32) * U32 * mag + lost).all())
