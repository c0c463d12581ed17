"""GPU tests of SiLU and GELU far from zero, where they are small beside 1 (ssd_linear's epilogue, ssd_linear_bwd's
slopes), against the formulas in 64 bits and relative to the value itself.

Tolerances, fixed before the first run. With u = z / sqrt 2 rounded (relative 2^-23), erfc(u) moves by up to
2 u^2 2^-23 = z^2 2^-23 of itself; erfc and the products are a few units more: (z^2 + 24) 2^-23 in fp32. In bf16 the
exponential's argument, up to 122 at z = -13, is off by 3 roundings (2 z^2 2^-24) and the polynomial by 2^-13, beside
half a step of 2^-8: 2^-8 + 2^-12 + z^2 2^-23. SiLU: an argument of |z| in an exponential, (2 |z| + 24) 2^-23. Values
below 2^-118 in magnitude may come out as zero: so far the exponentials of fp32 go."""
from __future__ import annotations

import math

import pytest

from tests.gpu_util import log
from tests.linear_plans import plan_of
from tests.test_gpu_linear import _act, _slope, _t

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -23


def _points(dtype, act):
    import torch
    z = torch.linspace(-13.0, 13.0, 4001, device="cuda") if act == "gelu" else torch.linspace(-80.0, 80.0, 4001, device="cuda")
    return z.to(_t(dtype))


def _rel(z, dtype, act):
    grow = z * z if act == "gelu" else 2 * z.abs()
    return (grow + 24) * STEP + (2.0 ** -8 + 2.0 ** -12 if dtype == "bf16" else 2.0 ** -24)


# up to 16 rows; a tile; a split sum, joined behind the products
@pytest.mark.parametrize("rows,k,n,split", [(16, 8, 1, False), (4001, 8, 3, False), (64, 2048, 5, True)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_values(ssd, rows, k, n, split, dtype, act):
    import torch
    log(f"[tails] {rows}x{k}x{n} {dtype} {act}")
    if rows > 16:
        assert plan_of(ssd, "fwd", dtype, rows, k, n)[1] == split
    points = _points(dtype, act)
    w = torch.zeros(n, k, device="cuda", dtype=points.dtype)
    w[:, k // 2] = 1.0
    for z in points.split(rows):
        x = torch.zeros(rows, k, device="cuda", dtype=points.dtype)
        x[:len(z), k // 2] = z
        y, pre = ssd.ssd_linear(x, w, act=act, want_preact=True)
        assert torch.equal(pre[:len(z), 0], z)
        ref = _act(z.double(), act)
        keep = ref.abs() >= 2.0 ** -118
        err = (y[:len(z)].double() - ref[:, None]).abs()
        bad = keep[:, None] & ~(err <= (_rel(z.double(), dtype, act) * ref.abs())[:, None])
        assert not bool(bad.any()), (z[bad.any(1)][:4].tolist(), float((err / ref.abs()[:, None])[bad].max()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_slopes(ssd, dtype, act):
    """The bias's gradient of one row of ones is the slope, in fp32: relative to its two terms, which cancel where it
    is zero."""
    import torch
    log(f"[tails] slopes {dtype} {act}")
    z = _points(dtype, act)
    one = torch.ones_like(z)[None]
    x, w = torch.zeros(1, 8, device="cuda", dtype=z.dtype), torch.zeros(len(z), 8, device="cuda", dtype=z.dtype)
    _, _, db = ssd.ssd_linear_bwd(one, x, w, act=act, preact=z[None], want_x=False, want_w=False, want_bias=True)
    d = z.double()
    if act == "gelu":
        size = 0.5 * torch.erfc(-d / math.sqrt(2))
        terms = size + d.abs() * torch.exp(-d * d / 2) / math.sqrt(2 * math.pi)
    else:
        size = torch.sigmoid(d)
        terms = size * (1 + d.abs() * torch.sigmoid(-d))
    ref = _slope(d, act)
    grow = d * d if act == "gelu" else 2 * d.abs()
    lim = (2 * grow + 32) * STEP * terms + (2.0 ** -12 * size if dtype == "bf16" and act == "gelu" else 0)
    bad = (ref.abs() >= 2.0 ** -118) & ~((db.double() - ref).abs() <= lim)
    assert not bool(bad.any()), (z[bad][:4].tolist(), float(((db.double() - ref).abs() / ref.abs())[bad].max()))
