"""GPU tests of the projections from 8-bit integers (ssd_int_quantize, ssd_linear_int) against the definition in 64 bits.

Tolerances, fixed before the first run. The codes and scales are exact: each is the definition's. The sum of the codes'
products is exact in 32 bits; rounding it to fp32, two scales, the bias and the residual are one rounding each (2^-24 of
the term), and a sum that is split is rounded once for each part (of magnitude up to the sum of magnitudes, 32 parts: their
sum of roundings is at most 2^-24 of the magnitudes for the parts and 32 * 2^-24 for adding them). Activations: slope at most
1.13, and 2^-20 of the value (fp32) or 2^-12 (bf16, before its rounding)."""
from __future__ import annotations

import numpy as np
import pytest

from tests.gpu_util import log

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U32 = 2.0 ** -24


def _t(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _codes(x):
    x = x.float().cpu().numpy().astype(np.float32)
    top = np.abs(x).max(-1)
    scale = (top * np.float32(1 / 127)).astype(np.float32)
    q = np.rint(x.astype(np.float64) / np.where(scale > 0, scale, 1).astype(np.float64)[..., None])
    return np.where(scale[..., None] > 0, np.clip(q, -127, 127), 0), scale


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,dim", [(1, 1), (1, 2048), (7, 33), (3, 8200), (1500, 768), (1030, 1001), (2, 40000), (1, 70001), (1030, 4096), (5, 16)])
def test_codes_are_exact(ssd, rows, dim, dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(rows * dim)
    x = torch.randn(rows, dim, device="cuda", generator=g)
    x *= torch.exp2(60 * torch.rand(rows, 1, device="cuda", generator=g) - 30)
    x = x.to(_t(dtype))
    if rows > 4:
        x[1] = 0
        x[2] = torch.round(x[2].float() / x[2].float().abs().max() * 254).to(x.dtype) / 2   # quotients half way between codes
        x[2, 0] = 127
    q, s = ssd.ssd_int_quantize(x)
    torch.cuda.synchronize()
    want, scale = _codes(x)
    assert np.array_equal(s.cpu().numpy(), scale)
    assert np.array_equal(q.cpu().numpy().astype(np.float64), want)


def test_codes_of_scales_of_few_bits(ssd):
    """The largest value is k 2^-149, and its scale rounded to 1, 2, 3 of those: a quotient of up to 190 stays 127."""
    import torch
    tops = np.array([1, 63, 64, 100, 190, 191, 317, 318, 400, 5000], np.int64)
    bits = np.stack([tops, tops // 2, np.zeros_like(tops)], 1).astype(np.int32)
    bits[:, 1] |= np.int32(-2 ** 31)
    x = torch.from_numpy(bits).cuda().view(torch.float32)
    q, s = ssd.ssd_int_quantize(x)
    torch.cuda.synchronize()
    want, scale = _codes(x)
    assert np.array_equal(s.cpu().numpy(), scale) and np.array_equal(q.cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_codes_of_extreme_rows(ssd, dtype):
    import torch
    x = torch.randn(8, 96, device="cuda").to(_t(dtype))
    x[0, 5], x[1, 6], x[2, 7] = float("nan"), float("inf"), float("-inf")
    x[3] = 0
    x[4] = x[4] * 1e-38
    x[5] = 1e38
    x[6] = 0
    x[6, 3] = 1e-40
    q, s = ssd.ssd_int_quantize(x)
    torch.cuda.synchronize()
    assert bool(torch.isnan(s[:3]).all()) and not bool(q[:3].any())
    assert float(s[3]) == 0 and not bool(q[3].any())
    want, scale = _codes(x[4:])
    assert np.array_equal(s[4:].cpu().numpy(), scale) and np.array_equal(q[4:].cpu().numpy().astype(np.float64), want)
    y = ssd.ssd_linear_int(q, s, q, torch.ones(8, device="cuda"), dtype=torch.float32)
    torch.cuda.synchronize()
    assert bool(torch.isnan(y[:3]).all()) and not bool(y[3].any())


def _act(z, act):
    import torch
    if act == "silu":
        return z * torch.sigmoid(z)
    return z * 0.5 * torch.special.erfc(-z / 2 ** 0.5) if act == "gelu" else z


def _check(ssd, rows, k, n, dtype, act="none", bias=False, residual=False, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + rows)
    xq = torch.randint(-127, 128, (rows, k), device="cuda", generator=g, dtype=torch.int8)
    wq = torch.randint(-127, 128, (n, k), device="cuda", generator=g, dtype=torch.int8)
    xs = torch.rand(rows, device="cuda", generator=g) / 50
    ws = torch.rand(n, device="cuda", generator=g) / (50 * k ** 0.5)
    b = torch.randn(n, device="cuda", generator=g) if bias else None
    r = torch.randn(rows, n, device="cuda", generator=g).to(_t(dtype)) if residual else None
    buf = torch.full((rows * n + 512,), 7.0, device="cuda").to(_t(dtype))
    y = ssd.ssd_linear_int(xq, xs, wq, ws, bias=b, act=act, residual=r, y=buf[:rows * n].view(rows, n))
    again = ssd.ssd_linear_int(xq, xs, wq, ws, bias=b, act=act, residual=r, dtype=_t(dtype))
    torch.cuda.synchronize()
    assert torch.equal(y, again) and bool((buf[rows * n:].float() == 7.0).all())
    sc = xs.double()[:, None] * ws.double()
    z = (xq.double() @ wq.double().t().contiguous()) * sc
    mag = (xq.double().abs() @ wq.double().abs().t().contiguous()) * sc
    size = z.abs()
    if b is not None:
        z, size = z + b.double(), size + b.double().abs()
    ref = _act(z, act)
    lim = 1.13 * U32 * (36 * mag + 6 * size) + (2.0 ** -12 if dtype == "bf16" else 2.0 ** -20) * ref.abs() * (act != "none")
    if r is not None:
        ref = ref + r.double()
        lim = lim + 2 * U32 * (ref.abs() + r.double().abs())
    err = (y.double() - ref).abs()
    assert bool((err <= lim + HALF[dtype] * ref.abs() + 1e-37).all()), (float((err - lim).max()), float(err.max()))


SHAPES = [(1, 16, 1), (1, 2048, 8512), (8, 2048, 8512), (16, 112, 16400), (17, 16, 5), (33, 64, 100), (100, 1008, 515), (300, 2048, 640),
          (64, 16384, 72), (700, 768, 3352), (2, 65536, 33), (1000, 144, 1003), (4096, 512, 1024)]


@pytest.mark.parametrize("rows,k,n", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_products(ssd, rows, k, n, dtype):
    log(f"[linear_int] {rows} {k} {n} {dtype}")
    _check(ssd, rows, k, n, dtype)
    i = SHAPES.index((rows, k, n))
    _check(ssd, rows, k, n, dtype, act=("none", "silu", "gelu")[i % 3], bias=i % 2 == 0, residual=i % 4 < 3, seed=1)


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k,n", [(5, 96, 70), (200, 256, 301), (600, 128, 512)])
def test_epilogues(ssd, act, dtype, rows, k, n):
    for bias in (False, True):
        for residual in (False, True):
            _check(ssd, rows, k, n, dtype, act, bias, residual, seed=2)


T128, T192, T256, T64 = (128, 128), (256, 192), (256, 256), (64, 64)
# (rows, in, out) that take each tile, split and not, alone and with another for the last columns
TILES = [(407, 416, 9624, T128, False, None), (840, 16464, 4608, T128, True, None), (839, 16464, 4607, T128, True, None),
         (8737, 416, 908, T192, False, None), (8737, 416, 907, T192, False, None), (341, 8448, 11536, T192, True, None),
         (1157, 416, 10024, T256, False, None), (1157, 416, 10023, T256, False, None), (8305, 7552, 480, T256, True, None),
         (3899, 448, 5396, T256, False, T128), (3847, 512, 6945, T256, False, T192), (3859, 496, 4868, T256, False, T64),
         (300, 96, 500, T64, False, None), (60, 4096, 200, T64, True, None)]


@pytest.mark.parametrize("rows,k,n,tile,split,rest", TILES)
def test_every_tile(ssd, rows, k, n, tile, split, rest):
    from tests import linear_plans
    assert linear_plans.plan_of(ssd, "mx", "bf16", rows, k, n) == (tile, split, rest)   # by bytes of a row, as 8-bit codes
    log(f"[linear_int] tile {rows} {k} {n}")
    _check(ssd, rows, k, n, "bf16", bias=True, seed=3)
    _check(ssd, rows, k, n, "f32", act="silu", residual=True, seed=3)


def test_largest_sums_are_exact(ssd):
    """in = 131072, every code -127 or 127: sums of 2113929216, next to the end of 32 bits."""
    import torch
    k = 131072
    for rows in (2, 40):
        xq = torch.full((rows, k), 127, device="cuda", dtype=torch.int8)
        wq = torch.full((24, k), 127, device="cuda", dtype=torch.int8)
        wq[1] = -127
        wq[2, ::2] = -127
        y = ssd.ssd_linear_int(xq, torch.ones(rows, device="cuda"), wq, torch.ones(24, device="cuda"), dtype=torch.float32)
        torch.cuda.synchronize()
        want = torch.full((rows, 24), 127.0 * 127 * k, device="cuda")
        want[:, 1], want[:, 2] = -127.0 * 127 * k, 0
        assert torch.equal(y, want)


def test_residual_in_place_and_no_rows(ssd):
    import torch
    xq, xs = ssd.ssd_int_quantize(torch.randn(50, 64, device="cuda"))
    wq, ws = ssd.ssd_int_quantize(torch.randn(40, 64, device="cuda"))
    r = torch.randn(50, 40, device="cuda").bfloat16()
    want = ssd.ssd_linear_int(xq, xs, wq, ws, residual=r)
    got = ssd.ssd_linear_int(xq, xs, wq, ws, residual=r, y=r)
    torch.cuda.synchronize()
    assert got is r and torch.equal(got, want)
    assert ssd.ssd_linear_int(xq[:0], xs[:0], wq, ws).shape == (0, 40)
    q, s = ssd.ssd_int_quantize(torch.empty(0, 64, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0,)


def test_captured_and_replayed(ssd):
    import torch
    x = torch.randn(90, 4096, device="cuda").bfloat16()
    wq, ws = ssd.ssd_int_quantize(torch.randn(130, 4096, device="cuda"))
    def run():
        return ssd.ssd_linear_int(*ssd.ssd_int_quantize(x), wq, ws, act="silu")
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for r in range(3):
        x.normal_()
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), r
