"""GPU tests of the projections (ssd_linear, ssd_linear_mx, ssd_linear_bwd) against the formulas in 64 bits.

Tolerances, fixed before the first run. Products of bf16 (or 8-bit) operands are exact in fp32; a sum over k passes
k / 32 matrix-core accumulations, each off by at most one unit of fp32 of the sum of the terms' magnitudes so far,
and a few partial sums: (k / 16 + 32) 2^-24 of that magnitude. fp32 operands: k / 4 accumulations and rounded
products, (k / 2 + 32) 2^-24. An activation has slope under 1.13 and is itself off by under 16 * 2^-24 of |z| + 1e-7.
8-bit operands: the scaled matrix-core product adds 8 consecutive k in fixed point, 13 bits below the largest of the 8
products (measured: beside 2^16, 2^3 is kept whole and 2^2 lost; products 8 or more apart in k keep 24 bits and more).
Each of the other 7 loses less than 2^-13 of the largest, so a sum is off by under 7 * 2^-13 of the sum of magnitudes.
Where all codes lie in one binade nothing is lost, and the bound above holds: that is tested by itself.
The stored value is off by at most half a step. In the backward with an activation in bf16, dz is an operand of the
products: each of its values is off by half a step, at most HALF of the sum of magnitudes."""
from __future__ import annotations

import math

import pytest

from tests.gpu_util import log

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _t(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _behind(t, fill):
    """t's values at the front of a larger allocation that holds `fill` behind them."""
    import torch
    buf = torch.full((t.numel() + 8192,), fill, device="cuda").to(t.dtype)
    buf[:t.numel()] = t.reshape(-1)
    return buf[:t.numel()].view(t.shape)


def _draw(m, k, n, dtype, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    def r(*s):
        return torch.randn(*s, device="cuda", generator=g)
    x, w = r(m, k).to(_t(dtype)), (r(n, k) * k ** -0.5).to(_t(dtype))
    return _behind(x, math.nan), _behind(w, math.nan), 0.5 * r(n), r(m, n).to(_t(dtype)), g


def _act(z, act):
    import torch
    if act == "silu":
        return z * torch.sigmoid(z)
    return z * 0.5 * torch.erfc(-z / math.sqrt(2)) if act == "gelu" else z


def _slope(z, act):
    import torch
    if act == "silu":
        s = torch.sigmoid(z)
        return s + z * s * torch.sigmoid(-z)
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def _sum_tol(k, dtype):
    return (k / 2 + 32 if dtype == "f32" else k / 16 + 32) * U32


def _check(got, ref, mag, k, dtype, act, what, extra=0.0):
    lim = _sum_tol(k, dtype) * mag * (1.0 if act == "none" else 1.13) + HALF[dtype] * ref.abs() + extra
    err = (got.double() - ref).abs()
    bad = ~(err <= lim)
    assert not bool(bad.any()), (what, int(bad.sum()), float((err / lim).max()))


def _forward(ssd, m, k, n, dtype, act, bias, res, seed=1, data=None):
    import torch
    x, w, b, r, _ = data or _draw(m, k, n, dtype, seed)
    b, r = (b if bias else None), (r if res else None)
    out = torch.full((m * n + 4096,), 7.0, device="cuda").to(_t(dtype))
    y, pre = ssd.ssd_linear(x, w, bias=b, act=act, residual=r, y=out[:m * n].view(m, n), want_preact=True)
    torch.cuda.synchronize()
    assert bool((out[m * n:].float() == 7.0).all()), "written past the end"
    z = x.double() @ w.double().t()
    mag = x.double().abs() @ w.double().abs().t()
    if bias:
        z, mag = z + b.double(), mag + b.double().abs()
    _check(pre, z, mag, k, dtype, "none", "preact")
    ref = _act(z, act)
    extra = 0 if act == "none" else 16 * U32 * z.abs() + 1e-7
    if res:
        ref = ref + r.double()
        extra = extra + 4 * U32 * r.double().abs()
    _check(y, ref, mag, k, dtype, act, "y", extra)
    again, _ = ssd.ssd_linear(x, w, bias=b, act=act, residual=r)
    torch.cuda.synchronize()
    assert torch.equal(again, y)
    return y


SIZES = [(1, 1, 1), (1, 8, 16), (1, 2048, 100), (2, 3, 5), (15, 72, 17), (16, 64, 4), (17, 128, 33), (33, 100, 3),
         (64, 520, 130), (64, 2048, 515), (65, 8, 1), (65, 64, 64), (100, 1003, 257), (127, 96, 129), (128, 256, 128),
         (129, 31, 130), (256, 2048, 256), (300, 4096, 200), (513, 136, 700), (1000, 64, 1000), (2000, 1536, 772)]


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear(ssd, m, k, n, dtype):
    log(f"[linear] {m}x{k}x{n} {dtype}")
    _forward(ssd, m, k, n, dtype, "none", False, False)
    _forward(ssd, m, k, n, dtype, "gelu", True, True)
    _forward(ssd, m, k, n, dtype, "silu", True, False)


@pytest.mark.parametrize("m,k,n", [(4096, 1024, 4360), (8192, 4096, 2048)])
def test_linear_large(ssd, m, k, n):
    log(f"[linear] {m}x{k}x{n} bf16")
    _forward(ssd, m, k, n, "bf16", "silu", True, True)


@pytest.mark.parametrize("dtype,m,k,n", [("bf16", 4096, 512, 4359), ("bf16", 4096, 520, 4364), ("f32", 4096, 100, 3301)])
def test_linear_columns_in_two_kernels(ssd, dtype, m, k, n):
    """Whole rounds of the large tile and a rest of the columns by a smaller one: the rest's offsets in every operand,
    with rows of y that are and are not multiples of 4."""
    log(f"[linear] {m}x{k}x{n} {dtype}")
    _forward(ssd, m, k, n, dtype, "none", False, False)
    _forward(ssd, m, k, n, dtype, "gelu", True, True)


def test_linear_leading_dimensions_and_no_rows(ssd):
    import torch
    x, w, b, _, _ = _draw(24, 64, 48, "bf16", 3)
    y, pre = ssd.ssd_linear(x, w, bias=b)
    y3, _ = ssd.ssd_linear(x.view(2, 3, 4, 64), w, bias=b)
    torch.cuda.synchronize()
    assert pre is None and y3.shape == (2, 3, 4, 48) and torch.equal(y3.view(24, 48), y)
    z, _ = ssd.ssd_linear(x[:0], w)
    assert z.shape == (0, 48)


def test_linear_infinities_stay_in_their_rows(ssd):
    import torch
    for m in (8, 200):
        x, w, _, _, _ = _draw(m, 256, 96, "bf16", 4)
        clean, _ = ssd.ssd_linear(x, w, act="silu")
        x[3, 17] = math.nan
        x[5, 200] = math.inf
        y, _ = ssd.ssd_linear(x, w, act="silu")
        torch.cuda.synchronize()
        keep = [i for i in range(m) if i not in (3, 5)]
        assert torch.equal(y[keep], clean[keep])
        assert bool(torch.isnan(y[3]).all()) and not bool(torch.isfinite(y[5]).all())


@pytest.mark.parametrize("m,k,n", [(1, 32, 1), (3, 96, 20), (16, 2048, 515), (40, 160, 33), (64, 4096, 100), (65, 32, 7),
                                   (100, 224, 130), (129, 128, 300), (700, 2048, 772), (2048, 1024, 2304),
                                   (4096, 512, 4359), (2048, 96, 4100)])
def test_linear_mx(ssd, m, k, n):
    import torch
    log(f"[linear mx] {m}x{k}x{n}")
    x, w, b, r, g = _draw(m, k, n, "bf16", 5)
    # blocks of very different size, so that every scale matters
    x = (x.float() * torch.exp2(16 * torch.rand(m, k // 32, device="cuda", generator=g) - 8).repeat_interleave(32, 1)).bfloat16()
    w = (w.float() * torch.exp2(16 * torch.rand(n, k // 32, device="cuda", generator=g) - 8).repeat_interleave(32, 1)).bfloat16()
    xq, xs = ssd.ssd_mx_quantize(x)
    wq, ws = ssd.ssd_mx_quantize(w)
    xq, wq = (_behind(t.view(torch.uint8), 0x7F).view(torch.float8_e4m3fn) for t in (xq, wq))
    xs, ws = (_behind(t.view(torch.uint8), 255).view(torch.float8_e8m0fnu) for t in (xs, ws))
    torch.cuda.synchronize()
    xv = xq.float().double() * xs.float().double().repeat_interleave(32, 1)
    wv = wq.float().double() * ws.float().double().repeat_interleave(32, 1)
    z, mag = xv @ wv.t(), xv.abs() @ wv.abs().t()
    lost = 7 * 2.0 ** -13
    y = ssd.ssd_linear_mx(xq, xs, wq, ws)
    torch.cuda.synchronize()
    _check(y, z, mag, k, "bf16", "none", "y", lost * mag)
    y = ssd.ssd_linear_mx(xq, xs, wq, ws, bias=b, act="gelu", residual=r)
    torch.cuda.synchronize()
    z, mag = z + b.double(), mag + b.double().abs()
    _check(y, _act(z, "gelu") + r.double(), mag, k, "bf16", "gelu", "y gelu",
           16 * U32 * z.abs() + 4 * U32 * r.double().abs() + 1e-7 + 1.13 * lost * mag)
    # codes of one binade, scales 2^-4 .. 2^4: products of a block differ by less than 4, and nothing is lost
    def narrow(*shape):
        code = torch.randint(0, 256, shape, device="cuda", generator=g) & 0x87 | 0x38
        scale = torch.randint(123, 132, (shape[0], shape[1] // 32), device="cuda", generator=g)
        return code.to(torch.uint8).view(torch.float8_e4m3fn), scale.to(torch.uint8).view(torch.float8_e8m0fnu)
    (xq, xs), (wq, ws) = narrow(m, k), narrow(n, k)
    xv = xq.float().double() * xs.float().double().repeat_interleave(32, 1)
    wv = wq.float().double() * ws.float().double().repeat_interleave(32, 1)
    y = ssd.ssd_linear_mx(xq, xs, wq, ws)
    torch.cuda.synchronize()
    _check(y, xv @ wv.t(), xv.abs() @ wv.abs().t(), k, "bf16", "none", "y narrow")


def _backward(ssd, m, k, n, dtype, act, seed=6):
    import torch
    x, w, _, dy, g = _draw(m, k, n, dtype, seed)
    dy = _behind(dy, math.nan)
    pre = _behind(torch.randn(m, n, device="cuda", generator=g).to(_t(dtype)), math.nan) if act != "none" else None
    dx, dw, db = ssd.ssd_linear_bwd(dy, x, w, act=act, preact=pre, want_bias=True)
    torch.cuda.synchronize()
    dz = dy.double() * (_slope(pre.double(), act) if act != "none" else 1.0)
    unit = 0.0 if act == "none" else HALF["bf16"] if dtype == "bf16" else 0.0
    off = 0.0 if act == "none" else 32 * U32  # the slope in fp32, against its own size of up to 1.13
    mz = dz.abs() + (0 if act == "none" else dy.double().abs())
    for got, ref, mag, depth, what in (
            (dx, dz @ w.double(), mz @ w.double().abs(), n, "dx"),
            (dw, dz.t() @ x.double(), mz.t() @ x.double().abs(), m, "dw")):
        _check(got, ref, mag, depth, dtype, "none", what, (unit + off) * mag)
    lim = (128 * U32 + off) * mz.sum(0) + 1e-30
    assert bool(((db.double() - dz.sum(0)).abs() <= lim).all()), "db"
    again = ssd.ssd_linear_bwd(dy, x, w, act=act, preact=pre, want_bias=True)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dw, db)))
    return dx, dw, db, (dy, x, w, pre)


@pytest.mark.parametrize("m,k,n", [(1, 1, 1), (1, 64, 48), (7, 33, 5), (64, 64, 64), (65, 100, 130), (300, 72, 17),
                                   (513, 520, 264), (2048, 768, 1000), (1000, 2048, 100)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_linear_bwd(ssd, m, k, n, dtype, act):
    log(f"[linear bwd] {m}x{k}x{n} {dtype} {act}")
    _backward(ssd, m, k, n, dtype, act)


def test_linear_bwd_parts(ssd):
    """Each gradient alone has the same bits as all together, and what it does not need may be left out."""
    import torch
    dx, dw, db, (dy, x, w, pre) = _backward(ssd, 200, 136, 72, "bf16", "silu")
    kw = dict(act="silu", preact=pre)
    a = ssd.ssd_linear_bwd(dy, x, w, want_w=False, **kw)
    b = ssd.ssd_linear_bwd(dy, x, w, want_x=False, **kw)
    c = ssd.ssd_linear_bwd(dy, x, w, want_x=False, want_w=False, want_bias=True, **kw)
    torch.cuda.synchronize()
    assert a[1] is None and a[2] is None and torch.equal(a[0], dx)
    assert b[0] is None and torch.equal(b[1], dw) and torch.equal(c[2], db)
    z = ssd.ssd_linear_bwd(dy[:0], x[:0], w, want_bias=True)
    torch.cuda.synchronize()
    assert z[0].shape == (0, 136) and float(z[1].abs().max()) == 0 and float(z[2].abs().max()) == 0


def test_linear_bwd_against_differences(ssd):
    import torch
    m, k, n = 9, 20, 12
    x, w, b, dy, g = _draw(m, k, n, "f32", 8)
    for act in ("silu", "gelu"):
        _, pre = ssd.ssd_linear(x, w, bias=b, act=act, want_preact=True)
        dx, dw, db = ssd.ssd_linear_bwd(dy, x, w, act=act, preact=pre, want_bias=True)
        def loss(xx, ww, bb):
            return float((dy.double() * _act(xx @ ww.t() + bb, act)).sum())
        e = 1e-4  # truncation ~ e^2
        for _ in range(4):
            ux, uw, ub = (torch.randn(*s, device="cuda", generator=g).double() for s in ((m, k), (n, k), (n,)))
            X, W, B = x.double(), w.double(), b.double()
            num = (loss(X + e * ux, W + e * uw, B + e * ub) - loss(X - e * ux, W - e * uw, B - e * ub)) / (2 * e)
            parts = [dx.double() * ux, dw.double() * uw, db.double() * ub]
            assert abs(num - float(sum(p.sum() for p in parts))) <= 1e-5 * float(sum(p.abs().sum() for p in parts))


def test_linear_on_another_stream_and_replayed(ssd):
    """Forward, backward and the 8-bit product: on a side stream, and captured and replayed with new inputs."""
    import torch
    x, w, b, dy, _ = _draw(130, 200, 264, "bf16", 9)
    wq, ws = ssd.ssd_mx_quantize(w[:, :192].contiguous())

    def every(**kw):
        y, pre = ssd.ssd_linear(x, w, bias=b, act="gelu", want_preact=True, **kw)
        g = ssd.ssd_linear_bwd(dy, x, w, act="gelu", preact=pre, want_bias=True, **kw)
        xq, xs = ssd.ssd_mx_quantize(x.view(-1)[:130 * 192].view(130, 192), **kw)
        return (y, pre) + g + (ssd.ssd_linear_mx(xq, xs, wq, ws, **kw),)
    want = every()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = every(stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = every()
    for k in range(3):
        x.copy_(torch.roll(x, 1 + k, 0))
        want = every()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_bwd_rows_of_dz_end_in_zeros(ssd, dtype):
    """dz lies at the workspace's front, its rows at whole 128-byte lines: behind column n there are zeros, and nothing
    of the next row of dy or of what lies behind its last."""
    import torch
    m, k, n = 70, 24, 72
    dy, _, _, pre, g = _draw(m, n, 8, dtype, 5)
    pre = torch.randn(m, n, device="cuda", generator=g).to(_t(dtype))
    pre = _behind(pre, math.nan)
    x, w = (torch.randn(*s, device="cuda", generator=g).to(_t(dtype)) for s in ((m, k), (n, k)))
    ws = torch.full((ssd.ssd_linear_bwd_workspace_bytes(m, k, n, "silu", int(dtype == "bf16")),), 0xff,
                    dtype=torch.uint8, device="cuda")
    assert ws.data_ptr() % 256 == 0
    ssd.ssd_linear_bwd(dy, x, w, act="silu", preact=pre, want_bias=True, workspace=ws)
    ld = (n * dy.element_size() + 127) // 128 * 128
    rows = ws[:m * ld].view(dy.dtype).view(m, -1)
    assert rows.shape[1] > n and torch.count_nonzero(rows[:, n:]) == 0
    ref = dy.double() * _slope(pre.double(), "silu")
    assert torch.all((rows[:, :n].double() - ref).abs() <= HALF[dtype] * ref.abs() + 2.0 ** -18 * dy.double().abs())


@pytest.mark.parametrize("m,k,n", [(1, 7, 1), (3, 65, 17), (5, 129, 3), (16, 7469, 100), (13, 1003, 515), (2, 4097, 33),
                                   (8, 8191, 40), (16, 63, 16), (4, 2050, 48), (7, 64 * 33 + 1, 20)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_of_few_rows_at_any_address(ssd, m, k, n, dtype):
    """Rows of an odd number of values are taken where they are, without a workspace, and a NaN of the row behind
    (or behind the last row) stays out of a row's end."""
    import torch
    log(f"[linear, few rows] {m}x{k}x{n} {dtype}")
    assert ssd.ssd_linear_workspace_bytes(m, k, n, int(dtype == "bf16")) == 0
    _forward(ssd, m, k, n, dtype, "none", False, False)
    _forward(ssd, m, k, n, dtype, "silu", True, True)
    x, w, _, _, _ = _draw(m, k, n, dtype, 9)
    ref, _ = ssd.ssd_linear(x, w)
    if m > 1:
        x[1] = math.nan
        y, _ = ssd.ssd_linear(x, w)
        assert bool(torch.isnan(y[1]).all()) and torch.equal(y[0], ref[0]) and torch.equal(y[2:], ref[2:])
        x[1] = 0
    if n > 1:
        w[1] = math.nan
        y, _ = ssd.ssd_linear(x, w)
        keep = [j for j in range(n) if j != 1]
        rows = [i for i in range(m) if i != 1]
        assert bool(torch.isnan(y[:, 1]).all()) and torch.equal(y[rows][:, keep], ref[rows][:, keep])


@pytest.mark.parametrize("m,k,n", [(1, 768, 16384), (16, 96, 16401), (7, 67, 16417), (13, 33, 20000), (3, 1500, 16385)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_of_few_rows_and_many_columns(ssd, m, k, n, dtype):
    log(f"[linear, few rows, many columns] {m}x{k}x{n} {dtype}")
    _forward(ssd, m, k, n, dtype, "none", False, False)
    _forward(ssd, m, k, n, dtype, "gelu", True, True)


@pytest.mark.parametrize("m,k,n", [(16, 96, 16401), (5, 1024, 16384)])
def test_linear_mx_of_few_rows_and_many_columns(ssd, m, k, n):
    test_linear_mx(ssd, m, k, n)


@pytest.mark.parametrize("dtype,m,k,n", [("f32", 17, 1, 5), ("f32", 20, 3, 40), ("f32", 33, 33, 3), ("f32", 777, 1003, 515),
                                         ("f32", 300, 2050, 260), ("f32", 40, 5001, 70), ("f32", 4096, 101, 3301),
                                         ("f32", 1024, 95, 3100), ("bf16", 17, 2, 5), ("bf16", 65, 66, 64), ("bf16", 100, 390, 100),
                                         ("bf16", 40, 4098, 130), ("bf16", 1000, 1022, 772), ("bf16", 4096, 514, 4364),
                                         ("bf16", 2048, 130, 4100), ("bf16", 3000, 62, 1000)])
def test_linear_of_rows_that_end_inside_16_bytes(ssd, dtype, m, k, n):
    """Rows at multiples of 4 bytes are taken as they are: what lies behind a row's end (the next row, or anything
    behind the last) stays out of it, NaN or not."""
    import torch
    log(f"[linear, ragged rows] {m}x{k}x{n} {dtype}")
    _forward(ssd, m, k, n, dtype, "none", False, False)
    _forward(ssd, m, k, n, dtype, "gelu", True, True)
    x, w, _, _, _ = _draw(m, k, n, dtype, 9)
    ref, _ = ssd.ssd_linear(x, w)
    rows, cols = torch.ones(m, dtype=torch.bool, device="cuda"), torch.ones(n, dtype=torch.bool, device="cuda")
    rows[1::3] = cols[1::2] = False
    x[~rows], w[~cols] = math.nan, math.nan
    y, _ = ssd.ssd_linear(x, w)
    assert torch.equal(y[rows][:, cols], ref[rows][:, cols]) and bool(torch.isnan(y[~rows]).all())
    assert bool(torch.isnan(y[:, ~cols]).all())
