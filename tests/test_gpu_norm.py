"""GPU tests of the norm family (ssd_rms_norm, ssd_rms_norm_mx, ssd_mx_quantize, ssd_rms_norm_bwd) against the
formulas in 64 bits.

Tolerances, fixed before the first run. A stored value is off by at most half a step, HALF[type] relative. The
fp32 arithmetic before it: a row's sum of squares adds at most 64 values per lane, then 6 + 16 partial sums, so
the root's factor is off by under (64 + 22) / 2 + 4 half-steps of fp32, and y by 3 more: 64 * 2^-24 covers it.
In the backward, each term of dh passes under 128 roundings, and a column's sum over the rows under 128
additions at these sizes; errors are relative to the sum of the terms' magnitudes, since the terms can cancel.
"""
from __future__ import annotations

import numpy as np
import pytest

from tests.gpu_util import log

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]
EPS = 1e-5


def _t(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _draw(rows, dim, dtype, rtype, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    def r(*s):
        return torch.randn(*s, device="cuda", generator=g)
    return r(rows, dim).to(_t(dtype)), (2 * r(rows, dim)).to(_t(rtype)), 1 + 0.1 * r(dim)


def _ref(x, res, w, groups):
    import torch
    h = x.double() + (res.double() if res is not None else 0)
    p = h.unflatten(-1, (groups, -1))
    inv = 1 / torch.sqrt((p * p).mean(-1) + EPS)
    return (p * inv[..., None]).flatten(-2) * w.double(), h, inv


def _close(got, ref, half, what):
    err = (got.double() - ref).abs()
    lim = ref.abs() * (half + 64 * U32) + 1e-38
    bad = err > lim
    assert not bool(bad.any()), (what, float((err - lim).max()), float((err / ref.abs().clamp(min=1e-30)).max()))


def _guarded(shape, dtype, seed=0):
    """A tensor of this shape at the front of a larger one, and a check that the rest was left alone."""
    import torch
    n = int(np.prod(shape))
    buf = torch.full((n + 4096,), 7.0, device="cuda").to(dtype)
    def check():
        assert bool((buf[n:].float() == 7.0).all()), "written past the end"
    return buf[:n].view(shape), check


SHAPES = [(1, 1, 1), (1, 2048, 1), (3, 7, 1), (2, 8, 2), (5, 31, 1), (1025, 100, 1), (4, 513, 1), (2000, 512, 1),
          (1100, 1000, 1), (1025, 2048, 8), (1024, 4096, 1), (7, 4095, 3), (1030, 4097, 1), (3, 16384, 1),
          (2, 16385, 1), (2, 20000, 2), (1, 40000, 1), (2, 65536, 1), (1030, 1536, 2)]


@pytest.mark.parametrize("rows,dim,groups", SHAPES)
@pytest.mark.parametrize("dtype,rtype", TYPES)
def test_norm_with_residual(ssd, rows, dim, groups, dtype, rtype):
    import torch
    log(f"[norm] {rows}x{dim} groups {groups} {dtype} residual {rtype}")
    x, res, w = _draw(rows, dim, dtype, rtype, 1)
    y, check_y = _guarded((rows, dim), _t(dtype))
    h, check_h = _guarded((rows, dim), _t(rtype))
    _, _, rstd = ssd.ssd_rms_norm(x, w, EPS, residual=res, groups=groups, residual_out=h, y=y, want_rstd=True)
    torch.cuda.synchronize()
    yr, hr, ir = _ref(x, res, w, groups)
    _close(h, hr, HALF[rtype], "h")
    # y comes from the h before its rounding, which is off by one fp32 rounding
    _close(y, yr, HALF[dtype], "y")
    _close(rstd, ir, 0, "rstd")
    check_y(), check_h()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,dim", [(1, 768), (6, 333), (1500, 2048)])
def test_norm_without_residual_and_in_place(ssd, dtype, rows, dim):
    import torch
    x, res, w = _draw(rows, dim, dtype, dtype, 2)
    y, h, rstd = ssd.ssd_rms_norm(x, w, EPS)
    assert h is None and rstd is None
    torch.cuda.synchronize()
    _close(y, _ref(x, None, w, 1)[0], HALF[dtype], "y")
    # the residual updated in place gives the same bits as out of place
    y1, h1, _ = ssd.ssd_rms_norm(x, w, EPS, residual=res)
    r2 = res.clone()
    y2, h2, _ = ssd.ssd_rms_norm(x, w, EPS, residual=r2, residual_out=r2)
    torch.cuda.synchronize()
    assert torch.equal(y1, y2) and torch.equal(h1, r2) and h2 is r2


def test_norm_of_no_rows_and_extreme_values(ssd):
    import torch
    w = torch.ones(64, device="cuda")
    y, _, _ = ssd.ssd_rms_norm(torch.empty(0, 64, device="cuda"), w, EPS)
    assert y.shape == (0, 64)
    x = torch.zeros(4, 64, device="cuda")
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    x[3] = 1e-30
    y, _, rstd = ssd.ssd_rms_norm(x, w, EPS, want_rstd=True)
    torch.cuda.synchronize()
    assert bool((y[0] == 0).all()) and bool(torch.isnan(y[1]).all())
    # infinity: the factor is 0, so its own place is NaN and the others 0
    assert bool(torch.isnan(y[2, 5])) and float(y[2].nan_to_num(0).abs().max()) == 0
    assert bool(((y[3] - 1e-30 / EPS ** 0.5).abs() <= 1e-30 / EPS ** 0.5 * 64 * U32).all())


def _e4m3_ref(v):
    """(codes' values, scale) of rows in 64 bits, blocks of 32, from the definition."""
    b = np.asarray(v, np.float64).reshape(-1, 32)
    top = np.abs(b).max(1)
    m, e = np.frexp(top)
    p = np.where(m > 0.875, e - 8, e - 9)
    p = np.maximum(np.where(top > 0, p, -127), -127)
    u = b * np.exp2(-p.astype(np.float64))[:, None]
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(u), 2.0 ** -6))) - 3)
    return np.round(u / step) * step, p


def _scale_exp(scale):
    import torch
    return scale.view(torch.uint8).cpu().numpy().astype(np.int64).reshape(-1) - 127


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,dim", [(1, 32), (3, 96), (1, 2048), (1000, 4096 + 32)])
def test_quantize_is_exact(ssd, dtype, rows, dim):
    """No arithmetic but the scaling by a power of two and one rounding: every code and scale is the definition's."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(rows * dim)
    x = torch.randn(rows, dim, device="cuda", generator=g)
    x *= torch.exp2(40 * torch.rand(rows, dim // 32, device="cuda", generator=g) - 20).repeat_interleave(32, 1)
    x = x.to(_t(dtype))
    x[0, :32] = 0
    if dim > 64:
        x[0, 32:64] = torch.tensor([448.0, -448.0, 1.0, -0.5] * 8, device="cuda").to(x.dtype)  # scale 1, exactly full
        x[0, 64:96] = torch.tensor([450.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10] * 8, device="cuda").to(x.dtype)
    q, s = ssd.ssd_mx_quantize(x)
    torch.cuda.synchronize()
    val, p = _e4m3_ref(x.float().cpu().numpy())
    assert np.array_equal(_scale_exp(s), p)
    assert np.array_equal(q.float().cpu().numpy().reshape(-1, 32), val)


def test_quantize_edges(ssd):
    import torch
    x = torch.zeros(6, 32, device="cuda")
    x[0, 7] = float("nan")
    x[1, 8] = float("inf")
    x[2, 9] = -float("inf")
    x[3, 0] = 3.0e38
    x[4, 0] = 1e-45
    x[5, :] = 2.0 ** -140
    q, s = ssd.ssd_mx_quantize(x)
    torch.cuda.synchronize()
    code, exp = q.view(torch.uint8).cpu().numpy(), s.view(torch.uint8).cpu().numpy().reshape(-1)
    assert (exp[:3] == 255).all() and (code[:3] == 0x7F).all()
    val, p = _e4m3_ref(x[3:].cpu().numpy())
    assert np.array_equal(exp[3:].astype(int) - 127, p)
    assert np.array_equal(q[3:].float().cpu().numpy(), val)
    e, _ = ssd.ssd_mx_quantize(torch.empty(0, 64, device="cuda"))
    assert e.shape == (0, 64)


@pytest.mark.parametrize("rows,dim,groups", [(1, 32, 1), (3, 2048, 1), (1025, 2048, 8), (2000, 1536, 1),
                                              (2, 32768 + 64, 1), (5, 192, 3)])
@pytest.mark.parametrize("dtype,rtype", TYPES)
def test_norm_mx(ssd, rows, dim, groups, dtype, rtype):
    import torch
    x, res, w = _draw(rows, dim, dtype, rtype, 3)
    q, s, h = ssd.ssd_rms_norm_mx(x, w, EPS, residual=res, groups=groups)
    torch.cuda.synchronize()
    yr, hr, _ = _ref(x, res, w, groups)
    _close(h, hr, HALF[rtype], "h")
    scale = np.exp2(_scale_exp(s).astype(np.float64))[:, None]
    y = yr.cpu().numpy().reshape(-1, 32)
    got = q.float().cpu().numpy().astype(np.float64).reshape(-1, 32) * scale
    top = np.abs(y).max(1, keepdims=True)
    slack = 64 * U32  # the fp32 y before its rounding
    assert (top <= 448 * scale * (1 + slack)).all() and (top >= 224 * scale * (1 - slack)).all()
    # half a step of e4m3 (2^-4 relative, 2^-10 scales below 2^-6 of them), and the fp32 error
    lim = np.maximum(np.abs(y) * 2.0 ** -4, scale * 2.0 ** -10) + np.abs(y) * slack
    assert (np.abs(got - y) <= lim).all(), float((np.abs(got - y) / lim).max())


def _bwd_ref(dy, h, w, rstd, dres, groups):
    import torch
    dy, h, w, inv = dy.double(), h.double(), w.double(), rstd.double()[..., None]
    hh = h.unflatten(-1, (groups, -1)) * inv
    g = (dy * w).unflatten(-1, (groups, -1))
    c = (g * hh).mean(-1, keepdim=True)
    dh = (inv * (g - hh * c)).flatten(-2)
    mag = (inv * (g.abs() + hh.abs() * (g * hh).abs().mean(-1, keepdim=True))).flatten(-2)
    if dres is not None:
        dh, mag = dh + dres.double(), mag + dres.double().abs()
    t = dy * hh.flatten(-2)
    return dh, mag, t.sum(0), t.abs().sum(0)


@pytest.mark.parametrize("rows,dim,groups", SHAPES)
@pytest.mark.parametrize("dtype,rtype", TYPES)
def test_norm_bwd(ssd, rows, dim, groups, dtype, rtype):
    import torch
    log(f"[norm bwd] {rows}x{dim} groups {groups} {dtype} residual {rtype}")
    dy, h, w = _draw(rows, dim, dtype, rtype, 4)
    dres = _draw(rows, dim, rtype, rtype, 5)[0]
    rstd = _ref(h, None, w, groups)[2].float()
    for d in (dres, None):
        dx, dh, dw = ssd.ssd_rms_norm_bwd(dy, h, w, rstd, d_residual_out=d, groups=groups)
        torch.cuda.synchronize()
        r, mag, rw, wmag = _bwd_ref(dy, h, w, rstd, d, groups)
        assert bool(((dx.double() - r).abs() <= HALF[dtype] * r.abs() + 128 * U32 * mag).all())
        assert (dh is None) == (dtype == rtype)
        if dh is not None:
            assert bool(((dh.double() - r).abs() <= HALF[rtype] * r.abs() + 128 * U32 * mag).all())
        assert bool(((dw.double() - rw).abs() <= 128 * U32 * wmag + 1e-38).all())
    again = ssd.ssd_rms_norm_bwd(dy, h, w, rstd, d_residual_out=None, groups=groups)
    assert torch.equal(again[2], dw) and torch.equal(again[0], dx)


def test_norm_bwd_against_differences(ssd):
    """Central differences of <dy, y> + <dres, h> in 64 bits along random directions of x and w."""
    import torch
    x, res, w = _draw(5, 96, "f32", "f32", 6)
    dy, dres, _ = _draw(5, 96, "f32", "f32", 7)
    _, h, rstd = ssd.ssd_rms_norm(x, w, EPS, residual=res, groups=3, want_rstd=True)
    dx, _, dw = ssd.ssd_rms_norm_bwd(dy, h, w, rstd, d_residual_out=dres, groups=3)
    g = torch.Generator(device="cuda").manual_seed(8)

    def loss(xx, ww):
        y, hh, _ = _ref(xx, res, ww, 3)
        return float((dy.double() * y).sum() + (dres.double() * hh).sum())
    e = 1e-4  # truncation ~ e^2, far below the fp32 gradient's own error
    for _ in range(4):
        ux = torch.randn(5, 96, device="cuda", generator=g).double()
        uw = torch.randn(96, device="cuda", generator=g).double()
        num = (loss(x.double() + e * ux, w.double() + e * uw) - loss(x.double() - e * ux, w.double() - e * uw)) / (2 * e)
        ana = float((dx.double() * ux).sum() + (dw.double() * uw).sum())
        mag = float((dx.double() * ux).abs().sum() + (dw.double() * uw).abs().sum())
        assert abs(num - ana) <= 1e-5 * mag, (num, ana)


def test_norm_bwd_of_no_rows(ssd):
    import torch
    z = torch.empty(0, 64, device="cuda")
    dx, _, dw = ssd.ssd_rms_norm_bwd(z, z, torch.ones(64, device="cuda"), torch.empty(0, 1, device="cuda"))
    torch.cuda.synchronize()
    assert dx.shape == (0, 64) and bool((dw == 0).all())


def test_norm_on_another_stream_and_replayed(ssd):
    """The forward and backward on a side stream, and captured in a graph that is replayed with new inputs and
    eager calls between the replays."""
    import torch
    x, res, w = _draw(300, 1000, "bf16", "f32", 9)
    dy, _, _ = _draw(300, 1000, "bf16", "f32", 10)

    def both(**kw):
        y, h, rstd = ssd.ssd_rms_norm(x, w, EPS, residual=res, want_rstd=True, **kw)
        return (y, h) + ssd.ssd_rms_norm_bwd(dy, h, w, rstd, **kw)
    want = both()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = both(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for k in range(3):
        x.copy_(torch.roll(x, k + 1, 0))
        want = both()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k
