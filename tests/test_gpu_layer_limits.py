"""GPU tests of the operators around the core at counts of rows whose threads pass 2^32, the most that one launch takes
along a dimension: the ends, both sides of that border, and the middle against the formulas in 64 bits."""
from __future__ import annotations

import ctypes

import pytest

from tests.gpu_util import log

pytestmark = pytest.mark.gpu

EPS = 1e-5
HALF, U32 = 2.0 ** -8, 2.0 ** -24   # of bf16, of fp32


@pytest.fixture(autouse=True)
def _free():
    import torch
    yield
    torch.cuda.empty_cache()


def _spots(n, border, width):
    """Starts of stretches of `width` of n rows: the first, around the border, the middle, the last."""
    return [0, border - width, border, n // 2, n - width]


@pytest.mark.parametrize("per", [8, 7])
def test_norm_of_many_groups(ssd, per):
    """2^26 + 8 (row, group) pairs, of a wavefront each."""
    import torch
    rows, groups = (1 << 23) + 1, 8
    dim = per * groups
    log(f"[limits] norm {rows} x {groups} x {per}")
    g = torch.Generator(device="cuda").manual_seed(per)
    x = torch.empty(rows, dim, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    w = torch.rand(dim, device="cuda", generator=g) + 0.5
    y, _, rstd = ssd.ssd_rms_norm(x, w, EPS, groups=groups, want_rstd=True)
    for r0 in range(0, rows, 1 << 20):
        h = x[r0:r0 + (1 << 20)].double().unflatten(1, (groups, per))
        inv = 1 / torch.sqrt((h * h).mean(-1) + EPS)
        ref = (h * inv[..., None]).flatten(1) * w.double()
        assert bool(((y[r0:r0 + (1 << 20)].double() - ref).abs() <= (HALF + 32 * U32) * ref.abs()).all()), r0
        assert bool(((rstd[r0:r0 + (1 << 20)].double() - inv).abs() <= 16 * U32 * inv).all()), r0


def test_norm_in_eight_bits_of_many_groups(ssd):
    """The same, with 3 groups (2^26 is no multiple of them) of 32 and a residual: equal bits to the rows by themselves."""
    import torch
    rows, groups = (1 << 26) // 3 + 2, 3
    dim = 32 * groups
    log(f"[limits] norm in 8 bits {rows} x {groups} x 32")
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty(rows, dim, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    res = torch.empty(rows, dim, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    w = torch.rand(dim, device="cuda", generator=g) + 0.5
    q, s, h = ssd.ssd_rms_norm_mx(x, w, EPS, residual=res, groups=groups)
    for r0 in _spots(rows, (1 << 26) // 3, 1):
        r1 = min(rows, r0 + 2)
        a, b, c = ssd.ssd_rms_norm_mx(x[r0:r1].clone(), w, EPS, residual=res[r0:r1].clone(), groups=groups)
        torch.cuda.synchronize()
        assert torch.equal(a.view(torch.uint8), q[r0:r1].view(torch.uint8)) and torch.equal(c, h[r0:r1])
        assert torch.equal(b.view(torch.uint8), s[r0:r1].view(torch.uint8))
    step = 1 << 21
    for r0 in range(0, rows, step):  # all of it: within half a step of e4m3, and the fp32 sum
        hh = (x[r0:r0 + step].float() + res[r0:r0 + step].float()).unflatten(1, (groups, 32))
        y = hh / torch.sqrt((hh * hh).mean(-1, keepdim=True) + EPS) * w.view(groups, 32)
        sc = s[r0:r0 + step].float()[..., None]
        got = q[r0:r0 + step].float().unflatten(1, (groups, 32)) * sc
        assert bool(((got - y).abs() <= torch.maximum(y.abs() * 2.0 ** -4, sc * 2.0 ** -10) + 256 * U32 * y.abs()).all()), r0


def test_norm_gradients_of_a_wide_row(ssd):
    """2^26 + 65536 columns: the sums over rows of that many."""
    import torch
    groups, per, rows = 1025, 65536, 2
    dim = groups * per
    log(f"[limits] norm backward {rows} x {groups} x {per}")
    g = torch.Generator(device="cuda").manual_seed(4)
    x, dy = (torch.empty(rows, dim, device="cuda").normal_(generator=g) for _ in range(2))
    w = torch.rand(dim, device="cuda", generator=g) + 0.5
    y, _, rstd = ssd.ssd_rms_norm(x, w, EPS, groups=groups, want_rstd=True)
    dx, _, dw = ssd.ssd_rms_norm_bwd(dy, x, w, rstd, groups=groups)
    hh = x.double().unflatten(1, (groups, per)) * rstd.double()[..., None]
    up = dy.double().unflatten(1, (groups, per))
    mag = (up * hh).abs().sum(0).flatten()
    assert bool(((dw.double() - (up * hh).sum(0).flatten()).abs() <= 64 * U32 * mag).all())
    up = up * w.double().view(groups, per)
    dot = (up * hh).mean(-1, keepdim=True)
    size = (up.abs() + hh.abs() * (up * hh).abs().mean(-1, keepdim=True)) * rstd.double()[..., None]
    ref = (up - hh * dot) * rstd.double()[..., None]
    assert bool(((dx.double().unflatten(1, (groups, per)) - ref).abs() <= 128 * U32 * size).all())


def test_quantize_of_many_values(ssd):
    """2^35 + 2^20 values, 8 to a thread."""
    import torch
    rows, dim = (1 << 15) + 1, 1 << 20
    log(f"[limits] quantize {rows} x {dim}")
    x = torch.zeros(rows, dim, device="cuda", dtype=torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(5)
    at = _spots(rows, 1 << 15, 1)
    for r in at:
        x[r].normal_(generator=g)
    q, s = ssd.ssd_mx_quantize(x)
    for r in at:
        a, b = ssd.ssd_mx_quantize(x[r].clone())
        torch.cuda.synchronize()
        assert torch.equal(a.view(torch.uint8), q[r].view(torch.uint8)), r
        assert torch.equal(b.view(torch.uint8), s[r].view(torch.uint8)), r
    for r0 in range(0, rows, 1 << 12):
        part = q[r0:r0 + (1 << 12)].view(torch.uint8)
        seen = torch.count_nonzero(part.view(torch.int64), dim=1) > 0  # (zeros are codes 0)
        assert torch.nonzero(seen).flatten().tolist() == sorted({r - r0 for r in at if 0 <= r - r0 < (1 << 12)})


def test_gradients_of_no_rows_are_zero(ssd):
    """2^32 fp32 weights, cleared without a row to sum."""
    import torch
    n = 1 << 16
    log(f"[limits] gradients of no rows, {n} x {n}")
    dw, db = torch.ones(n, n, device="cuda"), torch.ones(n, device="cuda")
    rc = ssd.raw_call("ssd_linear_bwd", None, None, None, 0, None, None, ctypes.c_void_p(dw.data_ptr()),
                      ctypes.c_void_p(db.data_ptr()), 0, n, n, ssd.SSD_F32, None, 0,
                      ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    for r in range(0, n, 1 << 12):
        assert float(dw[r:r + (1 << 12)].abs().max()) == 0, r
    assert float(db.abs().max()) == 0


@pytest.mark.parametrize("beam", [False, True])
def test_step_of_many_heads(ssd, beam):
    """2^24 + 64 (sequence, head) pairs, of a work-group each: the step in place and from parents' rows."""
    import torch
    rows, H, P, N = (1 << 18) + 1, 64, 1, 4
    log(f"[limits] step of {rows} x {H} heads, beam {beam}")
    g = torch.Generator(device="cuda").manual_seed(6)

    def draw(*shape):  # in [-1, 1)
        return 2 * torch.rand(*shape, device="cuda", generator=g) - 1
    state, x, z, conv = draw(rows, H, P, N), draw(rows, H, P), draw(rows, H, P), draw(rows, H * P, 3)
    dt, A = torch.rand(rows, H, device="cuda", generator=g), -torch.rand(H, device="cuda", generator=g)
    B, C, D, conv_w, conv_b = draw(rows, 1, N), draw(rows, 1, N), draw(H), draw(H * P, 4), draw(H * P)
    parent = torch.arange(rows - 1, -1, -1, device="cuda", dtype=torch.int32)
    frm = parent.long() if beam else torch.arange(rows, device="cuda")
    s0, c0 = state.double()[frm], conv.double()[frm]
    v = (c0 * conv_w.double()[:, :3]).sum(-1) + conv_w.double()[:, 3] * x.double().flatten(1) + conv_b.double()
    xv = (v / (1 + torch.exp(-v))).view(rows, H, P)
    new = torch.exp(dt.double() * A.double())[..., None, None] * s0 + (dt.double()[..., None] * xv)[..., None] * B.double()[:, None]
    ref = ((new * C.double()[:, None]).sum(-1) + D.double()[:, None] * xv) * (z.double() / (1 + torch.exp(-z.double())))
    kept = torch.cat([c0[..., 1:], x.double().flatten(1)[..., None]], -1)
    kw = dict(conv_w=conv_w, conv_b=conv_b, z=z)
    if beam:
        out, cout = torch.empty_like(state), torch.empty_like(conv)
        y = ssd.ssd_step_beam(state, out, parent, x, dt, A, B, C, D, conv_in=conv, conv_out=cout, **kw)
    else:
        out, cout = state, conv
        y = ssd.ssd_step_fused(state, conv, x, dt, A, B, C, D, **kw)
    torch.cuda.synchronize()
    assert torch.equal(cout.double(), kept)
    # fp32: under 32 roundings of magnitudes of at most 6 (states) and 29 (y)
    assert float((out.double() - new).abs().max()) < 2.0 ** -16
    assert float((y.double() - ref).abs().max()) < 2.0 ** -14
