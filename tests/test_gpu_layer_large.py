"""GPU tests of the operators around the core where a tensor holds more than 2^31 values: a few rows at its start, in
its middle and at its end hold values, the others zeros, and these are compared with the formulas in 64 bits.

Tolerances, fixed before the first run: a stored bf16 value is off by half a step (2^-8), sums in fp32 of up to 4096
values by under 2^-12 of the sum of magnitudes."""
from __future__ import annotations

import pytest

from tests.gpu_util import log

pytestmark = pytest.mark.gpu

HALF, SUM = 2.0 ** -8, 2.0 ** -12


def _near(a, ref, mag):
    assert bool(((a.double() - ref).abs() <= HALF * ref.abs() + SUM * mag).all())


def _sparse(rows, cols, at, scale=1.0, dtype=None):
    import torch
    t = torch.zeros(rows, cols, device="cuda", dtype=dtype or torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(rows % 1000 + cols)
    t[at] = (scale * torch.randn(len(at), cols, device="cuda", generator=g)).to(t.dtype)
    return t


def test_linear_and_its_gradients(ssd):
    import torch
    m, k, n = (1 << 17) + 3, 64, 32776
    at = [0, 65537, m - 1]
    log(f"[large] linear {m}x{k}x{n}")
    x, w, r = _sparse(m, k, at), _sparse(n, k, list(range(n)), 0.1), _sparse(m, n, at)
    y, _ = ssd.ssd_linear(x, w, residual=r)
    z, mag = x[at].double() @ w.double().t(), x[at].double().abs() @ w.double().abs().t()
    _near(y[at], z + r[at].double(), mag + r[at].double().abs())
    assert float(y[1].abs().max()) == 0 and float(y[m - 2].abs().max()) == 0
    q, s = ssd.ssd_mx_quantize(x)
    wq, ws = ssd.ssd_mx_quantize(w)
    y = ssd.ssd_linear_mx(q, s, wq, ws, y=y)
    xv = q[at].float().double() * s[at].float().double().repeat_interleave(32, 1)
    wv = wq.float().double() * ws.float().double().repeat_interleave(32, 1)
    _near(y[at], xv @ wv.t(), 8 * (xv.abs() @ wv.abs().t()))  # the 8-bit products' sums: 7 * 2^-13 of it
    del y
    pre = _sparse(m, n, at, 0.5)
    dx, dw, db = ssd.ssd_linear_bwd(r, x, w, act="silu", preact=pre, want_bias=True)
    p = pre[at].double()
    g = torch.sigmoid(p)
    dz = r[at].double() * (g + p * g * (1 - g))
    _near(dx[at], dz @ w.double(), 32 * (dz.abs() @ w.double().abs()))  # dz itself is rounded: 2^-8 of the magnitudes
    _near(dw, dz.t() @ x[at].double(), 32 * (dz.abs().t() @ x[at].double().abs()))
    assert bool(((db.double() - dz.sum(0)).abs() <= SUM * dz.abs().sum(0)).all())
    assert float(dx[1].abs().max()) == 0


def test_norms(ssd):
    import torch
    rows, dim = (1 << 20) + 1, 2080
    at = [0, 524289, rows - 1]
    log(f"[large] norm {rows}x{dim}")
    x, r = _sparse(rows, dim, at), _sparse(rows, dim, at, 2.0)
    w = torch.rand(dim, device="cuda") + 0.5
    y, ro, rstd = ssd.ssd_rms_norm(x, w, 1e-5, residual=r, want_rstd=True)
    h = x[at].double() + r[at].double()
    inv = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-5)
    _near(ro[at], h, h.abs())
    _near(y[at], h * inv * w.double(), (h * inv).abs())
    assert float(y[1].abs().max()) == 0
    q, s, _ = ssd.ssd_rms_norm_mx(x, w, 1e-5, residual=r, residual_out=r)
    v = q[at].float().double() * s[at].float().double().repeat_interleave(32, 1)
    top = (h * inv * w.double()).abs().unflatten(1, (-1, 32)).amax(-1).repeat_interleave(32, 1)
    assert bool(((v - h * inv * w.double()).abs() <= 2.0 ** -4 * (h * inv * w.double()).abs() + 2.0 ** -14 * top).all())
    del q, s, r
    dx, _, dw = ssd.ssd_rms_norm_bwd(x, ro, w, rstd)
    hh, gw = ro[at].double() * inv, x[at].double() * w.double()
    _near(dx[at], inv * (gw - hh * (gw * hh).mean(-1, keepdim=True)), inv * (gw.abs() + hh.abs() * (gw * hh).abs().mean(-1, keepdim=True)))
    assert bool(((dw.double() - (x[at].double() * hh).sum(0)).abs() <= SUM * (x[at].double() * hh).abs().sum(0)).all())


def test_beam_search(ssd):
    import torch
    b, k, v = 64, 16, (1 << 21) + 8
    log(f"[large] select {b}x{k}x{v}")
    logits = torch.full((b, k, v), -20.0, device="cuda", dtype=torch.bfloat16)
    spots = [(0, 3, 5), (40, 0, v - 1), (63, 15, v - 1), (63, 15, 0)]
    for i, j, t in spots:
        logits[i, j, t] = 20.0
    scores = torch.zeros(b, k, device="cuda")
    _, parent, token, _ = ssd.ssd_beam_select(logits, scores)
    # a spike is its beam's only likely token (two share the last beam's): score 0 and -log 2; without one -log v
    assert (int(parent[0, 0]), int(token[0, 0])) == (3, 5)
    assert (int(parent[40, 0]), int(token[40, 0])) == (40 * k, v - 1)
    assert parent[63, :2].tolist() == [63 * k + 15] * 2 and token[63, :2].tolist() == [0, v - 1]
    assert parent[1].tolist() == [k] * k and token[1].tolist() == list(range(k))  # all equal: the lowest
    del logits
    rows, H, P, N = 4200, 64, 64, 128
    log(f"[large] step from {rows} states")
    at = [0, 4097, rows - 1]
    state = _sparse(rows, H * P * N, at, dtype=torch.float32).view(rows, H, P, N)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, B, C = (torch.randn(rows, *s, device="cuda", generator=g).bfloat16() for s in ((H, P), (1, N), (1, N)))
    dt = torch.rand(rows, H, device="cuda", generator=g).bfloat16()
    A, D = -torch.rand(H, device="cuda", generator=g), torch.rand(H, device="cuda", generator=g)
    parent = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(state)
    y = ssd.ssd_step_beam(state, out, parent, x, dt, A, B, C, D)
    for row in at:
        i = rows - 1 - row
        own = state[row:row + 1].clone()
        ref = ssd.ssd_step(own, x[i:i + 1], dt[i:i + 1], A, B[i:i + 1], C[i:i + 1], D)
        assert torch.equal(out[i], own[0]) and torch.equal(y[i], ref[0])
