"""CPU tests of the argument checks of the operators around the core (norm, beam search, projections): each call
fails a host-side check, or is empty, so nothing is enqueued. Pointers are fake aligned addresses."""
from __future__ import annotations

import ctypes

import pytest

import ssd_sequence_mixing_amd as ssd

OK, ENULL, ESHAPE, EUNSUP, EWS, EALIGN = range(6)
F32, BF16 = ssd.SSD_F32, ssd.SSD_BF16
P = 0x10000
NONE = ctypes.c_size_t(-1).value


def norm(x=P, res=P, w=P, eps=1e-5, res_out=P, y=P, rstd=P, rows=8, dim=2048, groups=1, dtype=BF16, rdtype=F32):
    return ssd.raw_call("ssd_rms_norm", x, res, w, eps, res_out, y, rstd, rows, dim, groups, dtype, rdtype, None)


def norm_mx(x=P, res=P, w=P, eps=1e-5, res_out=P, q=P, s=P, rows=8, dim=2048, groups=1, dtype=BF16, rdtype=F32):
    return ssd.raw_call("ssd_rms_norm_mx", x, res, w, eps, res_out, q, s, rows, dim, groups, dtype, rdtype, None)


def norm_bwd(dy=P, h=P, w=P, rstd=P, dres=P, dx=P, dh=P, dw=P, rows=8, dim=2048, groups=1, dtype=BF16, rdtype=F32,
             ws=P, wsb=1 << 40):
    return ssd.raw_call("ssd_rms_norm_bwd", dy, h, w, rstd, dres, dx, dh, dw, rows, dim, groups, dtype, rdtype, ws,
                        wsb, None)


def quantize(x=P, q=P, s=P, rows=8, dim=2048, dtype=BF16):
    return ssd.raw_call("ssd_mx_quantize", x, q, s, rows, dim, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ENULL), (dict(w=None), ENULL), (dict(y=None), ENULL), (dict(res_out=None), ENULL),
    (dict(res=None), ENULL), (dict(rows=-1), ESHAPE), (dict(dim=0), ESHAPE), (dict(groups=0), ESHAPE),
    (dict(groups=3), ESHAPE), (dict(dtype=7), EUNSUP), (dict(rdtype=7), EUNSUP), (dict(dtype=F32, rdtype=BF16), EUNSUP),
    (dict(dim=65536 + 8), EUNSUP), (dict(rows=1 << 40), EUNSUP), (dict(rows=1 << 31), EUNSUP),
    (dict(x=P + 2), EALIGN), (dict(res=P + 4), EALIGN), (dict(w=P + 4), EALIGN), (dict(y=P + 8), EALIGN),
    (dict(rstd=P + 4), EALIGN), (dict(rows=0, x=None, res=None, w=None, y=None, res_out=None, rstd=None), OK),
])
def test_norm_checks(kw, code):
    assert norm(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ENULL), (dict(s=None), ENULL), (dict(dim=2040), ESHAPE), (dict(dim=96, groups=2), ESHAPE),
    (dict(q=P + 1), EALIGN), (dict(s=P + 1), EALIGN), (dict(rows=0), OK),
])
def test_norm_mx_checks(kw, code):
    assert norm_mx(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ENULL), (dict(q=None), ENULL), (dict(s=None), ENULL), (dict(dim=31), ESHAPE), (dict(rows=-1), ESHAPE),
    (dict(dtype=3), EUNSUP), (dict(rows=1 << 40), EUNSUP), (dict(x=P + 4), EALIGN), (dict(rows=0), OK),
])
def test_quantize_checks(kw, code):
    assert quantize(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), ENULL), (dict(h=None), ENULL), (dict(w=None), ENULL), (dict(rstd=None), ENULL),
    (dict(dx=None), ENULL), (dict(dw=None), ENULL), (dict(groups=5), ESHAPE), (dict(rdtype=BF16), EUNSUP),
    (dict(dtype=F32, rdtype=BF16), EUNSUP), (dict(dh=P + 4), EALIGN), (dict(ws=None), EWS), (dict(wsb=64), EWS),
    (dict(ws=P + 16), EALIGN),
])
def test_norm_bwd_checks(kw, code):
    assert norm_bwd(**kw) == code


def test_norm_bwd_workspace():
    q = ssd.load().ssd_rms_norm_bwd_workspace_bytes
    assert q(0, 2048, 1, BF16, BF16) == 0
    assert q(8, 2048, 1, BF16, F32) == 8 * 2048 * 4  # few rows: a work-group, and a share of dw, for each
    assert q(16384, 1536, 1, BF16, BF16) == 1024 * 1536 * 4
    assert q(8, 2048, 3, BF16, BF16) == NONE


def select(logits=P, scores=P, fin=None, eos=-1, out=P, parent=P, token=P, done=P, batch=2, beams=4, vocab=1000,
           dtype=BF16, ws=P, wsb=1 << 40):
    return ssd.raw_call("ssd_beam_select", logits, scores, fin, eos, out, parent, token, done, batch, beams, vocab,
                        dtype, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), ENULL), (dict(scores=None), ENULL), (dict(out=None), ENULL), (dict(parent=None), ENULL),
    (dict(token=None), ENULL), (dict(batch=-1), ESHAPE), (dict(beams=0), ESHAPE), (dict(vocab=0), ESHAPE),
    (dict(beams=17), EUNSUP), (dict(vocab=(1 << 28) + 1), EUNSUP), (dict(batch=1 << 40), EUNSUP), (dict(dtype=4), EUNSUP),
    (dict(eos=1000), ESHAPE), (dict(eos=-2), ESHAPE), (dict(fin=P), ESHAPE), (dict(logits=P + 2), EALIGN),
    (dict(parent=P + 4), EALIGN), (dict(ws=None), EWS), (dict(wsb=16), EWS), (dict(ws=P + 16), EALIGN),
    (dict(batch=0, logits=None, ws=None, wsb=0), OK),
])
def test_select_checks(kw, code):
    assert select(**kw) == code


def test_select_workspace():
    q = ssd.load().ssd_beam_select_workspace_bytes
    # 25 wavefronts of 2048 logits for each of 4 rows, 4 keys and one pair of sums from each
    assert q(1, 4, 50257) == -(-4 * 25 * 4 * 8 // 256) * 256 + -(-4 * 25 * 8 // 256) * 256
    assert q(0, 4, 100) == 0 and q(1, 17, 100) == NONE and q(1, 0, 100) == NONE


def step_beam(si=P, so=1 << 40, parent=P, src=4, ci=None, co=None, x=P, cw=None, cb=None, dt=P, A=P, B=P, C=P, D=P,
              y=P, batch=4, H=8, hd=64, N=128, G=1, dtype=BF16):
    return ssd.raw_call("ssd_step_beam", si, so, parent, src, ci, co, x, cw, cb, dt, None, 0, A, B, C, D, None, y,
                        batch, H, hd, N, G, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(si=None), ENULL), (dict(so=None), ENULL), (dict(parent=None), ENULL), (dict(x=None), ENULL),
    (dict(src=-1), ESHAPE), (dict(src=1 << 40), ESHAPE), (dict(N=12), EUNSUP), (dict(G=3), ESHAPE),
    (dict(ci=P), ENULL), (dict(co=P), ENULL), (dict(cb=P), ENULL), (dict(cw=P), ENULL), (dict(cw=P, co=P), ENULL),
    (dict(si=P + 4), EALIGN), (dict(parent=P + 4), EALIGN),
    (dict(so=P), EUNSUP), (dict(so=P + 4 * 8 * 64 * 128 * 4 - 16), EUNSUP),   # the states overlap
    (dict(ci=P, co=P, cw=P), EUNSUP), (dict(batch=0), OK),
])
def test_step_beam_checks(kw, code):
    assert step_beam(**kw) == code


def test_binding_refuses_what_the_library_would_misread():
    import torch
    x, w = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError):
        ssd.ssd_rms_norm(x, w[:32], 1e-5)
    with pytest.raises(ValueError):
        ssd.ssd_rms_norm(x, w, 1e-5, residual=torch.zeros(4, 32))
    with pytest.raises(ValueError):
        ssd.ssd_rms_norm(x, w, 1e-5, residual_out=x)
    with pytest.raises(TypeError):
        ssd.ssd_rms_norm(x.half(), w, 1e-5)
    with pytest.raises(ValueError):   # not on the GPU
        ssd.ssd_rms_norm(x, w, 1e-5)
    with pytest.raises(ValueError):
        ssd.ssd_rms_norm_bwd(x, x, w, torch.zeros(4, 2))
    with pytest.raises(ValueError):
        ssd.ssd_beam_select(torch.zeros(2, 3, 10), torch.zeros(2, 4))
    with pytest.raises(ValueError):
        ssd.ssd_beam_select(torch.zeros(2, 3, 10), torch.zeros(2, 3), finished=torch.zeros(2, 3))


def linear(x=P, w=P, b=None, act=0, r=None, y=P, pre=None, rows=100, k=64, n=48, dtype=BF16, ws=P, wsb=1 << 40):
    return ssd.raw_call("ssd_linear", x, w, b, act, r, y, pre, rows, k, n, dtype, ws, wsb, None)


def linear_mx(x=P, xs=P, w=P, ws_=P, b=None, act=0, r=None, y=P, rows=100, k=64, n=48, ws=P, wsb=1 << 40):
    return ssd.raw_call("ssd_linear_mx", x, xs, w, ws_, b, act, r, y, rows, k, n, ws, wsb, None)


def linear_bwd(dy=P, x=P, w=P, act=1, pre=P, dx=P, dw=P, db=P, rows=100, k=64, n=48, dtype=BF16, ws=P, wsb=1 << 40):
    return ssd.raw_call("ssd_linear_bwd", dy, x, w, act, pre, dx, dw, db, rows, k, n, dtype, ws, wsb, None)


COMMON = [(dict(rows=-1), ESHAPE), (dict(k=0), ESHAPE), (dict(n=-3), ESHAPE), (dict(act=3), EUNSUP), (dict(act=-1), EUNSUP),
          (dict(rows=(1 << 24) + 1), EUNSUP), (dict(k=1 << 21), EUNSUP), (dict(n=1 << 40), EUNSUP)]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(x=None), ENULL), (dict(w=None), ENULL), (dict(y=None), ENULL), (dict(dtype=5), EUNSUP),
    (dict(x=P + 2), EALIGN), (dict(w=P + 8), EALIGN), (dict(b=P + 4), EALIGN), (dict(r=P + 2), EALIGN),
    (dict(pre=P + 2), EALIGN), (dict(k=63, ws=None), EWS), (dict(k=63, wsb=100), EWS), (dict(k=63, ws=P + 16), EALIGN),
    (dict(rows=0, x=None, w=None, y=None), OK)])
def test_linear_checks(kw, code):
    assert linear(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(x=None), ENULL), (dict(xs=None), ENULL), (dict(w=None), ENULL), (dict(ws_=None), ENULL), (dict(y=None), ENULL),
    (dict(k=72), ESHAPE), (dict(xs=P + 4), EALIGN), (dict(ws_=P + 4), EALIGN), (dict(rows=0, y=None), OK)])
def test_linear_mx_checks(kw, code):
    assert linear_mx(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(dy=None), ENULL), (dict(x=None), ENULL), (dict(w=None), ENULL), (dict(pre=None), ENULL), (dict(dtype=5), EUNSUP),
    (dict(dx=P + 2), EALIGN), (dict(dw=P + 2), EALIGN), (dict(db=P + 4), EALIGN), (dict(pre=P + 2), EALIGN),
    (dict(ws=None), EWS), (dict(wsb=1000), EWS), (dict(ws=P + 128), EALIGN), (dict(rows=0, dw=None, db=None), OK)])
def test_linear_bwd_checks(kw, code):
    assert linear_bwd(**kw) == code


def test_linear_workspaces():
    q = ssd.load().ssd_linear_workspace_bytes
    assert q(8, 2048, 8512, BF16) == 0 and q(8192, 4096, 2048, BF16) == 0
    # rows of 1003 bf16 values: both operands copied to rows of 1008; fp32 ones and few rows are taken as they are
    copies = -(-64 * 1008 * 2 // 256) * 256 + -(-515 * 1008 * 2 // 256) * 256
    assert q(64, 1003, 515, BF16) - copies == q(64, 1008, 515, BF16)
    assert q(64, 1003, 515, F32) == q(64, 1004, 515, F32) and q(16, 1003, 515, BF16) == 0
    assert q(0, 1003, 515, F32) == 0 and q(-1, 64, 64, F32) == NONE and q(8, 64, 64, 9) == NONE
    q = ssd.load().ssd_linear_mx_workspace_bytes
    assert q(8, 96, 64) == 0 and q(8, 40, 64) == NONE
    for rows in (0, 1, 1 << 20, (1 << 20) + 1, 1 << 40, -1):
        for dim in (1, 7, 1 << 20, (1 << 20) + 1, 0):
            ssd.load().ssd_linear_bwd_workspace_bytes(rows, dim, dim, 1, BF16)


def test_linear_binding_refuses():
    import torch
    x, w = torch.zeros(4, 64), torch.zeros(8, 64)
    with pytest.raises(ValueError):
        ssd.ssd_linear(x, w[:, :32])
    with pytest.raises(ValueError):
        ssd.ssd_linear(x, w, bias=torch.zeros(64))
    with pytest.raises(ValueError):
        ssd.ssd_linear(x, w.bfloat16())
    with pytest.raises(ValueError):
        ssd.ssd_linear(x, w, residual=torch.zeros(4, 64))
    with pytest.raises(ValueError):
        ssd.ssd_linear(x, w, act="relu")
    with pytest.raises(ValueError):
        ssd.ssd_linear_bwd(torch.zeros(4, 8), x, w, act="silu")
    with pytest.raises(ValueError):
        ssd.ssd_linear_mx(x, x, w, w)
