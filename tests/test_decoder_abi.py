"""CPU tests of the argument checks of the gated recurrence, the embedding, the logits' processing and the 8-bit integer
projections: each call fails a host-side check, or is empty, so nothing is enqueued. Pointers are fake aligned addresses."""
from __future__ import annotations

import ctypes

import pytest

import ssd_sequence_mixing_amd as ssd

OK, ENULL, ESHAPE, EUNSUP, EWS, EALIGN = range(6)
F32, BF16 = ssd.SSD_F32, ssd.SSD_BF16
LOG, SIG, RATE = 0, 1, 2
NONE = ctypes.c_size_t(-1).value
M = 1 << 32   # addresses far apart
A = [k * M for k in range(1, 20)]


def fwd(x=A[0], ldx=64, f=A[1], ldf=64, i=A[2], ldi=64, decay=RATE, rate=A[3], reset=A[4], init=A[5], y=A[6], final=A[7], states=A[8],
        batch=2, T=300, dim=64, dtype=BF16, ws=A[9], wsb=1 << 31):
    return ssd.raw_call("ssd_gated_scan_fwd", x, ldx, f, ldf, i, ldi, decay, rate, reset, init, y, final, states, batch, T, dim, dtype, ws, wsb, None)


def bwd(dy=A[10], x=A[0], ldx=64, f=A[1], ldf=64, i=A[2], ldi=64, decay=RATE, rate=A[3], reset=A[4], states=A[8], dfin=A[11], dx=A[12],
        df=A[13], di=A[14], drate=A[15], d0=A[16], batch=2, T=300, dim=64, dtype=BF16, ws=A[9], wsb=1 << 31):
    return ssd.raw_call("ssd_gated_scan_bwd", dy, x, ldx, f, ldf, i, ldi, decay, rate, reset, states, dfin, dx, df, di, drate, d0, batch, T,
                        dim, dtype, ws, wsb, None)


def step(si=A[0], so=A[1], parent=A[2], src=8, x=A[3], ldx=64, f=A[4], ldf=64, i=A[5], ldi=64, decay=RATE, rate=A[6], y=A[7], rows=8,
         dim=64, dtype=BF16):
    return ssd.raw_call("ssd_gated_step", si, so, parent, src, x, ldx, f, ldf, i, ldi, decay, rate, y, rows, dim, dtype, None)


SHAPES = [(dict(batch=-1), ESHAPE), (dict(T=-1), ESHAPE), (dict(dim=0), ESHAPE), (dict(dim=(1 << 20) + 1, ldx=1 << 21, ldf=1 << 21, ldi=1 << 21), EUNSUP),
          (dict(T=1 << 31), EUNSUP), (dict(batch=1 << 26), EUNSUP), (dict(dtype=2), EUNSUP), (dict(decay=3), EUNSUP), (dict(decay=-1), EUNSUP),
          (dict(ldx=63), ESHAPE), (dict(ldf=0), ESHAPE), (dict(ldi=-64), ESHAPE), (dict(ldx=1 << 60), EUNSUP), (dict(x=A[0] + 1), EALIGN),
          (dict(f=A[1] + 1), EALIGN), (dict(i=A[2] + 1), EALIGN), (dict(dtype=F32, x=A[0] + 2), EALIGN), (dict(rate=A[3] + 4), EALIGN),
          (dict(reset=A[4] + 8), EALIGN), (dict(ws=None), EWS), (dict(wsb=64), EWS), (dict(ws=A[9] + 16), EALIGN), (dict(decay=LOG), EUNSUP)]


@pytest.mark.parametrize("kw,code", SHAPES + [
    (dict(x=None), ENULL), (dict(f=None), ENULL), (dict(y=None), ENULL), (dict(rate=None), ENULL), (dict(y=A[6] + 8), EALIGN),
    (dict(final=A[7] + 4), EALIGN), (dict(states=A[8] + 4), EALIGN), (dict(init=A[5] + 4), EALIGN),
    (dict(y=A[0]), EUNSUP), (dict(y=A[1] + 16), EUNSUP), (dict(final=A[5]), EUNSUP), (dict(states=A[6]), EUNSUP), (dict(final=A[8]), EUNSUP),
    (dict(x=A[6] - 1000, ldx=1024), EUNSUP), (dict(batch=0, x=None, f=None, y=None, i=None, init=None, final=None, ws=None, wsb=0), OK),
    (dict(T=0, x=None, f=None, y=None, i=None, init=None, final=None, rate=None), OK)])
def test_scan_checks(kw, code):
    if code in (EWS, EALIGN) and ("ws" in kw or "wsb" in kw) and ssd.load().ssd_gated_scan_fwd_workspace_bytes(2, 300, 64, BF16) == 0:
        pytest.skip("no workspace")
    assert fwd(**kw) == code


@pytest.mark.parametrize("kw,code", SHAPES + [
    (dict(dy=None), ENULL), (dict(x=None), ENULL), (dict(f=None), ENULL), (dict(states=None), ENULL), (dict(dx=None), ENULL),
    (dict(df=None), ENULL), (dict(di=None), ENULL), (dict(i=None), ENULL), (dict(rate=None), ENULL), (dict(drate=None), ENULL),
    (dict(decay=SIG, rate=None), EUNSUP), (dict(dx=A[10]), EUNSUP), (dict(df=A[12]), EUNSUP), (dict(di=A[2]), EUNSUP),
    (dict(drate=A[3]), EUNSUP), (dict(d0=A[11]), EUNSUP), (dict(d0=A[16] + 4), EALIGN), (dict(df=A[13] + 2), EALIGN),
    (dict(batch=0, T=0, dim=0), ESHAPE)])
def test_scan_gradient_checks(kw, code):
    assert bwd(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(si=None), ENULL), (dict(so=None), ENULL), (dict(x=None), ENULL), (dict(f=None), ENULL), (dict(y=None), ENULL), (dict(rate=None), ENULL),
    (dict(rows=-1), ESHAPE), (dict(dim=0), ESHAPE), (dict(src=-1), ESHAPE), (dict(parent=None, src=7), ESHAPE), (dict(src=1 << 31), EUNSUP),
    (dict(rows=1 << 31), EUNSUP), (dict(dtype=5), EUNSUP), (dict(decay=7), EUNSUP), (dict(decay=SIG), EUNSUP), (dict(ldf=8), ESHAPE),
    (dict(so=A[0]), EUNSUP), (dict(so=A[0] + 1024, parent=None), EUNSUP), (dict(y=A[0]), EUNSUP), (dict(y=A[3]), EUNSUP), (dict(so=A[7]), EUNSUP),
    (dict(si=A[0] + 4), EALIGN), (dict(parent=A[2] + 4), EALIGN), (dict(y=A[7] + 2), EALIGN), (dict(x=A[3] + 1), EALIGN),
    (dict(rows=0, si=None, so=None, x=None, f=None, y=None, parent=None, rate=None), OK)])
def test_step_checks(kw, code):
    assert step(**kw) == code


def embed(t=A[0], w=A[1], scale=1.0, y=A[2], rows=10, vocab=100, dim=64, dtype=BF16, out=F32):
    return ssd.raw_call("ssd_embedding", t, w, scale, y, rows, vocab, dim, dtype, out, None)


def embed_bwd(dy=A[0], t=A[1], scale=1.0, d=A[2], acc=0, rows=10, vocab=100, dim=64, dtype=BF16, out=F32, ws=A[3], wsb=1 << 31):
    return ssd.raw_call("ssd_embedding_bwd", dy, t, scale, d, acc, rows, vocab, dim, dtype, out, ws, wsb, None)


EMBED = [(dict(rows=-1), ESHAPE), (dict(vocab=0), ESHAPE), (dict(dim=0), ESHAPE), (dict(rows=1 << 31), EUNSUP), (dict(vocab=(1 << 20) + 1), EUNSUP),
         (dict(dim=(1 << 20) + 1), EUNSUP), (dict(dtype=2), EUNSUP), (dict(out=-1), EUNSUP)]


@pytest.mark.parametrize("kw,code", EMBED + [
    (dict(t=None), ENULL), (dict(w=None), ENULL), (dict(y=None), ENULL), (dict(t=A[0] + 4), EALIGN), (dict(w=A[1] + 2), EALIGN),
    (dict(y=A[1]), EUNSUP), (dict(y=A[0]), EUNSUP), (dict(rows=0, t=None, w=None, y=None), OK)])
def test_embedding_checks(kw, code):
    assert embed(**kw) == code


@pytest.mark.parametrize("kw,code", EMBED + [
    (dict(dy=None), ENULL), (dict(t=None), ENULL), (dict(d=None), ENULL), (dict(ws=None), EWS), (dict(wsb=256), EWS), (dict(ws=A[3] + 16), EALIGN),
    (dict(d=A[0]), EUNSUP), (dict(d=A[1]), EUNSUP), (dict(d=A[2] + 8), EALIGN), (dict(rows=0, dy=None, t=None, acc=1, ws=None, wsb=0), OK)])
def test_embedding_gradient_checks(kw, code):
    assert embed_bwd(**kw) == code


def logits(l=A[0], o=A[1], t=A[2], cap=50, n=A[3], p=A[4], rep=A[5], pres=A[6], freq=A[7], b=A[8], nb=1, m=A[9], nm=4, rows=4, vocab=1000, dtype=BF16):
    return ssd.raw_call("ssd_logits_process", l, o, t, cap, n, p, rep, pres, freq, b, nb, m, nm, rows, vocab, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(l=None), ENULL), (dict(o=None), ENULL), (dict(t=None), ENULL), (dict(rows=-1), ESHAPE), (dict(vocab=0), ESHAPE), (dict(cap=-1), ESHAPE),
    (dict(nb=2), ESHAPE), (dict(nm=3), ESHAPE), (dict(nb=0), ESHAPE), (dict(vocab=(1 << 28) + 1), EUNSUP), (dict(cap=1 << 31), EUNSUP),
    (dict(rows=1 << 24, nm=1), EUNSUP), (dict(dtype=9), EUNSUP), (dict(l=A[0] + 2), EALIGN), (dict(o=A[1] + 4), EALIGN), (dict(t=A[2] + 4), EALIGN),
    (dict(m=A[9] + 4), EALIGN), (dict(b=A[8] + 4), EALIGN), (dict(o=A[0] + 16), EUNSUP), (dict(o=A[2]), EUNSUP), (dict(o=A[9]), EUNSUP),
    (dict(rows=0, l=None, o=None, nm=1), OK)])
def test_logits_checks(kw, code):
    assert logits(**kw) == code


def quantize(x=A[0], q=A[1], s=A[2], rows=8, dim=100, dtype=BF16):
    return ssd.raw_call("ssd_int_quantize", x, q, s, rows, dim, dtype, None)


def linear(xq=A[0], xs=A[1], wq=A[2], ws_=A[3], b=A[4], act=0, r=A[5], y=A[6], rows=100, k=64, n=48, dtype=BF16, ws=A[7], wsb=1 << 31):
    return ssd.raw_call("ssd_linear_int", xq, xs, wq, ws_, b, act, r, y, rows, k, n, dtype, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ENULL), (dict(q=None), ENULL), (dict(s=None), ENULL), (dict(rows=-1), ESHAPE), (dict(dim=0), ESHAPE), (dict(dtype=2), EUNSUP),
    (dict(dim=(1 << 20) + 1), EUNSUP), (dict(rows=1 << 40), EUNSUP), (dict(q=A[0]), EUNSUP), (dict(s=A[1]), EUNSUP), (dict(x=A[0] + 2), EALIGN),
    (dict(rows=0, x=None), OK)])
def test_quantize_checks(kw, code):
    assert quantize(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(xq=None), ENULL), (dict(xs=None), ENULL), (dict(wq=None), ENULL), (dict(ws_=None), ENULL), (dict(y=None), ENULL), (dict(rows=-1), ESHAPE),
    (dict(k=0), ESHAPE), (dict(k=72), ESHAPE), (dict(n=0), ESHAPE), (dict(rows=(1 << 24) + 1), EUNSUP), (dict(k=131072 + 16), EUNSUP),
    (dict(n=(1 << 20) + 1), EUNSUP), (dict(act=3), EUNSUP), (dict(dtype=2), EUNSUP), (dict(xq=A[0] + 1), EALIGN), (dict(ws_=A[3] + 4), EALIGN),
    (dict(b=A[4] + 4), EALIGN), (dict(y=A[0]), EUNSUP), (dict(y=A[5] + 16), EUNSUP), (dict(k=8192, ws=None), EWS), (dict(k=8192, wsb=100), EWS),
    (dict(k=8192, ws=A[7] + 16), EALIGN), (dict(rows=0, xq=None, xs=None, wq=None, ws_=None, y=None), OK)])
def test_linear_checks(kw, code):
    assert linear(**kw) == code


def test_workspaces():
    lib = ssd.load()
    for q, args in ((lib.ssd_gated_scan_fwd_workspace_bytes, (BF16,)), (lib.ssd_gated_scan_bwd_workspace_bytes, (RATE, F32))):
        assert q(-1, 5, 8, *args) == NONE and q(1, 5, 0, *args) == NONE and q(1, 1 << 40, 8, *args) == NONE
        assert q(0, 5, 8, *args) < 1 << 20
    assert lib.ssd_gated_scan_bwd_workspace_bytes(1, 5, 8, 3, F32) == NONE
    q = lib.ssd_embedding_bwd_workspace_bytes
    assert q(0, 10, 8) == 0 and q(-1, 10, 8) == NONE and q(10, 0, 8) == NONE and q(10, 1 << 21, 8) == NONE
    assert q(100, 10, 8) >= 800
    q = lib.ssd_linear_int_workspace_bytes
    assert q(8, 2048, 8512) == 0 and q(8, 40, 64) == NONE and q(0, 64, 64) == 0 and q(60, 4096, 200) > 0


def test_binding_refuses():
    import torch
    x = torch.zeros(2, 5, 8)
    with pytest.raises(ValueError):
        ssd.ssd_gated_scan_fwd(x, x, decay="tanh")
    with pytest.raises(ValueError):
        ssd.ssd_gated_scan_fwd(x, x, decay="rate")
    with pytest.raises(ValueError):
        ssd.ssd_gated_scan_fwd(x, x, decay="log", rate=torch.zeros(8))
    with pytest.raises(TypeError):
        ssd.ssd_gated_scan_fwd(x.half(), x.half(), decay="log")
    with pytest.raises(ValueError):   # not on the GPU
        ssd.ssd_gated_scan_fwd(x, x, decay="log")
    with pytest.raises(ValueError):
        ssd.ssd_gated_step(torch.zeros(2, 8), torch.zeros(2, 8), x, x, decay="log")
    with pytest.raises(ValueError):
        ssd.ssd_embedding(torch.zeros(3, dtype=torch.int32), torch.zeros(8))
    with pytest.raises(TypeError):
        ssd.ssd_embedding(torch.zeros(3, dtype=torch.int32), torch.zeros(8, 4), dtype=torch.float16)
    with pytest.raises(ValueError):
        ssd.ssd_embedding_bwd(torch.zeros(3, 4), torch.zeros(3, dtype=torch.int32), 10, accumulate=True)
    with pytest.raises(ValueError):
        ssd.ssd_logits_process(torch.zeros(3, 40))
    with pytest.raises(ValueError):
        ssd.ssd_linear_int(torch.zeros(3, 40), torch.zeros(3), torch.zeros(4, 32), torch.zeros(4))
    with pytest.raises(ValueError):
        ssd.ssd_linear_int(torch.zeros(3, 32), torch.zeros(3), torch.zeros(4, 32), torch.zeros(4), act="relu")


def test_which_tokens_may_lie_apart():
    """The strides a recurrence's input may have (checked on the CPU: the device is given)."""
    import torch
    ssd.load()
    base = torch.zeros(2, 5, 3 * 8)
    dev = -1  # of a CPU tensor
    def ld(t, shape=None):
        return ssd._tokens(dev, "x", t, t.shape if shape is None else shape, torch.float32)[1]
    assert ld(base[..., :8]) == 24 and ld(base[..., 8:16]) == 24 and ld(torch.zeros(2, 5, 8)) == 8
    assert ld(base[:1, :, :8]) == 24 and ld(base[:, 0, :8]) == 5 * 24 and ld(base[:, :1, :8]) == 5 * 24
    assert ld(torch.zeros(1, 1, 8)) == 8 and ld(base[0, :, 3:11]) == 24
    for bad in (base[:, :3, :8], base[..., ::3], base.transpose(0, 1)[..., :8], torch.zeros(2, 1, 8).expand(2, 5, 8)):
        with pytest.raises(ValueError):
            ld(bad)
