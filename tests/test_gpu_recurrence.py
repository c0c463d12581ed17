"""GPU tests of the gated linear recurrence (ssd_gated_scan_fwd, ssd_gated_scan_bwd, ssd_gated_step) against the formulas
in 64 bits.

Tolerances, fixed before the first run. A decay a_t is within EPS = 2^-21 (1 + max |log a|) of itself (its exponential
2^-22, its logarithm 2^-22 of itself, one rounding to multiply by it), a coefficient c_t within 4 EPS. A state's term s
tokens back passes s decays, so with M_t = a M_(t-1) + |u_t| (the magnitudes) and K_t = a (K_(t-1) + M_(t-1)) (weighted by
their age) the state is within EPS (K_t + 8 M_t). The same goes for the gradient's g_t backward in time, and a product of
the two adds both errors. Stored values are off by half a step, HALF[type], beside that.
"""
from __future__ import annotations

import pytest

from tests.gpu_util import log

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = 1e-37


def _t(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _draw(batch, T, dim, dtype, decay, gated, resets, initial, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + 1000 * T + dim)
    def r(*s):
        return torch.randn(*s, device="cuda", generator=g)
    s = dict(decay=decay)
    s["x"] = r(batch, T, dim).to(_t(dtype))
    s["f"] = (-0.1 * torch.exp(1.5 * r(batch, T, dim)) if decay == "log" else 2 + r(batch, T, dim)).to(_t(dtype))
    s["rate"] = torch.log(0.9 + 0.099 * torch.rand(dim, device="cuda", generator=g)) if decay == "rate" else None
    s["in_gate"] = r(batch, T, dim).to(_t(dtype)) if gated else None
    s["reset"] = torch.rand(batch, T, device="cuda", generator=g) < 0.02 if resets else None
    s["initial_state"] = r(batch, dim) if initial else None
    s["dy"] = r(batch, T, dim).to(_t(dtype))
    s["d_final_state"] = r(batch, dim) if initial else None
    return s


def _parts(s):
    """log a, a (0 where reset), its unreset value, c, slope of c for log a, v, and the gates."""
    import torch
    f, x = s["f"].double(), s["x"].double()
    gate = torch.sigmoid(s["in_gate"].double()) if s["in_gate"] is not None else torch.ones_like(x)
    p = torch.sigmoid(f)
    if s["decay"] == "log":
        la, c = f, torch.ones_like(f)
        a = torch.exp(la)
        slope, per_f = torch.zeros_like(f), torch.ones_like(f)
    elif s["decay"] == "sigmoid":
        la, c = torch.nn.functional.logsigmoid(f), torch.sigmoid(-f)
        a = torch.exp(la)
        slope, per_f = -a, c
    else:
        la = s["rate"].double() * p
        a, c = torch.exp(la), torch.sqrt(-torch.expm1(2 * la))
        slope, per_f = torch.where(c > 0, -a * a / c, torch.zeros_like(c)), la * torch.sigmoid(-f)
    kept = a.clone()
    if s["reset"] is not None:
        kept[s["reset"].bool()] = 0
    return dict(la=la, a=a, kept=kept, c=c, slope=slope, per_f=per_f, x=x, v=gate * x, gate=gate, p=p,
                eps=2.0 ** -21 * (1 + float(la.abs().max()) if la.numel() else 1))


def _forward(s):
    """Per token h, its error's bound, magnitudes; and the states before each token (h, bound, magnitude)."""
    import torch
    q = _parts(s)
    B, T, D = q["x"].shape
    h = s["initial_state"].double() if s["initial_state"] is not None else torch.zeros(B, D, device="cuda", dtype=torch.float64)
    M, K = h.abs(), torch.zeros_like(h)
    out = {k: [] for k in ("h", "E", "M", "before", "before_E", "before_M")}
    for t in range(T):
        a, u = q["kept"][:, t], (q["c"] * q["v"])[:, t]
        for k, v in (("before", h), ("before_E", q["eps"] * (K + 8 * M)), ("before_M", M)):
            out[k].append(v)
        h, K, M = a * h + u, a * (K + M), a * M + u.abs()
        for k, v in (("h", h), ("E", q["eps"] * (K + 8 * M)), ("M", M)):
            out[k].append(v)
    return q, {k: torch.stack(v, 1) if v else torch.zeros(B, 0, D, device="cuda") for k, v in out.items()}, h


def _near(got, ref, lim, half, what):
    err = (got.double() - ref).abs()
    lim = lim + half * ref.abs() + TINY
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert not bool((~(err <= lim)).any()), (what, float((err - lim).max()), float((err / lim).max()))


def _check(ssd, s, dtype, name):
    import torch
    q, ref, last = _forward(s)
    B, T, D = s["x"].shape
    call = {k: s[k] for k in ("decay", "rate", "in_gate", "reset")}
    y, final, states = ssd.ssd_gated_scan_fwd(s["x"], s["f"], initial_state=s["initial_state"], want_states=True, **call)
    grads = ssd.ssd_gated_scan_bwd(s["dy"], s["x"], s["f"], states, d_final_state=s["d_final_state"], **call)
    again = ssd.ssd_gated_scan_fwd(s["x"], s["f"], initial_state=s["initial_state"], **call)
    more = ssd.ssd_gated_scan_bwd(s["dy"], s["x"], s["f"], states, d_final_state=s["d_final_state"], **call)
    torch.cuda.synchronize()
    assert again[2] is None and torch.equal(y, again[0]) and torch.equal(final, again[1]), "the same bits"
    assert all(a is b if a is None else torch.equal(a, b) for a, b in zip(grads, more)), "the same bits"
    half = HALF[dtype]
    _near(y, ref["h"], ref["E"], half, name + " y")
    _near(final, last, ref["E"][:, -1], 2.0 ** -24, name + " final")
    _near(states, ref["before"][:, ::ssd.GATED_CHUNK], ref["before_E"][:, ::ssd.GATED_CHUNK], 2.0 ** -24, name + " states")

    # backward: g_t = dy_t + kept_(t+1) g_(t+1)
    eps = q["eps"]
    back = s["d_final_state"].double() if s["d_final_state"] is not None else torch.zeros(B, D, device="cuda", dtype=torch.float64)
    bM, bK = back.abs(), torch.zeros_like(back)
    g, gE, gM = torch.empty_like(q["x"]), torch.empty_like(q["x"]), torch.empty_like(q["x"])
    for t in range(T - 1, -1, -1):
        g[:, t] = s["dy"][:, t].double() + back
        m = s["dy"][:, t].double().abs() + bM
        gM[:, t], gE[:, t] = m, eps * (bK + 8 * m)
        a = q["kept"][:, t]
        back, bK, bM = a * g[:, t], a * (bK + m), a * m
    dx, df, di, drate, d0 = grads
    _near(d0, back, eps * (bK + 8 * bM), 2.0 ** -24, name + " d_initial")
    c, gate, v = q["c"], q["gate"], q["v"]
    _near(dx, g * c * gate, c * gate * (gE + 8 * eps * gM), half, name + " dx")
    if di is not None:
        w = c * v * (1 - gate)
        _near(di, g * w, w.abs() * (gE + 16 * eps * gM), half, name + " di")
    terms = q["kept"] * ref["before"] + q["slope"] * v
    mag = q["kept"] * ref["before_M"] + (q["slope"] * v).abs()
    dla = g * terms
    lim = gE * mag + gM * (q["kept"] * ref["before_E"] + 16 * eps * mag)
    _near(df, dla * q["per_f"], (lim + 16 * eps * gM * mag) * q["per_f"].abs(), half, name + " df")
    if drate is not None:
        big = (gM * mag * q["p"]).sum((0, 1))
        _near(drate, (dla * q["p"]).sum((0, 1)), (lim * q["p"]).sum((0, 1)) + 512 * 2.0 ** -24 * big, 2.0 ** -24, name + " drate")


SHAPES = [(1, 1, 1), (2, 3, 7), (1, 127, 64), (3, 128, 65), (1, 129, 8), (2, 300, 515), (1, 1000, 40), (1, 257, 1536),
          (5, 64, 96), (9, 2, 200), (1, 2500, 24), (2, 640, 72)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("decay", ["log", "sigmoid", "rate"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_and_gradients(ssd, shape, decay, dtype):
    log(f"[recurrence] {shape} {decay} {dtype}")
    k = SHAPES.index(shape)
    _check(ssd, _draw(*shape, dtype, decay, k % 2 == 0, k % 3 == 0, k % 4 < 2), dtype, f"{shape} {decay} {dtype}")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("resets", [False, True])
@pytest.mark.parametrize("initial", [False, True])
@pytest.mark.parametrize("dtype,dim", [("bf16", 136), ("f32", 68), ("bf16", 51)])
def test_every_combination(ssd, gated, resets, initial, dtype, dim):
    for decay in ("log", "sigmoid", "rate"):
        _check(ssd, _draw(2, 270, dim, dtype, decay, gated, resets, initial, seed=7), dtype, f"{dim} {decay} {dtype}")


@pytest.mark.parametrize("T", [128 * 16, 128 * 17 + 5, 128 * 40 + 1])
def test_many_chunks(ssd, T):
    """States that live for thousands of tokens, handed from chunk to chunk many times."""
    import torch
    for dtype, dim in (("bf16", 64), ("f32", 33)):
        s = _draw(1, T, dim, dtype, "log", True, False, True, seed=T)
        s["f"] = (-0.001 * torch.rand_like(s["f"].float())).to(_t(dtype))
        _check(ssd, s, dtype, f"T {T} {dtype}")


@pytest.mark.parametrize("shape", [(2, 700, 3), (1, 513, 5), (3, 260, 1), (1, 1300, 9), (2, 400, 65)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_narrow_rows_of_several_chunks(ssd, shape, dtype):
    for decay in ("log", "sigmoid", "rate"):
        _check(ssd, _draw(*shape, dtype, decay, True, True, True, seed=13), dtype, f"{shape} {decay} {dtype}")


@pytest.mark.parametrize("B,T,D", [(1, 16384, 4160), (3, 9000, 1500), (5, 4000, 2600)])
def test_more_chunks_than_tickets(ssd, B, T, D):
    """So many chunks that a ticket is for two of them, with odd numbers of columns: parts have the bits of a call alone."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)
    x, f, dy = (torch.randn(B, T, D, device="cuda", generator=g).bfloat16() for _ in range(3))
    rate = torch.log(0.9 + 0.099 * torch.rand(D, device="cuda", generator=g))
    reset = torch.rand(B, T, device="cuda", generator=g) < 0.001
    y, final, st = ssd.ssd_gated_scan_fwd(x, f, decay="rate", rate=rate, reset=reset, want_states=True)
    grads = ssd.ssd_gated_scan_bwd(dy, x, f, st, decay="rate", rate=rate, reset=reset)
    for d in (0, D // 2 // 8 * 8, D - 40):
        part = [t[..., d:d + 40].contiguous() for t in (x, f, dy)]
        r = rate[d:d + 40].contiguous()
        yp, fp, sp = ssd.ssd_gated_scan_fwd(part[0], part[1], decay="rate", rate=r, reset=reset, want_states=True)
        gp = ssd.ssd_gated_scan_bwd(part[2], part[0], part[1], sp, decay="rate", rate=r, reset=reset)
        torch.cuda.synchronize()
        assert torch.equal(y[..., d:d + 40], yp) and torch.equal(final[:, d:d + 40], fp) and torch.equal(st[..., d:d + 40], sp)
        for a, b in ((grads[0], gp[0]), (grads[1], gp[1]), (grads[3], gp[3]), (grads[4], gp[4])):
            assert torch.equal(a[..., d:d + 40], b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 72, 37])
def test_views_of_one_projection(ssd, dtype, dim):
    """x, f and the gate as parts of one tensor, tokens apart, give the bits of contiguous copies; the rest of it
    is left alone, also by the step."""
    import torch
    s = _draw(2, 150, dim, dtype, "rate", True, True, True)
    wide = torch.full((2, 150, 3 * dim + 5), 7.0, device="cuda").to(_t(dtype))
    views = [wide[..., k * dim + k:(k + 1) * dim + k] for k in range(3)]
    for v, k in zip(views, ("x", "f", "in_gate")):
        v.copy_(s[k])
    kept = wide.clone()
    call = dict(decay="rate", rate=s["rate"], reset=s["reset"])
    a = ssd.ssd_gated_scan_fwd(s["x"], s["f"], in_gate=s["in_gate"], initial_state=s["initial_state"], want_states=True, **call)
    b = ssd.ssd_gated_scan_fwd(views[0], views[1], in_gate=views[2], initial_state=s["initial_state"], want_states=True, **call)
    ga = ssd.ssd_gated_scan_bwd(s["dy"], s["x"], s["f"], a[2], in_gate=s["in_gate"], **call)
    gb = ssd.ssd_gated_scan_bwd(s["dy"], views[0], views[1], b[2], in_gate=views[2], **call)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b)) and all(torch.equal(p, q) for p, q in zip(ga, gb))
    h1, h2 = torch.empty(2, dim, device="cuda"), torch.empty(2, dim, device="cuda")
    t = 3
    y1 = ssd.ssd_gated_step(s["initial_state"], h1, s["x"][:, t].contiguous(), s["f"][:, t].contiguous(), decay="rate", rate=s["rate"],
                            in_gate=s["in_gate"][:, t].contiguous())
    y2 = ssd.ssd_gated_step(s["initial_state"], h2, views[0][:, t], views[1][:, t], decay="rate", rate=s["rate"], in_gate=views[2][:, t])
    torch.cuda.synchronize()
    assert torch.equal(y1, y2) and torch.equal(h1, h2) and torch.equal(wide, kept)


def _guard(shape, dtype):
    import torch
    n = 1
    for v in shape:
        n *= v
    buf = torch.full((n + 4096,), 7.0, device="cuda").to(dtype)
    return buf[:n].view(shape), lambda: bool((buf[n:].float() == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(2, 131, 67), (1, 300, 96), (3, 1, 1)])
def test_nothing_behind_the_output(ssd, dtype, shape):
    import torch
    s = _draw(*shape, dtype, "sigmoid", True, False, False)
    y, fine = _guard(shape, _t(dtype))
    out, _, _ = ssd.ssd_gated_scan_fwd(s["x"], s["f"], decay="sigmoid", in_gate=s["in_gate"], y=y)
    want, _, _ = ssd.ssd_gated_scan_fwd(s["x"], s["f"], decay="sigmoid", in_gate=s["in_gate"])
    torch.cuda.synchronize()
    assert out is y and torch.equal(y, want) and fine()


def test_empty(ssd):
    import torch
    h0 = torch.randn(2, 24, device="cuda")
    x = torch.empty(2, 0, 24, device="cuda")
    y, final, states = ssd.ssd_gated_scan_fwd(x, x, decay="log", initial_state=h0, want_states=True)
    assert y.shape == (2, 0, 24) and torch.equal(final, h0) and states.shape == (2, 0, 24)
    _, final, _ = ssd.ssd_gated_scan_fwd(x, x, decay="log")
    assert not bool(final.any())
    rate = -torch.rand(24, device="cuda")
    g = ssd.ssd_gated_scan_bwd(x, x, x, states, decay="rate", rate=rate, d_final_state=h0)
    assert torch.equal(g[4], h0) and not bool(g[3].any())
    x = torch.empty(0, 5, 24, device="cuda")
    y, final, _ = ssd.ssd_gated_scan_fwd(x, x, decay="log")
    assert y.shape == (0, 5, 24) and final.shape == (0, 24)
    g = ssd.ssd_gated_scan_bwd(x, x, x, torch.empty(0, 1, 24, device="cuda"), decay="rate", rate=rate)
    assert not bool(g[3].any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["log", "sigmoid", "rate"])
def test_a_document_keeps_its_values_to_itself(ssd, decay, dtype):
    """Infinities and NaN in one document, channel or sequence reach no other: the rest has the bits that it has without
    them, forward and backward."""
    import torch
    s = _draw(2, 400, 40, dtype, decay, True, False, False, seed=3)
    s["reset"] = torch.zeros(2, 400, dtype=torch.bool, device="cuda")
    s["reset"][:, [100, 256, 300]] = True
    call = {k: s[k] for k in ("decay", "rate", "reset")}
    def both(x, dy):
        y, final, st = ssd.ssd_gated_scan_fwd(x, s["f"], in_gate=s["in_gate"], want_states=True, **call)
        g = ssd.ssd_gated_scan_bwd(dy, x, s["f"], st, in_gate=s["in_gate"], **call)
        torch.cuda.synchronize()
        return y, final, g
    y0, f0, g0 = both(s["x"], s["dy"])
    x, dy = s["x"].clone(), s["dy"].clone()
    x[0, 150, 5], x[0, 260, 6], x[0, 257, 7] = float("nan"), float("inf"), float("-inf")
    dy[0, 290, 9] = float("nan")
    y1, f1, g1 = both(x, dy)
    assert torch.equal(f0, f1)   # the last document, from token 300 on, and the others
    hurt = torch.zeros(2, 400, 40, dtype=torch.bool, device="cuda")
    hurt[0, 150:256, 5] = hurt[0, 260:300, 6] = hurt[0, 257:300, 7] = True
    assert torch.equal(y0[~hurt], y1[~hurt]) and bool((~torch.isfinite(y1[hurt])).all())
    back = hurt.clone()
    back[0, 256:291, 9] = True
    for a, b in zip(g0[:3], g1[:3]):
        assert torch.equal(a[~back], b[~back])
    assert torch.equal(g0[4], g1[4])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_gates(ssd, dtype):
    """Decays of 1 (a rate of 0, a gate far below zero) and 0, inputs shut out: finite, with finite gradients."""
    import torch
    t = _t(dtype)
    x = torch.randn(1, 200, 16, device="cuda").to(t)
    f = torch.full((1, 200, 16), -300.0, device="cuda").to(t)
    f[..., 4:8], f[..., 8:12] = 300.0, float("-inf")
    f[..., 12:] = float("inf")
    h0 = torch.randn(1, 16, device="cuda")
    for decay in ("sigmoid", "rate"):
        rate = torch.zeros(16, device="cuda") if decay == "rate" else None
        y, final, st = ssd.ssd_gated_scan_fwd(x, f, decay=decay, rate=rate, in_gate=f, initial_state=h0, want_states=True)
        g = ssd.ssd_gated_scan_bwd(x, x, f, st, decay=decay, rate=rate, in_gate=f)
        torch.cuda.synchronize()
        assert all(bool(torch.isfinite(v).all()) for v in (y, final, *[v for v in g if v is not None]))
        if decay == "rate":
            assert torch.equal(final, h0)  # decay 1, no input
        else:
            want = torch.where(torch.arange(16, device="cuda") // 4 % 2 == 1, h0, torch.zeros_like(h0))
            assert torch.equal(final, want)  # kept whole, or (decay 0, input gate 0) nothing
    y, final, _ = ssd.ssd_gated_scan_fwd(x, torch.full_like(f, float("-inf")), decay="log", initial_state=h0)
    torch.cuda.synchronize()
    assert torch.equal(y, x) and torch.equal(final, x[:, -1].float())


@pytest.mark.parametrize("decay", ["log", "sigmoid", "rate"])
def test_gradients_against_differences(ssd, decay):
    """fp32, small: the gradient along a random direction against central differences of the 64-bit formula."""
    import torch
    s = _draw(2, 140, 5, "f32", decay, True, True, True, seed=11)
    names = ["x", "f", "in_gate", "initial_state"] + (["rate"] if decay == "rate" else [])
    y, final, st = ssd.ssd_gated_scan_fwd(s["x"], s["f"], decay=decay, rate=s["rate"], in_gate=s["in_gate"], reset=s["reset"],
                                          initial_state=s["initial_state"], want_states=True)
    g = ssd.ssd_gated_scan_bwd(s["dy"], s["x"], s["f"], st, decay=decay, rate=s["rate"], in_gate=s["in_gate"], reset=s["reset"],
                               d_final_state=s["d_final_state"])
    torch.cuda.synchronize()
    grads = dict(x=g[0], f=g[1], in_gate=g[2], rate=g[3], initial_state=g[4])
    gen = torch.Generator(device="cuda").manual_seed(1)
    for n in names:
        way = torch.randn(s[n].shape, device="cuda", generator=gen).double()
        if n == "rate":
            way *= 0.01
        def value(step):
            v = dict(s)
            v[n] = s[n].double() + step * way
            _, ref, last = _forward(v)
            return float((ref["h"] * s["dy"].double()).sum() + (last * s["d_final_state"].double()).sum())
        # central differences in 64 bits: third derivatives of some 1e3 times 1e-8 / 6, beside fp32 gradients
        want, got = (value(1e-4) - value(-1e-4)) / 2e-4, float((grads[n].double() * way).sum())
        scale = float((grads[n].double() * way).abs().sum())
        assert abs(got - want) <= 2e-5 * scale, (n, got, want, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["log", "sigmoid", "rate"])
@pytest.mark.parametrize("rows,dim,gated", [(1, 1, True), (8, 1536, False), (5, 515, True), (3, 4096, True), (700, 33, False)])
def test_step(ssd, dtype, decay, rows, dim, gated):
    import torch
    s = _draw(rows, 1, dim, dtype, decay, gated, False, True, seed=5)
    src = rows + 2
    state = torch.randn(src, dim, device="cuda")
    parent = torch.randint(0, src, (rows,), device="cuda", dtype=torch.int32)
    if rows > 2:
        parent[0], parent[1] = -1, src   # a sequence begins
    before = torch.where(((parent >= 0) & (parent < src))[:, None], state[parent.clamp(0, src - 1).long()], torch.zeros(1, device="cuda"))
    _, ref, _ = _forward(dict(s, initial_state=before))
    args = (s["x"][:, 0], s["f"][:, 0])
    kw = dict(decay=decay, rate=s["rate"], in_gate=None if s["in_gate"] is None else s["in_gate"][:, 0])
    out, fine = _guard((rows, dim), torch.float32)
    y = ssd.ssd_gated_step(state, out, *args, parent=parent, **kw)
    torch.cuda.synchronize()
    _near(out, ref["h"][:, 0], ref["E"][:, 0], 2.0 ** -24, "state")
    _near(y, ref["h"][:, 0], ref["E"][:, 0], HALF[dtype], "y")
    assert fine()
    # in place, each row from its own
    own = before.clone()
    y2 = ssd.ssd_gated_step(own, own, *args, **kw)
    torch.cuda.synchronize()
    assert torch.equal(own, out) and torch.equal(y2, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_are_the_scan(ssd, dtype):
    """Token by token from the scan's state: the scan over both pieces."""
    import torch
    s = _draw(3, 150, 48, dtype, "rate", True, False, True, seed=9)
    kw = dict(decay="rate", rate=s["rate"])
    q, ref, last = _forward(s)
    _, state, _ = ssd.ssd_gated_scan_fwd(s["x"][:, :140].contiguous(), s["f"][:, :140].contiguous(), in_gate=s["in_gate"][:, :140].contiguous(),
                                         initial_state=s["initial_state"], **kw)
    for t in range(140, 150):
        y = ssd.ssd_gated_step(state, state, s["x"][:, t], s["f"][:, t], in_gate=s["in_gate"][:, t], **kw)
        torch.cuda.synchronize()
        _near(y, ref["h"][:, t], ref["E"][:, t], HALF[dtype], t)
    _near(state, last, ref["E"][:, -1], 2.0 ** -24, "final")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_replayed(ssd, dtype):
    """Forward and backward captured together, replayed with new inputs beside eager calls of the same workspace sizes;
    on a stream of their own."""
    import torch
    s = _draw(2, 700, 96, dtype, "rate", True, True, True, seed=21)
    call = {k: s[k] for k in ("decay", "rate", "in_gate", "reset")}
    def run(stream=None):
        y, final, st = ssd.ssd_gated_scan_fwd(s["x"], s["f"], initial_state=s["initial_state"], want_states=True, stream=stream, **call)
        return [y, final, st] + list(ssd.ssd_gated_scan_bwd(s["dy"], s["x"], s["f"], st, d_final_state=s["d_final_state"], stream=stream, **call))
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for r in range(4):
        s["x"].normal_()
        s["dy"].normal_()
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), r
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side)
    also = run()   # at the same time on the current stream
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, got, also))
