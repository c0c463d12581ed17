"""GPU tests of the operators together, as a Mamba-2 decoder runs them: a decode loop with beam search (norm, input
projection, decode step from the chosen beams' states, gated norm, output projection with the residual, logits,
selection), the same projections in 8 bits, and one training step of a layer, each against the plain formulas in
64 bits."""
from __future__ import annotations

import math

import pytest

from tests.gpu_util import log

pytestmark = pytest.mark.gpu

EPS = 1e-5


class Layer:
    """One layer's sizes and weights (fp32 draws, stored in `dtype`)."""

    def __init__(self, g, dtype, d=96, H=4, P=32, N=32, G=2):
        import torch
        self.d, self.H, self.P, self.N, self.G = d, H, P, N, G
        self.inner, self.bc = H * P, G * N
        def r(*s, sc=1.0):
            return sc * torch.randn(*s, device="cuda", generator=g)
        self.w_in = r(2 * self.inner + 2 * self.bc + H, d, sc=d ** -0.5).to(dtype)
        self.w_out = r(d, self.inner, sc=self.inner ** -0.5).to(dtype)
        self.norm1, self.norm2 = 1 + r(d, sc=0.1), 1 + r(self.inner, sc=0.1)
        self.A, self.D, self.dt_bias = -torch.exp(r(H, sc=0.5)), r(H), r(H) - 2
        self.conv_w, self.conv_b = r(self.inner, 4, sc=0.5), r(self.inner, sc=0.1)

    def split(self, zxbcdt):
        i, bc, b = self.inner, self.bc, zxbcdt.shape[0]
        z, x, B, C, dt = zxbcdt.split([i, i, bc, bc, self.H], -1)
        return (z.reshape(b, self.H, self.P).contiguous(), x.reshape(b, self.H, self.P).contiguous(),
                B.reshape(b, self.G, self.N).contiguous(), C.reshape(b, self.G, self.N).contiguous(), dt.contiguous())


def _decoder(dtype, seed=3, layers=2, vocab=517):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    ls = [Layer(g, dtype) for _ in range(layers)]
    embed = torch.randn(vocab, ls[0].d, device="cuda", generator=g).to(dtype)
    head = (3 * torch.randn(vocab, ls[0].d, device="cuda", generator=g) * ls[0].d ** -0.5).to(dtype)
    return ls, embed, head, torch.ones(ls[0].d, device="cuda")


def _step(ssd, model, tokens, states, parent):
    """One token through the decoder: logits, and the states of its beams. The residual stream is fp32."""
    import torch
    ls, embed, head, norm = model
    rows = tokens.numel()
    res = embed[tokens.reshape(-1).long()].float()
    delta = torch.zeros(rows, ls[0].d, device="cuda", dtype=embed.dtype)
    out = []
    for l, (s, c) in zip(ls, states):
        y, res, _ = ssd.ssd_rms_norm(delta, l.norm1, EPS, residual=res)
        z, x, B, C, dt = l.split(ssd.ssd_linear(y, l.w_in)[0])
        s2 = torch.empty(rows, *s.shape[1:], device="cuda")
        c2 = torch.empty(rows, *c.shape[1:], device="cuda", dtype=c.dtype)
        y = ssd.ssd_step_beam(s, s2, parent, x, dt, l.A, B, C, l.D, conv_in=c, conv_out=c2, conv_w=l.conv_w,
                              conv_b=l.conv_b, dt_bias=l.dt_bias, dt_softplus=1, z=z)
        y, _, _ = ssd.ssd_rms_norm(y.view(rows, l.inner), l.norm2, EPS, groups=l.G)
        delta, _ = ssd.ssd_linear(y, l.w_out)
        out.append((s2, c2))
    y, _, _ = ssd.ssd_rms_norm(delta, norm, EPS, residual=res)
    return ssd.ssd_linear(y, head)[0], out


def _norm64(h, w, groups=1):
    p = h.unflatten(-1, (groups, -1))
    return (p / (p.square().mean(-1, keepdim=True) + EPS).sqrt()).flatten(-2) * w.double()


def _step64(model, tokens, states, parent):
    import torch
    ls, embed, head, norm = model
    res = embed[tokens.reshape(-1).long()].double()
    p = parent.long()
    out = []
    for l, (s, c) in zip(ls, states):
        z, x, B, C, dt = l.split(_norm64(res, l.norm1) @ l.w_in.double().t())
        s, c = s[p], c[p]
        c = torch.cat([c, x.reshape(len(p), -1, 1)], -1)
        x = (c * l.conv_w.double()).sum(-1) + l.conv_b.double()
        x = (x * torch.sigmoid(x)).view(len(p), l.H, l.P)
        dt = torch.nn.functional.softplus(dt + l.dt_bias.double())
        grp = torch.arange(l.H, device="cuda") * l.G // l.H
        s = torch.exp(dt * l.A.double())[..., None, None] * s + (dt[..., None] * x)[..., None] * B[:, grp][:, :, None]
        y = (s * C[:, grp][:, :, None]).sum(-1) + l.D.double()[:, None] * x
        y = (y * z * torch.sigmoid(z)).flatten(1)
        res = res + _norm64(y, l.norm2, l.G) @ l.w_out.double().t()
        out.append((s, c[..., 1:]))
    return _norm64(res, norm) @ head.double().t(), out


def _new_states(ls, rows, dtype):
    import torch
    return [(torch.zeros(rows, l.H, l.P, l.N, device="cuda", dtype=torch.float64 if dtype == torch.float64 else torch.float32),
             torch.zeros(rows, l.inner, 3, device="cuda", dtype=dtype)) for l in ls]


def _search(ssd, model, dtype, b, k, steps, eos):
    """The loop: what was chosen at each step, and the scores."""
    import torch
    states = _new_states(model[0], 1, dtype)
    parent = torch.full((b * k,), -1, device="cuda", dtype=torch.int32)  # sequences begin: zero states
    tokens = torch.arange(b, device="cuda", dtype=torch.int32).repeat_interleave(k).view(b, k)
    scores = torch.full((b, k), -math.inf, device="cuda")
    scores[:, 0] = 0
    done, said = None, []
    for _ in range(steps):
        logits, states = _step(ssd, model, tokens, states, parent.reshape(-1))
        before = scores
        scores, parent, tokens, done_next = ssd.ssd_beam_select(logits.view(b, k, -1), scores, finished=done, eos=eos)
        said.append((before, done, scores, parent, tokens))
        done = done_next
    return said


def test_beam_search_decode(ssd):
    """fp32 storage: the kernels' scores against the same choices scored in 64 bits. Each step's error is the fp32
    rounding of a few thousand operations, some 1e-6 of values of size 1 to 30; over 6 steps 1e-3 covers it."""
    import torch
    b, k, steps, eos = 3, 4, 6, 5
    model = _decoder(torch.float32)
    said = _search(ssd, model, torch.float32, b, k, steps, eos)
    states = [(torch.zeros(b * k, *s.shape[1:], device="cuda", dtype=torch.float64),
               torch.zeros(b * k, *c.shape[1:], device="cuda", dtype=torch.float64)) for s, c in _new_states(model[0], 1, torch.float64)]
    parent = torch.arange(b * k, device="cuda", dtype=torch.int32)
    tokens = torch.arange(b, device="cuda", dtype=torch.int32).repeat_interleave(k).view(b, k)
    s64 = said[0][0].double()
    for t, (before, done, scores, par, tok) in enumerate(said):
        logits, states = _step64(model, tokens, states, parent.reshape(-1))
        cand = s64[..., None] + torch.log_softmax(logits.view(b, k, -1), -1)
        if done is not None:
            only = torch.full_like(cand, -math.inf)
            only[..., eos] = s64
            cand = torch.where(done[..., None], only, cand)
        best = cand.flatten(1).topk(k).values
        mine = cand.flatten(1).gather(1, ((par % k).long() * cand.shape[-1] + tok.long()))
        log(f"[decoder] step {t}: worst score error {float((scores.double() - mine).abs().max()):.1e}")
        assert float((scores.double() - mine).abs().max()) <= 1e-3
        assert float((best - mine).abs().max()) <= 1e-3      # the choice is a best one
        s64, parent, tokens = mine, par, tok


def test_beam_search_decode_replayed(ssd):
    """bf16 storage: two tokens captured into a graph and replayed with new scores, against eager."""
    import torch
    b, k = 2, 4
    model = _decoder(torch.bfloat16)
    states = [(torch.randn_like(s), torch.randn_like(c)) for s, c in _new_states(model[0], b * k, torch.bfloat16)]
    tokens = torch.randint(0, 500, (b, k), device="cuda", dtype=torch.int32)
    parent = torch.arange(b * k, device="cuda", dtype=torch.int32)
    scores = -5 * torch.rand(b, k, device="cuda")

    def run():
        logits, st = _step(ssd, model, tokens, states, parent)
        one = ssd.ssd_beam_select(logits.view(b, k, -1), scores, eos=3)
        logits, st = _step(ssd, model, one[2], st, one[1].view(-1))
        two = ssd.ssd_beam_select(logits.view(b, k, -1), one[0], finished=one[3], eos=3)
        return list(one) + list(two) + [t for pair in st for t in pair]
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for r in range(3):
        scores.sub_(torch.rand(b, k, device="cuda"))
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), r


def test_prompt_projections_in_8_bits(ssd):
    """Norm into 8 bits, both projections from 8 bits: against the 8-bit operands' own values in 64 bits (sums of fixed
    point in groups of 8: 7 * 2^-13 of the magnitudes; the result's half step), and within the codes' rounding of the
    unrounded layer: an operand's code is off by at most 2^-4, so a sum of k independent ones of two operands by about
    sqrt(2 / 3) 2^-4 = 5.1e-2 at the most, relative in norm."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(4)
    rows, d, n = 700, 512, 900
    x = torch.randn(rows, d, device="cuda", generator=g).bfloat16()
    res = torch.randn(rows, d, device="cuda", generator=g)
    w = torch.randn(n, d, device="cuda", generator=g) * d ** -0.5
    norm = 1 + 0.1 * torch.randn(d, device="cuda", generator=g)
    wq, ws = ssd.ssd_mx_quantize(w)
    q, s, h = ssd.ssd_rms_norm_mx(x, norm, EPS, residual=res)
    y = ssd.ssd_linear_mx(q, s, wq, ws, act="silu")
    torch.cuda.synchronize()
    qv = q.float().double() * s.float().double().repeat_interleave(32, 1)
    wv = wq.float().double() * ws.float().double().repeat_interleave(32, 1)
    z, mag = qv @ wv.t(), qv.abs() @ wv.abs().t()
    ref = z * torch.sigmoid(z)
    assert bool(((y.double() - ref).abs() <= 1.13 * (7 * 2.0 ** -13) * mag + 2.0 ** -8 * ref.abs() + 1e-5 * mag).all())
    full = _norm64(x.double() + res.double(), norm) @ w.double().t()
    assert float((z - full).norm() / full.norm()) <= 5.1e-2


def test_training_step_of_a_layer(ssd):
    """Forward and backward of norm (residual) -> projections -> chunked scan -> norm -> projection with the residual,
    with the framework's operators in fp32, against 64-bit autograd of the plain recurrence. Every gradient passes
    some hundred fp32 sums: 1e-4 relative in norm."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    b, T, d, H, P, N, G, chunk = 2, 70, 48, 4, 32, 32, 2, 64
    inner = H * P
    def r(*s, sc=1.0):
        return sc * torch.randn(*s, device="cuda", generator=g)
    x, res = r(b, T, d), r(b, T, d)
    w = dict(x=r(inner, d, sc=d ** -0.5), B=r(G * N, d, sc=d ** -0.5), C=r(G * N, d, sc=d ** -0.5), out=r(d, inner, sc=inner ** -0.5))
    bias, norm1, norm2 = r(inner, sc=0.3), 1 + r(d, sc=0.1), 1 + r(inner, sc=0.1)
    dt = torch.nn.functional.softplus(r(b, T, H) - 2)
    A, D = -torch.exp(r(H, sc=0.5)), r(H)
    dy = r(b, T, d)

    u, h, rstd1 = ssd.ssd_rms_norm(x, norm1, EPS, residual=res, want_rstd=True)
    X, preX = ssd.ssd_linear(u, w["x"], bias=bias, act="silu", want_preact=True)
    B, _ = ssd.ssd_linear(u, w["B"])
    C, _ = ssd.ssd_linear(u, w["C"])
    X4, B4, C4 = X.view(b, T, H, P), B.view(b, T, G, N), C.view(b, T, G, N)
    Y, _ = ssd.ssd_chunk_scan_fwd(X4, dt, A, B4, C4, D, chunk)
    v, _, rstd2 = ssd.ssd_rms_norm(Y.view(b, T, inner), norm2, EPS, groups=G, want_rstd=True)
    o, _ = ssd.ssd_linear(v, w["out"], residual=h)
    # backward; the residual's gradient is dy
    dv, dwo, _ = ssd.ssd_linear_bwd(dy, v, w["out"])
    dY, _, dn2 = ssd.ssd_rms_norm_bwd(dv, Y.view(b, T, inner), norm2, rstd2, groups=G)
    dX, ddt, dA, dB, dC, dD, _ = ssd.ssd_chunk_scan_bwd(X4, dt, A, B4, C4, D, chunk, dY.view(b, T, H, P))
    du1, dwx, dbx = ssd.ssd_linear_bwd(dX.view(b, T, inner), u, w["x"], act="silu", preact=preX, want_bias=True)
    du2, dwB, _ = ssd.ssd_linear_bwd(dB.view(b, T, G * N), u, w["B"])
    du3, dwC, _ = ssd.ssd_linear_bwd(dC.view(b, T, G * N), u, w["C"])
    dx, _, dn1 = ssd.ssd_rms_norm_bwd(du1 + du2 + du3, h, norm1, rstd1, d_residual_out=dy)
    torch.cuda.synchronize()

    leaves = {k: t.double().cpu().requires_grad_() for k, t in dict(
        x=x, res=res, wx=w["x"], wB=w["B"], wC=w["C"], wo=w["out"], bias=bias, n1=norm1, n2=norm2, dt=dt, A=A, D=D).items()}
    L = leaves
    hh = L["x"] + L["res"]
    uu = _norm64(hh, L["n1"])
    z = uu @ L["wx"].t() + L["bias"]
    XX = (z * torch.sigmoid(z)).view(b, T, H, P)
    BB, CC = (uu @ L["wB"].t()).view(b, T, G, N), (uu @ L["wC"].t()).view(b, T, G, N)
    grp = torch.arange(H) * G // H
    st, ys = torch.zeros(b, H, P, N, dtype=torch.float64), []
    for t in range(T):
        st = torch.exp(L["dt"][:, t] * L["A"])[..., None, None] * st + (L["dt"][:, t][..., None] * XX[:, t])[..., None] * BB[:, t][:, grp][:, :, None]
        ys.append((st * CC[:, t][:, grp][:, :, None]).sum(-1) + L["D"][:, None] * XX[:, t])
    YY = torch.stack(ys, 1).flatten(2)
    oo = _norm64(YY, L["n2"], G) @ L["wo"].t() + hh
    (oo * dy.double().cpu()).sum().backward()
    def rel(a, ref):
        return float((a.double().cpu() - ref).norm() / ref.norm())
    errs = dict(o=rel(o, oo.detach()), x=rel(dx, L["x"].grad), res=rel(dx, L["res"].grad), wx=rel(dwx, L["wx"].grad),
                wB=rel(dwB, L["wB"].grad), wC=rel(dwC, L["wC"].grad), wo=rel(dwo, L["wo"].grad), bias=rel(dbx, L["bias"].grad),
                n1=rel(dn1, L["n1"].grad), n2=rel(dn2, L["n2"].grad), dt=rel(ddt, L["dt"].grad), A=rel(dA, L["A"].grad), D=rel(dD, L["D"].grad))
    log("[layer] " + " ".join(f"{k} {v:.1e}" for k, v in errs.items()))
    assert all(v <= 1e-4 for v in errs.values()), errs
