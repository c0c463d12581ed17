"""GPU tests of a decoder whose mixer is the gated recurrence, from its tokens to its choice: a beam search (embedding, norm,
projections from 8-bit integers, the recurrence's step from the chosen beams' states, logits with penalties, a bias and a
mask, selection), a prompt through the scan and its continuation token by token, and a training step back to the table, each
against the plain formulas in 64 bits."""
from __future__ import annotations

import math

import pytest

from tests.gpu_util import log

pytestmark = pytest.mark.gpu

EPS = 1e-5


class Model:
    """Layers of norm -> one projection (x, gate, input gate) -> recurrence -> projection back, and tied ends."""

    def __init__(self, dtype, d=96, inner=160, vocab=530, layers=2, seed=3):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        def r(*s, sc=1.0):
            return sc * torch.randn(*s, device="cuda", generator=g)
        self.d, self.inner, self.vocab, self.dtype = d, inner, vocab, dtype
        self.table = r(vocab, d, sc=d ** -0.5).to(dtype)
        self.layers = [dict(norm=1 + r(d, sc=0.1), w_in=r(3 * inner, d, sc=d ** -0.5).to(dtype), b_in=r(3 * inner, sc=0.3),
                            w_out=r(d, inner, sc=inner ** -0.5).to(dtype),
                            rate=torch.log(0.9 + 0.099 * torch.rand(inner, device="cuda", generator=g))) for _ in range(layers)]
        self.norm = 1 + r(d, sc=0.1)


def _norm64(h, w):
    return h / (h.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()


def _mix64(l, zxf, state):
    """One token of the recurrence in 64 bits: (y, new state)."""
    import torch
    x, f, i = zxf.chunk(3, -1)
    la = l["rate"].double() * torch.sigmoid(f)
    state = torch.exp(la) * state + torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(i) * x
    return state, state


def test_prompt_then_decode(ssd):
    """fp32: a prompt through the scan, then tokens one by one, against 64 bits throughout. Each layer's error is the fp32
    rounding of some hundred operations on values of size 1 to 10: 2e-4 over two layers and 40 tokens."""
    import torch
    m = Model(torch.float32)
    g = torch.Generator(device="cuda").manual_seed(9)
    tokens = torch.randint(0, m.vocab, (3, 40), device="cuda", generator=g, dtype=torch.int32)
    scale = math.sqrt(m.d)

    def run(tok, states):
        h = ssd.ssd_embedding(tok, m.table, scale=scale)
        new = []
        for l, s in zip(m.layers, states):
            u, _, _ = ssd.ssd_rms_norm(h, l["norm"], EPS)
            p, _ = ssd.ssd_linear(u, l["w_in"], bias=l["b_in"])
            x, f, i = p.split(m.inner, -1)   # views of one projection
            if tok.dim() == 2:
                y, s, _ = ssd.ssd_gated_scan_fwd(x, f, decay="rate", rate=l["rate"], in_gate=i, initial_state=s)
            else:
                out = torch.empty(tok.shape[0], m.inner, device="cuda")
                y = ssd.ssd_gated_step(s, out, x, f, decay="rate", rate=l["rate"], in_gate=i)
                s = out
            new.append(s)
            h, _ = ssd.ssd_linear(y, l["w_out"], residual=h)
        u, _, _ = ssd.ssd_rms_norm(h, m.norm, EPS)
        return ssd.ssd_linear(u, m.table)[0], new

    logits, states = run(tokens[:, :30].contiguous(), [torch.zeros(3, m.inner, device="cuda") for _ in m.layers])
    said = [logits]
    for t in range(30, 40):
        logits, states = run(tokens[:, t].contiguous(), states)
        said.append(logits[:, None])
    said = torch.cat(said, 1)
    torch.cuda.synchronize()

    h = m.table.double()[tokens.long()] * scale
    for l, s in zip(m.layers, states):
        p = _norm64(h, l["norm"]) @ l["w_in"].double().t() + l["b_in"].double()
        st, ys = torch.zeros(3, m.inner, device="cuda", dtype=torch.float64), []
        for t in range(40):
            y, st = _mix64(l, p[:, t], st)
            ys.append(y)
        assert float((s.double() - st).abs().max()) <= 2e-4
        h = h + torch.stack(ys, 1) @ l["w_out"].double().t()
    want = _norm64(h, m.norm) @ m.table.double().t()
    log(f"[recurrent] worst logit error {float((said.double() - want).abs().max()):.1e}")
    assert float((said.double() - want).abs().max()) <= 2e-4


def _search(ssd, m, b, k, steps, eos, int_weights):
    """Beam search: every step's logits as they were chosen from, and the choices."""
    import torch
    rows = b * k
    states = [torch.zeros(rows, m.inner, device="cuda") for _ in m.layers]
    parent = torch.full((rows,), -1, device="cuda", dtype=torch.int32)
    tokens = torch.arange(b, device="cuda", dtype=torch.int32).repeat_interleave(k).view(b, k)
    scores = torch.full((b, k), -math.inf, device="cuda")
    scores[:, 0] = 0
    history = torch.full((rows, steps + 1), -1, device="cuda", dtype=torch.int32)
    history[:, 0] = tokens.view(-1)
    ones = torch.ones(rows, device="cuda")
    bias = torch.linspace(-0.5, 0.5, m.vocab, device="cuda")
    mask = torch.full((-(-m.vocab // 32),), -1, device="cuda", dtype=torch.int32)
    mask[3] = 0x0f0f0f0f
    done, said = None, []
    for t in range(steps):
        h = ssd.ssd_embedding(tokens.view(-1), m.table, scale=math.sqrt(m.d))
        new = []
        for l, s, w in zip(m.layers, states, int_weights):
            u, _, _ = ssd.ssd_rms_norm(h, l["norm"], EPS)
            p = ssd.ssd_linear_int(*ssd.ssd_int_quantize(u), *w[0], bias=l["b_in"], dtype=m.dtype)
            x, f, i = p.split(m.inner, -1)
            out = torch.empty_like(s)
            y = ssd.ssd_gated_step(s, out, x, f, decay="rate", rate=l["rate"], in_gate=i, parent=parent)
            new.append(out)
            h = ssd.ssd_linear_int(*ssd.ssd_int_quantize(y), *w[1], residual=h, dtype=m.dtype)
        u, _, _ = ssd.ssd_rms_norm(h, m.norm, EPS)
        raw, _ = ssd.ssd_linear(u, m.table)
        lengths = torch.full((rows,), t + 1, device="cuda", dtype=torch.int32)
        logits = ssd.ssd_logits_process(raw, tokens=history, lengths=lengths, repetition=1.3 * ones, presence=0.2 * ones,
                                        frequency=0.1 * ones, bias=bias, mask=mask)
        before = scores
        scores, parent, tokens, done_next = ssd.ssd_beam_select(logits.view(b, k, -1), scores, finished=done, eos=eos)
        said.append((raw, history, lengths, logits, before, done, scores, parent, tokens, list(new)))
        parent = parent.view(-1)
        history = history[parent.long()].contiguous()
        history[:, t + 1] = tokens.view(-1)
        states, done = new, done_next
    return said, bias, mask


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_beam_search(ssd, dtype):
    """The logits that were chosen from are the raw ones with the penalties of each beam's own history, the choice is the
    best of them, and the states are those of the chosen beams' tokens, by 64-bit definitions fed with the same values."""
    import torch
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    half = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
    b, k, steps, eos = 2, 4, 7, 5
    m = Model(dt)
    w = [(ssd.ssd_int_quantize(l["w_in"]), ssd.ssd_int_quantize(l["w_out"])) for l in m.layers]
    said, bias, mask = _search(ssd, m, b, k, steps, eos, w)
    torch.cuda.synchronize()
    at = torch.arange(m.vocab, device="cuda")
    allowed = (mask[at // 32] >> (at % 32)) & 1 != 0
    for t, (raw, history, lengths, logits, before, done, scores, parent, tokens, states) in enumerate(said):
        l = raw.double()
        n = torch.zeros_like(l)
        n.scatter_add_(1, history[:, :t + 1].long(), torch.ones_like(history[:, :t + 1], dtype=torch.float64))
        l = torch.where(n > 0, torch.where(l > 0, l / 1.3, l * 1.3) - (0.1 * n + 0.2), l) + bias.double()
        err = (logits.double() - l).abs()[:, allowed]
        assert bool((err <= half * l.abs()[:, allowed] + 1e-5).all()) and bool((logits[:, ~allowed] == -math.inf).all())
        cand = before.double()[..., None] + torch.log_softmax(logits.double().view(b, k, -1), -1)
        if done is not None:
            only = torch.full_like(cand, -math.inf)
            only[..., eos] = before.double()
            cand = torch.where(done[..., None], only, cand)
        mine = cand.flatten(1).gather(1, (parent.view(b, k) % k).long() * m.vocab + tokens.long())
        assert float((mine - cand.flatten(1).topk(k).values).abs().max()) <= 1e-4
        assert float((mine - scores.double()).abs().max()) <= 1e-4
    # two tokens of a beam: the last step's first layer's state from the one before it, by its parent
    old, parent, tokens = said[-2][9][0], said[-2][7].view(-1), said[-2][8]
    h = ssd.ssd_embedding(tokens.view(-1), m.table, scale=math.sqrt(m.d))
    u, _, _ = ssd.ssd_rms_norm(h, m.layers[0]["norm"], EPS)
    uq, us = ssd.ssd_int_quantize(u)
    wq, ws = w[0][0]
    p = (uq.double() @ wq.double().t()) * us.double()[:, None] * ws.double() + m.layers[0]["b_in"].double()
    p = p.to(dt).double()   # as the step reads it
    st, _ = _mix64(m.layers[0], p, old.double()[parent.long()])
    # a projection next to the middle of two bf16 values may be rounded to the other: 2^-8 of some parts of 3
    assert float((said[-1][9][0].double() - st).abs().max()) <= (1e-5 if dtype == "f32" else 0.05)


def test_beam_search_replayed(ssd):
    """A token's whole step captured into a graph and replayed with new tokens and scores, against eager."""
    import torch
    m = Model(torch.bfloat16)
    w = [(ssd.ssd_int_quantize(l["w_in"]), ssd.ssd_int_quantize(l["w_out"])) for l in m.layers]
    rows = 8
    tokens = torch.randint(0, m.vocab, (rows,), device="cuda", dtype=torch.int32)
    parent = torch.arange(rows, device="cuda", dtype=torch.int32)
    states = [torch.randn(rows, m.inner, device="cuda") for _ in m.layers]
    history = torch.randint(0, m.vocab, (rows, 30), device="cuda", dtype=torch.int32)
    rep, scores = torch.full((rows,), 1.2, device="cuda"), -torch.rand(2, 4, device="cuda")

    def run():
        h = ssd.ssd_embedding(tokens, m.table)
        out = []
        for l, s, q in zip(m.layers, states, w):
            u, _, _ = ssd.ssd_rms_norm(h, l["norm"], EPS)
            x, f, i = ssd.ssd_linear_int(*ssd.ssd_int_quantize(u), *q[0], bias=l["b_in"]).split(m.inner, -1)
            new = torch.empty_like(s)
            y = ssd.ssd_gated_step(s, new, x, f, decay="rate", rate=l["rate"], in_gate=i, parent=parent)
            out.append(new)
            h = ssd.ssd_linear_int(*ssd.ssd_int_quantize(y), *q[1], residual=h)
        u, _, _ = ssd.ssd_rms_norm(h, m.norm, EPS)
        logits = ssd.ssd_logits_process(ssd.ssd_linear(u, m.table)[0], tokens=history, repetition=rep)
        return out + list(ssd.ssd_beam_select(logits.view(2, 4, -1), scores, eos=3))
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for r in range(3):
        tokens.copy_(torch.randint(0, m.vocab, (rows,), device="cuda", dtype=torch.int32))
        parent.copy_(torch.randint(-1, rows, (rows,), device="cuda", dtype=torch.int32))
        scores.sub_(torch.rand(2, 4, device="cuda"))
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), r


def test_training_step(ssd):
    """Forward and backward of embedding -> norm -> projection -> scan over two documents -> projection with the residual ->
    logits with the tied table, in fp32, against 64-bit autograd of the plain recurrence: the table's gradient adds up from
    both ends. Every gradient passes some hundred fp32 sums: 1e-4 relative in norm."""
    import torch
    m = Model(torch.float32, d=48, inner=40, vocab=130, layers=1, seed=5)
    l = m.layers[0]
    g = torch.Generator(device="cuda").manual_seed(6)
    b, T = 2, 150
    tokens = torch.randint(0, m.vocab, (b, T), device="cuda", generator=g, dtype=torch.int32)
    tokens[1, 100:] = -1                                   # a shorter sequence, padded
    reset = torch.zeros(b, T, dtype=torch.bool, device="cuda")
    reset[:, 0] = reset[:, 70] = True
    dlogits = torch.randn(b, T, m.vocab, device="cuda", generator=g)
    scale = math.sqrt(m.d)

    h = ssd.ssd_embedding(tokens, m.table, scale=scale)
    u, _, rstd = ssd.ssd_rms_norm(h, l["norm"], EPS, want_rstd=True)
    p, _ = ssd.ssd_linear(u, l["w_in"], bias=l["b_in"])
    x, f, i = p.split(m.inner, -1)
    y, _, states = ssd.ssd_gated_scan_fwd(x, f, decay="rate", rate=l["rate"], in_gate=i, reset=reset, want_states=True)
    o, _ = ssd.ssd_linear(y, l["w_out"], residual=h)
    logits, _ = ssd.ssd_linear(o, m.table)
    # backward
    do, dtable, _ = ssd.ssd_linear_bwd(dlogits, o, m.table)
    dy, dw_out, _ = ssd.ssd_linear_bwd(do, y, l["w_out"])
    dx, df, di, drate, _ = ssd.ssd_gated_scan_bwd(dy, x, f, states, decay="rate", rate=l["rate"], in_gate=i, reset=reset)
    du, dw_in, db = ssd.ssd_linear_bwd(torch.cat([dx, df, di], -1), u, l["w_in"], want_bias=True)
    dh, _, dn = ssd.ssd_rms_norm_bwd(du, h, l["norm"], rstd, d_residual_out=do)
    ssd.ssd_embedding_bwd(dh, tokens, m.vocab, scale=scale, dtable=dtable, accumulate=True)
    torch.cuda.synchronize()

    leaf = {k: v.double().cpu().requires_grad_() for k, v in dict(table=m.table, **l).items()}
    there = (tokens >= 0).cpu()
    hh = torch.where(there[..., None], leaf["table"][tokens.clamp(min=0).long().cpu()] * scale, torch.zeros((), dtype=torch.float64))
    uu = hh / (hh.square().mean(-1, keepdim=True) + EPS).sqrt() * leaf["norm"]
    xx, ff, ii = (uu @ leaf["w_in"].t() + leaf["b_in"]).chunk(3, -1)
    la = leaf["rate"] * torch.sigmoid(ff)
    a, v = torch.exp(la), torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(ii) * xx
    st, ys = torch.zeros(b, m.inner, dtype=torch.float64), []
    for t in range(T):
        st = torch.where(reset[:, t, None].cpu(), torch.zeros_like(st), a[:, t] * st) + v[:, t]
        ys.append(st)
    oo = torch.stack(ys, 1) @ leaf["w_out"].t() + hh
    want = oo @ leaf["table"].t()
    (want * dlogits.double().cpu()).sum().backward()
    def rel(got, ref):
        return float((got.double().cpu() - ref).norm() / ref.norm())
    errs = dict(logits=rel(logits, want.detach()), table=rel(dtable, leaf["table"].grad), norm=rel(dn, leaf["norm"].grad),
                w_in=rel(dw_in, leaf["w_in"].grad), b_in=rel(db, leaf["b_in"].grad), w_out=rel(dw_out, leaf["w_out"].grad),
                rate=rel(drate, leaf["rate"].grad))
    log("[recurrent] " + " ".join(f"{k} {e:.1e}" for k, e in errs.items()))
    assert all(e <= 1e-4 for e in errs.values()), errs
