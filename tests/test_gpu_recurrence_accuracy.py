"""GPU tests of how far a decay is off, one token at a time: with x = 0 and a state of 1, the state that follows is the
decay; with a state of 0 and x = 1 it is the input's coefficient, or the input's gate.

Tolerances, in steps u = 2^-24, from the operations (the exponential and the reciprocal of the hardware are within 2 u of
themselves, a product, sum or root's rounding 1 u, the root's reciprocal 2 u):
  e^x, fine        the exponent in two parts: 2 u, and 2 u for putting the second in; 4 u
  e^x, bf16 scan   |x| u for the product's rounding, |x| u / 4 for log2 e itself, 2 u; (2 + 1.3 |x|) u
  sigmoid(x)       e u_e / (1 + e), and 1 + 2 u: 7 u fine, (5 + 1.3 |x|) u for x < 0 in the bf16 scan
  e^(rate s)       log a is off by that and 2.3 u of itself: (2 + |log a| (u_s + 2.3)) u
  sqrt(1 - a^2)    half of log a's error, half of 1 - a^2's own (5 u by its series; beyond it, from a^2 = 0.61 down, or
                   0.78 in the bf16 scan, a's 2 u are 6 u or 14 u there) and 3.5 u: (u_s + 2.3) / 2 + 8, or + 12
Second orders are below 0.1 u."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _type(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _sizes(form, f):
    """Bounds in u of e^f and sigmoid(f)."""
    import torch
    fine = form != "bf16 scan"
    e = torch.full_like(f, 4.0) if fine else 2 + 1.3 * f.abs()
    s = torch.full_like(f, 7.0) if fine else 5 + 1.3 * f.abs()
    return e, s


def _one_token(ssd, form, state, x, f, **kw):
    import torch
    if form.endswith("step"):
        out = torch.empty_like(state)
        ssd.ssd_gated_step(state, out, x, f, **kw)
    else:
        kw = dict(kw, in_gate=None if kw.get("in_gate") is None else kw["in_gate"][:, None])
        _, out, _ = ssd.ssd_gated_scan_fwd(x[:, None], f[:, None], initial_state=state, **kw)
    torch.cuda.synchronize()
    return out.double()


def _within(got, want, lim, what):
    err = (got - want).abs() / want.abs().clamp(min=2.0 ** -120) / U
    print(f"[accuracy] {what}: {float(err.max()):.2f} u, of the bound {float((err / lim).max()):.2f}", flush=True)
    assert bool((err <= lim + 0.1).all()), what


@pytest.mark.parametrize("form", ["bf16 scan", "f32 scan", "bf16 step", "f32 step"])
@pytest.mark.parametrize("reach", [1, 8, 30, 80])
def test_decays_and_gates(ssd, form, reach):
    import torch
    t = _type(form[:4].strip())
    g = torch.Generator(device="cuda").manual_seed(reach)
    shape = (64, 2048)
    one, zero = torch.ones(shape, device="cuda"), torch.zeros(shape, device="cuda")
    f = (reach * (2 * torch.rand(shape, device="cuda", generator=g) - 1)).to(t)
    f64 = f.double()
    e, s = _sizes(form, f64)
    neg = -f.abs()
    _within(_one_token(ssd, form, one, zero.to(t), neg, decay="log"), torch.exp(neg.double()), e, f"{form} e^f to {reach}")
    _within(_one_token(ssd, form, one, zero.to(t), f, decay="sigmoid"), torch.sigmoid(f64), s, f"{form} sigmoid to {reach}")
    _within(_one_token(ssd, form, zero, one.to(t), f, decay="sigmoid"), torch.sigmoid(-f64), 2 * s, f"{form} 1 - sigmoid to {reach}")
    gate = _one_token(ssd, form, zero, one.to(t), neg, decay="log", in_gate=f)
    _within(gate, torch.sigmoid(f64), s, f"{form} input gate to {reach}")


@pytest.mark.parametrize("form", ["bf16 scan", "f32 scan", "bf16 step", "f32 step"])
@pytest.mark.parametrize("most", [0.01, 1.0, 8.0, 30.0])
def test_decays_by_rates(ssd, form, most):
    import torch
    t = _type(form[:4].strip())
    g = torch.Generator(device="cuda").manual_seed(7)
    shape = (64, 2048)
    one, zero = torch.ones(shape, device="cuda"), torch.zeros(shape, device="cuda")
    f = (4 * torch.randn(shape, device="cuda", generator=g)).clamp(-8, 8).to(t)
    rate = -most * torch.rand(2048, device="cuda", generator=g)
    la = rate.double() * torch.sigmoid(f.double())
    _, s = _sizes(form, f.double())
    a = _one_token(ssd, form, one, zero.to(t), f, decay="rate", rate=rate)
    _within(a, torch.exp(la), 2 + la.abs() * (s + 2.3), f"{form} rates to {most}")
    c = _one_token(ssd, form, zero, one.to(t), f, decay="rate", rate=rate)
    _within(c, torch.sqrt(-torch.expm1(2 * la)), (s + 2.3) / 2 + (12 if form == "bf16 scan" else 8), f"{form} coefficients of rates to {most}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_positive_rate_counts_as_zero(ssd, dtype):
    """The bits of a rate of 0, forward, backward and in the step."""
    import torch
    t = _type(dtype)
    g = torch.Generator(device="cuda").manual_seed(8)
    x, f, i, dy = (torch.randn(2, 300, 40, device="cuda", generator=g).to(t) for _ in range(4))
    h0 = torch.randn(2, 40, device="cuda", generator=g)
    some = torch.randn(40, device="cuda", generator=g)
    some[5], some[6] = 1e30, float("inf")
    def run(rate):
        call = dict(decay="rate", rate=rate, in_gate=i)
        y, final, st = ssd.ssd_gated_scan_fwd(x, f, initial_state=h0, want_states=True, **call)
        out = torch.empty_like(h0)
        ys = ssd.ssd_gated_step(h0, out, x[:, 0], f[:, 0], decay="rate", rate=rate, in_gate=i[:, 0])
        grads = ssd.ssd_gated_scan_bwd(dy, x, f, st, **call)
        torch.cuda.synchronize()
        return [y, final, st, ys, out, *grads]
    assert bool((some > 0).any())
    for a, b in zip(run(some), run(some.clamp(max=0))):
        assert torch.equal(a, b)
    assert torch.equal(run(some)[1][:, some > 0], h0[:, some > 0])
