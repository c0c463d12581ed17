"""GPU tests of the gated linear recurrence with the largest finite gates, torch.finfo(t).min and max: they count as the
infinities do, in the scan, its gradients and the step."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu


def _type(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _gates(t, shape, largest):
    """Columns of -largest, largest, and ordinary values."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    f = torch.randn(*shape, device="cuda", generator=g).to(t)
    f[..., 0::3], f[..., 1::3] = -largest, largest
    return f


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["log", "sigmoid", "rate"])
@pytest.mark.parametrize("dim", [2, 24])
def test_largest_gates_are_infinite_ones(ssd, decay, dtype, dim):
    import torch
    t, B, T = _type(dtype), 2, 150
    top = torch.finfo(t).max
    g = torch.Generator(device="cuda").manual_seed(4)
    x, dy = (torch.randn(B, T, dim, device="cuda", generator=g).to(t) for _ in range(2))
    h0 = torch.randn(B, dim, device="cuda", generator=g)
    rate = -torch.rand(dim, device="cuda", generator=g) if decay == "rate" else None
    def run(largest):
        f, i = _gates(t, (B, T, dim), largest), _gates(t, (B, T, dim), largest).flip(-1).contiguous()
        if decay == "log":
            f = -f.abs()
        call = dict(decay=decay, rate=rate, in_gate=i)
        y, final, st = ssd.ssd_gated_scan_fwd(x, f, initial_state=h0, want_states=True, **call)
        grads = ssd.ssd_gated_scan_bwd(dy, x, f, st, **call)
        state = torch.empty_like(h0)
        ys = ssd.ssd_gated_step(h0, state, x[:, 0], f[:, 0], **dict(call, in_gate=i[:, 0]))
        torch.cuda.synchronize()
        return [y, final, st, ys, state] + [v for v in grads if v is not None]
    got, want = run(top), run(float("inf"))
    for k, (a, b) in enumerate(zip(got, want)):
        assert bool(torch.isfinite(a).all()), k
        assert torch.equal(a, b), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["log", "sigmoid", "rate"])
def test_the_step_is_the_scan_of_one_token(ssd, decay, dtype):
    """Decays and gates of 0, 1 and e^rate (twice 2^-20 apart at most, with their rounding): state' = a state + c v."""
    import torch
    t, B, dim = _type(dtype), 3, 24
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(B, 1, dim, device="cuda", generator=g).to(t)
    h0 = torch.randn(B, dim, device="cuda", generator=g)
    rate = -torch.rand(dim, device="cuda", generator=g) if decay == "rate" else None
    f = torch.full((B, 1, dim), torch.finfo(t).min, device="cuda").to(t)
    if decay != "log":
        f[..., ::2] = torch.finfo(t).max
    call = dict(decay=decay, rate=rate)
    _, final, _ = ssd.ssd_gated_scan_fwd(x, f, in_gate=f, initial_state=h0, **call)
    state = torch.empty_like(h0)
    ssd.ssd_gated_step(h0, state, x[:, 0], f[:, 0], in_gate=f[:, 0], **call)
    torch.cuda.synchronize()
    assert bool(((final - state).abs() <= 2.0 ** -19 * (h0.abs() + x[:, 0].float().abs())).all())
