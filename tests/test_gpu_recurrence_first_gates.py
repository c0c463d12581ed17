"""GPU tests of the gated linear recurrence with log-decays: the gate of a document's first token decides nothing, since
what it would let in is left out. Whatever it is, states, outputs and gradients have the bits of an ordinary gate, and
the gate's own gradient is zero."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [1, 3, 24, 65])
@pytest.mark.parametrize("value", ["nan", "inf", "-inf", "200"])
def test_the_first_gate_of_a_document(ssd, dim, dtype, value):
    import torch
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    B, T = 2, 300
    g = torch.Generator(device="cuda").manual_seed(9)
    def r(*s):
        return torch.randn(*s, device="cuda", generator=g)
    x, i, dy = (r(B, T, dim).to(t) for _ in range(3))
    f = -r(B, T, dim).abs().to(t)
    h0, dfin = r(B, dim), r(B, dim)
    reset = torch.rand(B, T, device="cuda", generator=g) < 0.2   # at every place of a group, and next to each other
    reset[:, 0] = True
    wild = torch.where(reset[..., None], torch.full_like(f, float(value)), f)
    def run(f):
        call = dict(decay="log", in_gate=i, reset=reset)
        y, final, st = ssd.ssd_gated_scan_fwd(x, f, initial_state=h0, want_states=True, **call)
        dx, df, di, _, d0 = ssd.ssd_gated_scan_bwd(dy, x, f, st, d_final_state=dfin, **call)
        torch.cuda.synchronize()
        return [y, final, st, dx, di, d0, df]
    for k, (a, b) in enumerate(zip(run(f), run(wild))):
        assert torch.equal(a, b), k
    assert not bool(run(wild)[-1][reset].any())
