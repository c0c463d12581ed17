"""GPU tests of the gated linear recurrence: an undefined or infinite decay stays in its document, forward and backward."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

T, D = 700, 40
STARTS = (5, 20, 130, 131, 256, 390, 513)   # of documents, in every sequence
# (token whose gate is replaced, channel). A chunk has 128 tokens, a wavefront 16 of them, a group of lanes 2 (bf16) or 4
# (fp32): before a reset of its own group, of its wavefront, of its chunk and of a later chunk; a reset itself, right
# behind one in its group, and later
PLACES = [(4, 0), (3, 1), (10, 2), (19, 3), (40, 4), (129, 5), (130, 6), (131, 7), (132, 8), (255, 9), (256, 10), (257, 11), (260, 12),
          (300, 13), (389, 14), (391, 15), (395, 16), (512, 17), (514, 18), (600, 19)]


def _type(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _inputs(dtype, decay):
    import torch
    g = torch.Generator(device="cuda").manual_seed(17)
    def r(*s):
        return torch.randn(*s, device="cuda", generator=g)
    t = _type(dtype)
    s = dict(x=r(2, T, D).to(t), i=r(2, T, D).to(t), dy=r(2, T, D).to(t), h0=r(2, D), dfin=r(2, D),
             f=(-0.1 * torch.exp(r(2, T, D)) if decay == "log" else 2 + r(2, T, D)).to(t),
             rate=torch.log(0.9 + 0.099 * torch.rand(D, device="cuda", generator=g)) if decay == "rate" else None,
             reset=torch.zeros(2, T, dtype=torch.bool, device="cuda"))
    s["reset"][:, list(STARTS)] = True
    return s


def _both(ssd, s, f, decay):
    import torch
    call = dict(decay=decay, rate=s["rate"], in_gate=s["i"], reset=s["reset"])
    y, final, states = ssd.ssd_gated_scan_fwd(s["x"], f, initial_state=s["h0"], want_states=True, **call)
    g = ssd.ssd_gated_scan_bwd(s["dy"], s["x"], f, states, d_final_state=s["dfin"], **call)
    torch.cuda.synchronize()
    return y, final, states, g


@pytest.mark.parametrize("value", ["nan", "inf"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["log", "sigmoid", "rate"])
def test_undefined_decays_stay_in_their_document(ssd, decay, dtype, value):
    """Whatever lies outside the gate's document (and, forward, before the gate) has the bits that it has with an ordinary
    gate; behind an undefined decay the document is undefined to its end."""
    import torch
    s = _inputs(dtype, decay)
    f = s["f"].clone()
    hurt = torch.zeros(2, T, D, dtype=torch.bool, device="cuda")   # y: from the token to its document's end
    back = hurt.clone()                                            # gradients: the whole document
    for t, d in PLACES:
        first, end = max([0, *[k for k in STARTS if k <= t]]), min([T, *[k for k in STARTS if k > t]])
        f[1, t, d] = float(value)
        hurt[1, t:end, d] = back[1, first:end, d] = True
    y0, final0, states0, g0 = _both(ssd, s, s["f"], decay)
    y1, final1, states1, g1 = _both(ssd, s, f, decay)
    assert torch.equal(y0[~hurt], y1[~hurt])
    assert torch.equal(final0[~hurt[:, -1]], final1[~hurt[:, -1]])
    entering = torch.zeros_like(states0, dtype=torch.bool)
    entering[:, 1:] = hurt[:, 127::128][:, :entering.shape[1] - 1]
    assert torch.equal(states0[~entering], states1[~entering])
    for a, b in zip(g0[:3], g1[:3]):
        assert torch.equal(a[~back], b[~back])
    assert torch.equal(g0[4][~back[:, 0]], g1[4][~back[:, 0]])
    if decay == "rate":
        touched = back.any(1).any(0)
        assert torch.equal(g0[3][~touched], g1[3][~touched])
    if value == "nan":
        for t, d in PLACES:
            end = min([T, *[k for k in STARTS if k > t]])
            assert bool(torch.isnan(y1[1, t:end, d]).all()) or s["reset"][1, t] and decay == "log", (t, d)
