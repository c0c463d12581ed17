"""GPU tests of the gated linear recurrence: marks that reset nothing change nothing, also where a state is undefined or
infinite and the decays behind it underflow.

Tolerance: with and without marks the same operations run on the same values, but where a product's rounding falls away in
a sum. Terms are at most as large as the tensor's largest value (the decays are far below 1: nothing grows), a value
passes fewer than 32 of them, so 2^-18 of the largest; both are rounded to their type, half a step each."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu


def _type(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _same(a, b):
    import torch
    fine = torch.isfinite(a)
    if not torch.equal(torch.isnan(a), torch.isnan(b)) or not torch.equal(torch.isinf(a), torch.isinf(b)):
        return False
    x, y = a[fine].double(), b[fine].double()
    return bool(((x - y).abs() <= torch.finfo(a.dtype).eps * (x.abs() + y.abs()) / 2 + 2.0 ** -18 * y.abs().max()).all())


@pytest.mark.parametrize("value", [None, "nan", "inf"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["log", "sigmoid", "rate"])
def test_no_reset_set(ssd, decay, dtype, value):
    import torch
    B, T, D = 2, 520, 24
    t = _type(dtype)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, dy = (torch.randn(B, T, D, device="cuda", generator=g).to(t) for _ in range(2))
    # decays of e^-20 to e^-60 a token: the product of a few is zero
    f = (-20 - 40 * torch.rand(B, T, D, device="cuda", generator=g)).to(t)
    rate = None
    if decay == "rate":
        f, rate = -f / 10, torch.full((D,), -40.0, device="cuda")
    at = [(0, 3), (15, 4), (16, 5), (127, 6), (128, 7), (300, 8)]
    if value is not None:
        for k, d in at:
            x[0, k, d] = float(value)
            dy[1, T - 1 - k, d] = float(value)
    none = torch.zeros(B, T, dtype=torch.bool, device="cuda")
    def both(reset):
        call = dict(decay=decay, rate=rate, reset=reset)
        y, final, st = ssd.ssd_gated_scan_fwd(x, f, want_states=True, **call)
        grads = ssd.ssd_gated_scan_bwd(dy, x, f, st, **call)
        torch.cuda.synchronize()
        return [y, final, st] + [v for v in grads if v is not None]
    with_marks, without = both(none), both(None)
    for k, (a, b) in enumerate(zip(with_marks, without)):
        assert _same(a, b), k
    if value is not None:
        for k, d in at:   # never finite again, forward and backward
            assert not bool(torch.isfinite(with_marks[0][0, k:, d]).any()), (k, d)
            assert not bool(torch.isfinite(with_marks[3][1, :T - k, d]).any()), (k, d)
