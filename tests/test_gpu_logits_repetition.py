"""GPU tests of ssd_logits_process with repetition penalties of every size.

Tolerance: l * repetition, or l times the number nearest to 1 / repetition, are two roundings to fp32 at most (2^-24 of the value
each, or 2^-149 where it is as small as that) and one to the logit's type, half a step."""
from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [64, 1003, 40000])
def test_repetitions_of_every_size(ssd, vocab, dtype):
    import torch
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(vocab)
    rep = torch.tensor([1.0, 1.1, 1.2, 1.3, 0.7, 3.0, 1e-39, 1e-30, 1e30, 3e38, 2.0 ** -149, 7.1], device="cuda")
    rows = len(rep)
    logits = 5 * torch.randn(rows, vocab, device="cuda", generator=g)
    logits[:, 3], logits[:, 4], logits[:, 5], logits[:, 6] = float("inf"), float("-inf"), 0.0, -0.0
    logits[:, 7], logits[:, 8] = 1e-3, 1e-30
    logits = logits.to(t)
    tokens = torch.arange(vocab, device="cuda", dtype=torch.int32).expand(rows, -1).contiguous()
    got = ssd.ssd_logits_process(logits, tokens=tokens, repetition=rep)
    torch.cuda.synchronize()
    l, r = logits.float().cpu().numpy(), rep.cpu().numpy()[:, None]
    l, r, got = l.astype(np.float64), r.astype(np.float64), got.double().cpu().numpy()
    want = np.where(l > 0, l / r, l * r)
    top = float(torch.finfo(t).max)
    assert np.array_equal(np.isinf(got), np.abs(want) > top)
    fine = np.abs(want) <= top
    lim = (2 * 2.0 ** -24 + torch.finfo(t).eps / 2) * np.abs(want) + 2 * 2.0 ** -149 + (2.0 ** -134 if dtype == "bf16" else 0)
    assert (np.abs(got[fine] - want[fine]) <= lim[fine]).all()
