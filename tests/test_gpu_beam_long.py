"""GPU tests of ssd_beam_select at vocabularies whose rows are more than one pass of 2048 logits a wavefront.

Tolerance. A term e^-d is 2^(d log2 e) of a difference and a product rounded to fp32 (each 2^-24 of d log2 e, the
constant 2^-26), and 2^x itself is off by 2^-23: under (d + 1) 2^-22 of the term. Terms of d < 15 make the sums here, 2^-18
at most. 32 of them a lane and 6 partial sums are added in fp32, 38 * 2^-24 = 2^-18.7, and what lies beyond 2048
logits in 64 bits. A score of up to 32 is rounded to fp32, 2^-20. All three: 7.1e-6, under 2^-17, where all errors had one
sign; the fault that these tests are for is 2^-15 and more."""
from __future__ import annotations

import math

import pytest

from tests.gpu_util import log

pytestmark = pytest.mark.gpu

TOL = 2.0 ** -17


def _sums(logits):
    """log sum exp in 64 bits, by parts (a row's doubles would be large)."""
    import torch
    top = logits.amax(-1).double()
    total = torch.zeros_like(top)
    for part in logits.split(1 << 24, dim=-1):
        total += torch.exp(part.double() - top[..., None]).sum(-1)
    return top + torch.log(total)


def test_sums_of_many_equal_logits(ssd):
    """2^28 logits, all but one in 2^22 the same: added one behind the other in 32 bits, every addition would round the
    same way, and the two beams' sums would be off by 3e-5 in opposite directions, more than the scores differ."""
    import torch
    v = 1 << 28
    log(f"[select] 1x2x{v} bf16")
    logits = torch.empty(1, 2, v, device="cuda", dtype=torch.bfloat16)
    for k, d in enumerate((0.67578125, 2.8125)):
        logits[0, k] = -d
        logits[0, k, ::1 << 22] = 0.0
    lse = [math.log(64 + (v - 64) * math.exp(-d)) for d in (0.67578125, 2.8125)]
    assert float((_sums(logits)[0].cpu() - torch.tensor(lse, dtype=torch.float64)).abs().max()) < 1e-9
    for gap in (2e-5, -2e-5):   # of the beams' best candidates, the first beam's being the larger or the smaller
        scores = torch.tensor([[lse[0] + gap - 8, lse[1] - 8]], device="cuda", dtype=torch.float32)
        cand = [float(scores[0, k]) - lse[k] for k in (0, 1)]
        assert abs(cand[0] - cand[1] - gap) < 4e-6  # the scores' own rounding
        out, parent, token, _ = ssd.ssd_beam_select(logits, scores)
        first = 0 if gap > 0 else 1
        assert parent[0].tolist() == [first, first] and token[0].tolist() == [0, 1 << 22]
        assert float((out[0].cpu().double() - cand[first]).abs().max()) <= TOL


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,k,v", [(2, 3, 131073), (1, 4, (1 << 20) + 77), (1, 2, (1 << 24) - 3)])
def test_scores_of_long_rows(ssd, dtype, b, k, v):
    """Maxima that rise and fall from one pass to the next, rows with nothing in most of their passes, and a row's
    largest values in its last ones."""
    import torch
    log(f"[select] {b}x{k}x{v} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(v)
    logits = 1.5 * torch.randn(b, k, v, device="cuda", generator=g)
    logits += 4 * torch.randn(b, k, (v + 2047) // 2048, device="cuda", generator=g).repeat_interleave(2048, -1)[..., :v]
    logits[0, 0, :v - 5000] = -math.inf
    logits[-1, -1] = torch.arange(v, device="cuda") * (30.0 / v)
    logits = logits.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    lse = _sums(logits)
    scores = lse.float() - 3 * torch.rand(b, k, device="cuda", generator=g)
    out, parent, token, _ = ssd.ssd_beam_select(logits, scores)
    torch.cuda.synchronize()
    cand = torch.cat([(scores.double()[..., j:j + 1] + logits[:, j].double() - lse[:, j:j + 1]) for j in range(k)], -1)
    best, at = torch.topk(cand, 2 * k)
    assert float((out.double() - best[:, :k]).abs().max()) <= TOL
    flat = (parent.long() - torch.arange(b, device="cuda")[:, None] * k) * v + token.long()
    assert bool(((cand.gather(1, flat) - best[:, :k]).abs() <= TOL).all())
    for i in range(b):
        assert len(set(flat[i].tolist())) == k
