"""GPU test that ssd_rms_norm_mx's codes are the nearest to the exact h inv w, not to its fp32 value.

The rows hold small whole numbers, so that their squares add up exactly; the weights put every product next to the
middle between two e4m3 values, as near as an fp32 weight can (some 2^-25 of it), where a product rounded to fp32
first goes to either side. The kernel keeps it to 48 bits: codes have to be the definition's in 64 bits wherever the
product lies further than 2^-44 of itself from the middle."""
from __future__ import annotations

import numpy as np
import pytest

from tests.gpu_util import log

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -10


@pytest.mark.parametrize("dim", [64, 2048, 4096 + 32, 32768])
@pytest.mark.parametrize("dtype,rtype", [("bf16", None), ("bf16", "f32"), ("f32", "f32")])
def test_codes_next_to_the_middle(ssd, dim, dtype, rtype):
    import torch
    log(f"[mx codes] {dim} {dtype} residual {rtype}")
    r = np.random.default_rng(dim)
    rows = 24
    h = np.tile(r.integers(1, 5, dim), (rows, 1)).astype(np.float64)
    h *= r.choice([-1, 1], (rows, dim))            # signs differ from row to row: one set of weights serves all
    inv = 1 / np.sqrt((h[0] * h[0]).mean() + EPS)  # the same for every row
    # a block's largest is 416 of its scale, the others middles of neighbouring codes below 256
    code = r.integers(8 * 8, 15 * 8 - 1, dim)      # 2^e (1 + m / 8) with e = code / 8 - 7
    middle = np.exp2(code // 8 - 7.0) * (1 + (code % 8 + 0.5) / 8)
    middle[::32] = 416.0
    w = (middle / (np.abs(h[0]) * inv)).astype(np.float32)
    exact = h * inv * w.astype(np.float64)
    u = np.abs(exact)
    step = np.exp2(np.floor(np.log2(u)) - 3)
    away = np.abs(np.abs(u / step - np.floor(u / step) - 0.5)) * step / u
    sure = away > 2.0 ** -44
    assert sure.mean() > 0.99
    want = np.round(exact / step) * step
    t = {"bf16": torch.bfloat16, "f32": torch.float32}
    x = torch.from_numpy(h).to(t[dtype]).cuda()
    res = None
    if rtype is not None:
        res = torch.from_numpy(h - 1).to(t[rtype]).cuda()
        x = torch.ones_like(x)
    q, s, _ = ssd.ssd_rms_norm_mx(x, torch.from_numpy(w).cuda(), EPS, residual=res)
    got = q.float().double() * s.float().double().repeat_interleave(32, 1)
    got = got.cpu().numpy()
    assert np.array_equal(got[sure], want[sure]), int((got[sure] != want[sure]).sum())
    # the same from an fp32 product would differ in many places: the inputs are what they are meant to be
    y = (h.astype(np.float32) * np.float32(inv)).astype(np.float32) * w
    st = np.exp2(np.floor(np.log2(np.abs(y.astype(np.float64)))) - 3)
    assert (np.round(y.astype(np.float64) / st) * st != want)[sure].mean() > 0.1
