"""GPU tests of beam search: ssd_beam_select against a selection in 64 bits, and ssd_step_beam, bit for bit, against
gathered states and ssd_step_fused.

Tolerance of a score, fixed before the first run: a wavefront adds 32 exponentials a lane and 6 partial sums in fp32,
each exponential off by under 2^-20 relative where it counts, so a log-sum-exp is off by under 5e-6; a score of up to
64 in magnitude is rounded to fp32 (4e-6): 1e-5. Two candidates of different beams closer than that may change
places, which the test allows; everything else has to be equal."""
from __future__ import annotations

import math

import numpy as np
import pytest

from tests.gpu_util import log

pytestmark = pytest.mark.gpu

TOL = 1e-5


def _candidates(logits, scores, finished, eos):
    l = logits.float().cpu().numpy().astype(np.float64)
    s = scores.cpu().numpy().astype(np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    s = np.where(np.isnan(s), -np.inf, s)
    with np.errstate(all="ignore"):
        top = l.max(-1, keepdims=True)
        lse = top + np.log(np.exp(l - top).sum(-1, keepdims=True))
        cand = s[..., None] + (l - lse)
    cand = np.where(np.isfinite(lse) & ~np.isnan(cand), cand, -np.inf)
    if finished is not None:
        f = finished.cpu().numpy().astype(bool)
        only = np.full_like(cand, -np.inf)
        if eos >= 0:
            only[..., eos] = s
        cand = np.where(f[..., None], only, cand)
    return cand


def _check(ssd, logits, scores, finished=None, eos=-1):
    import torch
    b, k, v = logits.shape
    out, parent, token, done = ssd.ssd_beam_select(logits, scores, finished=finished, eos=eos)
    torch.cuda.synchronize()
    out, parent, token, done = (t.cpu().numpy() for t in (out, parent, token, done))
    cand = _candidates(logits, scores, finished, eos).reshape(b, k * v)
    fin = None if finished is None else finished.cpu().numpy().astype(bool).reshape(-1)
    for i in range(b):
        order = np.argsort(-cand[i], kind="stable")[:k]
        ref = cand[i][order]
        flat = (parent[i] - i * k) * v + token[i]
        assert ((flat >= 0) & (flat < k * v)).all()
        assert len(set(flat.tolist())) == k
        got = cand[i][flat]
        inf = np.isinf(ref)
        assert np.array_equal(np.isinf(out[i]), inf), (out[i], ref)
        assert np.array_equal(np.isinf(got), inf)
        assert np.all(np.abs(out[i][~inf] - ref[~inf]) <= TOL), (i, out[i], ref)
        assert np.all(np.abs(got[~inf] - ref[~inf]) <= TOL), (i, flat, order)
        edge = np.sort(cand[i])[::-1][:k + 1]
        with np.errstate(invalid="ignore"):
            gaps = np.diff(edge[np.isfinite(edge)])
        if not np.any((gaps != 0) & (np.abs(gaps) < TOL)):
            assert np.array_equal(flat, order), (i, flat, order, ref)
        for j in range(k):
            assert bool(done[i, j]) == bool((fin is not None and fin[parent[i, j]]) or token[i, j] == eos)


def _draw(b, k, v, dtype, seed, scale=3.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = (scale * torch.randn(b, k, v, device="cuda", generator=g)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return logits, -20 * torch.rand(b, k, device="cuda", generator=g), g


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b,k,v", [(1, 1, 1), (3, 4, 1), (2, 3, 2), (2, 16, 7), (5, 1, 64), (3, 5, 2041), (2, 2, 2047),
                                   (2, 8, 2049), (1, 16, 4100), (4, 4, 50257), (1, 16, 131065), (2, 3, 140001),
                                   (70, 2, 1000)])
def test_select(ssd, dtype, b, k, v):
    import torch
    log(f"[select] {b}x{k}x{v} {dtype}")
    logits, scores, g = _draw(b, k, v, dtype, v)
    _check(ssd, logits, scores)
    # a new sequence: only the first beam is in use
    scores[0, 1:] = -math.inf
    _check(ssd, logits, scores)
    # finished beams and forbidden tokens
    fin = torch.rand(b, k, device="cuda", generator=g) < 0.4
    logits.masked_fill_(torch.rand(b, k, v, device="cuda", generator=g) < 0.3, -math.inf)
    _check(ssd, logits, scores, fin, eos=v // 2)
    _check(ssd, logits, scores, fin.to(torch.uint8), eos=v - 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k", [1, 4, 16])
def test_select_ties_and_order(ssd, dtype, k):
    """Constant rows, few distinct values, rising and falling rows: ties go to the lowest index, and a wavefront's
    filter lets many through."""
    import torch
    v = 5003
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    scores = torch.full((4, k), -1.0, device="cuda")
    ramp = torch.arange(v, device="cuda", dtype=torch.float32)
    rows = torch.stack([torch.zeros(v, device="cuda"), ramp % 3, ramp / 16, -ramp / 16])
    logits = rows[:, None].expand(4, k, v).to(t).contiguous()
    out, parent, token, _ = ssd.ssd_beam_select(logits, scores)
    torch.cuda.synchronize()
    base = torch.arange(4, device="cuda")[:, None] * k
    l = logits.double()
    # the beams of a sequence are equal here, so one beam's log-sum-exp is every beam's and all ties are exact
    cand = (l - torch.logsumexp(l[:, :1], -1, keepdim=True) - 1.0)
    best, at = torch.sort(cand.cpu().reshape(4, -1), dim=-1, descending=True, stable=True)
    assert torch.equal(token.cpu().long(), at[:, :k] % v)
    assert torch.equal((parent - base).cpu().long(), at[:, :k] // v)
    assert float((out.cpu() - best[:, :k]).abs().max()) <= TOL


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_select_of_the_types_extremes(ssd, dtype):
    """Tokens forbidden by the type's lowest value instead of -inf: among others, for a whole row and for a whole
    sequence (every token then has log-probability -log V); and its largest value."""
    import torch
    logits, scores, g = _draw(5, 3, 4500, dtype, 12)
    low, high = torch.finfo(logits.dtype).min, torch.finfo(logits.dtype).max
    logits.masked_fill_(torch.rand(5, 3, 4500, device="cuda", generator=g) < 0.5, low)
    logits[1, 1] = low
    logits[2] = low
    logits[3, 0, 2100] = high
    logits[4, 2] = low
    logits[4, 2, 7] = high
    _check(ssd, logits, scores)


def test_select_of_values_that_are_not_numbers(ssd):
    import torch
    logits, scores, g = _draw(6, 4, 3001, "f32", 11)
    nan, inf = math.nan, math.inf
    logits[0, 1, 5] = nan              # one logit of a row
    logits[1, :] = -inf                # nothing is left of any row
    logits[2, 0] = -inf                # nothing of one
    logits[3, 2, 17] = inf             # an infinite sum
    scores[4, 1] = nan
    scores[5, :] = -inf                # no beam in use
    _check(ssd, logits, scores)
    logits[:, :, 1:] = -inf            # one token allowed
    logits[:, :, 0] = 0
    _check(ssd, logits, scores)
    fin = torch.zeros(6, 4, dtype=torch.bool, device="cuda")
    fin[1] = True                      # all finished
    fin[2, 0] = True
    logits[2, 0] = nan                 # a finished beam's logits are not read
    _check(ssd, logits, scores, fin, eos=7)
    out = ssd.ssd_beam_select(torch.empty(0, 4, 10, device="cuda"), torch.empty(0, 4, device="cuda"))
    assert out[0].shape == (0, 4)


def _step_inputs(rows, src, H, P, N, G, dtype, seed, conv=True):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    def r(*s, dt=torch.float32, sc=1.0):
        return (sc * torch.randn(*s, device="cuda", generator=g)).to(dt)
    d = dict(state_in=r(src, H, P, N), parent=torch.randint(0, max(src, 1), (rows,), device="cuda", generator=g).int(),
             x=r(rows, H, P, dt=t), dt=r(rows, H, dt=t), A=-torch.exp(2 * torch.rand(H, device="cuda", generator=g)),
             B=r(rows, G, N, dt=t, sc=N ** -0.5), C=r(rows, G, N, dt=t, sc=N ** -0.5), D=r(H))
    kw = dict(dt_bias=r(H) - 4, dt_softplus=1, z=r(rows, H, P, dt=t))
    if conv:
        kw.update(conv_w=r(H * P, 4, sc=0.5), conv_b=r(H * P, sc=0.5))
        d["conv_in"] = r(src, H * P, 3, dt=t)
    return d, kw


def _by_gather(ssd, d, kw):
    """The rows of the parents copied, then ssd_step_fused / ssd_step_gated in place."""
    import torch
    p = d["parent"].long()
    ok = (p >= 0) & (p < d["state_in"].shape[0])
    if d["state_in"].shape[0]:
        state = torch.where(ok[:, None, None, None], d["state_in"][p.clamp(0, d["state_in"].shape[0] - 1)], 0.0)
    else:
        state = torch.zeros(len(p), *d["state_in"].shape[1:], device="cuda")
    args = (d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"])
    if "conv_in" not in d:
        return ssd.ssd_step_gated(state, *args, **kw), state, None
    if d["conv_in"].shape[0]:
        conv = torch.where(ok[:, None, None], d["conv_in"][p.clamp(0, d["conv_in"].shape[0] - 1)], torch.zeros((), dtype=d["x"].dtype, device="cuda")).contiguous()
    else:
        conv = torch.zeros(len(p), *d["conv_in"].shape[1:], dtype=d["x"].dtype, device="cuda")
    return ssd.ssd_step_fused(state.contiguous(), conv, *args, **kw), state, conv


def _beam(ssd, d, kw, **more):
    import torch
    rows = d["x"].shape[0]
    so = torch.full((rows, *d["state_in"].shape[1:]), math.nan, device="cuda")
    if "conv_in" in d:
        co = torch.full((rows, *d["conv_in"].shape[1:]), math.nan, device="cuda").to(d["x"].dtype)
        more.update(conv_in=d["conv_in"], conv_out=co)
    y = ssd.ssd_step_beam(d["state_in"], so, d["parent"], d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], **kw, **more)
    return y, so, more.get("conv_out")


def _same(a, b):
    import torch
    return all((p is None and q is None) or torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,src,H,P,N,G,conv", [(1, 1, 1, 1, 4, 1, True), (8, 8, 4, 64, 128, 2, True),
                                                   (12, 3, 8, 50, 64, 8, True), (5, 9, 2, 33, 256, 1, False),
                                                   (6, 6, 24, 64, 128, 1, False), (3, 0, 2, 16, 16, 1, True)])
def test_step_beam_is_gather_and_step(ssd, dtype, rows, src, H, P, N, G, conv):
    import torch
    d, kw = _step_inputs(rows, src, H, P, N, G, dtype, 21, conv)
    before = d["state_in"].clone()
    got, want = _beam(ssd, d, kw), _by_gather(ssd, d, kw)
    torch.cuda.synchronize()
    assert _same(got, want) and torch.equal(before, d["state_in"])


def test_step_beam_bad_parents_start_from_zero(ssd):
    import torch
    d, kw = _step_inputs(6, 4, 3, 20, 32, 1, "bf16", 22)
    d["parent"] = torch.tensor([-1, 4, 2 ** 31 - 1, -2 ** 31, 3, 0], dtype=torch.int32, device="cuda")
    got, want = _beam(ssd, d, kw), _by_gather(ssd, d, kw)
    torch.cuda.synchronize()
    assert _same(got, want)


def test_step_beam_refuses_in_place_and_partial_convolutions(ssd):
    import torch
    d, kw = _step_inputs(4, 4, 2, 16, 32, 1, "f32", 23, conv=False)
    args = (d["parent"], d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"])
    with pytest.raises(ssd.SSDError) as e:
        ssd.ssd_step_beam(d["state_in"], d["state_in"], *args, **kw)
    assert e.value.code == 3
    out = torch.empty_like(d["state_in"])
    conv = torch.zeros(4, 32, 3, device="cuda")
    with pytest.raises(ssd.SSDError):
        ssd.ssd_step_beam(d["state_in"], out, *args, conv_in=conv, conv_out=conv.clone(), **kw)
    w = torch.zeros(32, 4, device="cuda")
    with pytest.raises(ssd.SSDError):
        ssd.ssd_step_beam(d["state_in"], out, *args, conv_in=conv, conv_w=w, **kw)
    with pytest.raises(ssd.SSDError):
        ssd.ssd_step_beam(d["state_in"], out, *args, conv_in=conv, conv_out=conv, conv_w=w, **kw)
    with pytest.raises(ValueError):
        ssd.ssd_step_beam(d["state_in"], out, d["parent"].long(), *args[1:], **kw)


def test_beam_search_step_on_a_stream_and_replayed(ssd):
    """Selection and step together, two states swapped, captured for two tokens and replayed against eager."""
    import torch
    b, k, v = 3, 4, 4099
    d, kw = _step_inputs(b * k, b * k, 4, 32, 64, 2, "bf16", 24)
    logits, scores, g = _draw(b, k, v, "bf16", 25)

    def token(src, conv, sc, fin, **on):
        sc, parent, tok, fin = ssd.ssd_beam_select(logits, sc, finished=fin, eos=3, **on)
        so, co = torch.empty_like(src), torch.empty_like(conv)
        y = ssd.ssd_step_beam(src, so, parent.view(-1), d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], conv_in=conv,
                              conv_out=co, **kw, **on)
        return y, so, co, sc, fin, parent, tok

    def two():
        one = token(d["state_in"], d["conv_in"], scores, None)
        return one + token(one[1], one[2], one[3], one[4])
    want = two()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = two()
    s.synchronize()
    assert _same(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = two()
    for r in range(3):
        logits.copy_(torch.roll(logits, 1 + r, 2))
        d["state_in"].mul_(0.5)
        want = two()
        graph.replay()
        torch.cuda.synchronize()
        assert _same(out, want), r


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_select_takes_both_zeros_as_one(ssd, dtype):
    """-0 and 0 are equal logits: the lower index goes first, in whole tiles, in the rest of a row and across tiles."""
    import torch
    for v, minus, plus in ((100, 3, 7), (5000, 10, 1500), (5000, 40, 4999), (300, 299, 17), (70000, 2047, 69999)):
        logits = torch.full((1, 2, v), -9.0, device="cuda", dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
        logits[:, :, minus], logits[:, :, plus] = -0.0, 0.0
        scores = torch.tensor([[0.0, -math.inf]], device="cuda")
        _, parent, token, _ = ssd.ssd_beam_select(logits, scores)
        assert token[0].tolist() == sorted((minus, plus)) and parent[0].tolist() == [0, 0]
