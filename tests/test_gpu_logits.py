"""GPU tests of ssd_logits_process against its definition in 64 bits, entry by entry.

Tolerances, fixed before the first run: a touched logit passes at most five fp32 roundings of values no larger than
|l| (1 + repetition) + frequency g + presence + |bias| (8 * 2^-24 of that covers them) and is stored in its type; an
untouched one keeps its bits; masked ones are -inf."""
from __future__ import annotations

import math

import pytest

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _t(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _mask(rows, vocab, g, density):
    import torch
    allowed = torch.rand(rows, vocab, device="cuda", generator=g) < density
    bits = torch.nn.functional.pad(allowed, (0, -vocab % 32)).view(rows, -1, 32).long()
    words = (bits << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).int(), allowed


def _run(ssd, rows, vocab, cap, dtype, bias="none", mask="none", seed=0, in_place=False, wild=True):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + vocab)
    def u(*s):
        return torch.rand(*s, device="cuda", generator=g)
    logits = (3 * torch.randn(rows, vocab, device="cuda", generator=g)).to(_t(dtype))
    tokens = torch.randint(0, vocab, (rows, cap), device="cuda", generator=g, dtype=torch.int32)
    if cap > 4:
        tokens[:, ::3] = tokens[:, :1]   # one token often
        if wild:
            tokens[:, 1::7] = -1
            tokens[:, 2::11] = vocab
    lengths = (u(rows) * (cap + 1)).int().clamp(max=cap)
    prompt = (u(rows) * (cap + 1)).int()
    rep, pres, freq = 0.5 + 1.5 * u(rows), u(rows), 0.5 * u(rows)
    b = None if bias == "none" else torch.randn(1 if bias == "one" else rows, vocab, device="cuda", generator=g)
    m, allowed = (None, None) if mask == "none" else _mask(1 if mask == "one" else rows, vocab, g, 0.4)
    buf = torch.full((rows * vocab + 512,), 7.0, device="cuda").to(_t(dtype))
    out = buf[:rows * vocab].view(rows, vocab)
    before = logits.clone()
    if in_place:
        out.copy_(logits)
        logits = out
    got = ssd.ssd_logits_process(logits, tokens=tokens, lengths=lengths, prompt=prompt, repetition=rep, presence=pres, frequency=freq,
                                 bias=b, mask=m, out=out)
    torch.cuda.synchronize()
    assert got is out and bool((buf[rows * vocab:].float() == 7.0).all())
    l = before.double()
    at = torch.arange(cap, device="cuda")
    ok = (at < lengths[:, None]) & (tokens >= 0) & (tokens < vocab)
    n, said = torch.zeros_like(l), torch.zeros_like(l)
    n.scatter_add_(1, tokens.clamp(0, vocab - 1).long(), ok.double())
    said.scatter_add_(1, tokens.clamp(0, vocab - 1).long(), (ok & (at >= prompt[:, None])).double())
    r = rep.double()[:, None]
    ref = torch.where(n > 0, torch.where(l > 0, l / r, l * r), l)
    ref = ref - torch.where(said > 0, freq.double()[:, None] * said + pres.double()[:, None], torch.zeros_like(l))
    size = l.abs() * (1 + r + 1 / r) + freq.double()[:, None] * said + pres.double()[:, None]
    if b is not None:
        ref, size = ref + b.double(), size + b.double().abs()
    lim = 8 * 2.0 ** -24 * size + HALF[dtype] * ref.abs()
    touched = (n > 0) | (b is not None)
    err = (out.double() - ref).abs()
    if allowed is not None:
        allowed = allowed.expand_as(l)
        assert bool((out[~allowed] == -math.inf).all())
    else:
        allowed = torch.ones_like(touched)
    assert bool((err <= lim)[allowed].all()), float((err - lim)[allowed].max())
    assert torch.equal(out[allowed & ~touched], before[allowed & ~touched])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,cap", [(1, 1, 1), (3, 5, 9), (4, 50257, 512), (2, 4096, 100), (5, 4097, 33), (3, 8191, 3), (7, 65536, 2000),
                                            (300, 1003, 64), (2, 131072, 8000)])
def test_penalties(ssd, dtype, rows, vocab, cap):
    _run(ssd, rows, vocab, cap, dtype)
    _run(ssd, rows, vocab, cap, dtype, in_place=True, seed=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bias", ["none", "one", "rows"])
@pytest.mark.parametrize("mask", ["none", "one", "rows"])
@pytest.mark.parametrize("rows,vocab", [(3, 1001), (5, 12345), (4, 8192), (2, 31)])
def test_bias_and_masks(ssd, dtype, bias, mask, rows, vocab):
    _run(ssd, rows, vocab, 40, dtype, bias=bias, mask=mask, seed=2)
    _run(ssd, rows, vocab, 40, dtype, bias=bias, mask=mask, seed=3, in_place=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_a_history_and_bits_kept(ssd, dtype):
    import torch
    vocab = 5003
    logits = torch.randn(3, vocab, device="cuda").to(_t(dtype))
    logits[0, 5], logits[1, 6], logits[2, 7] = float("nan"), float("inf"), float("-inf")
    kind = torch.int16 if dtype == "bf16" else torch.int32
    out = ssd.ssd_logits_process(logits)
    none = ssd.ssd_logits_process(logits, tokens=torch.empty(3, 0, device="cuda", dtype=torch.int32), repetition=torch.ones(3, device="cuda"))
    empty = ssd.ssd_logits_process(logits, tokens=torch.zeros(3, 4, device="cuda", dtype=torch.int32),
                                   lengths=torch.tensor([0, -5, 0], device="cuda", dtype=torch.int32), presence=torch.ones(3, device="cuda"))
    torch.cuda.synchronize()
    for o in (out, none, empty):
        assert torch.equal(o.view(kind), logits.view(kind))
    # a mask that leaves nothing, also where the logits are NaN or infinite
    shut = ssd.ssd_logits_process(logits, mask=torch.zeros(157, device="cuda", dtype=torch.int32))
    torch.cuda.synchronize()
    assert bool((shut == -math.inf).all())
    # lengths beyond the capacity count as the capacity; without lengths all of it counts
    tokens = torch.tensor([[5, 5, 9]], device="cuda", dtype=torch.int32)
    zeros = torch.zeros(1, 64, device="cuda").to(_t(dtype))
    freq = torch.ones(1, device="cuda")
    want = torch.zeros(1, 64, device="cuda")
    want[0, 5], want[0, 9] = -2, -1
    for lengths in (None, torch.tensor([1000], device="cuda", dtype=torch.int32)):
        got = ssd.ssd_logits_process(zeros, tokens=tokens, lengths=lengths, frequency=freq)
        torch.cuda.synchronize()
        assert torch.equal(got.float(), want)


def test_no_rows(ssd):
    import torch
    assert ssd.ssd_logits_process(torch.empty(0, 100, device="cuda")).shape == (0, 100)


def test_captured_and_replayed(ssd):
    import torch
    logits = torch.randn(6, 20011, device="cuda").bfloat16()
    tokens = torch.randint(0, 20011, (6, 300), device="cuda", dtype=torch.int32)
    lengths = torch.full((6,), 100, device="cuda", dtype=torch.int32)
    rep = torch.full((6,), 1.3, device="cuda")
    def run():
        return ssd.ssd_logits_process(logits.view(2, 3, -1), tokens=tokens, lengths=lengths, repetition=rep, presence=rep)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for r in range(3):
        logits.normal_()
        lengths.add_(50)
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        assert out.shape == (2, 3, 20011) and torch.equal(out, want), r
