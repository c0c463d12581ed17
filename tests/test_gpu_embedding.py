"""GPU tests of ssd_embedding and ssd_embedding_bwd against the formulas in 64 bits.

Tolerances, fixed before the first run: a looked-up value is one product, rounded to fp32 and to its type. A gradient is
a sum of n terms in fp32: at most n roundings of a partial sum that is no larger than the terms' magnitudes, n 2^-24 of
them, then the scale's, the old value's and the type's rounding."""
from __future__ import annotations

import pytest

from tests.gpu_util import log

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U32 = 2.0 ** -24


def _t(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _tokens(rows, vocab, kind, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + rows)
    if kind == "one":
        return torch.full((rows,), vocab // 2, device="cuda", dtype=torch.int32)
    if kind == "none":
        return torch.full((rows,), -1, device="cuda", dtype=torch.int32)
    t = (torch.exp(torch.rand(rows, device="cuda", generator=g) * torch.log(torch.tensor(vocab + 1.0))) - 1).int().clamp(max=vocab - 1)
    if kind == "even":
        t = torch.randint(0, vocab, (rows,), device="cuda", generator=g, dtype=torch.int32)
    if kind == "wild":  # padding and tokens behind the table
        t[torch.rand(rows, device="cuda", generator=g) < 0.3] = -1
        t[torch.rand(rows, device="cuda", generator=g) < 0.1] = vocab
        t[torch.rand(rows, device="cuda", generator=g) < 0.05] = 2 ** 31 - 1
        t[torch.rand(rows, device="cuda", generator=g) < 0.05] = -2 ** 31
    return t


@pytest.mark.parametrize("rows,vocab,dim", [(1, 1, 1), (1, 50257, 2048), (37, 100, 7), (300, 259, 1003), (1000, 5000, 96), (5, 3, 4100), (70000, 1000, 36)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_lookup(ssd, rows, vocab, dim, dtype, out):
    import torch
    table = torch.randn(vocab, dim, device="cuda").to(_t(dtype))
    tokens = _tokens(rows, vocab, "wild")
    buf = torch.full((rows * dim + 512,), 7.0, device="cuda").to(_t(out))
    for scale in (1.0, dim ** 0.5):
        y = ssd.ssd_embedding(tokens, table, scale=scale, y=buf[:rows * dim].view(rows, dim))
        torch.cuda.synchronize()
        there = (tokens >= 0) & (tokens < vocab)
        scale32 = float(torch.tensor(scale, dtype=torch.float32))
        ref = torch.where(there[:, None], table[tokens.clamp(0, vocab - 1).long()].double() * scale32, torch.zeros((), device="cuda", dtype=torch.float64))
        assert bool(((y.double() - ref).abs() <= ref.abs() * (HALF[out] + 2 * U32)).all())
        assert bool((buf[rows * dim:].float() == 7.0).all())
    if dtype == out:
        y = ssd.ssd_embedding(tokens.view(1, rows), table)
        torch.cuda.synchronize()
        assert y.shape == (1, rows, dim) and y.dtype == table.dtype and torch.equal(y[0][there], table[tokens[there].long()])


def _gradient(ssd, rows, vocab, dim, dtype, grad, kind, scale=1.0, accumulate=False):
    import torch
    g = torch.Generator(device="cuda").manual_seed(rows + dim)
    tokens = _tokens(rows, vocab, kind)
    dy = torch.randn(rows, dim, device="cuda", generator=g).to(_t(dtype))
    there = (tokens >= 0) & (tokens < vocab)
    dy[~there] = float("nan")   # nothing is taken from these
    buf = torch.full((vocab * dim + 512,), 7.0, device="cuda").to(_t(grad))
    d = buf[:vocab * dim].view(vocab, dim)
    old = torch.randn(vocab, dim, device="cuda", generator=g).to(_t(grad))
    d.copy_(old)
    scale32 = float(torch.tensor(scale, dtype=torch.float32))
    ssd.ssd_embedding_bwd(dy, tokens, vocab, scale=scale, dtable=d, accumulate=accumulate)
    fresh = None if accumulate else ssd.ssd_embedding_bwd(dy, tokens, vocab, scale=scale, dtype=_t(grad))
    torch.cuda.synchronize()
    ref = torch.zeros(vocab, dim, device="cuda", dtype=torch.float64)
    mag, many = torch.zeros_like(ref), torch.zeros(vocab, device="cuda", dtype=torch.float64)
    t = tokens[there].long()
    ref.index_add_(0, t, dy[there].double())
    mag.index_add_(0, t, dy[there].double().abs())
    many.index_add_(0, t, torch.ones_like(t, dtype=torch.float64))
    ref, mag = ref * scale32, mag * abs(scale32)
    lim = (many[:, None] + 3) * U32 * mag
    if accumulate:
        ref = ref + old.double()
        lim = lim + 2 * U32 * (mag + old.double().abs())
    err = (d.double() - ref).abs()
    assert not bool((~(err <= lim + HALF[grad] * ref.abs())).any()), float((err - lim).max())
    assert bool((buf[vocab * dim:].float() == 7.0).all())
    untouched = many == 0
    assert torch.equal(d[untouched], old[untouched] if accumulate else torch.zeros_like(d[untouched]))
    if fresh is not None:
        assert torch.equal(fresh, d), "the same bits"
    return d


SHAPES = [(1, 1, 1), (1, 50257, 64), (15, 100, 7), (16, 10, 8), (17, 10, 8), (300, 259, 1003), (1000, 5000, 96), (5000, 131072, 20),
          (16384, 50257, 64), (16385, 300, 36), (40000, 70, 12), (140000, 200000, 4), (30000, 600000, 5)]


@pytest.mark.parametrize("rows,vocab,dim", SHAPES)
@pytest.mark.parametrize("dtype,grad", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
def test_gradient(ssd, rows, vocab, dim, dtype, grad):
    log(f"[embedding] {rows} {vocab} {dim} {dtype} {grad}")
    _gradient(ssd, rows, vocab, dim, dtype, grad, "words", scale=dim ** 0.5)
    _gradient(ssd, rows, vocab, dim, dtype, grad, "wild")


@pytest.mark.parametrize("kind", ["one", "none", "even"])
@pytest.mark.parametrize("rows,vocab,dim", [(1, 3, 5), (16, 3, 64), (31, 7, 100), (4096, 1, 300), (20000, 11, 260), (50000, 2, 8), (9000, 9000, 16)])
def test_gradient_of_skewed_tokens(ssd, kind, rows, vocab, dim):
    """One token for all rows, none, or all tokens alike: sums that go over many pieces of the sorted list, or none."""
    _gradient(ssd, rows, vocab, dim, "f32", "f32", kind)
    _gradient(ssd, rows, vocab, dim, "bf16", "f32", kind, scale=0.5, accumulate=True)


@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,dim", [(0, 10, 8), (1, 10, 8), (700, 300, 33), (20000, 500, 64)])
def test_gradient_added(ssd, grad, rows, vocab, dim):
    _gradient(ssd, rows, vocab, dim, "bf16", grad, "wild", scale=2.0, accumulate=True)


def test_gradient_of_no_rows(ssd):
    import torch
    d = torch.full((100, 33), 5.0, device="cuda").bfloat16()
    ssd.ssd_embedding_bwd(torch.empty(0, 33, device="cuda"), torch.empty(0, device="cuda", dtype=torch.int32), 100, dtable=d)
    torch.cuda.synchronize()
    assert not bool(d.any())


def test_gradient_by_differences(ssd):
    """The sum of dy * embedding is linear in the table: its change along a direction is the gradient's product with it."""
    import torch
    tokens = _tokens(500, 60, "wild")
    dy, way = torch.randn(500, 24, device="cuda"), torch.randn(60, 24, device="cuda")
    d = ssd.ssd_embedding_bwd(dy, tokens, 60, scale=3.0)
    y = ssd.ssd_embedding(tokens, way, scale=3.0)
    torch.cuda.synchronize()
    a, b = float((d.double() * way.double()).sum()), float((y.double() * dy.double()).sum())
    assert abs(a - b) <= 1e-5 * float((y.double() * dy.double()).abs().sum())


def test_captured_and_replayed(ssd):
    import torch
    rows, vocab, dim = 20000, 500, 96
    dy, tokens = torch.randn(rows, dim, device="cuda").bfloat16(), _tokens(rows, vocab, "wild")
    table = torch.randn(vocab, dim, device="cuda").bfloat16()
    def run():
        return ssd.ssd_embedding(tokens, table), ssd.ssd_embedding_bwd(dy, tokens, vocab, dtype=torch.float32)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for r in range(4):
        tokens.copy_(_tokens(rows, vocab, ("wild", "one", "even", "none")[r], seed=r))
        dy.normal_()
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), r
