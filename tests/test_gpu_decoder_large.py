"""GPU tests of the recurrence, the embedding, the logits' processing and the integer products on tensors of more than
2^31 values: parts of the results, from the front and from behind the 2^31st value, have the bits of a call on that part
alone (or are checked against the definition)."""
from __future__ import annotations

import pytest

from tests.gpu_util import log

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    import torch
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_scan_of_many_values(ssd):
    import torch
    B, T, D = 1, 50000, 43100   # 2.16e9 values, a step of 11034000 bytes between chunks
    log(f"[large] scan {B} {T} {D}")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(B, T, D, device="cuda", generator=g, dtype=torch.bfloat16)
    f = torch.randn(B, T, D, device="cuda", generator=g, dtype=torch.bfloat16).add_(2)
    assert x.numel() > 2 ** 31
    y, final, states = ssd.ssd_gated_scan_fwd(x, f, decay="sigmoid", want_states=True)
    for d0 in (0, D - 100):
        a, b = x[..., d0:d0 + 100].contiguous(), f[..., d0:d0 + 100].contiguous()
        yp, fp, sp = ssd.ssd_gated_scan_fwd(a, b, decay="sigmoid", want_states=True)
        torch.cuda.synchronize()
        assert torch.equal(y[..., d0:d0 + 100], yp) and torch.equal(final[:, d0:d0 + 100], fp) and torch.equal(states[..., d0:d0 + 100], sp)
    dx, df, _, _, d0_ = ssd.ssd_gated_scan_bwd(y, x, f, states, decay="sigmoid")
    for d0 in (0, D - 100):
        cut = [t[..., d0:d0 + 100].contiguous() for t in (y, x, f, states)]
        dxp, dfp, _, _, dp = ssd.ssd_gated_scan_bwd(*cut, decay="sigmoid")
        torch.cuda.synchronize()
        assert torch.equal(dx[..., d0:d0 + 100], dxp) and torch.equal(df[..., d0:d0 + 100], dfp) and torch.equal(d0_[:, d0:d0 + 100], dp)


def test_scan_of_tokens_far_apart(ssd):
    """Tokens 2^21 values apart: a sequence of 1100 spans 2^31 values and more."""
    import torch
    T, D, ld = 1100, 70, 1 << 21
    log(f"[large] tokens {ld} apart")
    wide = torch.empty(1, T, ld, device="cuda", dtype=torch.bfloat16)
    x, f = wide[..., ld - 70:], wide[..., 5:75]
    x.normal_(), f.normal_()
    y, final, states = ssd.ssd_gated_scan_fwd(x, f, decay="sigmoid", want_states=True)
    yp, fp, sp = ssd.ssd_gated_scan_fwd(x.contiguous(), f.contiguous(), decay="sigmoid", want_states=True)
    g = ssd.ssd_gated_scan_bwd(y, x, f, states, decay="sigmoid")
    gp = ssd.ssd_gated_scan_bwd(y, x.contiguous(), f.contiguous(), states, decay="sigmoid")
    torch.cuda.synchronize()
    assert torch.equal(y, yp) and torch.equal(final, fp) and torch.equal(states, sp)
    assert torch.equal(g[0], gp[0]) and torch.equal(g[1], gp[1])


def test_step_of_many_rows(ssd):
    import torch
    rows, D = 300000, 7000   # 2.1e9 values
    log(f"[large] step {rows} {D}")
    state = torch.empty(rows, D, device="cuda").normal_()
    x = torch.empty(rows, D, device="cuda", dtype=torch.bfloat16).normal_()
    last = state[-50:].clone()
    y = ssd.ssd_gated_step(state, state, x, x, decay="sigmoid")
    yp = ssd.ssd_gated_step(last, last, x[-50:], x[-50:], decay="sigmoid")
    torch.cuda.synchronize()
    assert torch.equal(y[-50:], yp) and torch.equal(state[-50:], last)


def test_embedding_of_many_values(ssd):
    import torch
    V, D, rows = 1 << 20, 2056, 1 << 20   # table and rows of 2.16e9 values each
    log(f"[large] embedding {rows} {V} {D}")
    table = torch.empty(V, D, device="cuda", dtype=torch.bfloat16).normal_()
    tokens = torch.randint(0, V, (rows,), device="cuda", dtype=torch.int32)
    tokens[-3:] = V - 1
    y = ssd.ssd_embedding(tokens, table, scale=2.0)
    torch.cuda.synchronize()
    for r in (0, rows // 2, rows - 1):
        assert torch.equal(y[r], table[int(tokens[r])] * 2)
    del table
    d = ssd.ssd_embedding_bwd(y, tokens, V, dtype=torch.float32)
    torch.cuda.synchronize()
    order = torch.sort(tokens, stable=True)
    for v in (int(order.values[0]), int(order.values[rows // 3]), V - 1):
        mine = (tokens == v).nonzero()[:, 0]
        want = y[mine].double().sum(0)
        assert float((d[v].double() - want).abs().max()) <= (len(mine) + 2) * 2.0 ** -24 * float(y[mine].double().abs().sum(0).max())
    unused = torch.ones(V, dtype=torch.bool, device="cuda")
    unused[tokens.long()] = False
    assert not bool(d[unused.nonzero()[-1000:, 0]].any())


def test_logits_of_many_values(ssd):
    import torch
    rows, V = 17000, 131071   # 2.2e9 values
    log(f"[large] logits {rows} {V}")
    l = torch.empty(rows, V, device="cuda", dtype=torch.bfloat16).normal_()
    tokens = torch.randint(0, V, (rows, 20), device="cuda", dtype=torch.int32)
    freq = torch.ones(rows, device="cuda")
    mask = torch.full((4096,), -1, device="cuda", dtype=torch.int32)
    mask[1000] = 5
    y = ssd.ssd_logits_process(l, tokens=tokens, frequency=freq, mask=mask)
    part = ssd.ssd_logits_process(l[-8:].contiguous(), tokens=tokens[-8:].contiguous(), frequency=freq[-8:].contiguous(), mask=mask)
    torch.cuda.synchronize()
    assert torch.equal(y[-8:], part) and bool((y[-1, 32001] == -float("inf")))
    t = int(tokens[-1, 0])
    n = int((tokens[-1] == t).sum())
    if t // 32 != 1000:
        assert float(y[-1, t]) == float((l[-1, t].float() - n).bfloat16())


def test_integer_products_of_many_values(ssd):
    import torch
    rows, k, n = 33000, 64, 65540   # y: 2.16e9 values
    log(f"[large] integer product {rows} {k} {n}")
    x = torch.empty(rows, 65536, device="cuda", dtype=torch.bfloat16).normal_()   # 2.16e9 values to quantise
    q, s = ssd.ssd_int_quantize(x)
    qp, sp = ssd.ssd_int_quantize(x[-5:].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(q[-5:], qp) and torch.equal(s[-5:], sp)
    xq = q[:, -k:].contiguous()
    del x, q
    wq, ws = ssd.ssd_int_quantize(torch.randn(n, k, device="cuda"))
    y = ssd.ssd_linear_int(xq, s, wq, ws)
    torch.cuda.synchronize()
    want = (xq[-20:].double() @ wq.double().t().contiguous()) * s[-20:].double()[:, None] * ws.double()
    assert bool(((y[-20:].double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -20) + 1e-30).all())
