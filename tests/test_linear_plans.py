"""CPU test that the sizes of the GPU tests of the projections' tiles reach the tiles that they are there for."""
from __future__ import annotations

import ssd_sequence_mixing_amd as ssd
from tests.linear_plans import BACKWARD, EIGHT_BITS, FORWARD, T64, T128, T192, T256, plan_of


def test_forward_cases_take_their_tiles():
    for dtype, m, k, n, *want in FORWARD:
        assert plan_of(ssd, "fwd", dtype, m, k, n) == tuple(want), (dtype, m, k, n)
    for m, k, n, *want in EIGHT_BITS:
        assert plan_of(ssd, "mx", "bf16", m, k, n) == tuple(want), (m, k, n)


def test_backward_cases_take_their_tiles():
    for dtype, m, k, n, dx, dw in BACKWARD:
        assert dx is None or plan_of(ssd, "dx", dtype, m, k, n) == dx, (dtype, m, k, n)
        assert dw is None or plan_of(ssd, "dw", dtype, m, k, n) == dw, (dtype, m, k, n)


def test_cases_cover_every_tile():
    """Split and not, of each type; the smallest tile has tests of its own."""
    for dtype, tiles in (("bf16", (T128, T192, T256)), ("f32", (T128, T192))):
        reached = {(t, s) for d, _, _, _, t, s, _ in FORWARD if d == dtype}
        assert reached >= {(t, s) for t in tiles for s in (False, True)}
        assert {r for d, _, _, _, _, _, r in FORWARD if d == dtype and r} >= {T64, T128, T192}
        for i in (4, 5):
            reached = {c[i][:2] for c in BACKWARD if c[0] == dtype and c[i]}
            assert reached >= {(t, s) for t in tiles for s in (False, True)}, (dtype, i)
    assert {c[3] for c in EIGHT_BITS} == {T128, T192, T256}
