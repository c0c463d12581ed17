"""CPU tests of what the operators around the core refuse: selections of more wavefronts than one launch takes, and
products whose outputs lie on their inputs. Pointers are fake aligned addresses; every call fails a host-side check."""
from __future__ import annotations

import pytest

import ssd_sequence_mixing_amd as ssd
from tests.test_layer_abi import EUNSUP, EWS, NONE, P, linear, linear_bwd, linear_mx, select

MOST = (1 << 26) - 4  # wavefronts of 2048 logits


@pytest.mark.parametrize("batch,beams,vocab", [
    (MOST // 32, 16, 2049),          # 2 of them a row
    (MOST // 64, 1, 131072),         # 64
    (MOST // (64 * 4), 4, 1 << 28),  # 64 longer ones
    ((1 << 21) - 1, 16, 2048)])
def test_select_takes_as_many_wavefronts_as_one_launch(batch, beams, vocab):
    need = ssd.load().ssd_beam_select_workspace_bytes(batch, beams, vocab)
    assert need != NONE
    assert select(batch=batch, beams=beams, vocab=vocab, wsb=need - 1) == EWS


@pytest.mark.parametrize("batch,beams,vocab", [
    (MOST // 32 + 1, 16, 2049), ((1 << 21) - 1, 16, 6000), (MOST // 64 + 1, 1, 131072),
    (MOST // (64 * 4) + 1, 4, 1 << 28), ((1 << 21) - 1, 16, 1 << 28)])
def test_select_refuses_more(batch, beams, vocab):
    assert ssd.load().ssd_beam_select_workspace_bytes(batch, beams, vocab) == NONE
    assert select(batch=batch, beams=beams, vocab=vocab) == EUNSUP


FAR = 1 << 44   # apart from everything at P


@pytest.mark.parametrize("kw,code", [
    (dict(y=P + 16), EUNSUP), (dict(x=FAR), EUNSUP), (dict(w=FAR), EUNSUP), (dict(x=FAR, w=FAR, b=P), EUNSUP),
    (dict(x=FAR, w=FAR, r=P + 16), EUNSUP), (dict(x=FAR, w=FAR, y=FAR << 1, pre=FAR), EUNSUP),
    (dict(x=FAR, w=FAR, y=FAR << 1, r=P, pre=P), EUNSUP), (dict(w=FAR, x=P + 100 * 48 * 2 - 16), EUNSUP)])
def test_linear_refuses_outputs_on_inputs(kw, code):
    assert linear(**kw) == code


@pytest.mark.parametrize("kw", [dict(), dict(x=FAR), dict(w=FAR, x=FAR), dict(x=FAR, xs=FAR, w=FAR),
                                dict(x=FAR, xs=FAR, w=FAR, ws_=FAR, b=P), dict(x=FAR, xs=FAR, w=FAR, ws_=FAR, r=P + 32)])
def test_linear_mx_refuses_outputs_on_inputs(kw):
    assert linear_mx(**kw) == EUNSUP


@pytest.mark.parametrize("kw", [dict(), dict(dy=FAR), dict(dy=FAR, x=FAR), dict(dy=FAR, x=FAR, w=FAR),
                                dict(dx=FAR, dw=FAR), dict(dx=FAR, dw=FAR, db=FAR, dy=FAR << 1, x=FAR << 1, w=FAR << 1, pre=FAR),
                                dict(dx=None, dw=None), dict(dx=None, db=None, dy=FAR, pre=FAR),
                                dict(dw=None, db=None, dy=FAR, pre=FAR)])
def test_linear_bwd_refuses_outputs_on_inputs(kw):
    assert linear_bwd(**kw) == EUNSUP
