"""CPU test of the sizes that ssd_beam_select refuses: more wavefronts than one launch takes. Pointers are fake aligned
addresses; every call fails a host-side check."""
from __future__ import annotations

import pytest

import ssd_sequence_mixing_amd as ssd
from tests.test_layer_abi import EUNSUP, EWS, NONE, select

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
