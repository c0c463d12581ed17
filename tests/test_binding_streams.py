"""CPU test of the streams that the operators around the core take: one of the tensors' device, as an object or as its
address. A stand-in takes a stream's place; nothing is launched."""
from __future__ import annotations

import pytest

import ssd_sequence_mixing_amd as ssd


class _Stream:
    def __init__(self, index):
        self.device_index, self.cuda_stream = index, 0x40


def test_stream_of_another_device_is_refused():
    ssd.load()
    with pytest.raises(ValueError, match="stream of cuda:1"):
        ssd._stream_on(0, _Stream(1))


def test_streams_of_the_device():
    ssd.load()
    assert ssd._stream_on(0, _Stream(0)) == 0x40
    assert ssd._stream_on(1, _Stream(1)) == 0x40
    assert ssd._stream_on(0, 0x80) == 0x80
