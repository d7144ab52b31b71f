"""CPU: what the binding takes as a stream."""
import enum

from fp8_fine_grained_fp8bs_amd import fp8bs


class Handle(int):
    pass


class Known(enum.IntEnum):
    DEFAULT = 0


class Stream:
    cuda_stream = 64


def test_handles():
    for handle, value in ((0, 0), (128, 128), (Handle(192), 192), (Known.DEFAULT, 0), (Stream(), 64)):
        assert fp8bs._stream(handle) == value
        assert fp8bs._stream_later(handle) == value
