"""The model operators' Python layer takes tensors of the current device alone: the C ABI launches there (stand-ins for
tensors of a second device, on the CPU)."""
import pytest
import torch

from compensated_bit_reproducible_gb300 import api


class Elsewhere:
    """What the checks look at of a tensor on device 1."""
    is_cuda, dtype, shape = True, torch.float32, (4, 8)

    def __init__(self, dims=2):
        self.dims = dims

    def get_device(self):
        return 1

    def dim(self):
        return self.dims

    def numel(self):
        return 4 if self.dims == 1 else 32

    def stride(self):
        return (8, 1)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


@pytest.mark.parametrize("check", [lambda t: api._mat(t, 0), lambda t: api._vec(t, torch.float32, 4, 0),
                                   lambda t: api._stream_on(t.get_device(), None)])
def test_tensors_of_another_device(monkeypatch, check):
    monkeypatch.setattr(api, "_device", lambda: 0)
    with pytest.raises(AssertionError):
        check(Elsewhere(1))


def test_the_current_device_may_be_another_than_the_first(monkeypatch):
    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(api, "_device", lambda: 1)
    assert api._stream_on(1, Stream()) == 77
    assert api._mat(Elsewhere(), 1) == (1 << 20, 4, 8, 8)
    assert api._vec(Elsewhere(1), torch.float32, 4, 1) == 1 << 20
