"""Token strides that the binding measures (no GPU: the tensors only stand for CUDA ones).  A stride
of 0 means "the row's width" in the C ABI, so one that was measured may never be passed on: the
kernels would read B * N rows of a tensor that holds one."""

import pytest
import torch

from tests._sana import _lib


class OnGpu:
    """A CPU tensor that says it is a CUDA tensor."""

    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


def stride(t, width=256):
    return _lib._token_stride(OnGpu(t), "x", width)


@pytest.mark.parametrize("shape", [(4, 1, 256), (1, 7, 256), (4, 7, 256)])
def test_expanded_tensors_are_refused(shape):
    with pytest.raises(ValueError, match="rows of their own"):
        stride(torch.zeros(1, 1, 256).expand(shape))


@pytest.mark.parametrize("t", [
    torch.zeros(4, 1, 256).expand(4, 7, 256),                        # one token of each sequence, repeated
    torch.zeros(1, 7, 256).expand(4, 7, 256),                        # one sequence for the whole batch
    torch.zeros(1024).as_strided((1, 4, 256), (1024, 128, 1)),       # rows that overlap
    torch.zeros(1024).as_strided((4, 1, 256), (128, 256, 1)),
    torch.zeros(4096).as_strided((2, 3, 256), (384, 128, 1)),
])
def test_rows_that_share_elements_are_refused(t):
    with pytest.raises(ValueError):
        stride(t)


def test_slices_and_single_rows_keep_their_strides():
    packed = torch.zeros(3, 5, 1024)
    assert stride(packed[:, :, 256:512]) == 1024
    assert stride(packed[:, :1, 256:512]) == 5 * 1024        # a token of each sequence
    assert stride(packed[:1, :, :256]) == 1024
    assert stride(torch.zeros(3, 5, 256)) == 256
    # one row, or none: its strides say nothing
    assert stride(torch.zeros(1, 1, 256).as_strided((1, 1, 256), (0, 0, 1))) == 256
    assert stride(packed[:1, :1, :256]) == 256
    assert stride(torch.zeros(2, 0, 256)) == 256 and stride(torch.zeros(0, 4, 256)) == 256
    assert stride(torch.zeros(1, 1, 256).expand(0, 4, 256)) == 256
