"""The largest shapes that the convolution's gradients take: those whose grids
would count more threads than 32 bits hold are refused with every other wrong
argument, before the first launch.  CPU only (addresses that are never read)."""
import ctypes

import pytest

from state_space_model_amd import ConvDesc, lib

INVALID, UNSUP = 1, 5


def call(batch, seqlen, channels, width, io=1, x=True):
    d = ConvDesc(batch, seqlen, channels, width, io, 1)
    p = [ctypes.c_void_p(0x100000000000 + (i << 40)) for i in range(11)]   # x .. workspace
    p[0] = p[0] if x else None
    st = lib.ssd_conv1d_backward(ctypes.byref(d), io, *p, ctypes.c_size_t(1 << 62), None)
    return st, lib.ssd_conv1d_backward_workspace_bytes(ctypes.byref(d))


@pytest.mark.parametrize("channels", [(1 << 29) - 63, 1 << 29, (1 << 31) - 1])
@pytest.mark.parametrize("seqlen", [0, 1])
def test_more_channels_than_the_sum_of_the_parts_counts(channels, seqlen):
    """Eight threads to a channel."""
    assert call(1, seqlen, channels, 4) == (UNSUP, 0)


@pytest.mark.parametrize("batch,channels,width", [(16, (1 << 27) - 7, 3), (65535, 65537, 2),
                                                  (3, (1 << 29) - 64, 4)])
def test_more_windows_than_an_empty_sequence_hands_on(batch, channels, width):
    """A thread to an element of the window."""
    assert batch * channels * (width - 1) > (1 << 32) - 256
    assert call(batch, 0, channels, width) == (UNSUP, 0)


def test_the_largest_shapes_are_looked_at():
    """Their pointers are: a missing x is what is refused."""
    st, need = call(1, 1, (1 << 29) - 64, 4, x=False)
    assert st == INVALID and need > 0
    assert call(65535, 1, 65537, 2, x=False)[0] == INVALID
    # an empty sequence needs no x, but never a missing dw
    d = ConvDesc(16, 0, (1 << 27) - 8, 3, 1, 1)
    p = [ctypes.c_void_p(0x100000000000 + (i << 40)) for i in range(11)]
    p[7] = None
    assert lib.ssd_conv1d_backward(ctypes.byref(d), 1, *p, ctypes.c_size_t(1 << 62), None) == INVALID
