"""Layouts that the calls on tensors refuse before any launch.  CPU only: the
device tensors here are descriptions without memory."""
import pytest
import torch

import state_space_model_amd as ssd


class Described(torch.Tensor):
    """Sizes, strides, type and device of a tensor that has no memory."""

    @staticmethod
    def __new__(cls, *size, strides=None, dtype=torch.float32, device="cuda:0"):
        return torch.Tensor._make_wrapper_subclass(cls, size, strides=strides, dtype=dtype,
                                                   device=device)

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError(func)


@pytest.mark.parametrize("t", [
    torch.zeros(14)[::2], torch.zeros(1).expand(7), torch.zeros(5, 7)[:, 3]],
    ids=["every_second", "expanded", "a_column"])
def test_row_stride_of_one_row_that_is_not_dense(t):
    """A gate of one dimension is one row: its elements must be adjacent."""
    with pytest.raises(ValueError, match="evenly spaced"):
        ssd._row_stride(t, "z")


def test_row_stride_of_one_dense_row():
    assert ssd._row_stride(torch.zeros(20)[3:10], "z") == 7
    # one element and none have no neighbours
    assert ssd._row_stride(torch.zeros(14)[::14], "z") == 1
    assert ssd._row_stride(torch.zeros(()), "z") == 1
    assert ssd._row_stride(torch.zeros(14)[:0:2], "z") == 0


@pytest.mark.parametrize("strides", [(2,), (0,)], ids=["every_second", "expanded"])
def test_gated_norm_refuses_a_row_that_is_not_dense(strides):
    """The gate in all three forms, and the gate's gradient as a buffer."""
    y, w, bad = Described(8), Described(8), Described(8, strides=strides)
    for call in (lambda: ssd.ssd_gated_norm(y, bad, w),
                 lambda: ssd.ssd_gated_norm_q8(y, bad, w),
                 lambda: ssd.ssd_gated_norm_backward(y, bad, w, dout=y),
                 lambda: ssd.ssd_gated_norm_backward(y, y, w, dout=y, grads={"dz": bad})):
        with pytest.raises(ValueError, match="evenly spaced"):
            call()
