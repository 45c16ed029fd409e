"""Layouts that the calls on tensors refuse before any launch, and the device
they launch on.  CPU only: the device tensors here are descriptions without
memory."""
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


def block_calls(m):
    """Every call on tensors between two scans, on the descriptions m makes."""
    x, w, c3, i8 = m(4, 128), m(128), m(2, 4, 128), lambda *n: m(*n, dtype=torch.int8)
    grads = lambda **shapes: {k: m(*v) for k, v in shapes.items()}
    return {
        "add_norm": lambda: ssd.ssd_add_norm(x, w, y=x, residual_out=x),
        "add_norm_q8": lambda: ssd.ssd_add_norm_q8(x, w, q=i8(4, 128), qscale=m(4), residual_out=x),
        "add_norm_backward": lambda: ssd.ssd_add_norm_backward(
            x, w, dy=x, workspace=x, grads=grads(dx=(4, 128), dresidual=(4, 128), dweight=(128,))),
        "gated_norm": lambda: ssd.ssd_gated_norm(x, x, w, out=x),
        "gated_norm_q8": lambda: ssd.ssd_gated_norm_q8(x, x, w, q=i8(4, 128), qscale=m(4)),
        "gated_norm_backward": lambda: ssd.ssd_gated_norm_backward(
            x, x, w, dout=x, workspace=x, grads=grads(dy=(4, 128), dz=(4, 128), dweight=(128,))),
        "quantize_q8": lambda: ssd.ssd_quantize_q8(x, q=i8(4, 128), qscale=m(4)),
        "linear_q8": lambda: ssd.ssd_linear_q8(i8(4, 128), m(4), i8(5, 128), m(5), out=m(4, 5)),
        "conv1d_backward": lambda: ssd.ssd_conv1d_backward(
            c3, m(128, 4), dy=c3, workspace=x, grads=grads(
                dx=(2, 4, 128), dweight=(128, 4), dbias=(128,), dstate=(2, 128, 3)))}


def scan_calls(m):
    x, dt, a, bc = m(2, 64, 2, 64), m(2, 64, 2), m(2), m(2, 64, 1, 64)
    st = m(2, 2, 64, 64)
    scan = dict(y=x, final_state=st, chunk=64)
    return {
        "chunk_scan": lambda: ssd.ssd_chunk_scan(x, dt, a, bc, bc, workspace=x, **scan),
        "chunk_scan_noalloc": lambda: ssd.ssd_chunk_scan_noalloc(x, dt, a, bc, bc, **scan),
        "chunk_scan_ablation": lambda: ssd.ssd_chunk_scan(
            x, dt, a, bc, bc, workspace=x, variant=ssd.SSD_VARIANT_BF16_DECAY, **scan),
        "step": lambda: ssd.ssd_step(st, m(2, 2, 64), m(2, 2), a, m(2, 1, 64), m(2, 1, 64),
                                     y_t=m(2, 2, 64)),
        "conv1d": lambda: ssd.ssd_conv1d(m(2, 4, 128), m(128, 4), y=m(2, 4, 128),
                                         state_out=m(2, 128, 3)),
        "conv1d_step": lambda: ssd.ssd_conv1d_step(m(2, 128, 3), m(2, 128), m(128, 4),
                                                   y_t=m(2, 128))}


def all_calls(device="cuda:0"):
    m = lambda *size, **kw: Described(*size, device=device, **kw)
    return {**block_calls(m), **scan_calls(m)}


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("name", all_calls())
def test_a_call_launches_with_its_tensors_device_current(name, index, monkeypatch):
    """Device 0 is current.  A call on tensors of device 1 asks for that
    device's stream, makes that device current and device 0 again afterwards,
    also when it fails (as here, at the null pointers of these tensors)."""
    asked, made_current = [], []
    stream = lambda i: asked.append(i) or 0
    monkeypatch.setattr(ssd, "_raw_stream", stream)
    monkeypatch.setattr(ssd, "_current_device", lambda: 0)
    monkeypatch.setattr(ssd, "_set_device", made_current.append)
    ssd._calls.connect(ssd.SSDError, stream, lambda: 0, made_current.append)
    try:
        with pytest.raises(ssd.SSDError):
            all_calls(f"cuda:{index}")[name]()
    finally:
        monkeypatch.undo()
        ssd._calls.connect(ssd.SSDError, ssd._raw_stream, ssd._current_device, ssd._set_device)
    assert asked == [index]
    assert made_current == ([] if index == 0 else [1, 0])
