"""The operators between two scans refuse wrong arguments before any launch:
shapes in the binding, everything else in the C ABI (fake device addresses
that are never dereferenced).  CPU only."""
import ctypes

import pytest
import torch

import state_space_model_amd as ssd
from state_space_model_amd import AddNormDesc, ConvDesc, GatedNormDesc, LinearQ8Desc, lib

OK, INVALID, SHAPE, DTYPE, ALIGN, UNSUP, WS, HIP = range(8)
BASE = 0x7F0000000000
NAN, INF = float("nan"), float("inf")


def addr(i):
    return BASE + (i << 32)


def call(fn, desc, n, *tail, **over):
    """fn(desc, n pointers, tail, stream) with pointers 0..n-1 at disjoint
    addresses unless overridden as p<i>."""
    ptrs = [ctypes.c_void_p(over.get(f"p{i}", addr(i + 1))) for i in range(n)]
    return fn(ctypes.byref(desc) if desc is not None else None, *ptrs, *tail, None)


def add_desc(rows=5, cols=100, io=1, scale=1.0, eps=1e-5):
    return AddNormDesc(rows, cols, io, scale, eps)


ADD_BAD = [(dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(io=2), DTYPE),
           (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID),
           (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(cols=16385), UNSUP),
           (dict(rows=1 << 31), UNSUP)]


@pytest.mark.parametrize("kw,code", ADD_BAD)
def test_add_norm_descriptors(kw, code):
    d = add_desc(**kw)
    ws = ctypes.c_size_t(1 << 40)
    assert call(lib.ssd_add_norm, d, 5) == code
    assert call(lib.ssd_add_norm_q8, d, 6) == code
    assert call(lib.ssd_add_norm_backward, d, 8, ws) == code
    assert lib.ssd_add_norm_backward_workspace_bytes(ctypes.byref(d)) == 0
    assert call(lib.ssd_add_norm, None, 5) == INVALID


def test_add_norm_arguments():
    d = add_desc()
    f = lambda **o: call(lib.ssd_add_norm, d, 5, **o)     # x, residual, weight, y, residual_out
    for p in ("p0", "p2", "p3"):
        assert f(**{p: 0}) == INVALID
    assert f(p0=addr(1) + 1) == ALIGN and f(p1=addr(2) + 2) == ALIGN and f(p4=addr(5) + 1) == ALIGN
    assert f(p3=addr(1)) == INVALID                       # y over x
    assert f(p4=addr(2) + 4) == INVALID                   # residual_out shifted into residual
    assert f(p4=addr(4)) == INVALID                       # two outputs
    g = lambda **o: call(lib.ssd_add_norm_q8, d, 6, **o)  # x, residual, weight, q, qscale, res_out
    assert g(p3=0) == INVALID and g(p4=0) == INVALID and g(p3=addr(4) + 8) == ALIGN
    assert g(p4=addr(4) + 512) == INVALID                 # scales inside the padded rows
    need = lib.ssd_add_norm_backward_workspace_bytes(ctypes.byref(d))
    assert need >= 4 * 100
    # residual_out, weight, dy, dresidual_out, dx, dresidual, dweight, workspace
    h = lambda w=need, **o: call(lib.ssd_add_norm_backward, d, 8, ctypes.c_size_t(w), **o)
    assert h(p0=0) == INVALID and h(p6=0) == INVALID and h(p2=0) == INVALID
    assert h(p7=0) == WS and h(w=need - 1) == WS and h(p7=addr(8) + 4) == ALIGN
    assert h(p4=addr(3)) == INVALID and h(p5=addr(4) + 4) == INVALID and h(p6=addr(8)) == INVALID
    # nothing to do: no pointer is needed
    assert lib.ssd_add_norm(ctypes.byref(add_desc(rows=0)), *[None] * 5, None) == OK


def gated_desc(rows=5, cols=96, groups=2, z=96, dz=96, io=1, eps=1e-5):
    return GatedNormDesc(rows, cols, groups, z, dz, io, eps)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(groups=0), SHAPE), (dict(groups=5), SHAPE),
    (dict(z=95), SHAPE), (dict(io=-1), DTYPE), (dict(eps=NAN), INVALID),
    (dict(cols=16386 * 2, z=16386 * 2, dz=16386 * 2), UNSUP), (dict(rows=1 << 30), UNSUP)])
def test_gated_norm_descriptors(kw, code):
    d = gated_desc(**kw)
    ws = ctypes.c_size_t(1 << 50)
    if kw != dict(rows=1 << 30):
        assert call(lib.ssd_gated_norm, d, 4) == code
        assert call(lib.ssd_gated_norm_q8, d, 5) == code
    else:                                                 # rows * groups beyond the grid
        assert call(lib.ssd_gated_norm, d, 4) == code
    assert call(lib.ssd_gated_norm_backward, d, 8, ws) == code
    assert lib.ssd_gated_norm_backward_workspace_bytes(ctypes.byref(d)) == 0


def test_gated_norm_arguments():
    d = gated_desc(z=200, dz=300)
    f = lambda **o: call(lib.ssd_gated_norm, d, 4, **o)   # y, z, weight, out
    for p in ("p0", "p1", "p2", "p3"):
        assert f(**{p: 0}) == INVALID
    assert f(p1=addr(2) + 1) == ALIGN and f(p3=addr(1)) == INVALID
    assert f(p3=addr(2) + 4 * 400 + 100) == INVALID       # inside z's span
    wide = gated_desc(cols=16384 * 2, z=16384 * 2)
    assert call(lib.ssd_gated_norm_q8, wide, 5) == UNSUP
    assert call(lib.ssd_gated_norm_q8, gated_desc(cols=1025, groups=1025, z=1025), 5) == UNSUP
    need = lib.ssd_gated_norm_backward_workspace_bytes(ctypes.byref(d))
    # y, z, weight, dout, dy, dz, dweight, workspace
    h = lambda w=need, **o: call(lib.ssd_gated_norm_backward, d, 8, ctypes.c_size_t(w), **o)
    for i in range(7):
        assert h(**{f"p{i}": 0}) == INVALID
    assert h(p7=0) == WS and h(w=need - 1) == WS
    assert h(p5=addr(5)) == INVALID and h(p4=addr(4)) == INVALID and h(p5=addr(6) + 1) == ALIGN
    assert call(lib.ssd_gated_norm_backward, gated_desc(dz=95), 8, ctypes.c_size_t(1 << 40)) == SHAPE


def test_quantize_and_linear_arguments():
    qz = lambda r, c, t, v=addr(1), q=addr(2), s=addr(3): lib.ssd_quantize_q8(
        r, c, t, ctypes.c_void_p(v), ctypes.c_void_p(q), ctypes.c_void_p(s), None)
    assert qz(5, 100, 7) == DTYPE and qz(-1, 100, 0) == SHAPE and qz(5, 0, 0) == SHAPE
    assert qz(5, 130945, 0) == UNSUP and qz(1 << 31, 8, 0) == UNSUP
    assert qz(5, 100, 0, v=0) == INVALID and qz(5, 100, 0, q=0) == INVALID and qz(5, 100, 0, s=0) == INVALID
    assert qz(5, 100, 0, q=addr(2) + 8) == ALIGN and qz(5, 100, 0, v=addr(1) + 2) == ALIGN
    assert qz(5, 100, 1, q=addr(1) + 16) == INVALID and qz(0, 100, 0, v=0) == OK
    ok = dict(rows=5, cols=256, outs=9, out_dtype=1)
    lin = lambda o={}, **kw: call(lib.ssd_linear_q8, LinearQ8Desc(**{**ok, **kw}), 5, **o)
    assert lin(rows=-1) == SHAPE and lin(cols=0) == SHAPE and lin(outs=0) == SHAPE
    assert lin(cols=192) == SHAPE and lin(out_dtype=4) == DTYPE
    assert lin(cols=131072) == UNSUP and lin(rows=1 << 31) == UNSUP and lin(outs=1 << 31) == UNSUP
    for i in range(5):
        assert lin({f"p{i}": 0}) == INVALID
    assert lin({"p0": addr(1) + 8}) == ALIGN and lin({"p2": addr(3) + 4}) == ALIGN
    assert lin({"p1": addr(2) + 2}) == ALIGN and lin({"p4": addr(5) + 1}) == ALIGN
    assert lin({"p4": addr(3)}) == INVALID and lin({"p4": addr(1)}) == INVALID
    assert lin({f"p{i}": 0 for i in range(5)}, rows=0) == OK


def test_conv_backward_arguments():
    d = lambda **kw: ConvDesc(*{**dict(b=2, t=9, c=24, k=4, io=1, silu=1), **kw}.values())
    need = lib.ssd_conv1d_backward_workspace_bytes(ctypes.byref(d()))
    assert need > 0
    names = ["x", "w", "bias", "state", "dy", "dso", "dx", "dw", "dbias", "dstate", "ws"]

    def f(desc=None, dyt=0, bytes_=need, **o):
        ptrs = [ctypes.c_void_p(o.get(n, addr(i + 1))) for i, n in enumerate(names)]
        return lib.ssd_conv1d_backward(ctypes.byref(desc or d()), dyt, *ptrs, ctypes.c_size_t(bytes_), None)

    assert f(d(io=3)) == DTYPE and f(d(t=-1)) == SHAPE and f(d(c=0)) == SHAPE and f(d(k=5)) == UNSUP
    assert f(dyt=2) == DTYPE and f(d(io=0), dyt=1) == DTYPE
    for n in ("x", "w", "dy", "dx", "dw"):
        assert f(**{n: 0}) == INVALID
    assert f(ws=0) == WS and f(bytes_=need - 1) == WS
    assert f(x=addr(1) + 8) == ALIGN and f(dw=addr(8) + 2) == ALIGN
    assert f(dx=addr(5)) == INVALID and f(dstate=addr(4)) == INVALID and f(dw=addr(11)) == INVALID
    assert lib.ssd_conv1d_backward(None, 0, *[None] * 11, ctypes.c_size_t(0), None) == INVALID
    assert lib.ssd_conv1d_backward_workspace_bytes(ctypes.byref(d(k=7))) == 0


Z = torch.zeros


@pytest.mark.parametrize("fn,match", [
    (lambda: ssd.ssd_add_norm(Z(2, 8), Z(7)), "weight must have shape"),
    (lambda: ssd.ssd_add_norm(Z(2, 8), Z(8), Z(2, 9)), "residual must have shape"),
    (lambda: ssd.ssd_add_norm(Z(2, 8), Z(8), y=Z(2, 7)), "y must have shape"),
    (lambda: ssd.ssd_add_norm_q8(Z(2, 8), Z(8), q=Z(2, 8)), "q must have shape"),
    (lambda: ssd.ssd_add_norm_q8(Z(2, 8), Z(8), qscale=Z(3)), "qscale must have shape"),
    (lambda: ssd.ssd_add_norm(Z(2, 8), Z(8)), "device tensor"),
    (lambda: ssd.ssd_add_norm_backward(Z(2, 8), Z(8), dy=Z(2, 4)), "dy must have shape"),
    (lambda: ssd.ssd_add_norm_backward(Z(2, 8), Z(8), dy=Z(2, 8), grads={"dw": Z(8)}), "unknown gradient"),
    (lambda: ssd.ssd_add_norm_backward(Z(2, 8), Z(8), dy=Z(2, 8), grads={"dx": Z(8)}), "dx must have shape"),
    (lambda: ssd.ssd_gated_norm(Z(2, 8), Z(2, 7), Z(8)), "z must have shape"),
    (lambda: ssd.ssd_gated_norm(Z(2, 8), Z(2, 8), Z(8)), "device tensor"),
    (lambda: ssd.ssd_gated_norm_backward(Z(2, 8), Z(2, 8), Z(8), dout=Z(1, 8)), "dout must have shape"),
    (lambda: ssd.ssd_quantize_q8(Z(2, 8), q=Z(2, 8)), "q must have shape"),
    (lambda: ssd.ssd_linear_q8(Z(2, 128), Z(3), Z(5, 128), Z(5)), "qscale must have shape"),
    (lambda: ssd.ssd_linear_q8(Z(2, 128), Z(2), Z(5, 64), Z(5)), "wq must have shape"),
    (lambda: ssd.ssd_linear_q8(Z(2, 128), Z(2), Z(5, 128), Z(4)), "wscale must have shape"),
    (lambda: ssd.ssd_conv1d_backward(Z(2, 6, 8), Z(8, 4), dy=Z(2, 6, 7)), "dy must have shape"),
    (lambda: ssd.ssd_conv1d_backward(Z(2, 6, 8), Z(7, 4), dy=Z(2, 6, 8)), "weight"),
    (lambda: ssd.ssd_conv1d_backward(Z(2, 6, 8), Z(8, 4), dy=Z(2, 6, 8), dstate_out=Z(2, 8, 4)),
     "dstate_out must have shape"),
], ids=range(19))
def test_binding_refuses_before_launch(fn, match):
    with pytest.raises(ValueError, match=match):
        fn()


def test_binding_refuses_types():
    with pytest.raises(TypeError):
        ssd.ssd_add_norm(Z(2, 8).half(), Z(8))
    with pytest.raises(TypeError):
        ssd.ssd_quantize_q8(Z(2, 8, dtype=torch.int8))


def test_row_strides_of_a_sliced_gate():
    """The row stride the binding reads off a slice of columns, and the layouts
    it refuses."""
    t = torch.zeros(3, 4, 100)
    assert ssd._row_stride(t[..., 10:30], "z") == 100
    assert ssd._row_stride(t[:1, :, 10:30], "z") == 100
    assert ssd._row_stride(t[:, :1, 10:30], "z") == 400
    assert ssd._row_stride(torch.zeros(1, 1, 7), "z") == 7
    assert ssd._row_stride(torch.zeros(7), "z") == 7
    for bad in (t[:, ::2, 10:30][:, :, ::2], t[:, :3, 10:30], t.transpose(0, 1)[..., :5],
                torch.zeros(1, 20).expand(5, 20)):
        with pytest.raises(ValueError, match="evenly spaced"):
            ssd._row_stride(bad, "z")


@pytest.mark.parametrize("exc,fn", [
    (TypeError, lambda: ssd.ssd_add_norm([1.0], Z(8))),
    (TypeError, lambda: ssd.ssd_add_norm_backward(Z(2, 8), Z(8), dy=Z(2, 8), grads=[Z(8)])),
    (TypeError, lambda: ssd.ssd_linear_q8(Z(2, 128), Z(2), Z(5, 128), Z(5), out_dtype=torch.float16)),
    (TypeError, lambda: ssd.ssd_add_norm(Z(2, 8), Z(8), eps="small")),
    (ValueError, lambda: ssd.ssd_add_norm(Z(()), Z(8))),
    (ValueError, lambda: ssd.ssd_gated_norm_q8(Z(()), Z(()), Z(8))),
    (ValueError, lambda: ssd.ssd_quantize_q8(Z(()))),
    (ValueError, lambda: ssd.ssd_conv1d_backward(Z(2, 6, 8), Z(8, 0), dy=Z(2, 6, 8))),
    (ValueError, lambda: ssd.ssd_conv1d_backward(Z(2, 6, 8), Z(8, 4), dy=Z(2, 6, 8),
                                                 grads={3: Z(8)}))])
def test_binding_refuses_what_is_no_tensor_or_has_no_columns(exc, fn):
    with pytest.raises(exc):
        fn()


def test_linear_refuses_more_than_a_grid_counts():
    """512 threads per 16 outputs, 256 per 64 x 64 tile, below 2^32 in all."""
    lin = lambda r, o: call(lib.ssd_linear_q8, LinearQ8Desc(r, 128, o, 1), 5)
    assert lin(1, (1 << 27) - 15) == UNSUP and lin(1, 1 << 27) == UNSUP
    assert lin((1 << 30) + 1, 1) == UNSUP and lin(1 << 18, 1 << 18) == UNSUP
    # the largest that one token has: its pointers are looked at
    assert call(lib.ssd_linear_q8, LinearQ8Desc(1, 128, (1 << 27) - 16, 1), 5, p0=0) == INVALID
