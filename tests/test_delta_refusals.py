"""The gated delta rule and the residual add with dropout refuse wrong
arguments before any launch: the C ABI (fake device addresses that are never
dereferenced) and the calls on tensors (tensors without memory).  CPU only."""
import ctypes

import pytest
import torch

import state_space_model_amd as ssd
from state_space_model_amd import DeltaDesc, DropoutAddNormDesc, lib
from test_block_layouts import Described
from test_block_refusals import addr, call

OK, INVALID, SHAPE, DTYPE, ALIGN, UNSUP, WS, HIP = range(8)
NAN, INF = float("nan"), float("inf")


def desc(batch=2, seqlen=70, nheads=4, headdim=16, dstate=24, ngroups=2, strides=None, grads=None,
         io=1, softplus=1, sigmoid=1, norm=1, lo=0.0, hi=INF, eps=1e-6, scale=0.2):
    gn, hp = ngroups * dstate, nheads * headdim
    return DeltaDesc(batch, seqlen, nheads, headdim, dstate, ngroups, *(strides or (gn, gn, hp)),
                     *(grads or (gn, gn, hp)), io, softplus, sigmoid, norm, lo, hi, eps, scale)


def scan(d, ws=None, **over):
    # q, k, v, dt, dt_bias, A, beta, initial_state, y, final_state, workspace
    need = lib.ssd_delta_scan_workspace_bytes(ctypes.byref(d)) if d is not None else 0
    return call(lib.ssd_delta_scan, d, 11, ctypes.c_size_t(need if ws is None else ws), **over)


def step(d, **over):
    # state, q, k, v, dt, dt_bias, A, beta, y
    return call(lib.ssd_delta_step, d, 9, **over)


def back(d, ws=None, **over):
    # q, k, v, dt, dt_bias, A, beta, h0, dy, dfinal, dq, dk, dv, ddt, dbeta, dA, ddt_bias, dh0, workspace
    need = lib.ssd_delta_scan_backward_workspace_bytes(ctypes.byref(d)) if d is not None else 0
    return call(lib.ssd_delta_scan_backward, d, 19, ctypes.c_size_t(need if ws is None else ws), **over)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), SHAPE), (dict(nheads=0), SHAPE), (dict(headdim=0), SHAPE), (dict(dstate=0), SHAPE),
    (dict(ngroups=0), SHAPE), (dict(ngroups=3), SHAPE), (dict(io=2), DTYPE), (dict(io=-1), DTYPE),
    (dict(lo=NAN), INVALID), (dict(lo=1.0, hi=0.5), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID),
    (dict(headdim=12), UNSUP), (dict(headdim=264), UNSUP), (dict(dstate=136), UNSUP), (dict(dstate=20), UNSUP),
    (dict(strides=(47, 48, 64)), SHAPE), (dict(strides=(48, 47, 64)), SHAPE), (dict(strides=(48, 48, 63)), SHAPE),
    (dict(strides=(1 << 25, 48, 64)), UNSUP), (dict(strides=(48, 1 << 40, 64)), UNSUP),
    (dict(strides=(48, 48, 1 << 25)), UNSUP), (dict(batch=1 << 40), UNSUP),
    (dict(batch=(1 << 62), nheads=2, ngroups=1), UNSUP)])
def test_descriptors(kw, code):
    d = desc(**kw)
    assert scan(d, 1 << 50) == code and step(d) == code and back(d, 1 << 50) == code
    assert lib.ssd_delta_scan_workspace_bytes(ctypes.byref(d)) == 0
    assert lib.ssd_delta_scan_backward_workspace_bytes(ctypes.byref(d)) == 0


def test_lengths_and_gradient_strides():
    assert scan(desc(seqlen=-1), 1 << 50) == SHAPE and back(desc(seqlen=-1), 1 << 50) == SHAPE
    assert scan(desc(seqlen=1 << 32), 1 << 50) == UNSUP          # 2^26 chunks of 8 rows
    assert back(desc(seqlen=1 << 24), 1 << 62) == UNSUP          # 2^27 rows of the keys' gradients
    for g in ((47, 48, 64), (48, 47, 64), (48, 48, 63)):
        assert back(desc(grads=g)) == SHAPE
    assert scan(None) == INVALID and step(None) == INVALID and back(None) == INVALID


def test_scan_arguments():
    d = desc()
    for p in ("p0", "p1", "p2", "p3", "p5", "p6", "p8"):
        assert scan(d, **{p: 0}) == INVALID, p
    for p in ("p0", "p1", "p2", "p7", "p8", "p9"):
        assert scan(d, **{p: addr(int(p[1:]) + 1) + 8}) == ALIGN, p
    for p in ("p3", "p4", "p5", "p6"):
        assert scan(d, **{p: addr(int(p[1:]) + 1) + 2}) == ALIGN, p
    assert scan(d, p10=addr(11) + 16) == ALIGN
    assert scan(desc(strides=(52, 48, 64))) == ALIGN and scan(desc(strides=(48, 48, 68))) == ALIGN
    assert scan(d, p10=0) == WS
    assert scan(d, ws=lib.ssd_delta_scan_workspace_bytes(ctypes.byref(d)) - 1) == WS
    assert scan(d, p8=addr(3)) == INVALID                        # y over v
    assert scan(d, p9=addr(9)) == INVALID                        # two outputs
    assert scan(d, p9=addr(8) + 16) == INVALID                   # final state shifted into the initial
    assert scan(d, p10=addr(1)) == INVALID                       # workspace over q
    none = dict.fromkeys((f"p{i}" for i in range(11)), 0)
    assert scan(desc(batch=0), **none) == OK and scan(desc(seqlen=0), **none) == OK
    assert scan(desc(seqlen=0), **dict(none, p7=addr(8), p9=addr(8))) == OK      # in place


def test_step_arguments():
    d = desc(seqlen=0)
    for p in ("p0", "p1", "p2", "p3", "p4", "p6", "p7", "p8"):
        assert step(d, **{p: 0}) == INVALID, p
    for p in ("p0", "p1", "p2", "p3", "p8"):
        assert step(d, **{p: addr(int(p[1:]) + 1) + 8}) == ALIGN, p
    assert step(d, p4=addr(5) + 1) == ALIGN and step(d, p7=addr(8) + 2) == ALIGN
    assert step(d, p8=addr(1)) == INVALID and step(d, p0=addr(4)) == INVALID and step(d, p8=addr(4)) == INVALID
    assert step(desc(batch=0), **dict.fromkeys((f"p{i}" for i in range(9)), 0)) == OK


def test_gradient_arguments():
    d = desc()
    for i in (0, 1, 2, 3, 5, 6, 8, 10, 11, 12, 13, 14, 15):
        assert back(d, **{f"p{i}": 0}) == INVALID, i
    for i in (0, 1, 2, 7, 8, 9, 10, 11, 12, 17):
        assert back(d, **{f"p{i}": addr(i + 1) + 8}) == ALIGN, i
    for i in (3, 4, 5, 6, 13, 14, 15, 16):
        assert back(d, **{f"p{i}": addr(i + 1) + 2}) == ALIGN, i
    assert back(d, p18=0) == WS and back(d, p18=addr(19) + 128) == ALIGN
    assert back(d, ws=lib.ssd_delta_scan_backward_workspace_bytes(ctypes.byref(d)) - 1) == WS
    assert back(desc(grads=(52, 48, 64))) == ALIGN
    # an output over an input, over another output, into the workspace
    assert back(d, p10=addr(1)) == INVALID and back(d, p12=addr(9)) == INVALID
    assert back(d, p11=addr(11)) == INVALID and back(d, p13=addr(12)) == INVALID
    assert back(d, p14=addr(14)) == INVALID and back(d, p17=addr(10)) == INVALID
    assert back(d, p12=addr(19)) == INVALID
    # columns of one tensor: apart, overlapping, with other strides
    one = dict(grads=(160, 160, 160))
    at = lambda k: addr(11) + 2 * k              # noqa: E731
    bad = desc(**one)
    assert back(bad, p10=at(0), p11=at(40), p12=at(96)) == INVALID      # dk inside dq
    assert back(bad, p10=at(0), p11=at(48), p12=at(104)) == INVALID     # dv past the row's end
    assert back(desc(grads=(160, 160, 168)), p10=at(0), p11=at(48), p12=at(96)) == INVALID
    none = dict.fromkeys((f"p{i}" for i in range(19)), 0)
    assert back(desc(seqlen=0), **none) == INVALID               # dA is always written


def tensors(Bt=2, T=5, H=4, G=2, P=16, N=24, dtype=torch.bfloat16, lead=None):
    lead = (Bt, T) if lead is None else lead
    m = lambda *s, **k: Described(*s, **k)       # noqa: E731
    return dict(q=m(*lead, G, N, dtype=dtype), k=m(*lead, G, N, dtype=dtype), v=m(*lead, H, P, dtype=dtype),
                dt=m(*lead, H), A=m(H), beta=m(*lead, H))


def run(t, **kw):
    return ssd.ssd_delta_scan(t["q"], t["k"], t["v"], t["dt"], t["A"], t["beta"], **kw)


@pytest.mark.parametrize("name,shape,kind", [
    ("q", (2, 5, 2, 16), ValueError), ("k", (2, 4, 2, 24), ValueError), ("dt", (2, 5, 2), ValueError),
    ("beta", (2, 5), ValueError), ("A", (2,), ValueError), ("v", (2, 5, 64), ValueError),
    ("q", (2, 5, 48), ValueError)])
def test_shapes(name, shape, kind):
    t = tensors()
    t[name] = Described(*shape, dtype=t[name].dtype)
    with pytest.raises(kind):
        run(t)
    with pytest.raises(kind):
        ssd.ssd_delta_scan_backward(*(t[n] for n in ("q", "k", "v", "dt", "A", "beta")),
                                    dy=Described(2, 5, 4, 16, dtype=torch.bfloat16))


def test_types_devices_and_layouts():
    for name, other in (("q", torch.float32), ("k", torch.float16), ("v", torch.float16), ("dt", torch.bfloat16),
                        ("beta", torch.float64), ("A", torch.bfloat16)):
        t = tensors()
        t[name] = Described(*t[name].shape, dtype=other)
        with pytest.raises(TypeError):
            run(t)
    t = tensors()
    for name in t:
        with pytest.raises(ValueError, match="device tensor|must be on"):
            run({**t, name: torch.zeros(t[name].shape, dtype=t[name].dtype)})
        with pytest.raises(ValueError, match="must be on|device"):
            run({**t, name: Described(*t[name].shape, dtype=t[name].dtype, device="cuda:1")})
    s = lambda *st: Described(2, 5, 2, 24, strides=st, dtype=torch.bfloat16)     # noqa: E731
    for bad in (s(240, 48, 24, 2), s(240, 48, 32, 1), s(300, 48, 24, 1), s(240, 24, 24, 1), s(0, 48, 24, 1)):
        with pytest.raises(ValueError, match="dense heads and evenly spaced"):
            run({**t, "q": bad})
        with pytest.raises(ValueError, match="dense heads and evenly spaced"):
            ssd.ssd_delta_scan_backward(*(t[n] for n in ("q", "k", "v", "dt", "A", "beta")),
                                        dy=Described(2, 5, 4, 16, dtype=torch.bfloat16), grads={"dk": bad})
    with pytest.raises(ValueError):
        run(t, initial_state=Described(2, 4, 24, 16))
    with pytest.raises(TypeError):
        run(t, initial_state=Described(2, 4, 16, 24, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        run(t, y=Described(2, 5, 4, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="unknown gradient"):
        ssd.ssd_delta_scan_backward(*(t[n] for n in ("q", "k", "v", "dt", "A", "beta")),
                                    dy=Described(2, 5, 4, 16, dtype=torch.bfloat16), grads={"dx": None})
    with pytest.raises(TypeError):
        ssd.ssd_delta_scan_backward(*(t[n] for n in ("q", "k", "v", "dt", "A", "beta")), dy=Described(2, 5, 4, 16))
    o = tensors(lead=(2,))
    with pytest.raises(ValueError):
        ssd.ssd_delta_step(Described(2, 4, 24, 16), o["q"], o["k"], o["v"], o["dt"], o["A"], o["beta"])
    with pytest.raises(TypeError):
        ssd.ssd_delta_step(Described(2, 4, 16, 24, dtype=torch.bfloat16), o["q"], o["k"], o["v"], o["dt"], o["A"],
                           o["beta"])


def drop_desc(rows=5, cols=100, io=1, scale=1.0, eps=1e-5, p=0.1):
    return DropoutAddNormDesc(rows, cols, io, scale, eps, p)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(io=2), DTYPE), (dict(eps=-1.0), INVALID),
    (dict(scale=INF), INVALID), (dict(cols=16385), UNSUP), (dict(rows=1 << 31), UNSUP), (dict(p=-0.1), INVALID),
    (dict(p=1.0), INVALID), (dict(p=NAN), INVALID), (dict(p=INF), INVALID)])
def test_dropout_descriptors(kw, code):
    d = drop_desc(**kw)
    assert call(lib.ssd_dropout_add_norm, d, 6) == code
    assert call(lib.ssd_dropout_add_norm_backward, d, 9, ctypes.c_size_t(1 << 40)) == code
    assert lib.ssd_dropout_add_norm_backward_workspace_bytes(ctypes.byref(d)) == 0
    assert call(lib.ssd_dropout_add_norm, None, 6) == INVALID


def test_dropout_arguments():
    d = drop_desc()
    f = lambda **o: call(lib.ssd_dropout_add_norm, d, 6, **o)    # x, residual, weight, rng, y, residual_out
    for p in ("p0", "p2", "p3", "p4"):
        assert f(**{p: 0}) == INVALID
    assert f(p3=addr(4) + 4) == ALIGN and f(p0=addr(1) + 1) == ALIGN
    assert f(p4=addr(1)) == INVALID and f(p5=addr(2) + 4) == INVALID and f(p5=addr(4)) == INVALID
    assert call(lib.ssd_dropout_add_norm, drop_desc(scale=3e38, p=0.5), 6) == INVALID   # 6e38 is no float
    need = lib.ssd_dropout_add_norm_backward_workspace_bytes(ctypes.byref(d))
    # residual_out, weight, dy, dresidual_out, rng, dx, dresidual, dweight, workspace
    h = lambda w=need, **o: call(lib.ssd_dropout_add_norm_backward, d, 9, ctypes.c_size_t(w), **o)   # noqa: E731
    for p in ("p0", "p1", "p2", "p4", "p7"):
        assert h(**{p: 0}) == INVALID
    assert h(p8=0) == WS and h(w=need - 1) == WS and h(p4=addr(5) + 4) == ALIGN
    assert h(p5=addr(3)) == INVALID and h(p6=addr(4) + 4) == INVALID and h(p7=addr(5)) == INVALID
    assert lib.ssd_dropout_add_norm(ctypes.byref(drop_desc(rows=0)), *[None] * 6, None) == OK


def test_dropout_tensors():
    x, w, rng = Described(4, 128), Described(128), Described(2, dtype=torch.int64)
    for bad in (Described(3, dtype=torch.int64), Described(1, 2, dtype=torch.int64)):
        with pytest.raises(ValueError):
            ssd.ssd_dropout_add_norm(x, w, p=0.1, rng=bad)
    with pytest.raises(TypeError):
        ssd.ssd_dropout_add_norm(x, w, p=0.1, rng=Described(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        ssd.ssd_dropout_add_norm(x, w, p=0.1, rng=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        ssd.ssd_dropout_add_norm(x, w, p=0.1, rng=None)
    with pytest.raises(ValueError):
        ssd.ssd_dropout_add_norm_backward(x, w, dy=Described(4, 127), p=0.1, rng=rng)
    with pytest.raises(ValueError):
        ssd.ssd_dropout_add_norm(x, w, p=0.1, rng=Described(2, dtype=torch.int64, device="cuda:1"))
