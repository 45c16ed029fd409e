"""Gradients of the gated delta rule's scan on the GPU against automatic
derivatives of its float64 definition (oracle.delta) and against differences."""
import math

import pytest
import torch

from delta_cases import close, grad_bars, make, on_device
from gpu_util import announce, need_gpu
from oracle import delta
from test_gpu_delta import args, options

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
NAMES = {"dinitial_state": "dh0"}

SHAPES = [(1, 1, 1, 1, 8, 8), (2, 63, 2, 1, 16, 16), (1, 64, 2, 2, 64, 128), (1, 65, 3, 3, 64, 128),
          (2, 130, 4, 2, 128, 64), (1, 140, 4, 1, 24, 72), (3, 129, 2, 2, 40, 40),
          (1, 70, 2, 2, 256, 128), (2, 17, 5, 5, 136, 120), (1, 80, 2, 2, 72, 104),
          (4, 66, 16, 4, 72, 40), (3, 130, 40, 8, 48, 128),             # chains in pairs
          (9, 70, 16, 2, 72, 104), (5, 65, 60, 20, 16, 64), (2, 129, 70, 70, 128, 128)]  # chains that own columns


def cotangents(seed, x, final=True):
    g = torch.Generator().manual_seed(seed)
    Bt, T, H, P = x["v"].shape
    N = x["q"].shape[-1]
    dy = torch.randn(Bt, T, H, P, generator=g).to(x["v"].dtype)
    return dy, torch.randn(Bt, H, P, N, generator=g) / math.sqrt(N) if final else None


def reference(x, dy, dfinal, **opts):
    limit = opts.get("limit", (0.0, math.inf))
    f = {n: delta.f64(t) for n, t in x.items()}
    ref, states, dstates = delta.gradients(f, delta.f64(dy), delta.f64(dfinal), **opts)
    ref["rates"] = delta.rates(f["dt"], f["dt_bias"], opts.get("softplus", True), limit)
    if "ddt_bias" not in ref:
        ref["ddt_bias"] = ref["ddt"].sum((0, 1))
    if "dh0" not in ref:   # without an initial state: that of zeros
        f["h0"] = torch.zeros_like(states[-1])
        ref["dh0"] = delta.gradients(f, delta.f64(dy), delta.f64(dfinal), **opts)[0]["dh0"]
    return ref, states, dstates


def check(got, x, dy, ref, states, dstates, scale=None, norm=True):
    N = x["q"].shape[-1]
    bars = grad_bars(x, dy, ref, states, dstates, 1 / math.sqrt(N) if scale is None else scale, norm)
    assert set(got) == set(bars)
    for n, bar in bars.items():
        io = x["v"].dtype if n in ("dq", "dk", "dv") else F32
        assert got[n].dtype == io, n
        close(got[n], ref[NAMES.get(n, n)], bar, n)


@pytest.mark.parametrize("io", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients(shape, io):
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta_scan_backward {shape} {io}")
    T = shape[1]
    x, u = make(T + 1, *shape, io=io, h0=T % 2 == 0, bias=T % 3 != 0, pad=8 * (T % 4))
    dy, dfinal = cotangents(T, x, T % 4 != 1)
    d = on_device(x, u)
    got = ssd.ssd_delta_scan_backward(*args(d), **options(d), dy=dy.cuda(),
                                      dfinal_state=None if dfinal is None else dfinal.cuda())
    check(got, x, dy, *reference(x, dy, dfinal))


@pytest.mark.parametrize("io", [F32, BF16], ids=["f32", "bf16"])
def test_options(io):
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta gradients, options {io}")
    shape = (2, 100, 2, 1, 32, 48)
    x, u = make(7, *shape, io=io, bias=False, spread=0.3)
    x["dt"], x["beta"], x["A"] = -x["dt"].abs(), torch.sigmoid(x["beta"]), torch.ones(2)
    dy, dfinal = cotangents(1, x)
    lim = (-math.inf, math.inf)
    d = on_device(x, u)
    got = ssd.ssd_delta_scan_backward(*args(d), initial_state=d["h0"], dy=dy.cuda(), dfinal_state=dfinal.cuda(),
                                      dt_softplus=False, dt_limit=lim, beta_sigmoid=False, qk_norm=False, scale=0.3)
    ref = reference(x, dy, dfinal, softplus=False, limit=lim, sigmoid=False, norm=False, scale=0.3)
    check(got, x, dy, *ref, scale=0.3, norm=False)
    x, u = make(8, *shape, io=io)
    d = on_device(x, u)
    got = ssd.ssd_delta_scan_backward(*args(d), **options(d), dy=dy.cuda(), dfinal_state=dfinal.cuda(),
                                      dt_limit=(0.4, 0.7), norm_eps=0.5)
    check(got, x, dy, *reference(x, dy, dfinal, limit=(0.4, 0.7), eps=0.5))
    clipped = (delta.rates(x["dt"], x["dt_bias"], limit=(0.4, 0.7)) == 0.4)
    assert clipped.any() and not got["ddt"].cpu()[clipped].any()


def test_hard_gates_and_padding():
    """Everything forgotten, nothing written, and tokens that change nothing at the ends of rows."""
    need_gpu()
    import state_space_model_amd as ssd
    announce("delta gradients, hard gates")
    shape = (2, 190, 4, 2, 16, 32)
    x, u = make(9, *shape, bias=False)
    x["A"] = torch.tensor([-1.0, -16.0, -1e-3, 0.0])
    x["dt"][:, 3::7] = 40.0
    x["dt"][:, 4::7] = -60.0
    x["beta"][:, ::5] = 30.0
    x["beta"][:, 1::5] = -120.0
    x["dt"][1, 77:] = x["beta"][1, 77:] = -math.inf
    dy, dfinal = cotangents(2, x)
    d = on_device(x, u)
    got = ssd.ssd_delta_scan_backward(*args(d), **options(d), dy=dy.cuda(), dfinal_state=dfinal.cuda())
    f = {n: t if t is None else t.clone() for n, t in x.items()}
    f["dt"][1, 77:] = f["beta"][1, 77:] = -1e4   # the same gates, whose derivatives have no inf - inf
    check(got, x, dy, *reference(f, dy, dfinal))
    for n in ("ddt", "dbeta", "dk", "dv"):
        assert not got[n][1, 77:].any(), n


@pytest.mark.parametrize("name", ["q", "k", "v", "dt", "beta", "A", "dt_bias", "h0"])
def test_against_differences(name):
    """The directional derivative against a difference of the float64 definition along it: its
    truncation is below 1e-8 of the loss, the gradients' own error 1e-5 of the terms' lengths."""
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta gradients, differences {name}")
    x, u = make(30, 1, 70, 2, 1, 16, 24)
    dy, dfinal = cotangents(3, x)
    d = on_device(x, u)
    got = ssd.ssd_delta_scan_backward(*args(d), **options(d), dy=dy.cuda(), dfinal_state=dfinal.cuda())
    grad = got["dinitial_state" if name == "h0" else "d" + name].double().cpu()
    f = {n: delta.f64(t) for n, t in x.items()}
    way = torch.randn(grad.shape, generator=torch.Generator().manual_seed(4), dtype=torch.float64)

    def loss(step):
        y, states = delta.scan(**{**f, name: f[name] + step * way})
        return float((y * dy.double()).sum() + (states[-1] * dfinal.double()).sum())

    h = 1e-5
    slope = (loss(h) - loss(-h)) / (2 * h)
    assert abs(float((grad * way).sum()) - slope) <= 1e-5 * float(grad.norm() * way.norm())


def test_slices_of_one_gradient():
    """dq, dk and dv written into columns of one tensor, whose other columns stay; a workspace of the
    caller's with anything in it; the same bits again."""
    need_gpu()
    import state_space_model_amd as ssd
    announce("delta gradients, slices")
    shape = (2, 75, 4, 2, 24, 40)
    x, u = make(31, *shape, io=BF16)
    dy, dfinal = cotangents(5, x)
    d = on_device(x, u)
    kw = dict(**options(d), dy=dy.cuda(), dfinal_state=dfinal.cuda())
    want = ssd.ssd_delta_scan_backward(*args(d), **kw)
    du = torch.full((2, 75, u.shape[-1] + 16), 7.0, device="cuda", dtype=BF16)
    w = 2 * 40
    grads = {"dq": du[..., 8:8 + w].unflatten(-1, (2, 40)), "dk": du[..., 8 + w:8 + 2 * w].unflatten(-1, (2, 40)),
             "dv": du[..., 8 + 2 * w:-8].unflatten(-1, (4, 24))}
    ws = torch.full((1 << 26,), 255, device="cuda", dtype=torch.uint8)
    got = ssd.ssd_delta_scan_backward(*args(d), **kw, grads=grads, workspace=ws)
    for n, t in want.items():
        assert torch.equal(t, got[n]), n
    assert bool((du[..., :8] == 7).all()) and bool((du[..., -8:] == 7).all())


def test_nothing_to_do():
    need_gpu()
    import state_space_model_amd as ssd
    announce("delta gradients, empty")
    x, u = make(32, 2, 5, 2, 1, 16, 16)
    dy, dfinal = cotangents(6, x)
    d = on_device(x, u)
    cut = [t[:, :0].contiguous() if t.dim() > 1 else t for t in args(d)]
    got = ssd.ssd_delta_scan_backward(*cut, **options(d), dy=dy[:, :0].cuda(), dfinal_state=dfinal.cuda())
    assert torch.equal(got["dinitial_state"].cpu(), dfinal) and not got["dA"].any() and not got["ddt_bias"].any()
    assert not ssd.ssd_delta_scan_backward(*cut, dy=dy[:, :0].cuda())["dinitial_state"].any()


def test_graph():
    """Captured after eager calls on the same tensors, replayed on other inputs with eager calls between."""
    need_gpu()
    import state_space_model_amd as ssd
    announce("delta gradients, graph")
    shape = (1, 100, 4, 2, 64, 128)
    sets = []
    for i in range(3):
        x, u = make(40 + i, *shape, io=BF16)
        dy, dfinal = cotangents(i, x)
        sets.append(dict(on_device(x, u), dy=dy.cuda(), dfinal=dfinal.cuda()))
    run = lambda d: ssd.ssd_delta_scan_backward(  # noqa: E731
        *args(d), **options(d), dy=d["dy"], dfinal_state=d["dfinal"])
    want = [run(d) for d in sets]
    live = {n: t.clone() for n, t in sets[0].items()}
    run(live)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(live)
    for i in (1, 2, 0, 1):
        for n, t in live.items():
            t.copy_(sets[i][n])
        graph.replay()
        torch.cuda.synchronize()
        again = run(sets[i])
        for n, t in got.items():
            assert torch.equal(t, want[i][n]) and torch.equal(again[n], t), (i, n)
