"""Gradients of the gated delta rule on the GPU, element by element within bars from the terms that
each is a sum of (delta_magnitudes), over every kind of chain."""
import math

import pytest
import torch

import delta_magnitudes as dm
from delta_cases import close, make, on_device
from gpu_util import announce, need_gpu
from test_gpu_delta import args, options
from test_gpu_delta_gradients import cotangents

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16

# The gradients' chains in bfloat16: every group of 16 value columns alone, in pairs of them (a pair's
# second group may lie past the last column: 40 and 72 values), columns owned
ALONE = [(1, 1, 1, 1, 8, 8), (2, 63, 2, 1, 16, 16), (1, 65, 3, 3, 64, 128), (2, 130, 4, 2, 128, 64),
         (1, 140, 4, 1, 24, 72), (3, 129, 2, 2, 40, 40), (2, 17, 5, 5, 136, 120)]
PAIRS = [(3, 70, 16, 4, 40, 72), (2, 130, 20, 20, 64, 128), (2, 66, 20, 5, 72, 40), (2, 129, 16, 8, 128, 64),
         (1, 200, 64, 16, 40, 128)]
OWNED = [(3, 130, 40, 8, 48, 128), (9, 70, 16, 2, 72, 104), (5, 65, 60, 20, 16, 64), (5, 67, 16, 16, 56, 40)]
SHAPES = ALONE + PAIRS + OWNED


def hard(kind, T, io, N=40, seed=51):
    """Everything forgotten, nothing written, A of none to many."""
    Bt, H, G, P = kind
    x, u = make(seed, Bt, T, H, G, P, N, io=io, bias=False)
    x["A"] = torch.tensor([-1.0, -16.0, -1e-3, -0.25]).repeat(H // 4)
    x["dt"][:, 3::7] = 40.0
    x["dt"][:, 4::7] = -60.0
    x["beta"][:, ::5] = 30.0
    x["beta"][:, 1::5] = -120.0
    return (x, u, *cotangents(4, x))


def raw(io):
    """Logarithms of decays and write strengths as they are, keys and queries of any length."""
    x, u = make(7, 2, 100, 2, 1, 32, 48, io=io, bias=False, spread=0.3)
    x["dt"], x["beta"], x["A"] = -x["dt"].abs(), torch.sigmoid(x["beta"]), torch.ones(2)
    lim = (-math.inf, math.inf)
    return (x, u, *cotangents(1, x), dict(softplus=False, limit=lim, sigmoid=False, norm=False, scale=0.3),
            dict(dt_softplus=False, dt_limit=lim, beta_sigmoid=False, qk_norm=False, scale=0.3))


def check(got, x, dy, dfinal, **opts):
    grads, terms = dm.reference(x, dy, dfinal, **opts)
    bars = dm.bars(x, grads, terms)
    assert set(got) == set(bars)
    for n, bar in bars.items():
        close(got[n], grads[n], bar.numpy(), n)


def run(x, u, dy, dfinal, **kw):
    import state_space_model_amd as ssd
    d = on_device(x, u)
    return ssd.ssd_delta_scan_backward(*args(d), **options(d), dy=dy.cuda(),
                                       dfinal_state=None if dfinal is None else dfinal.cuda(), **kw)


@pytest.mark.parametrize("io", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients(shape, io):
    need_gpu()
    announce(f"delta gradients' terms {shape} {io}")
    T = shape[1]
    x, u = make(T + 1, *shape, io=io, h0=T % 2 == 0, bias=T % 3 != 0)
    dy, dfinal = cotangents(T, x, T % 4 != 1)
    check(run(x, u, dy, dfinal), x, dy, dfinal)


@pytest.mark.parametrize("io,kind", [(F32, (2, 4, 2, 16)), (BF16, (2, 4, 2, 16)), (BF16, (3, 16, 4, 40)),
                                     (BF16, (3, 32, 8, 64))], ids=str)
def test_hard_gates(io, kind):
    need_gpu()
    announce(f"delta gradients' terms, hard gates {kind} {io}")
    x, u, dy, dfinal = hard(kind, 70, io)
    check(run(x, u, dy, dfinal), x, dy, dfinal)


@pytest.mark.parametrize("io", [F32, BF16], ids=["f32", "bf16"])
def test_options(io):
    need_gpu()
    announce(f"delta gradients' terms, options {io}")
    x, u, dy, dfinal, opts, kw = raw(io)
    check(run(x, u, dy, dfinal, **kw), x, dy, dfinal, **opts)
    T = 100
    x, u = make(T + 1, 2, T, 2, 1, 32, 48, io=io, h0=T % 2 == 0, bias=T % 3 != 0)
    dy, dfinal = cotangents(T, x, T % 4 != 1)
    check(run(x, u, dy, dfinal, dt_limit=(0.4, 0.7), norm_eps=0.5), x, dy, dfinal, limit=(0.4, 0.7), eps=0.5)
