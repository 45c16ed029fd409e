"""The gradients' chains of the gated delta rule that share their value columns in pairs (bfloat16; the
scans of the same sizes run in pairs or alone): hard gates, padding, values that are not finite, two
calls at once and replays."""
import math

import pytest
import torch

import test_gpu_delta_chains as chains
from delta_cases import make, on_device
from gpu_util import announce, need_gpu
from test_gpu_delta import args, options
from test_gpu_delta_gradients import cotangents

pytestmark = pytest.mark.gpu
# rows, heads, groups, values: 192 pairs, the second of each head half past the last column; 240 whole ones
KINDS = [(3, 16, 4, 40), (3, 20, 5, 64)]


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_hard_gates(kind):
    chains.test_hard_gates(kind)


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_padding(kind):
    chains.test_padding(kind)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_bad_values_stay_in_their_sequence(kind, bad):
    chains.test_bad_values_stay_in_their_sequence(kind, bad)


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_two_at_once_and_replays(kind):
    chains.test_two_at_once_and_replays(kind)


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_gradients_of_padding(kind):
    """Padded tokens, dirty gradient buffers and workspace: the bits of the shorter sequence, zeros after it."""
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta pairs, gradients of padding {kind}")
    Bt, H, G, P = kind
    x, u = make(54, Bt, 192, H, G, P, 40, io=torch.bfloat16)
    x["dt"][:, 100:] = x["beta"][:, 100:] = -math.inf
    dy, dfinal = cotangents(9, x)
    dy[:, 100:] = 0
    d = on_device(x, u)
    kw = dict(**options(d), dfinal_state=dfinal.cuda())
    want = ssd.ssd_delta_scan_backward(*[t[:, :100].contiguous() if t.dim() > 1 else t for t in args(d)],
                                       dy=dy[:, :100].contiguous().cuda(), **kw)
    got = ssd.ssd_delta_scan_backward(*args(d), dy=dy.cuda(), **kw)
    for n in ("dq", "dk", "dv", "ddt", "dbeta"):
        assert torch.equal(got[n][:, :100], want[n]) and not got[n][:, 100:].any(), n
    for n in ("dA", "ddt_bias", "dinitial_state"):
        assert torch.equal(got[n], want[n]), n
    dirty = {n: torch.full_like(t, math.nan) for n, t in got.items()}
    ws = torch.full((1 << 28,), 255, device="cuda", dtype=torch.uint8)
    again = ssd.ssd_delta_scan_backward(*args(d), dy=dy.cuda(), **kw, grads=dirty, workspace=ws)
    assert all(torch.equal(again[n], got[n]) for n in got)
