"""What is not finite among the gated delta rule's gates and values: a NaN reaches everything that
depends on it and nothing else; infinite gates are gates like large ones."""
import math

import pytest
import torch

from delta_cases import make, on_device
from gpu_util import announce, need_gpu
from test_gpu_delta import args, options
from test_gpu_delta_gradients import cotangents

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
# type, rows, heads, groups, values: float32; bfloat16 chains alone, in pairs, columns owned
KINDS = [(F32, 3, 4, 2, 16), (BF16, 3, 4, 2, 16), (BF16, 3, 32, 8, 64), (BF16, 5, 32, 8, 64)]
N, T = 40, 150
ROW, TOKEN, HEAD, COL = 1, 70, 3, 5
# with softplus and the default limits; the logarithm of the decay
MODES = {"rates": {}, "logs": dict(dt_softplus=False, dt_limit=(-math.inf, math.inf))}
WHERE = [(name, mode) for name in ("dt", "beta", "v") for mode in MODES] + [("dt_bias", "rates")]


def planted(kind, name, mode):
    io, Bt, H, G, P = kind
    x, u = make(80, Bt, T, H, G, P, N, io=io, bias=mode == "rates")
    if mode == "logs":
        x["A"], x["dt"] = torch.ones(H), -x["dt"].abs()
    clean = on_device(x, u)
    if name == "v":
        x["v"][ROW, TOKEN, HEAD, COL] = math.nan
    elif name == "dt_bias":
        x["dt_bias"][HEAD] = math.nan
    else:
        x[name][ROW, TOKEN, HEAD] = math.nan
    return x, clean, on_device(x, u)


def others(t, name):
    """All of t [Bt, T, H, ..] or [Bt, H, ..] that the NaN must not reach."""
    heads = [h for h in range(t.shape[2 if t.shape[1] == T else 1]) if h != HEAD]
    own = t[:, :, heads] if t.shape[1] == T else t[:, heads]
    rows = [b for b in range(t.shape[0]) if b != ROW]
    return [own] if name == "dt_bias" else [own, t[rows]]


@pytest.mark.parametrize("name,mode", WHERE)
@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_nan_reaches_what_depends_on_it(kind, name, mode):
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta NaN in {name} {kind} {mode}")
    io, Bt, H, G, P = kind
    x, clean, d = planted(kind, name, mode)
    kw = MODES[mode]
    want, wfinal = ssd.ssd_delta_scan(*args(clean), **options(clean), **kw)
    y, final = ssd.ssd_delta_scan(*args(d), **options(d), **kw)
    rows = slice(None) if name == "dt_bias" else slice(ROW, ROW + 1)
    first = 0 if name == "dt_bias" else TOKEN
    cols = slice(COL, COL + 1) if name == "v" else slice(None)
    assert y[rows, first:, HEAD, cols].isnan().all() and final[rows, HEAD, cols].isnan().all()
    for got, ref in ((y, want), (final, wfinal)):
        for g, r in zip(others(got, name), others(ref, name)):
            assert torch.equal(g, r)
    if name == "v":   # the head's other columns
        keep = [p for p in range(P) if p != COL]
        assert torch.equal(y[..., keep], want[..., keep]) and torch.equal(final[:, :, keep], wfinal[:, :, keep])
    assert torch.equal(y[:, :64][rows], want[:, :64][rows]) or name == "dt_bias"

    dy, dfinal = cotangents(7, x)
    kw = dict(kw, dy=dy.cuda(), dfinal_state=dfinal.cuda())
    ref = ssd.ssd_delta_scan_backward(*args(clean), **options(clean), **kw)
    got = ssd.ssd_delta_scan_backward(*args(d), **options(d), **kw)
    # of a value: its write strength, and the decays that its write meets; of a gate: its own
    # gradient and the head's
    assert got["dbeta"][rows, TOKEN, HEAD].isnan().all()
    assert got["ddt"][rows, TOKEN, HEAD].isnan().all() or name == "v"
    assert got["dA"][HEAD].isnan() and got["ddt_bias"][HEAD].isnan()
    keep = [h for h in range(H) if h != HEAD]
    assert torch.equal(got["dA"][keep], ref["dA"][keep]) and torch.equal(got["ddt_bias"][keep], ref["ddt_bias"][keep])
    for n in ("dv", "ddt", "dbeta", "dinitial_state"):
        for g, r in zip(others(got[n], name), others(ref[n], name)):
            assert torch.equal(g, r), n
    per = H // G
    groups = [g for g in range(G) if g != HEAD // per]
    for n in ("dq", "dk"):
        assert torch.equal(got[n][:, :, groups], ref[n][:, :, groups]), n


@pytest.mark.parametrize("name,mode", WHERE)
@pytest.mark.parametrize("io", [F32, BF16], ids=["f32", "bf16"])
def test_nan_in_a_step(io, name, mode):
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta step, NaN in {name} {io} {mode}")
    x, clean, d = planted((io, 3, 4, 2, 16), name, mode)
    out = []
    for t in (clean, d):
        state = t["h0"].clone()
        y = ssd.ssd_delta_step(state, t["q"][:, TOKEN], t["k"][:, TOKEN], t["v"][:, TOKEN],
                               t["dt"][:, TOKEN].contiguous(), t["A"], t["beta"][:, TOKEN].contiguous(),
                               dt_bias=t["dt_bias"], **MODES[mode])
        out.append((y, state))
    rows = slice(None) if name == "dt_bias" else slice(ROW, ROW + 1)
    cols = slice(COL, COL + 1) if name == "v" else slice(None)
    for got, ref in zip(out[1], out[0]):
        assert got[rows, HEAD, cols].isnan().all()
        hit = torch.zeros_like(got, dtype=torch.bool)
        hit[rows, HEAD, cols] = True
        assert torch.equal(got[~hit], ref[~hit])


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_infinite_gates_are_gates(kind, mode):
    """The bits of large finite gates: outputs, states, and every gradient, A's among them (the
    gradient of a decay that forgets everything is 0, however large the rate)."""
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta infinite gates {kind} {mode}")
    io, Bt, H, G, P = kind
    x, u = make(81, Bt, T, H, G, P, N, io=io, bias=mode == "rates")
    kw = MODES[mode]
    if mode == "logs":
        x["A"], x["dt"] = torch.ones(H), -x["dt"].abs()
    dy, dfinal = cotangents(8, x)
    out = []
    for rate, write in ((math.inf, math.inf), (1e30, 1e4)):
        x["dt"][:, 5::31] = -rate                  # keeps all; as a logarithm forgets all
        if mode == "rates":
            x["dt"][:, 11::37] = rate
            x["dt"][0, 100:] = -rate
        x["beta"][:, 3::17] = write
        x["beta"][:, 7::19] = -write
        d = on_device(x, u)
        y, final = ssd.ssd_delta_scan(*args(d), **options(d), **kw)
        grads = ssd.ssd_delta_scan_backward(*args(d), **options(d), **kw, dy=dy.cuda(), dfinal_state=dfinal.cuda())
        state = d["h0"].clone()
        t = 11 if mode == "rates" else 5
        step = ssd.ssd_delta_step(state, d["q"][:, t], d["k"][:, t], d["v"][:, t], d["dt"][:, t].contiguous(),
                                  d["A"], d["beta"][:, t].contiguous(), dt_bias=d["dt_bias"], **kw)
        out.append({"y": y, "final": final, "step": step, "state": state, **grads})
    for n in out[0]:
        assert out[0][n].isfinite().all(), n
        assert torch.equal(out[0][n], out[1][n]), n
