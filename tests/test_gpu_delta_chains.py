"""The gated delta rule's kinds of chain in bfloat16 (columns shared by four wavefronts, shared in
pairs, owned): hard gates, padding, values that are not finite, two calls at once and replays."""
import math

import pytest
import torch

from delta_cases import close, make, on_device, oracle_of, state_bar, y_bar
from gpu_util import announce, need_gpu
from test_gpu_delta import args, options
from test_gpu_delta_gradients import check, cotangents, reference

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
# rows, heads, groups, values: 8 chains alone, 192 in pairs (the gradients' owned), 320 owned
KINDS = [(2, 4, 2, 16), (3, 32, 8, 64), (5, 32, 8, 64)]
N = 40


def hard(kind, T, seed):
    Bt, H, G, P = kind
    x, u = make(seed, Bt, T, H, G, P, N, io=BF16, bias=False)
    x["A"] = torch.tensor([-1.0, -16.0, -1e-3, 0.0]).repeat(H // 4)
    x["dt"][:, 3::7] = 40.0
    x["dt"][:, 4::7] = -60.0
    x["beta"][:, ::5] = 30.0
    x["beta"][:, 1::5] = -120.0
    return x, u


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_hard_gates(kind):
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta chains, hard gates {kind}")
    T = 135
    x, u = hard(kind, T, 50)
    d = on_device(x, u)
    y, final = ssd.ssd_delta_scan(*args(d), **options(d))
    want, states = oracle_of(x)
    close(final, states[-1], state_bar(states, T, N), "final state")
    close(y, want, y_bar(want, states, T, N, BF16, 1 / math.sqrt(N)), "y")


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_hard_gates_gradients(kind):
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta chains, hard gates' gradients {kind}")
    x, u = hard(kind, 70, 51)
    dy, dfinal = cotangents(4, x)
    d = on_device(x, u)
    got = ssd.ssd_delta_scan_backward(*args(d), **options(d), dy=dy.cuda(), dfinal_state=dfinal.cuda())
    check(got, x, dy, *reference(x, dy, dfinal))


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_padding(kind):
    """Padded tokens change no bit of the state: the same as the shorter sequence's."""
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta chains, padding {kind}")
    Bt, H, G, P = kind
    x, u = make(52, Bt, 192, H, G, P, N, io=BF16)
    x["dt"][:, 100:] = x["beta"][:, 100:] = -math.inf
    d = on_device(x, u)
    _, final = ssd.ssd_delta_scan(*args(d), **options(d))
    cut = [t[:, :100].contiguous() if t.dim() > 1 else t for t in args(d)]
    _, short = ssd.ssd_delta_scan(*cut, **options(d))
    assert torch.equal(final, short)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_bad_values_stay_in_their_sequence(kind, bad):
    """In the last token of a ragged chunk, of one row's last group's keys: the heads of that group
    and row, in that chunk."""
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta chains, {bad} {kind}")
    Bt, H, G, P = kind
    x, u = make(53, Bt, 130, H, G, P, N, io=BF16)
    dy, dfinal = cotangents(7, x)
    clean = on_device(x, u)
    kw = dict(dy=dy.cuda(), dfinal_state=dfinal.cuda())
    want, wfinal = ssd.ssd_delta_scan(*args(clean), **options(clean))
    wgrad = ssd.ssd_delta_scan_backward(*args(clean), **options(clean), **kw)
    u[1, 129, 2 * G * N - 3] = bad
    d = on_device(x, u)
    y, final = ssd.ssd_delta_scan(*args(d), **options(d))
    grad = ssd.ssd_delta_scan_backward(*args(d), **options(d), **kw)
    per = H // G
    assert not y[1, 129, H - per:].isfinite().all()
    for got, ref in ((y, want), (final, wfinal), *((grad[n], wgrad[n]) for n in ("dv", "ddt", "dbeta", "dinitial_state"))):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[2:], ref[2:])
    assert torch.equal(y[1, :, :H - per], want[1, :, :H - per]) and torch.equal(y[1, :128], want[1, :128])
    assert torch.equal(final[1, :H - per], wfinal[1, :H - per])
    for n in ("dv", "ddt", "dbeta"):
        assert torch.equal(grad[n][1, :, :H - per], wgrad[n][1, :, :H - per]), n
    for n in ("dq", "dk"):
        assert torch.equal(grad[n][0], wgrad[n][0]) and torch.equal(grad[n][1, :, :G - 1], wgrad[n][1, :, :G - 1]), n


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_two_at_once_and_replays(kind):
    """Scans and gradients of two inputs on two streams, and both in graphs, replayed in turn with
    eager calls between."""
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta chains, two at once {kind}")
    Bt, H, G, P = kind
    sets = []
    for i in range(2):
        x, u = make(60 + i, Bt, 150, H, G, P, N, io=BF16)
        dy, dfinal = cotangents(i, x)
        sets.append(dict(on_device(x, u), dy=dy.cuda(), dfinal=dfinal.cuda()))

    def run(d):
        y, final = ssd.ssd_delta_scan(*args(d), **options(d))
        g = ssd.ssd_delta_scan_backward(*args(d), **options(d), dy=d["dy"], dfinal_state=d["dfinal"])
        return [y, final] + [g[n] for n in sorted(g)]

    want = [run(d) for d in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = []
        for s, d in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(run(d))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    graphs = [torch.cuda.CUDAGraph() for _ in sets]
    outs = []
    for g, d in zip(graphs, sets):
        with torch.cuda.graph(g):
            outs.append(run(d))
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
        torch.cuda.synchronize()
        again = run(sets[1 - i])
        assert all(torch.equal(p, q) for p, q in zip(outs[i], want[i]))
        assert all(torch.equal(p, q) for p, q in zip(again, want[1 - i]))
