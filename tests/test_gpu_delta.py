"""The gated delta rule (scan and step) on the GPU against its float64
definition (oracle.delta), token by token."""
import math

import pytest
import torch

from delta_cases import close, make, on_device, oracle_of, state_bar, y_bar
from gpu_util import announce, need_gpu

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16

# Bt, T, H, G, P, N
SHAPES = [(1, 1, 1, 1, 8, 8), (2, 63, 2, 1, 16, 16), (1, 64, 2, 2, 64, 128), (1, 65, 3, 3, 64, 128),
          (2, 130, 4, 2, 128, 64), (1, 200, 2, 1, 24, 72), (3, 129, 6, 2, 40, 40),
          (1, 300, 2, 2, 256, 128), (2, 17, 5, 5, 136, 120), (1, 80, 2, 2, 72, 104),
          (4, 130, 16, 4, 72, 40), (3, 200, 40, 8, 48, 128),             # chains in pairs
          (9, 140, 16, 2, 72, 104), (5, 65, 60, 20, 16, 64), (2, 193, 70, 70, 128, 128)]  # chains that own columns


def options(x):
    return dict(dt_bias=x["dt_bias"], initial_state=x["h0"])


def args(x):
    return tuple(x[n] for n in ("q", "k", "v", "dt", "A", "beta"))


@pytest.mark.parametrize("io", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_scan(shape, io):
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta_scan {shape} {io}")
    Bt, T, H, G, P, N = shape
    x, u = make(T, *shape, io=io, h0=T % 2 == 0, bias=T % 3 != 0, pad=8 * (T % 4))
    d = on_device(x, u)
    y, final = ssd.ssd_delta_scan(*args(d), **options(d))
    want, states = oracle_of(x)
    assert y.dtype == io and final.dtype == F32
    close(final, states[-1], state_bar(states, T, N), "final state")
    close(y, want, y_bar(want, states, T, N, io, 1 / math.sqrt(N)), "y")


@pytest.mark.parametrize("io", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_step(shape, io):
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta_step {shape} {io}")
    Bt, T, H, G, P, N = shape
    T = min(T, 5)
    x, u = make(100 + P, Bt, T, H, G, P, N, io=io, pad=8)
    d = on_device(x, u)
    state = d["h0"].clone()
    want, states = oracle_of(x)
    for t in range(T):
        y = ssd.ssd_delta_step(state, d["q"][:, t], d["k"][:, t], d["v"][:, t],
                               d["dt"][:, t].contiguous(), d["A"], d["beta"][:, t].contiguous(),
                               dt_bias=d["dt_bias"])
        close(y, want[:, t], y_bar(want[:, t], states, T, N, io, 1 / math.sqrt(N)), f"y {t}")
    close(state, states[-1], state_bar(states, T, N), "state")


@pytest.mark.parametrize("io", [F32, BF16], ids=["f32", "bf16"])
def test_options(io):
    """Raw gates (the logarithm of the decay through A = 1), no normalisation, a scale, clipped rates."""
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta options {io}")
    shape = (2, 100, 2, 1, 32, 48)
    T, N = shape[1], shape[5]
    x, u = make(7, *shape, io=io, bias=False, spread=0.3)
    x["dt"], x["beta"], x["A"] = -x["dt"].abs(), torch.sigmoid(x["beta"]), torch.ones(2)
    lim = (-math.inf, math.inf)
    d = on_device(x, u)
    y, final = ssd.ssd_delta_scan(*args(d), initial_state=d["h0"], dt_softplus=False, dt_limit=lim,
                                  beta_sigmoid=False, qk_norm=False, scale=0.3)
    want, states = oracle_of(x, softplus=False, limit=lim, sigmoid=False, norm=False, scale=0.3)
    length = 0.3 * float(x["q"].double().square().sum(-1).max().sqrt())
    close(final, states[-1], state_bar(states, T, N), "final state")
    close(y, want, y_bar(want, states, T, N, io, length), "y")
    s = d["h0"].clone()
    ssd.ssd_delta_step(s, d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["dt"][:, 0].contiguous(),
                       d["A"], d["beta"][:, 0].contiguous(), dt_softplus=False, dt_limit=lim,
                       beta_sigmoid=False, qk_norm=False, scale=0.3)
    close(s, states[1], state_bar(states[:2], 1, N), "state after a step")
    x, u = make(8, *shape, io=io)
    d = on_device(x, u)
    y, final = ssd.ssd_delta_scan(*args(d), **options(d), dt_limit=(0.2, 0.4), norm_eps=0.5)
    want, states = oracle_of(x, limit=(0.2, 0.4), eps=0.5)
    close(final, states[-1], state_bar(states, T, N), "final state, clipped")
    close(y, want, y_bar(want, states, T, N, io, 1 / math.sqrt(N)), "y, clipped")


def test_hard_gates():
    """Decays from none to all at once, writes of nothing and of everything, equal keys."""
    need_gpu()
    import state_space_model_amd as ssd
    announce("delta hard gates")
    shape = (1, 190, 4, 1, 16, 32)
    T, N = shape[1], shape[5]
    x, u = make(9, *shape, bias=False)
    x["A"] = torch.tensor([-1.0, -16.0, -1e-3, 0.0])
    x["dt"][:, 3::7] = 40.0          # forgets all (A = -16: e^-640), between tokens that keep all
    x["dt"][:, 4::7] = -60.0
    x["beta"][:, ::5] = 30.0
    x["beta"][:, 1::5] = -120.0
    u[:, 100:140, N:2 * N] = u[:, 100:101, N:2 * N]  # the same key forty times
    d = on_device(x, u)
    y, final = ssd.ssd_delta_scan(*args(d), **options(d))
    want, states = oracle_of(x)
    close(final, states[-1], state_bar(states, T, N), "final state")
    close(y, want, y_bar(want, states, T, N, F32, 1 / math.sqrt(N)), "y")


def test_far_decay_sums():
    """A chunk that begins by forgetting a great deal and then keeps everything: exponents are
    differences of sums far from zero."""
    need_gpu()
    import state_space_model_amd as ssd
    announce("delta far sums")
    shape = (1, 128, 2, 2, 16, 16)
    x, u = make(10, *shape, bias=False)
    x["A"] = torch.tensor([-1.0, -1.0])
    x["dt"][:] = -9.0
    x["dt"][:, 0::64] = 20000.0
    d = on_device(x, u)
    y, final = ssd.ssd_delta_scan(*args(d), **options(d))
    want, states = oracle_of(x)
    close(final, states[-1], state_bar(states, 128, 16), "final state")
    close(y, want, y_bar(want, states, 128, 16, F32, 0.25), "y")


@pytest.mark.parametrize("io", [F32, BF16], ids=["f32", "bf16"])
def test_continuation_and_batch(io):
    """A sequence split at any token, the state carried in place, and a row's bits in any batch."""
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta continuation {io}")
    shape = (3, 150, 4, 2, 64, 64)
    T, N = shape[1], shape[5]
    x, u = make(11, *shape, io=io)
    d = on_device(x, u)
    want, states = oracle_of(x)
    whole, final = ssd.ssd_delta_scan(*args(d), **options(d))
    one = {n: t[1:2] if t is not None and t.dim() > 1 else t for n, t in d.items()}
    y1, f1 = ssd.ssd_delta_scan(*args(one), **options(one))
    assert torch.equal(y1[0], whole[1]) and torch.equal(f1[0], final[1])
    state, ys = d["h0"].clone(), []
    for lo, hi in ((0, 1), (1, 65), (65, 66), (66, 150)):
        part = [t[:, lo:hi] if t.dim() > 1 else t for t in args(d)]
        part[3], part[5] = part[3].contiguous(), part[5].contiguous()
        if part[0].shape[0] > 1:   # tokens of several rows are not evenly spaced: as a batch of copies
            part[:3] = [t.contiguous() for t in part[:3]]
        y, s = ssd.ssd_delta_scan(*part, dt_bias=d["dt_bias"], initial_state=state, final_state=state)
        assert s.data_ptr() == state.data_ptr()
        ys.append(y)
    close(state, states[-1], state_bar(states, T, N), "state of the pieces")
    close(torch.cat(ys, 1), want, y_bar(want, states, T, N, io, 1 / math.sqrt(N)), "y of the pieces")


def test_padded_tokens():
    """Tokens with dt = beta = -inf leave the state to the bit and other rows alone."""
    need_gpu()
    import state_space_model_amd as ssd
    announce("delta padding")
    x, u = make(12, 2, 100, 2, 2, 16, 16)
    lens = (37, 100)
    x["dt"][0, 37:] = -math.inf
    x["beta"][0, 37:] = -math.inf
    d = on_device(x, u)
    _, final = ssd.ssd_delta_scan(*args(d), **options(d))
    for b, n in enumerate(lens):
        _, states = oracle_of({m: t if t is None or t.dim() == 1 else t[b:b + 1] if m == "h0" else
                               t[b:b + 1, :n] for m, t in x.items()})
        close(final[b:b + 1], states[-1], state_bar(states, n, 16), f"row {b}")
    s = d["h0"].clone()
    ssd.ssd_delta_step(s, d["q"][:, 50], d["k"][:, 50], d["v"][:, 50], d["dt"][:, 50].contiguous(),
                       d["A"], d["beta"][:, 50].contiguous(), dt_bias=d["dt_bias"])
    assert torch.equal(s[0], d["h0"][0]) and not torch.equal(s[1], d["h0"][1])


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_bad_values_stay_in_their_sequence(bad):
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta {bad}")
    x, u = make(13, 2, 150, 4, 2, 16, 16)
    clean = on_device(x, u)
    want, wfinal = ssd.ssd_delta_scan(*args(clean), **options(clean))
    u[0, 70, 3] = bad                    # q of batch row 0, group 0: heads 0 and 1, from its chunk on
    d = on_device(x, u)
    y, final = ssd.ssd_delta_scan(*args(d), **options(d))
    assert torch.equal(y[1], want[1]) and torch.equal(y[0, :, 2:], want[0, :, 2:])
    assert torch.equal(y[0, :64], want[0, :64]) and torch.equal(final, wfinal)
    assert not y[0, 70, :2].isfinite().any()


def test_nothing_to_do():
    need_gpu()
    import state_space_model_amd as ssd
    announce("delta empty")
    x, u = make(14, 2, 5, 2, 1, 16, 16)
    d = on_device(x, u)
    cut = [t[:, :0] if t.dim() > 1 else t for t in args(d)]
    cut[3], cut[5] = cut[3].contiguous(), cut[5].contiguous()
    y, final = ssd.ssd_delta_scan(*cut, **options(d))
    assert y.shape == (2, 0, 2, 16) and torch.equal(final, d["h0"])
    _, final = ssd.ssd_delta_scan(*cut)
    assert not final.any()
    y, none = ssd.ssd_delta_scan(*args(d), return_final_state=False)
    assert none is None and y.shape == (2, 5, 2, 16)
    nobody = [t[:0] if t.dim() > 1 else t for t in args(d)]
    y, final = ssd.ssd_delta_scan(*nobody)
    assert y.shape[0] == 0 and final.shape == (0, 2, 16, 16)
    first = [t[:0, 0] if t.dim() > 1 else t for t in args(d)]
    assert ssd.ssd_delta_step(final, *first).shape == (0, 2, 16)


def test_far_offsets():
    """Tokens whose strides take the last one past 2^32 bytes, and a state beyond them."""
    need_gpu()
    import state_space_model_amd as ssd
    announce("delta far offsets")
    T, stride = 140, 1 << 24         # 140 x 2^24 bfloat16 = 4.7 GB
    base = torch.empty((T - 1) * stride + 256, dtype=BF16, device="cuda")
    x, _ = make(15, 1, T, 1, 1, 16, 16, io=BF16, h0=False)
    d = {n: None if t is None else t.cuda() for n, t in x.items()}
    for i, n in enumerate("qkv"):
        far = base.as_strided((1, T, 1, 16), (T * stride, stride, 16, 1), 16 * i)
        far.copy_(d[n])
        d[n] = far
    y, final = ssd.ssd_delta_scan(*args(d), **options(d))
    want, states = oracle_of(x)
    close(final, states[-1], state_bar(states, T, 16), "final state")
    close(y, want, y_bar(want, states, T, 16, BF16, 0.25), "y")


def test_streams_and_graphs():
    """Another stream than the default one; a captured scan and step, replayed on new inputs with
    eager calls between."""
    need_gpu()
    import state_space_model_amd as ssd
    announce("delta graphs")
    shape = (2, 100, 4, 2, 64, 128)
    sets = [on_device(*make(20 + i, *shape, io=BF16)) for i in range(3)]
    want = [ssd.ssd_delta_scan(*args(d), **options(d)) for d in sets]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = ssd.ssd_delta_scan(*args(sets[0]), **options(sets[0]))
    side.synchronize()
    assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[0][1])

    def step(d, s):
        return ssd.ssd_delta_step(s, d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["dt0"], d["A"],
                                  d["beta0"], dt_bias=d["dt_bias"])

    for d in sets:
        d["dt0"], d["beta0"] = d["dt"][:, 0].contiguous(), d["beta"][:, 0].contiguous()
    live = {n: t.clone() for n, t in sets[0].items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, final = ssd.ssd_delta_scan(*args(live), **options(live))
        y1 = step(live, final)
    for i in (1, 2, 0, 1):
        for n, t in live.items():
            t.copy_(sets[i][n])
        graph.replay()
        torch.cuda.synchronize()
        s = want[i][1].clone()
        ref = step(sets[i], s)
        assert torch.equal(y, want[i][0]) and torch.equal(final, s) and torch.equal(y1, ref), i
