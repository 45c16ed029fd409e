"""The gated delta rule's y is a float32 sum rounded once: with orthogonal keys, no decay and values
that are powers of two every step of it is exact, and y has to be the float32 value's own rounding."""
import math

import pytest
import torch

from delta_cases import on_device
from gpu_util import announce, need_gpu
from test_gpu_delta import args

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
# rows, heads, groups, values: chains alone, in pairs, columns owned (bfloat16)
KINDS = [(2, 4, 2, 24), (3, 32, 8, 40), (5, 32, 8, 64)]


def near_ties(g, *shape):
    """Float32 numbers half-way between two bfloat16 numbers, 2^-22 above or below."""
    i = torch.randint(0, 128, shape, generator=g)
    side = 2 * torch.randint(0, 2, shape, generator=g) - 1
    return (1 + (2 * i + 1) / 256.0 + side * 2.0 ** -22).to(F32)


def case(kind, T, N, io, seed):
    """N / 2 tokens of T write, each to an axis of its own; the initial state holds the other axes'
    values; every token reads one axis that is known by then."""
    Bt, H, G, P = kind
    g = torch.Generator().manual_seed(seed)
    half = N // 2
    writers = torch.randperm(T, generator=g)[:half].sort().values.tolist()
    u = torch.zeros(Bt, T, 2 * G * N + H * P)
    x = {"q": u[..., :G * N].unflatten(-1, (G, N)), "k": u[..., G * N:2 * G * N].unflatten(-1, (G, N)),
         "v": u[..., 2 * G * N:].unflatten(-1, (H, P)), "dt": torch.full((Bt, T, H), -math.inf),
         "A": -torch.ones(H), "beta": torch.zeros(Bt, T, H), "dt_bias": None, "h0": torch.zeros(Bt, H, P, N)}
    x["v"].copy_(torch.pow(2.0, torch.randint(-2, 3, (Bt, T, H, P), generator=g)))
    x["v"].mul_(2 * torch.randint(0, 2, (Bt, T, H, P), generator=g) - 1)
    x["h0"][..., half:] = near_ties(g, Bt, H, P, N - half)
    axis, reads = {t: i for i, t in enumerate(writers)}, []
    for t in range(T):
        x["k"][:, t, :, axis.get(t, 0)] = 1.0
        known = list(range(sum(w <= t for w in writers))) + list(range(half, N))
        reads.append(known[int(torch.randint(0, len(known), (1,), generator=g))])
        x["q"][:, t, :, reads[-1]] = 1.0
    x["beta"][:, writers] = near_ties(g, Bt, half, H)
    return x, u, axis, reads


def expected(x, axis, reads):
    """y [Bt,T,H,P] in float32, each the value that the axis read holds."""
    held = x["h0"].clone()
    ys = []
    for t, n in enumerate(reads):
        if t in axis:
            held[..., axis[t]] = x["beta"][:, t, :, None] * x["v"][:, t].float()   # times a power of two
        ys.append(held[..., n].clone())
    return torch.stack(ys, 1), held


OPTIONS = dict(beta_sigmoid=False, qk_norm=False)


@pytest.mark.parametrize("io", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N", [40, 64, 104, 128])
@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_y_is_rounded_once(kind, N, io):
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta rounding {kind} {N} {io}")
    x, u, axis, reads = case(kind, 130, N, io, N)
    d = on_device(x, u.to(io))
    y, final = ssd.ssd_delta_scan(*args(d), initial_state=d["h0"], scale=1.0, **OPTIONS)
    want, held = expected(x, axis, reads)
    assert torch.equal(final.cpu(), held)
    assert torch.equal(y.cpu(), want.to(io))


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_scaled_y_is_rounded_once(kind):
    """The same where the scale of the queries holds the last bits, and states are powers of two."""
    need_gpu()
    import state_space_model_amd as ssd
    announce(f"delta rounding, scale {kind}")
    x, u, axis, reads = case(kind, 130, 128, BF16, 3)
    x["beta"] = (x["beta"] != 0).float()
    x["h0"] = x["h0"].round()
    for scale in near_ties(torch.Generator().manual_seed(5), 4).tolist():
        d = on_device(x, u.to(BF16))
        y, _ = ssd.ssd_delta_scan(*args(d), initial_state=d["h0"], scale=scale, **OPTIONS)
        want, _ = expected(x, axis, reads)
        assert torch.equal(y.cpu(), (scale * want).to(BF16))


def test_steps_round_once():
    need_gpu()
    import state_space_model_amd as ssd
    announce("delta rounding, steps")
    x, u, axis, reads = case((2, 4, 2, 24), 40, 72, BF16, 9)
    d = on_device(x, u.to(BF16))
    state, (want, held) = d["h0"].clone(), expected(x, axis, reads)
    for t in range(40):
        y = ssd.ssd_delta_step(state, d["q"][:, t], d["k"][:, t], d["v"][:, t], d["dt"][:, t].contiguous(), d["A"],
                               d["beta"][:, t].contiguous(), scale=1.0, **OPTIONS)
        assert torch.equal(y.cpu(), want[:, t].to(BF16)), t
    assert torch.equal(state.cpu(), held)
