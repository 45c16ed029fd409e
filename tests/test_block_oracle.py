"""The float64 forms of the operators between two scans (oracle.block) against
central differences of their own forwards, against torch's automatic
derivatives, and against mistakes planted in them.  CPU only."""
import numpy as np
import pytest
import torch

import oracle
from oracle import block

EPS = 1e-5


def rng(seed):
    return np.random.default_rng(seed)


def directional(loss, args, grads, seed, h=1e-6):
    """Central difference of loss along a random direction against <grad, v>;
    with |loss'''| of order one the difference is good to about h^2 + 1e-16/h."""
    r = rng(seed)
    for k in grads:
        v = r.standard_normal(args[k].shape)
        hi, lo = dict(args), dict(args)
        hi[k], lo[k] = args[k] + h * v, args[k] - h * v
        num = (loss(**hi) - loss(**lo)) / (2 * h)
        ana = float((grads[k] * v).sum())
        scale = np.abs(grads[k] * v).sum() + 1.0
        assert abs(num - ana) <= 1e-7 * scale, (k, num, ana)


@pytest.mark.parametrize("d,residual", [(1, True), (7, False), (64, True)])
def test_add_norm_gradients_against_differences(d, residual):
    r = rng(d)
    args = dict(x=r.standard_normal((3, d)), weight=1 + 0.1 * r.standard_normal(d),
                residual=r.standard_normal((3, d)))
    dy, dro = r.standard_normal((3, d)), r.standard_normal((3, d))

    def loss(x, weight, residual):
        y, ro = block.add_norm(x, weight, residual, 0.5, EPS)
        return (dy * y).sum() + (dro * ro).sum()

    _, ro = block.add_norm(**args, scale=0.5, eps=EPS)
    g = block.add_norm_backward(ro, args["weight"], dy, dro, 0.5, EPS)
    directional(loss, args, {"x": g["dx"], "residual": g["dresidual"], "weight": g["dweight"]}, 1)


@pytest.mark.parametrize("groups", [1, 2, 8])
def test_gated_norm_gradients_against_differences(groups):
    r = rng(groups)
    args = dict(y=r.standard_normal((3, 16)), z=2 * r.standard_normal((3, 16)),
                weight=1 + 0.1 * r.standard_normal(16))
    dout = r.standard_normal((3, 16))
    g = block.gated_norm_backward(args["y"], args["z"], args["weight"], dout, EPS, groups)
    directional(lambda y, z, weight: (dout * block.gated_norm(y, z, weight, EPS, groups)).sum(),
                args, {"y": g["dy"], "z": g["dz"], "weight": g["dweight"]}, 2)


@pytest.mark.parametrize("T,K,silu", [(1, 4, True), (2, 4, True), (9, 4, False), (5, 2, True),
                                      (6, 3, True)])
def test_conv_gradients_against_differences_of_the_convolution(T, K, silu):
    """The forward here is the oracle's convolution, not the one inside the
    gradient."""
    r = rng(10 * T + K)
    f32 = lambda *s: r.standard_normal(s).astype(np.float32).astype(np.float64)
    args = dict(x=f32(2, T, 3), weight=f32(3, K), bias=f32(3), state=f32(2, 3, K - 1))
    dy, dso = f32(2, T, 3), f32(2, 3, K - 1)
    g = block.conv1d_backward(args["x"], args["weight"], args["bias"], dy, args["state"], dso, silu)
    # one-token pieces through float64 conv1d_step would round inputs: use the
    # definition, and pin it to the oracle's convolution at the point itself
    z = np.zeros((2, T, 3))

    def forward(x, weight, bias, state):
        xp = np.concatenate([state.transpose(0, 2, 1), x], 1)
        z = bias + sum(weight[:, i] * xp[:, i:i + T] for i in range(K))
        return (block.silu(z) if silu else z), xp[:, T:].transpose(0, 2, 1)

    t32 = {k: torch.from_numpy(v.astype(np.float32)) for k, v in args.items()}
    y_o, st_o = oracle.conv1d(t32["x"], t32["weight"], t32["bias"], t32["state"], silu=silu)
    y, st = forward(**args)
    assert np.abs(y - y_o).max() <= 1e-12 and np.array_equal(st, st_o)
    directional(lambda **a: (dy * forward(**a)[0]).sum() + (dso * forward(**a)[1]).sum(), args,
                {"x": g["dx"], "weight": g["dweight"], "bias": g["dbias"], "state": g["dstate"]}, 3)


def test_norm_gradients_against_automatic_derivatives():
    r = rng(5)
    v = torch.tensor(r.standard_normal((4, 12)), requires_grad=True)
    z = torch.tensor(r.standard_normal((4, 12)), requires_grad=True)
    w = torch.tensor(1 + 0.1 * r.standard_normal(12), requires_grad=True)
    dout = r.standard_normal((4, 12))
    g = v * z * torch.sigmoid(z)
    u = g.view(4, 3, 4)
    n = (u * torch.rsqrt(u.pow(2).mean(-1, keepdim=True) + EPS)).view(4, 12) * w
    (n * torch.from_numpy(dout)).sum().backward()
    got = block.gated_norm_backward(v.detach().numpy(), z.detach().numpy(), w.detach().numpy(),
                                    dout, EPS, 3)
    for a, b in ((got["dy"], v.grad), (got["dz"], z.grad), (got["dweight"], w.grad)):
        assert np.abs(a - b.numpy()).max() <= 1e-13


@pytest.mark.parametrize("mistake", ["no_mean", "gate_slope", "group", "no_eps_in_slope"])
def test_planted_mistakes_are_seen(mistake):
    """Each slip in a copy of the gated norm's gradient fails the difference
    test that the unbroken one passes."""
    r = rng(6)
    args = dict(y=r.standard_normal((3, 16)), z=2 * r.standard_normal((3, 16)),
                weight=1 + 0.1 * r.standard_normal(16))
    dout = r.standard_normal((3, 16))
    eps = 0.5 if mistake == "no_eps_in_slope" else EPS

    def broken():
        y, z, w = args["y"], args["z"], args["weight"]
        g = y * block.silu(z)
        u, dn = g.reshape(3, 2, 8), (dout * w).reshape(3, 2, 8)
        if mistake == "group":
            u, dn = g.reshape(3, 1, 16), (dout * w).reshape(3, 1, 16)
        ms = (u * u).mean(-1, keepdims=True)
        c = 1 / np.sqrt(ms + eps)
        c3 = c / ms if mistake == "no_eps_in_slope" else c ** 3
        m = 0 if mistake == "no_mean" else (dn * u).mean(-1, keepdims=True)
        dg = (c * dn - c3 * u * m).reshape(3, 16)
        slope = block.logistic(z) if mistake == "gate_slope" else block.silu_slope(z)
        return {"y": dg * block.silu(z), "z": dg * y * slope}

    loss = lambda y, z, weight: (dout * block.gated_norm(y, z, weight, eps, 2)).sum()
    good = block.gated_norm_backward(args["y"], args["z"], args["weight"], dout, eps, 2)
    directional(loss, args, {"y": good["dy"], "z": good["dz"]}, 7)
    with pytest.raises(AssertionError):
        directional(loss, args, broken(), 7)
