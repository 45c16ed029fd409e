"""The float64 oracle of the gated delta rule pinned by closed forms, by
differences and with planted mistakes (CPU)."""
import math

import pytest
import torch

from delta_cases import make
from oracle import delta

CHANGES = ["dt", "beta", "A", "q", "k", "v", "h0", "dt_bias"]


def small(seed=1, **kw):
    x, _ = make(seed, 2, 7, 4, 2, 8, 8, **kw)
    return {n: delta.f64(t) for n, t in x.items()}


def test_equal_keys_are_an_average():
    """One unit key, no decay: S k follows v by the share b, S k = s, s' = s + b (v - s)."""
    x = small(h0=False, bias=False)
    x["k"][:] = 0.0
    x["k"][..., 3] = 2.0
    x["A"] = torch.zeros(4, dtype=torch.float64)
    _, states = delta.scan(**x, eps=0.0)
    s, b = torch.zeros(2, 4, 8, dtype=torch.float64), torch.sigmoid(x["beta"])
    for t in range(7):
        s = s + b[:, t, :, None] * (x["v"][:, t] - s)
        assert torch.allclose(states[t + 1][..., 3], s, atol=1e-14)
        assert not states[t + 1][..., [0, 1, 2, 4, 5, 6, 7]].any()


def test_whole_writes_to_orthogonal_keys_are_read_back():
    x = small(h0=False, bias=False)
    x["k"] = torch.eye(8, dtype=torch.float64)[:7].expand(2, 7, 8)[:, :, None].repeat(1, 1, 2, 1) * 3.0
    x["q"], x["beta"] = x["k"].clone(), torch.full_like(x["beta"], 1e3)
    y, _ = delta.scan(**x, eps=0.0, scale=1.0)
    assert torch.allclose(y, x["v"], atol=1e-14)


def test_decay_alone_and_tokens_that_change_nothing():
    x = small()
    x["beta"][:] = -math.inf
    _, states = delta.scan(**x)
    rate = delta.rates(x["dt"], x["dt_bias"])
    whole = torch.exp((rate * x["A"]).sum(1))
    assert torch.allclose(states[-1], whole[..., None, None] * x["h0"], atol=1e-14)
    x["dt"][:] = -math.inf
    _, states = delta.scan(**x)
    assert all(torch.equal(s, x["h0"]) for s in states)


@pytest.mark.parametrize("name", CHANGES)
def test_gradients_against_differences(name):
    x = small(3)
    g = torch.Generator().manual_seed(5)
    r = lambda t: torch.randn(t.shape, generator=g, dtype=torch.float64)  # noqa: E731
    dy, dfinal, way = r(x["v"]), r(x["h0"]), r(x[name])
    grads, _, _ = delta.gradients(x, dy, dfinal)

    def loss(step):
        y, states = delta.scan(**{**x, name: x[name] + step * way})
        return float((y * dy).sum() + (states[-1] * dfinal).sum())

    h = 1e-5
    slope = (loss(h) - loss(-h)) / (2 * h)
    got = float((grads["d" + name] * way).sum())
    assert abs(got - slope) <= 1e-7 * max(1.0, abs(slope)), (got, slope)


@pytest.mark.parametrize("slip", ["decay_after_write", "no_removal", "undecayed_removal", "key_not_unit",
                                  "group", "before_write"])
def test_planted_mistakes_show(slip):
    """A recurrence with one mistake is far from the oracle on the inputs that the tests use."""
    x = small(4)
    y, states = delta.scan(**x)
    q, k = delta.unit(x["q"], 1e-6) / math.sqrt(8), x["k"] if slip == "key_not_unit" else delta.unit(x["k"], 1e-6)
    spread = (lambda t: t.repeat(1, 1, 2, 1)) if slip == "group" else (lambda t: t.repeat_interleave(2, 2))
    q, k = spread(q), spread(k)
    a = torch.exp(delta.rates(x["dt"], x["dt_bias"]) * x["A"])[..., None, None]
    b = torch.sigmoid(x["beta"])[..., None]
    s, ys = x["h0"], []
    for t in range(7):
        kt, old = k[:, t, :, None, :], s
        if slip != "decay_after_write":
            s = a[:, t] * s
        held = ((old if slip == "undecayed_removal" else s) * kt).sum(-1)
        if slip == "no_removal":
            held = 0.0
        if slip == "before_write":
            ys.append((s * q[:, t, :, None, :]).sum(-1))
        s = s + (b[:, t] * (x["v"][:, t] - held))[..., None] * kt
        if slip == "decay_after_write":
            s = a[:, t] * s
        if slip != "before_write":
            ys.append((s * q[:, t, :, None, :]).sum(-1))
    off = max(float((torch.stack(ys, 1) - y).abs().max()), float((s - states[-1]).abs().max()))
    assert off > 1e-2
