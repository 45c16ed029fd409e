"""The bars of the gated delta rule's gradients (delta_magnitudes) on the CPU: the terms add up to the
automatic derivatives, and a gradient that is zero, negated or lacks a term is far outside its bar."""
import math

import pytest
import torch

import delta_magnitudes as dm
from delta_cases import make
from test_gpu_delta_gradients import cotangents
from test_gpu_delta_terms import ALONE, OWNED, PAIRS, hard, raw

F32, BF16 = torch.float32, torch.bfloat16


def inputs(shape, io):
    T = shape[1]
    x, _ = make(T + 1, *shape, io=io, h0=T % 2 == 0, bias=T % 3 != 0)
    return (x, *cotangents(T, x, T % 4 != 1))


def over(off, bar):
    """The largest error against its bar; nothing where both are 0."""
    return float(torch.where(off == 0, 0.0, off.abs() / bar).max())


def check(x, dy, dfinal, **opts):
    """Returns the terms that are not far below the rest, each of which has to show."""
    grads, terms = dm.reference(x, dy, dfinal, **opts)
    shown = set()
    bars = dm.bars(x, grads, terms)
    assert set(bars) == set(grads) - {"dh0"} | {"dinitial_state"}
    for n, parts in terms.items():
        ref, bar = grads[n], bars[n]
        assert bar.shape == ref.shape and bool((bar >= 0).all()), n
        assert over(sum(p.v for p in parts) - ref, bar) < 1e-3, n
        if ref.any():
            assert over(ref, bar) > 200 and over(2 * ref, bar) > 200, n
        for i, p in enumerate(parts):
            if float(p.v.abs().max()) > 1e-2 * float(ref.abs().max()):
                assert over(p.v, bar) > 2, (n, i)
                shown.add((n, i))
        # typical elements too: the bar against the gradient's root mean square
        rms = float(ref.square().mean().sqrt()) + dm.TINY
        part = 5e-3 if x["v"].dtype == BF16 and n in ("dq", "dk", "dv") else 5e-4
        assert float(bar.square().mean().sqrt()) <= part * rms + dm.TINY, n
    return shown, {(n, i) for n, parts in terms.items() for i in range(len(parts))}


@pytest.mark.parametrize("io", [F32, BF16], ids=["f32", "bf16"])
def test_bars_show_mistakes(io):
    """Zeros, the other sign and every missing term, and each term in several shapes of every kind."""
    for shapes in (ALONE, PAIRS, OWNED):
        counts = {}
        for shape in shapes:
            shown, every = check(*inputs(shape, io))
            for t in every:
                counts[t] = counts.get(t, 0) + (t in shown)
        assert min(counts.values()) >= 2, counts


@pytest.mark.parametrize("io", [F32, BF16], ids=["f32", "bf16"])
def test_bars_of_other_gates(io):
    x, u, dy, dfinal = hard((2, 4, 2, 16), 70, io)
    check(x, dy, dfinal)
    x, u, dy, dfinal, opts, _ = raw(io)
    check(x, dy, dfinal, **opts)
    x, dy, dfinal = inputs((2, 100, 2, 1, 32, 48), io)
    check(x, dy, dfinal, limit=(0.4, 0.7), eps=0.5)


def test_magnitudes_bound_float32():
    """The chunked products in float32, one after the other, stay within their bars."""
    g = torch.Generator().manual_seed(1)
    a, b = torch.randn(64, 200, generator=g), torch.randn(200, 64, generator=g)
    want = dm.Sum(a.double()) @ dm.Sum(b.double())
    got = torch.zeros(64, 64)
    for k in range(200):
        got = got + a[:, k:k + 1] * b[k:k + 1]
    assert bool(((got - want.v).abs() <= 8 * math.sqrt(200) * dm.U * want.m).all())
