"""The residual add with dropout and norm on the GPU against its float64
definition (oracle.dropout).  Bars as in test_gpu_block; the mask is exact."""
import math

import numpy as np
import pytest
import torch

from gpu_util import announce, need_gpu
from oracle import block, dropout
from oracle.block import f64
from test_gpu_block import EPS, U, WIDTHS, close, dev, gen, io_u, norm_u, randn, sum_u

pytestmark = pytest.mark.gpu
SEED, OFFSET = (0x1234567 << 32) + 0x89ABCDEF, (5 << 32) + 77


def state(seed=SEED, offset=OFFSET):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", WIDTHS + [6, 70, 1026, 2563])
def test_forward(d, io):
    need_gpu()
    import state_space_model_amd as ssd
    g = gen(d)
    rows, s, p = (7 if d > 4096 else 33), 0.5, 0.3
    x, r, w = randn(g, rows, d, io=io), 3 * randn(g, rows, d), 1 + 0.1 * randn(g, d)
    announce(f"dropout_add_norm {io} {rows}x{d}")
    keep = dropout.kept(rows, d, p, SEED, OFFSET)
    for residual in (r, None):
        y, ro = ssd.ssd_dropout_add_norm(dev(x), dev(w), dev(residual), p=p, rng=state(), scale=s, eps=EPS)
        res64 = None if residual is None else f64(residual)
        ref, ref_r = dropout.add_norm(f64(x), res64, f64(w), s, p, keep, EPS)
        # the mask: without a residual what is dropped is zero, and only that (no x is)
        if residual is None:
            assert np.array_equal(f64(ro) != 0, keep)
        mag = keep * np.abs(s / (1 - p) * f64(x)) + (0 if residual is None else np.abs(f64(r)))
        c = np.abs(1 / np.sqrt((ref_r ** 2).mean(-1, keepdims=True) + EPS) * f64(w))
        close(ro, ref_r, 3 * U * mag, "residual_out")     # the scale's rounding too
        close(y, ref, norm_u(d) * mag * c + io_u(io) * 1.01 * np.abs(ref), "y")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d", [(1, 1), (1, 2560), (2, 63), (33, 256), (300, 768), (1030, 130),
                                    (70, 2048), (40, 4099), (3, 8200), (5, 16384), (700, 71)])
def test_gradients(rows, d, io):
    need_gpu()
    import state_space_model_amd as ssd
    g = gen(rows + d)
    r, w, p, s = 2 * randn(g, rows, d), 1 + 0.1 * randn(g, d), 0.25, 0.5
    dy, dro = randn(g, rows, d, io=io), randn(g, rows, d)
    announce(f"dropout_add_norm_backward {io} {rows}x{d}")
    keep = dropout.kept(rows, d, p, SEED, OFFSET)
    for dres_out in (dro, None):
        kw = dict(dy=dev(dy), p=p, rng=state(), scale=s, eps=EPS)
        got = ssd.ssd_dropout_add_norm_backward(dev(r), dev(w), dresidual_out=dev(dres_out), **kw)
        ref = dropout.add_norm_backward(f64(r), f64(w), f64(dy), None if dres_out is None else f64(dro),
                                        s, p, keep, EPS)
        c = 1 / np.sqrt((f64(r) ** 2).mean(-1, keepdims=True) + EPS)
        pm, xh = np.abs(f64(dy) * f64(w)), np.abs(f64(r) * c)
        mag = c * (pm + xh * (pm * xh).mean(-1, keepdims=True)) + (0 if dres_out is None else np.abs(f64(dro)))
        close(got["dresidual"], ref["dresidual"], 4 * norm_u(d) * mag, "dresidual")
        close(got["dx"], ref["dx"], keep * (4 * norm_u(d) * mag + io_u(io) * 1.01 * np.abs(ref["dx"])), "dx")
        close(got["dweight"], ref["dweight"], (sum_u(rows) + norm_u(d)) * np.abs(f64(dy) * xh).sum(0), "dweight")
    buf = dev(dro)
    again = ssd.ssd_dropout_add_norm_backward(dev(r), dev(w), dresidual_out=buf, grads={"dresidual": buf}, **kw)
    first = ssd.ssd_dropout_add_norm_backward(dev(r), dev(w), dresidual_out=dev(dro), **kw)
    for k in first:
        assert torch.equal(first[k], again[k]), k


def test_forward_and_gradients_share_the_mask():
    """Differences of the float64 forward along x at the mask of the GPU's forward."""
    need_gpu()
    import state_space_model_amd as ssd
    announce("dropout differences")
    g = gen(5)
    x, r, w, dy, dro, way = (randn(g, 9, 77) for _ in range(6))
    w, p = w[0].clone(), 0.4
    _, ro = ssd.ssd_dropout_add_norm(dev(x), dev(w), p=p, rng=state())
    keep = f64(ro) != 0
    _, ro = ssd.ssd_dropout_add_norm(dev(x), dev(w), dev(r), p=p, rng=state())
    got = ssd.ssd_dropout_add_norm_backward(ro, dev(w), dy=dev(dy), dresidual_out=dev(dro), p=p, rng=state())

    def loss(step):
        y, out = dropout.add_norm(f64(x) + step * f64(way), f64(r), f64(w), 1.0, p, keep, EPS)
        return (y * f64(dy)).sum() + (out * f64(dro)).sum()

    slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
    grad = f64(got["dx"])
    assert abs((grad * f64(way)).sum() - slope) <= 1e-5 * np.linalg.norm(grad) * np.linalg.norm(f64(way))


def test_without_dropout_and_with_nearly_all():
    need_gpu()
    import state_space_model_amd as ssd
    announce("dropout p = 0 and p -> 1")
    g = gen(6)
    x, r, w = dev(randn(g, 40, 300, io="bf16")), dev(randn(g, 40, 300)), dev(randn(g, 300))
    for scale in (1.0, 0.3):
        want = ssd.ssd_add_norm(x, w, r, scale=scale)
        got = ssd.ssd_dropout_add_norm(x, w, r, p=0.0, rng=state(), scale=scale)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    dy = dev(randn(g, 40, 300, io="bf16"))
    want = ssd.ssd_add_norm_backward(r, w, dy=dy)
    got = ssd.ssd_dropout_add_norm_backward(r, w, dy=dy, p=0.0, rng=state())
    assert all(torch.equal(want[k], got[k]) for k in want)
    _, ro = ssd.ssd_dropout_add_norm(x, w, r, p=1 - 2.0 ** -33, rng=state())
    assert torch.equal(ro, r)


def test_dropped_values_reach_nothing():
    """A NaN or an infinity that is dropped is not seen; one that is kept stays in its row."""
    need_gpu()
    import state_space_model_amd as ssd
    announce("dropout of bad values")
    x = torch.ones(6, 130, device="cuda")
    r, w = torch.full((6, 130), 2.0, device="cuda"), torch.ones(130, device="cuda")
    keep = torch.from_numpy(dropout.kept(6, 130, 0.5, SEED, OFFSET)).cuda()
    clean = ssd.ssd_dropout_add_norm(x, w, r, p=0.5, rng=state())
    bad = torch.where(keep, x, torch.full_like(x, math.nan))
    bad[0, 3::2] = torch.where(keep[0, 3::2], x[0, 3::2], torch.full_like(x[0, 3::2], math.inf))
    got = ssd.ssd_dropout_add_norm(bad, w, r, p=0.5, rng=state())
    assert torch.equal(clean[0], got[0]) and torch.equal(clean[1], got[1])
    c = int(keep[2].nonzero()[0])
    bad[2, c] = math.nan
    y, _ = ssd.ssd_dropout_add_norm(bad, w, r, p=0.5, rng=state())
    others = [0, 1, 3, 4, 5]
    assert torch.equal(y[others], clean[0][others]) and y[2].isnan().all()


def test_rows_of_any_batch_and_many():
    """The mask goes by a row's number: leading dimensions do not matter; rows past one launch's grid."""
    need_gpu()
    import state_space_model_amd as ssd
    announce("dropout rows")
    w = torch.ones(8, device="cuda")
    rows = (1 << 23) + 5                 # four rows to a workgroup, 2^21 rows to a launch
    x = torch.ones(rows, 8, device="cuda")
    _, a = ssd.ssd_dropout_add_norm(x, w, p=0.5, rng=state())
    _, b = ssd.ssd_dropout_add_norm(x.view(5, -1, 1, 8) if rows % 5 == 0 else x[None], w, p=0.5, rng=state())
    assert torch.equal(a, b.view(rows, 8))
    for lo in (0, (1 << 21) - 2, (1 << 21), (1 << 23) - 1, rows - 3):
        n = min(4, rows - lo)
        c = np.zeros((n, 2, 4), np.uint64)
        c[..., 0], c[..., 1] = np.arange(2)[None], (lo + np.arange(n))[:, None]
        c[..., 2], c[..., 3] = dropout.halves(OFFSET)
        keep = dropout.philox(c, dropout.halves(SEED)).reshape(n, 8) >= 2 ** 31
        assert np.array_equal(a[lo:lo + n].cpu().numpy() != 0, keep), lo
    assert abs(float((a != 0).float().mean()) - 0.5) < 5 * 0.5 / math.sqrt(rows * 8)
    y, ro = ssd.ssd_dropout_add_norm(x[:0], w, p=0.5, rng=state())
    assert y.shape == (0, 8)
    assert not ssd.ssd_dropout_add_norm_backward(x[:0], w, dy=x[:0], p=0.5, rng=state())["dweight"].any()


def test_graph_with_an_advancing_offset():
    """Captured with the offset's advance; every replay has another mask, that of an eager call."""
    need_gpu()
    import state_space_model_amd as ssd
    announce("dropout graph")
    g = gen(8)
    x, r, w, dy = dev(randn(g, 50, 770, io="bf16")), dev(randn(g, 50, 770)), dev(randn(g, 770)), \
        dev(randn(g, 50, 770, io="bf16"))
    rng = state()

    def step(rng):
        y, ro = ssd.ssd_dropout_add_norm(x, w, r, p=0.2, rng=rng)
        return y, ro, ssd.ssd_dropout_add_norm_backward(ro, w, dy=dy, p=0.2, rng=rng)

    step(rng)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(rng)
        rng[1:].add_(1)
    seen = []
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        want = step(state(offset=OFFSET + i))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i
        assert all(torch.equal(got[2][k], want[2][k]) for k in want[2]), i
        seen.append(got[1].clone())
    assert all(not torch.equal(seen[0], s) for s in seen[1:])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = step(state())
    side.synchronize()
    assert torch.equal(other[1], seen[0])
