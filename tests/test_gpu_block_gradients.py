"""The norms' gradients against their float64 definitions (oracle.block) over
the range of sizes that their forwards take, and where a workgroup takes
several rows.  Bars as in test_gpu_block, whose terms scale with the inputs."""
import numpy as np
import pytest
import torch

from gpu_util import announce, need_gpu
from oracle import block
from oracle.block import f64
from test_gpu_block import EPS, U, close, dev, gated_case, gen, io_u, norm_u, randn, silu_bar, sum_u

pytestmark = pytest.mark.gpu


def check_add_norm(r, w, dy, dro, eps, io):
    import state_space_model_amd as ssd
    rows, d = r.shape
    got = ssd.ssd_add_norm_backward(dev(r), dev(w), dy=dev(dy), dresidual_out=dev(dro), scale=0.25,
                                    eps=eps)
    r64, w64, dy64 = f64(r), f64(w), f64(dy)
    ref = block.add_norm_backward(r64, w64, dy64, None if dro is None else f64(dro), 0.25, eps)
    c = 1 / np.sqrt((r64 ** 2).mean(-1, keepdims=True) + eps)
    p, xh = np.abs(dy64 * w64), np.abs(r64 * c)
    mag = c * (p + xh * (p * xh).mean(-1, keepdims=True)) + (0 if dro is None else np.abs(f64(dro)))
    close(got["dresidual"], ref["dresidual"], 4 * norm_u(d) * mag, "dresidual")
    close(got["dx"], ref["dx"], norm_u(d) * mag + io_u(io) * 1.01 * np.abs(ref["dx"]), "dx")
    close(got["dweight"], ref["dweight"], (sum_u(rows) + norm_u(d)) * np.abs(dy64 * xh).sum(0),
          "dweight")


def check_gated_norm(y, z, w, dout, groups, eps, io):
    import state_space_model_amd as ssd
    rows, d = y.shape
    got = ssd.ssd_gated_norm_backward(dev(y), dev(z), dev(w), dout=dev(dout), groups=groups, eps=eps)
    y64, z64, w64, d64 = f64(y), f64(z), f64(w), f64(dout)
    ref = block.gated_norm_backward(y64, z64, w64, d64, eps, groups)
    width = d // groups
    s, act, sb = block.logistic(z64), np.abs(block.silu(z64)), silu_bar(z64)
    g = (y64 * block.silu(z64)).reshape(rows, groups, width)
    g_err = (np.abs(y64) * sb).reshape(g.shape)
    ms = (g * g).mean(-1, keepdims=True) + eps
    c = 1 / np.sqrt(ms)
    rel = 3 * norm_u(width) + 3 * (np.abs(g) * g_err).mean(-1, keepdims=True) / ms
    p = np.abs(d64 * w64).reshape(g.shape)
    gh, gh_err = np.abs(g) * c, g_err * c
    mean = (p * gh).mean(-1, keepdims=True)
    mag = (c * (p + gh * mean)).reshape(rows, d)
    err = (c * (gh_err * mean + gh * (p * gh_err).mean(-1, keepdims=True)) +
           rel * c * (p + 2 * gh * mean)).reshape(rows, d)
    slope = s * (1 + np.abs(z64) * (1 - s))
    close(got["dy"], ref["dy"], err * act + mag * sb + 4 * U * mag * act +
          io_u(io) * 1.01 * np.abs(ref["dy"]), "dy")
    close(got["dz"], ref["dz"], np.abs(y64) * (err * slope + 2 * mag * (sb + 4 * U * slope)) +
          io_u(io) * 1.01 * np.abs(ref["dz"]), "dz")
    close(got["dweight"], ref["dweight"],
          (np.abs(d64) * ((gh_err + rel * gh).reshape(rows, d) +
                          sum_u(rows) * gh.reshape(rows, d))).sum(0), "dweight")


# sizes whose squares stay inside float32, far from one on both sides; with eps
# = 0 the inverse root mean square is as large as the rows are small
SIZES = [(1e15, EPS), (1e17, EPS), (1e-14, 0.0), (1e-16, 0.0)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size,eps", SIZES)
@pytest.mark.parametrize("d", [130, 768, 2560])
def test_add_norm_gradients_of_large_and_small_rows(d, size, eps, io):
    need_gpu()
    announce(f"add_norm_backward {io} 9x{d} of size {size}, eps {eps}")
    g = gen(d)
    check_add_norm(size * randn(g, 9, d), 1 + 0.1 * randn(g, d), randn(g, 9, d, io=io), None, eps, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size,eps", SIZES)
@pytest.mark.parametrize("d,groups", [(130, 1), (1536, 2), (2560, 1)])
def test_gated_norm_gradients_of_large_and_small_rows(d, groups, size, eps, io):
    need_gpu()
    announce(f"gated_norm_backward {io} 9x{d} groups {groups} of size {size}, eps {eps}")
    g, y, w, z = gated_case(9, d, io, d, 0)
    check_gated_norm(y * size, z, w, randn(g, 9, d, io=io), groups, eps, io)


# Rows beyond one per workgroup (512 workgroups over all groups; four wavefronts
# with a row each, or a workgroup per row), so that every workgroup takes
# several, some one more than others, and the second launch adds all the parts.
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d", [(1300, 2048), (1100, 4099), (700, 8200), (2600, 130), (5003, 768)])
def test_add_norm_gradients_of_many_rows(rows, d, io):
    need_gpu()
    announce(f"add_norm_backward {io} {rows}x{d}")
    g = gen(rows + d)
    check_add_norm(2 * randn(g, rows, d), 1 + 0.1 * randn(g, d), randn(g, rows, d, io=io),
                   randn(g, rows, d), EPS, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d,groups", [(700, 4096, 1), (1100, 8192, 2), (1541, 5120, 1),
                                           (9001, 96, 3), (3001, 1536, 4)])
def test_gated_norm_gradients_of_many_rows(rows, d, groups, io):
    need_gpu()
    announce(f"gated_norm_backward {io} {rows}x{d} groups {groups}")
    g, y, w, z = gated_case(rows, d, io, rows + d, 0)
    check_gated_norm(y, z, w, randn(g, rows, d, io=io), groups, EPS, io)
