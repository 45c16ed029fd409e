"""The convolution's gradients where the tokens are split into runs of other
lengths than the shortest, and the 8-bit product of two column steps on its
persistent tiles.  Bars as in test_gpu_block."""
import numpy as np
import pytest
import torch

from gpu_util import announce, need_gpu
from oracle import block
from oracle.block import f64
from test_gpu_block import U, close, dev, gen, io_u, randn, silu_bar, sum_u
from test_gpu_block import test_linear_q8_large as linear_q8_large

pytestmark = pytest.mark.gpu

# (batch, tokens, channels, taps, io, dy, state): runs of 27, 28, 30, 49 and 187
# tokens (768 workgroups of 512 channels over batch and runs), so that a run
# ends one, two or three tokens past a multiple of four and the next one begins
# there, with its taps and pending sums formed anew
RUNS = [(1, 20700, 36, 4, "f32", "f32", True), (1, 20737, 36, 3, "bf16", "f32", False),
        (8, 600, 2049, 4, "bf16", "f32", True), (8, 600, 2049, 4, "f32", "f32", False),
        (2, 9300, 515, 4, "f32", "f32", True), (2, 9300, 515, 2, "bf16", "bf16", True),
        (1, 143600, 36, 4, "bf16", "f32", True)]


@pytest.mark.parametrize("case", RUNS, ids=lambda c: "_".join(map(str, c)))
def test_conv1d_backward_of_long_runs(case):
    need_gpu()
    import state_space_model_amd as ssd
    Bt, T, D, K, io, dyt, has_state = case
    announce(f"conv1d_backward {case}")
    g = gen(300 + RUNS.index(case))
    x, dy = randn(g, Bt, T, D, io=io), randn(g, Bt, T, D, io=dyt)
    w, bias = torch.rand(D, K, generator=g) - 0.5, torch.rand(D, generator=g) - 0.5
    st, dso = ((randn(g, Bt, D, K - 1, io=io) for _ in range(2)) if has_state else (None, None))
    got = ssd.ssd_conv1d_backward(dev(x), dev(w), dev(bias), dy=dev(dy), state=dev(st),
                                  dstate_out=dev(dso))
    # 512 channels at a time: they do not meet, and float64 on the host stays small
    for c0 in range(0, D, 512):
        c = slice(c0, min(c0 + 512, D))
        part = {"dx": got["dx"][..., c], "dstate": got["dstate"][:, c], "dweight": got["dweight"][c],
                "dbias": got["dbias"][c]}
        n64 = lambda t: None if t is None else f64(t[:, c])
        check(part, f64(x[..., c]), f64(w[c]), f64(bias[c]), f64(dy[..., c]), n64(st), n64(dso), io)


def check(got, x, w, bias, dy, st, dso, io):
    (Bt, T, D), K = x.shape, w.shape[1]
    ref = block.conv1d_backward(x, w, bias, dy, st, dso, True)
    z, xa, w = ref["z"], np.abs(ref["xp"]), np.abs(w)
    zmag = np.abs(bias) + sum(w[:, i] * xa[:, i:i + T] for i in range(K))
    s = block.logistic(z)
    # |dz| error: the slope's own, and the slope's change with z's error
    dz_err = np.abs(dy) * (2 * silu_bar(z) + 8 * U * s * (1 + np.abs(z)) + K * U * zmag)
    dz = np.abs(ref["dz"])
    bar, dw_bar = np.zeros_like(xa), np.zeros_like(w)
    for i in range(K):
        bar[:, i:i + T] += w[:, i] * (dz_err + (K + 2) * U * dz)
        dw_bar[:, i] = (xa[:, i:i + T] * (dz_err + sum_u(Bt * T) * dz)).sum((0, 1))
    if dso is not None:
        bar[:, T:] += 2 * U * np.abs(dso).transpose(0, 2, 1)
    close(got["dx"], ref["dx"], 2 * bar[:, K - 1:] + io_u(io) * 1.01 * np.abs(ref["dx"]), "dx")
    close(got["dstate"], ref["dstate"], 2 * bar[:, :K - 1].transpose(0, 2, 1) +
          io_u(io) * 1.01 * np.abs(ref["dstate"]), "dstate")
    close(got["dweight"], ref["dweight"], dw_bar, "dweight")
    close(got["dbias"], ref["dbias"], (dz_err + sum_u(Bt * T) * dz).sum((0, 1)), "dbias")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("m,n", [(4352, 10752), (4099, 10560)])
def test_linear_q8_of_two_column_steps(m, n, io):
    """256 columns: a persistent workgroup's next tile is requested while the
    first step of the present one is multiplied.  Whole lines of outputs, with
    whole and cut tiles."""
    linear_q8_large(m, n, 256, io)
