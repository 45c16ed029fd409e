"""GPU parity of the operators between two scans (norms and their gradients,
8-bit rows and their product, the convolution's gradients) against their
float64 definitions (oracle.block).

Bars, with u = 2^-24 (float32) and every reference magnitude taken before any
cancellation:
  - a float32 sum of n terms in lanes and trees: (n / 64 + 32) u times the sum
    of the terms' magnitudes (64 partial sums at least, each a chain);
  - a mean square over d columns therefore moves 1/rms by half of that
    relatively; a product adds u per factor: norm_u(d) below;
  - silu and its slope on the hardware exponential and reciprocal: (16 + |z|) u
    of s (1 + |z|) (the exponent -z log2 e is rounded before 2^x);
  - the final rounding to bfloat16 (8 significant bits): 2^-8 of the value, to
    float32: u;
  - q8: rounding to an integer may differ from the float64 one by a whole step
    only where the float64 quotient lies within its error of a half.
"""
import numpy as np
import pytest
import torch

from gpu_util import announce, need_gpu
from oracle import block
from oracle.block import f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def norm_u(d):
    return (d / 128 + 32) * U


def io_u(io):
    return 2.0 ** -8 if io == "bf16" else U


def sum_u(n):
    return (n / 16 + 96) * U


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, io="f32"):
    return torch.randn(*shape, generator=g).to(DT[io])


def close(got, ref, bar, what):
    g = f64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert np.isfinite(g).all(), what
    bad = np.abs(g - ref) > bar + 1e-30
    assert not bad.any(), (what, int(bad.sum()), float((np.abs(g - ref) / (bar + 1e-30)).max()))


def dev(t):
    return None if t is None else t.to("cuda")


# widths: one column, below and above a lane group, odd, not multiples of the
# vectors, the package's, the widest
WIDTHS = [1, 3, 8, 63, 64, 130, 255, 256, 257, 768, 1000, 1025, 2048, 2560, 4099, 5120, 8200, 16383,
          16384]


# --------------------------------------------------------------------------
# add norm
# --------------------------------------------------------------------------
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", WIDTHS)
def test_add_norm(d, io):
    need_gpu()
    import state_space_model_amd as ssd
    g = gen(d)
    rows, s = (7 if d > 4096 else 33), 0.5
    x, r, w = randn(g, rows, d, io=io), 3 * randn(g, rows, d), 1 + 0.1 * randn(g, d)
    announce(f"add_norm {io} {rows}x{d}")
    for residual in (r, None):
        y, ro = ssd.ssd_add_norm(dev(x), dev(w), dev(residual), scale=s, eps=EPS)
        res64 = None if residual is None else f64(residual)
        ref, ref_r = block.add_norm(f64(x), f64(w), res64, s, EPS)
        mag = np.abs(s * f64(x)) + (0 if residual is None else np.abs(f64(r)))
        c = np.abs(1 / np.sqrt((ref_r ** 2).mean(-1, keepdims=True) + EPS) * f64(w))
        close(ro, ref_r, 2 * U * mag, "residual_out")
        close(y, ref, norm_u(d) * mag * c + io_u(io) * 1.01 * np.abs(ref), "y")
    # in place, over leading dimensions: the same bits
    y3, ro3 = ssd.ssd_add_norm(dev(x).view(1, rows, d), dev(w), scale=s, eps=EPS,
                               residual=(rr := dev(r).view(1, rows, d)), residual_out=rr)
    y2, ro2 = ssd.ssd_add_norm(dev(x), dev(w), dev(r), scale=s, eps=EPS)
    assert ro3 is rr and torch.equal(ro3[0], ro2) and torch.equal(y3[0], y2)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d", [(1, 1), (1, 2560), (2, 63), (33, 256), (300, 768), (1030, 130),
                                    (70, 2048), (40, 4099), (3, 8200), (5, 16384)])
def test_add_norm_backward(rows, d, io):
    need_gpu()
    import state_space_model_amd as ssd
    g = gen(rows + d)
    r, w = 2 * randn(g, rows, d), 1 + 0.1 * randn(g, d)
    dy, dro = randn(g, rows, d, io=io), randn(g, rows, d)
    announce(f"add_norm_backward {io} {rows}x{d}")
    for dres_out in (dro, None):
        got = ssd.ssd_add_norm_backward(dev(r), dev(w), dy=dev(dy), dresidual_out=dev(dres_out),
                                        scale=0.25, eps=EPS)
        ref = block.add_norm_backward(f64(r), f64(w), f64(dy),
                                      None if dres_out is None else f64(dro), 0.25, EPS)
        c = 1 / np.sqrt((f64(r) ** 2).mean(-1, keepdims=True) + EPS)
        p, xh = np.abs(f64(dy) * f64(w)), np.abs(f64(r) * c)
        mag = c * (p + xh * (p * xh).mean(-1, keepdims=True))
        mag = mag + (0 if dres_out is None else np.abs(f64(dro)))
        close(got["dresidual"], ref["dresidual"], 4 * norm_u(d) * mag, "dresidual")
        close(got["dx"], ref["dx"], norm_u(d) * mag + io_u(io) * 1.01 * np.abs(ref["dx"]), "dx")
        close(got["dweight"], ref["dweight"],
              (sum_u(rows) + norm_u(d)) * np.abs(f64(dy) * xh).sum(0), "dweight")
    # the residual's gradient in place; runs repeat bit for bit
    buf = dev(dro)
    again = ssd.ssd_add_norm_backward(dev(r), dev(w), dy=dev(dy), dresidual_out=buf, scale=0.25,
                                      eps=EPS, grads={"dresidual": buf})
    first = ssd.ssd_add_norm_backward(dev(r), dev(w), dy=dev(dy), dresidual_out=dev(dro),
                                      scale=0.25, eps=EPS)
    for k in first:
        assert torch.equal(first[k], again[k]), k


# --------------------------------------------------------------------------
# gated norm
# --------------------------------------------------------------------------
GATED = [(1, 1, 1, 0), (5, 3, 3, 2), (33, 64, 1, 7), (17, 130, 2, 0), (9, 768, 8, 1), (21, 1000, 1, 24),
         (12, 1536, 1, 280), (6, 4099, 1, 0), (40, 4096, 8, 1), (8, 5120, 1, 5456), (10, 5120, 4, 0),
         (3, 8200, 1, 3), (4, 16384, 2, 0), (2, 40000, 4, 8)]


def gated_case(rows, d, io, seed, zpad):
    g = gen(seed)
    y, w = randn(g, rows, d, io=io), 1 + 0.1 * randn(g, d)
    z = (3 * torch.randn(rows, d + zpad, generator=g)).to(DT[io])
    return g, y, w, z


def silu_bar(z):
    s = block.logistic(z)
    return (16 + np.abs(z)) * U * s * (1 + np.abs(z))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d,groups,zpad", GATED)
def test_gated_norm(rows, d, groups, zpad, io):
    need_gpu()
    import state_space_model_amd as ssd
    _, y, w, zf = gated_case(rows, d, io, d + rows, zpad)
    z = dev(zf)[:, zpad // 2:zpad // 2 + d]       # a slice of columns, off the vectors
    announce(f"gated_norm {io} {rows}x{d} groups {groups} zpad {zpad}")
    out = ssd.ssd_gated_norm(dev(y), z, dev(w), groups=groups, eps=EPS)
    y64, z64, w64 = f64(y), f64(z), f64(w)
    ref = block.gated_norm(y64, z64, w64, EPS, groups)
    width = d // groups
    gate = np.abs(y64) * (np.abs(block.silu(z64)) + silu_bar(z64) / U * 0)
    v = (y64 * block.silu(z64)).reshape(rows, groups, width)
    dv = (np.abs(y64) * silu_bar(z64)).reshape(rows, groups, width)
    ms = (v * v).mean(-1, keepdims=True) + EPS
    c = 1 / np.sqrt(ms)
    # the mean square's own error: of its sum, and of each g
    rel = norm_u(width) + (np.abs(v) * dv).mean(-1, keepdims=True) / ms
    bar = (c * (dv + rel * np.abs(v))).reshape(rows, d) * np.abs(w64)
    close(out, ref, bar + io_u(io) * 1.01 * np.abs(ref) + 4 * U * np.abs(ref), "out")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d,groups,zpad", GATED + [(515, 96, 1, 0), (1500, 64, 2, 3)])
def test_gated_norm_backward(rows, d, groups, zpad, io):
    need_gpu()
    import state_space_model_amd as ssd
    g, y, w, zf = gated_case(rows, d, io, 2 * d + rows, zpad)
    dout = randn(g, rows, d, io=io)
    z = dev(zf)[:, zpad // 2:zpad // 2 + d]
    # dz into a slice of a larger buffer whose other columns must stay
    dzf = torch.full((rows, d + zpad), 7.0, device="cuda", dtype=DT[io])
    dz = dzf[:, zpad // 2:zpad // 2 + d]
    announce(f"gated_norm_backward {io} {rows}x{d} groups {groups} zpad {zpad}")
    got = ssd.ssd_gated_norm_backward(dev(y), z, dev(w), dout=dev(dout), groups=groups, eps=EPS,
                                      grads={"dz": dz})
    y64, z64, w64, d64 = f64(y), f64(z), f64(w), f64(dout)
    ref = block.gated_norm_backward(y64, z64, w64, d64, EPS, groups)
    width = d // groups
    s = block.logistic(z64)
    act = np.abs(block.silu(z64))
    gv = (y64 * block.silu(z64)).reshape(rows, groups, width)
    dgv = (np.abs(y64) * silu_bar(z64)).reshape(rows, groups, width)
    ms = (gv * gv).mean(-1, keepdims=True) + EPS
    c = 1 / np.sqrt(ms)
    rel = 3 * norm_u(width) + 3 * (np.abs(gv) * dgv).mean(-1, keepdims=True) / ms
    p = np.abs(d64 * w64).reshape(gv.shape)
    gh, dgh = np.abs(gv) * c, dgv * c
    mean = (p * gh).mean(-1, keepdims=True)
    mag = (c * (p + gh * mean)).reshape(rows, d)
    err = (c * (dgh * mean + gh * (p * dgh).mean(-1, keepdims=True)) +
           rel * c * (p + 2 * gh * mean)).reshape(rows, d)
    sb = silu_bar(z64)
    slope = s * (1 + np.abs(z64) * (1 - s))
    close(got["dy"], ref["dy"], err * act + mag * sb + 4 * U * mag * act +
          io_u(io) * 1.01 * np.abs(ref["dy"]), "dy")
    close(dz, ref["dz"], np.abs(y64) * (err * slope + 2 * mag * (sb + 4 * U * slope)) +
          io_u(io) * 1.01 * np.abs(ref["dz"]), "dz")
    ghm = gh.reshape(rows, d)
    close(got["dweight"], ref["dweight"],
          (np.abs(d64) * ((dgh + rel * gh).reshape(rows, d) + sum_u(rows) * ghm)).sum(0), "dweight")
    if zpad:
        keep = torch.ones(d + zpad, dtype=torch.bool)
        keep[zpad // 2:zpad // 2 + d] = False
        assert (dzf[:, keep.cuda()] == 7.0).all()
    again = ssd.ssd_gated_norm_backward(dev(y), z, dev(w), dout=dev(dout), groups=groups, eps=EPS)
    for k in ("dy", "dz", "dweight"):
        assert torch.equal(again[k], got[k]), k


def test_gradients_against_differences_of_the_forward():
    """Central differences of the float64 forward along a random direction
    against the kernels' float32 gradients: both agree to float32 rounding of
    sums of |gradient * direction|."""
    need_gpu()
    import state_space_model_amd as ssd
    announce("gradients against differences")
    rng = np.random.default_rng(3)
    rows, d, h = 19, 300, 1e-5
    y, z = rng.standard_normal((rows, d)).astype(np.float32), rng.standard_normal((rows, d)).astype(np.float32)
    w, dout = (1 + 0.1 * rng.standard_normal(d)).astype(np.float32), rng.standard_normal((rows, d)).astype(np.float32)
    t = {k: torch.from_numpy(v).cuda() for k, v in dict(y=y, z=z, w=w, dout=dout).items()}
    got = ssd.ssd_gated_norm_backward(t["y"], t["z"], t["w"], dout=t["dout"], groups=3, eps=EPS)
    base = dict(y=y.astype(np.float64), z=z.astype(np.float64), weight=w.astype(np.float64))
    loss = lambda **a: (dout * block.gated_norm(**a, eps=EPS, groups=3)).sum()
    for name, key in (("y", "dy"), ("z", "dz"), ("weight", "dweight")):
        v = rng.standard_normal(base[name].shape)
        hi, lo = dict(base), dict(base)
        hi[name], lo[name] = base[name] + h * v, base[name] - h * v
        num = (loss(**hi) - loss(**lo)) / (2 * h)
        g64 = f64(got[key])
        assert abs(num - (g64 * v).sum()) <= (64 * U + 1e-8) * (np.abs(g64 * v).sum() + 1), name


# --------------------------------------------------------------------------
# 8-bit rows
# --------------------------------------------------------------------------
def check_q8(q, qscale, ref, bar, k):
    """q against the float64 values `ref` (known to +-bar before quantising)."""
    kp = (k + 127) // 128 * 128
    assert q.shape == (*ref.shape[:-1], kp) and q.dtype == torch.int8
    q64, s64 = f64(q), f64(qscale)
    assert not q64[..., k:].any()
    assert np.abs(q64).max() <= 127
    amax = np.abs(ref).max(-1)
    rel = (bar / np.where(amax > 0, amax, 1)[..., None]).max(-1)
    assert (np.abs(s64 - amax / 127) <= (rel + 4 * U) * amax / 127 + 1e-37).all()
    quot = ref / np.where(amax > 0, amax, 1)[..., None] * 127
    slack = (bar / np.where(amax > 0, amax, 1)[..., None] + rel[..., None] + 4 * U) * 127
    assert (np.abs(q64[..., :k] - quot) <= 0.5 + slack).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,k", [(1, 1), (3, 7), (9, 128), (5, 129), (40, 768), (7, 2560), (2, 5121),
                                    (2, 20000), (1, 130944)])
def test_quantize_q8(rows, k, io):
    need_gpu()
    import state_space_model_amd as ssd
    v = randn(gen(k), rows, k, io=io) * (1 + torch.arange(rows)[:, None]).to(DT[io])
    announce(f"quantize_q8 {io} {rows}x{k}")
    q, s = ssd.ssd_quantize_q8(dev(v))
    check_q8(q, s, f64(v), np.zeros((rows, k)), k)


def test_quantize_q8_rows_without_a_scale():
    """Zero rows, rows below 2^-100, the smallest kept row, the largest finite
    one, and rows with an infinity or a NaN anywhere."""
    need_gpu()
    import state_space_model_amd as ssd
    announce("quantize_q8 special rows")
    k = 300
    v = torch.zeros(9, k)
    v[1] = 2.0 ** -101
    v[2] = 2.0 ** -100
    v[3, 7] = torch.finfo(torch.float32).max
    v[4] = 1.0
    v[4, 299] = float("inf")
    v[5, 0] = float("-inf")
    v[6] = 1.0
    v[6, 150] = float("nan")
    v[7, 5] = -3.0
    v[8, 3] = 2.0 ** -149
    q, s = ssd.ssd_quantize_q8(dev(v))
    q, s = q.cpu(), s.cpu()
    for row in (0, 1, 8):
        assert not q[row].any() and s[row] == 0
    assert (q[2, :k] == 127).all() and s[2] > 0
    assert q[3, 7] == 127 and q[3].count_nonzero() == 1 and torch.isfinite(s[3])
    for row in (4, 5, 6):
        assert not q[row].any() and torch.isnan(s[row])
    assert q[7, 5] == -127 and abs(float(s[7]) - 3 / 127) < 1e-8
    # and what a product makes of them
    wq, ws = ssd.ssd_quantize_q8(torch.ones(5, k, device="cuda"))
    out = ssd.ssd_linear_q8(q.cuda(), s.cuda(), wq, ws, out_dtype=torch.float32).cpu()
    # (row 3 stands for 127 (max / 127), which rounds past the largest float)
    assert torch.isnan(out[4:7]).all() and torch.isfinite(out[[0, 1, 2, 7, 8]]).all()
    assert not out[0].any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d", [(1, 5), (3, 128), (33, 768), (1, 2560), (6, 4099), (3, 16384)])
def test_add_norm_q8(rows, d, io):
    need_gpu()
    import state_space_model_amd as ssd
    g = gen(d)
    x, r, w = randn(g, rows, d, io=io), 3 * randn(g, rows, d), 1 + 0.1 * randn(g, d)
    announce(f"add_norm_q8 {io} {rows}x{d}")
    q, s, ro = ssd.ssd_add_norm_q8(dev(x), dev(w), dev(r), scale=0.5, eps=EPS)
    ref, ref_r = block.add_norm(f64(x), f64(w), f64(r), 0.5, EPS)
    mag = np.abs(0.5 * f64(x)) + np.abs(f64(r))
    c = np.abs(1 / np.sqrt((ref_r ** 2).mean(-1, keepdims=True) + EPS) * f64(w))
    check_q8(q, s, ref, norm_u(d) * mag * c, d)
    _, ro2 = ssd.ssd_add_norm(dev(x), dev(w), dev(r), scale=0.5, eps=EPS)
    assert torch.equal(ro, ro2)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d,groups", [(1, 5, 1), (5, 96, 3), (33, 1536, 1), (4, 5120, 1), (7, 4096, 8),
                                           (2, 1000, 8), (2, 16384, 2), (1, 6000, 1000)])
def test_gated_norm_q8(rows, d, groups, io):
    need_gpu()
    import state_space_model_amd as ssd
    _, y, w, z = gated_case(rows, d, io, d, 0)
    announce(f"gated_norm_q8 {io} {rows}x{d} groups {groups}")
    q, s = ssd.ssd_gated_norm_q8(dev(y), dev(z), dev(w), groups=groups, eps=EPS)
    y64, z64, w64 = f64(y), f64(z), f64(w)
    ref = block.gated_norm(y64, z64, w64, EPS, groups)
    width = d // groups
    v = (y64 * block.silu(z64)).reshape(rows, groups, width)
    dv = (np.abs(y64) * silu_bar(z64)).reshape(rows, groups, width)
    ms = (v * v).mean(-1, keepdims=True) + EPS
    rel = norm_u(width) + (np.abs(v) * dv).mean(-1, keepdims=True) / ms
    bar = ((dv + rel * np.abs(v)) / np.sqrt(ms)).reshape(rows, d) * np.abs(w64)
    check_q8(q, s, ref, bar, d)


# --------------------------------------------------------------------------
# product of 8-bit rows
# --------------------------------------------------------------------------
LINEAR = [(1, 1, 128), (1, 16, 128), (1, 10576, 2560), (2, 33, 256), (7, 257, 384), (16, 2560, 5120),
          (17, 80, 1024), (31, 1003, 896), (33, 64, 128), (64, 2560, 1536), (65, 300, 2560),
          (100, 129, 640), (128, 128, 128), (200, 515, 768), (255, 257, 384), (256, 256, 512),
          (300, 1000, 1152), (513, 770, 640), (1000, 2561, 256), (2049, 300, 128)]


def ints(g, *shape):
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int32).to(torch.int8)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", LINEAR)
def test_linear_q8(m, n, k, io):
    """Every 8-bit value, -128 included: the integer sum is exact, so only the
    two scalings (and the conversion of sums beyond 2^24) round."""
    need_gpu()
    import state_space_model_amd as ssd
    g = gen(m + n + k)
    q, wq = ints(g, m, k), ints(g, n, k)
    qs, ws = torch.rand(m, generator=g) + 0.01, torch.rand(n, generator=g) + 0.01
    announce(f"linear_q8 {io} {m}x{n}x{k}")
    out = ssd.ssd_linear_q8(dev(q), dev(qs), dev(wq), dev(ws), out_dtype=DT[io])
    ref = (f64(q) @ f64(wq).T) * f64(qs)[:, None] * f64(ws)       # sums below 2^53: exact
    close(out, ref, (4 * U + (io_u(io) * 1.01 if io == "bf16" else 0)) * np.abs(ref), "out")


# tiles of 256 tokens and 160 to 256 outputs, more of them than compute units, with
# whole and cut ones, whole and cut lines
LINEAR_LARGE = [(4000, 2400, 2560), (2600, 4099, 640), (1500, 9000, 640), (4100, 10570, 512),
                (4352, 5376, 384), (4097, 2560, 1280)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", LINEAR_LARGE)
def test_linear_q8_large(m, n, k, io):
    """As test_linear_q8, the exact sums formed in float64 on the GPU; a second
    call gives the same bits."""
    need_gpu()
    import state_space_model_amd as ssd
    g = gen(m + n + k)
    q, wq = dev(ints(g, m, k)), dev(ints(g, n, k))
    qs, ws = dev(torch.rand(m, generator=g) + 0.01), dev(torch.rand(n, generator=g) + 0.01)
    announce(f"linear_q8 large {io} {m}x{n}x{k}")
    out = ssd.ssd_linear_q8(q, qs, wq, ws, out_dtype=DT[io])
    ref = (q.double() @ wq.double().t().contiguous()) * qs.double()[:, None] * ws.double()
    bar = (4 * U + (io_u(io) * 1.01 if io == "bf16" else 0)) * ref.abs()
    bad = (out.double() - ref).abs() > bar
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
    assert torch.equal(out, ssd.ssd_linear_q8(q, qs, wq, ws, out_dtype=DT[io]))


def test_linear_q8_extreme_sum():
    """The widest rows of -128 reach 2^31 - 2^21 without overflow."""
    need_gpu()
    import state_space_model_amd as ssd
    announce("linear_q8 extreme sum")
    k = 130944
    q = torch.full((3, k), -128, dtype=torch.int8, device="cuda")
    q[1] = 127
    one = torch.ones(3, device="cuda")
    wq = torch.full((40, k), -128, dtype=torch.int8, device="cuda")
    out = ssd.ssd_linear_q8(q, one, wq, torch.ones(40, device="cuda"), out_dtype=torch.float32)
    want = torch.tensor([16384.0 * k, -128.0 * 127 * k, 16384.0 * k]).double()
    assert ((out.cpu().double() - want[:, None]).abs() <= 2 * U * want.abs()[:, None]).all()


def test_linear_q8_rows_do_not_depend_on_the_batch():
    need_gpu()
    import state_space_model_amd as ssd
    g = gen(4)
    q, wq = dev(ints(g, 700, 640)), dev(ints(g, 500, 640))
    qs, ws = dev(torch.rand(700, generator=g)), dev(torch.rand(500, generator=g))
    announce("linear_q8 batch invariance")
    full = ssd.ssd_linear_q8(q, qs, wq, ws, out_dtype=torch.float32)
    for rows in (1, 5, 16, 40, 100, 300):
        part = ssd.ssd_linear_q8(q[:rows].contiguous(), qs[:rows].contiguous(), wq, ws,
                                 out_dtype=torch.float32)
        assert torch.equal(part, full[:rows]), rows


def test_offsets_beyond_32_bits():
    """Outputs and inputs of more than 2^32 bytes: the last rows equal a small
    call on those rows alone."""
    need_gpu()
    import state_space_model_amd as ssd
    g = torch.Generator(device="cuda").manual_seed(5)
    announce("offsets beyond 32 bits: linear_q8 70001 x 40000 x 128")
    q = torch.randint(-128, 128, (70001, 128), generator=g, device="cuda").to(torch.int8)
    wq = torch.randint(-128, 128, (40000, 128), generator=g, device="cuda").to(torch.int8)
    qs, ws = torch.rand(70001, generator=g, device="cuda"), torch.rand(40000, generator=g, device="cuda")
    out = ssd.ssd_linear_q8(q, qs, wq, ws)
    tail = ssd.ssd_linear_q8(q[-3:].contiguous(), qs[-3:].contiguous(), wq, ws)
    assert torch.equal(out[-3:], tail)
    assert torch.equal(out[:3], ssd.ssd_linear_q8(q[:3].contiguous(), qs[:3].contiguous(), wq, ws))
    del out, tail, q, wq
    rows, d = 300000, 8192
    announce(f"offsets beyond 32 bits: norms {rows}x{d}")
    x = torch.randn(rows, d, generator=g, device="cuda").bfloat16()
    w = torch.rand(d, generator=g, device="cuda")
    y, ro = ssd.ssd_add_norm(x, w, scale=0.5)
    y1, ro1 = ssd.ssd_add_norm(x[-2:].contiguous(), w, scale=0.5)
    assert torch.equal(y[-2:], y1) and torch.equal(ro[-2:], ro1)
    del ro, ro1
    o = ssd.ssd_gated_norm(x, y, w, groups=2)
    o1 = ssd.ssd_gated_norm(x[-2:].contiguous(), y[-2:].contiguous(), w, groups=2)
    assert torch.equal(o[-2:], o1)
    gr = ssd.ssd_gated_norm_backward(x, y, w, dout=o, groups=2)
    g1 = ssd.ssd_gated_norm_backward(x[-2:].contiguous(), y[-2:].contiguous(), w,
                                     dout=o[-2:].contiguous(), groups=2)
    assert torch.equal(gr["dy"][-2:], g1["dy"]) and torch.equal(gr["dz"][-2:], g1["dz"])


def test_more_rows_than_one_grid_holds():
    """2^21 + 3 rows: the rows past the first launch's equal a small call."""
    need_gpu()
    import state_space_model_amd as ssd
    announce("rows beyond one launch")
    g = torch.Generator(device="cuda").manual_seed(6)
    rows, d = (1 << 21) + 3, 64
    x = torch.randn(rows, d, generator=g, device="cuda").bfloat16()
    r = torch.randn(rows, d, generator=g, device="cuda")
    zf = torch.randn(rows, d + 6, generator=g, device="cuda").bfloat16()
    w = torch.rand(d, generator=g, device="cuda")
    tail = slice(rows - 5, rows)
    t = lambda v: v[tail].contiguous()
    for full, part in ((ssd.ssd_add_norm(x, w, r), ssd.ssd_add_norm(t(x), w, t(r))),
                       (ssd.ssd_add_norm_q8(x, w, r), ssd.ssd_add_norm_q8(t(x), w, t(r))),
                       ([ssd.ssd_gated_norm(x, zf[:, :d], w, groups=2)],
                        [ssd.ssd_gated_norm(t(x), zf[tail, :d], w, groups=2)]),
                       (ssd.ssd_gated_norm_q8(x, zf[:, :d], w, groups=2),
                        ssd.ssd_gated_norm_q8(t(x), zf[tail, :d], w, groups=2)),
                       (ssd.ssd_quantize_q8(x), ssd.ssd_quantize_q8(t(x)))):
        for a, b in zip(full, part):
            assert torch.equal(a[tail], b)


# --------------------------------------------------------------------------
# convolution gradients
# --------------------------------------------------------------------------
CONV = [
    # (Bt, T, D, k, io, dy, state, dstate_out, bias, silu)
    (1, 1, 1, 4, "f32", "f32", True, True, True, True),
    (2, 2, 5, 4, "f32", "f32", True, True, True, True),
    (2, 3, 8, 4, "bf16", "f32", True, True, True, True),
    (1, 17, 12, 4, "f32", "f32", False, False, True, True),
    (3, 33, 40, 3, "f32", "f32", True, False, False, True),
    (2, 64, 13, 2, "f32", "f32", False, True, True, False),
    (1, 129, 256, 4, "bf16", "bf16", True, True, True, True),
    (2, 257, 100, 4, "bf16", "f32", False, False, True, True),
    (4, 75, 259, 3, "bf16", "f32", True, True, True, True),
    (1, 1000, 64, 4, "f32", "f32", True, True, True, True),
    (5, 300, 516, 4, "bf16", "bf16", False, True, False, True),
    (1, 2111, 36, 2, "bf16", "f32", True, True, True, True),
    (70, 5, 6, 4, "f32", "f32", True, True, True, True),
]


@pytest.mark.parametrize("case", CONV, ids=lambda c: "_".join(map(str, c)))
def test_conv1d_backward(case):
    need_gpu()
    import state_space_model_amd as ssd
    Bt, T, D, K, io, dyt, has_state, has_dso, has_bias, silu = case
    g = gen(100 + CONV.index(case))
    x, dy = randn(g, Bt, T, D, io=io), randn(g, Bt, T, D, io=dyt)
    w, bias = torch.rand(D, K, generator=g) - 0.5, torch.rand(D, generator=g) - 0.5
    st = randn(g, Bt, D, K - 1, io=io) if has_state else None
    dso = randn(g, Bt, D, K - 1, io=io) if has_dso else None
    bias = bias if has_bias else None
    announce(f"conv1d_backward {case}")
    run = lambda: ssd.ssd_conv1d_backward(dev(x), dev(w), dev(bias), dy=dev(dy), state=dev(st),
                                          dstate_out=dev(dso), silu=silu)
    got = run()
    n64 = lambda t: None if t is None else f64(t)
    ref = block.conv1d_backward(f64(x), f64(w), n64(bias), f64(dy), n64(st), n64(dso), silu)
    # |dz| error: the slope's own, and the slope's change with z's error
    z, dy64, w64 = ref["z"], np.abs(f64(dy)), np.abs(f64(w))
    xa = np.abs(ref["xp"])
    zmag = (0 if bias is None else np.abs(f64(bias))) + sum(w64[:, i] * xa[:, i:i + T] for i in range(K))
    if silu:
        s = block.logistic(z)
        dz_err = dy64 * (2 * silu_bar(z) + 8 * U * s * (1 + np.abs(z)) + K * U * zmag)
    else:
        dz_err = 0 * dy64
    dz = np.abs(ref["dz"])
    bar = np.zeros_like(ref["xp"])
    dw_bar, terms = np.zeros_like(w64), (Bt * T)
    for i in range(K):
        bar[:, i:i + T] += w64[:, i] * (dz_err + (K + 2) * U * dz)
        dw_bar[:, i] = (xa[:, i:i + T] * (dz_err + sum_u(terms) * dz)).sum((0, 1))
    if dso is not None:
        bar[:, T:] += 2 * U * np.abs(f64(dso)).transpose(0, 2, 1)
    close(got["dx"], ref["dx"], 2 * bar[:, K - 1:] + io_u(io) * 1.01 * np.abs(ref["dx"]), "dx")
    close(got["dstate"], ref["dstate"], 2 * bar[:, :K - 1].transpose(0, 2, 1) +
          io_u(io) * 1.01 * np.abs(ref["dstate"]), "dstate")
    close(got["dweight"], ref["dweight"], dw_bar, "dweight")
    close(got["dbias"], ref["dbias"], (dz_err + sum_u(terms) * dz).sum((0, 1)), "dbias")
    again = run()
    for k in got:
        assert torch.equal(got[k], again[k]), k


# --------------------------------------------------------------------------
# empty problems, streams, graphs
# --------------------------------------------------------------------------
def test_empty_problems():
    need_gpu()
    import state_space_model_amd as ssd
    announce("empty problems")
    c = dict(device="cuda")
    w = torch.ones(24, **c)
    y, ro = ssd.ssd_add_norm(torch.empty(0, 24, **c), w)
    assert y.shape == (0, 24) and ro.shape == (0, 24)
    q, s = ssd.ssd_gated_norm_q8(torch.empty(0, 24, **c), torch.empty(0, 24, **c), w)
    assert q.shape == (0, 128) and s.shape == (0,)
    out = ssd.ssd_linear_q8(q, s, torch.zeros(5, 128, dtype=torch.int8, **c), torch.ones(5, **c))
    assert out.shape == (0, 5)
    dirty = torch.full((24,), 9.0, **c)
    ssd.ssd_add_norm_backward(torch.empty(0, 24, **c), w, dy=torch.empty(0, 24, **c),
                              grads={"dweight": dirty})
    assert not dirty.any()
    dirty = torch.full((24,), 9.0, **c)
    ssd.ssd_gated_norm_backward(torch.empty(0, 24, **c), torch.empty(0, 24, **c), w,
                                dout=torch.empty(0, 24, **c), grads={"dweight": dirty})
    assert not dirty.any()
    # an empty sequence hands the window's gradient on
    dso = torch.randn(2, 24, 3, **c)
    g = ssd.ssd_conv1d_backward(torch.empty(2, 0, 24, **c), torch.ones(24, 4, **c),
                                dy=torch.empty(2, 0, 24, **c), dstate_out=dso)
    assert torch.equal(g["dstate"], dso) and not g["dweight"].any() and not g["dbias"].any()
    g = ssd.ssd_conv1d_backward(torch.empty(2, 0, 24, **c), torch.ones(24, 4, **c),
                                dy=torch.empty(2, 0, 24, **c))
    assert not g["dstate"].any()
    g = ssd.ssd_conv1d_backward(torch.empty(0, 6, 24, **c), torch.ones(24, 4, **c),
                                dy=torch.empty(0, 6, 24, **c))
    assert not g["dweight"].any() and not g["dbias"].any()


def test_non_finite_rows_stay_in_their_rows():
    """A NaN or an infinity in one token reaches that token's outputs only (and
    the weight's gradient)."""
    need_gpu()
    import state_space_model_amd as ssd
    announce("non-finite rows")
    g = gen(8)
    x, w = randn(g, 5, 700), 1 + 0.1 * randn(g, 700)
    x[2, 13] = float("nan")
    x[4, 699] = float("inf")
    y, ro = ssd.ssd_add_norm(dev(x), dev(w))
    assert torch.isnan(y[2]).all() and torch.isnan(y[4, 699])
    assert torch.isfinite(y[[0, 1, 3]]).all() and torch.isfinite(ro[:, :13]).all()
    q, s, _ = ssd.ssd_add_norm_q8(dev(x), dev(w))
    assert torch.isnan(s[[2, 4]]).all() and torch.isfinite(s[[0, 1, 3]]).all()
    q, s = ssd.ssd_gated_norm_q8(dev(x), torch.ones(5, 700, device="cuda"), dev(w), groups=7)
    assert torch.isnan(s[[2, 4]]).all() and torch.isfinite(s[[0, 1, 3]]).all()
    # the gate's far ends: silu(-inf) -> -0, silu(large) -> z
    z = torch.full((5, 700), -200.0)
    z[1] = 200.0
    z[3] = -3e38
    out = ssd.ssd_gated_norm(torch.ones(5, 700, device="cuda"), dev(z), dev(w))
    assert torch.isfinite(out).all() and not out[3].any()
    gr = ssd.ssd_gated_norm_backward(torch.ones(5, 700, device="cuda"), dev(z), dev(w),
                                     dout=torch.ones(5, 700, device="cuda"))
    assert torch.isfinite(gr["dy"]).all() and torch.isfinite(gr["dz"]).all()


def test_side_stream_and_graph_replay():
    """Calls on another stream than the tensors', and captured in a HIP graph
    replayed between eager work, give the eager bits."""
    need_gpu()
    import state_space_model_amd as ssd
    announce("side stream and graph")
    g = gen(9)
    x, w, r = dev(randn(g, 64, 768, io="bf16")), dev(1 + 0.1 * randn(g, 768)), dev(randn(g, 64, 768))
    wq, ws = ssd.ssd_quantize_q8(dev(randn(g, 100, 768)))
    dy = dev(randn(g, 64, 768, io="bf16"))
    z = dev(randn(g, 64, 768, io="bf16"))
    xs, cw = dev(randn(g, 2, 32, 768, io="bf16")), dev(randn(g, 768, 4))

    def work():
        q, s, ro = ssd.ssd_add_norm_q8(x, w, r)
        gn = ssd.ssd_gated_norm_backward(x, z, w, dout=dy)
        ab = ssd.ssd_add_norm_backward(ro, w, dy=dy, dresidual_out=r)
        cb = ssd.ssd_conv1d_backward(xs, cw, dy=xs)
        return [ssd.ssd_linear_q8(q, s, wq, ws), ro, *gn.values(), *ab.values(), *cb.values()]

    eager = work()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = work()
    torch.cuda.synchronize()
    for a, b in zip(eager, other):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for replay in range(4):
        for t in captured:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, captured):
            assert torch.equal(a, b), replay
        work()
        torch.cuda.synchronize()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [2, 63, 64, 65, 66, 127, 128, 129, 131, 192, 255, 256, 257])
def test_narrow_rows(d, io):
    """Rows of up to one wavefront's lanes, where a lane holds one, two or four
    columns: on both sides of each change, even and odd."""
    test_add_norm(d, io)
    test_add_norm_backward(37, d, io)
    test_add_norm_q8(9, d, io)
    test_gated_norm(33, 3 * d, 3, 5, io)
    test_gated_norm_backward(41, 2 * d, 2, 3, io)
    test_gated_norm_q8(9, d, 1, io)
    test_quantize_q8(9, d, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(33, 2560, 640), (40, 129, 128), (100, 3352, 768), (129, 2111, 384),
                                   (17, 1001, 4992), (150, 2533, 1024)])
def test_linear_q8_few_tiles(m, n, k, io):
    """Columns split over wavefronts and turned from workgroup to workgroup: up
    to one tile per compute unit and up to two, shares of none to ten steps."""
    test_linear_q8(m, n, k, io)


def test_calls_check_what_they_are_given():
    """Wrong types, layouts and buffers on the device are refused before any
    launch; a caller's buffers come back as they are; nothing is leaked."""
    need_gpu()
    import sys

    import state_space_model_amd as ssd
    announce("checks of the calls")
    c = dict(device="cuda")
    x, r, w = torch.randn(6, 40, **c), torch.randn(6, 40, **c), torch.ones(40, **c)
    for exc, f in (
            (TypeError, lambda: ssd.ssd_add_norm(x, w.bfloat16())),
            (TypeError, lambda: ssd.ssd_add_norm(x, w, r.bfloat16())),
            (ValueError, lambda: ssd.ssd_add_norm(x, w.cpu())),
            (ValueError, lambda: ssd.ssd_add_norm(torch.randn(40, 6, **c).t(), w)),
            (TypeError, lambda: ssd.ssd_gated_norm(x, r.bfloat16(), w)),
            (ValueError, lambda: ssd.ssd_gated_norm(x, torch.randn(40, 6, **c).t(), w)),
            (TypeError, lambda: ssd.ssd_add_norm_q8(x, w, q=torch.empty(6, 128, **c))),
            (TypeError, lambda: ssd.ssd_linear_q8(torch.empty(6, 128, **c), w[:6],
                                                  torch.empty(5, 128, **c, dtype=torch.int8), w[:5]))):
        with pytest.raises(exc):
            f()
    for status, f in (
            (5, lambda: ssd.ssd_add_norm(torch.zeros(2, 16385, **c), torch.ones(16385, **c))),
            (1, lambda: ssd.ssd_add_norm(x, w, r, y=x)),
            (1, lambda: ssd.ssd_add_norm(x, w, r, eps=-1.0)),
            (2, lambda: ssd.ssd_gated_norm(x, r, w, groups=3)),
            (6, lambda: ssd.ssd_add_norm_backward(
                torch.zeros(40, 40, **c), w, dy=torch.zeros(40, 40, **c),
                workspace=torch.empty(16, **c, dtype=torch.uint8)))):
        with pytest.raises(ssd.SSDError) as e:
            f()
        assert e.value.status == status
    dw = torch.empty(40, **c)
    out = torch.empty_like(x)
    assert ssd.ssd_gated_norm(x, r, w, out=out) is out
    assert ssd.ssd_gated_norm_backward(x, r, w, dout=x, grads={"dweight": dw})["dweight"] is dw

    def work():
        ssd.ssd_add_norm(x, w, r)
        ssd.ssd_linear_q8(*ssd.ssd_gated_norm_q8(x, r, w), *ssd.ssd_quantize_q8(x))
        ssd.ssd_gated_norm_backward(x, r, w, dout=x, grads={"dweight": dw})
        with pytest.raises(ssd.SSDError):
            ssd.ssd_add_norm(x, w, r, y=x)
    work()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated(), [sys.getrefcount(t) for t in (x, r, w, dw, ssd.SSDError)]
    for _ in range(50):
        work()
    torch.cuda.synchronize()
    assert before == (torch.cuda.memory_allocated(),
                      [sys.getrefcount(t) for t in (x, r, w, dw, ssd.SSDError)])
