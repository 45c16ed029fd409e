"""The operators between two scans of a Mamba-2 stack: what is measured of them.

A block reads a float32 residual stream, normalises it, projects it, convolves
it, scans it, normalises the scan's output with its gate and projects it back.
The scan and the convolution's forward pass are the library's already; the
cases here are the rest of that path, in serving and in training:

  add_norm          r' = r + scale x; y = r' / rms(r') * weight
  add_norm_grad     its gradients with respect to x, r and the weight
  gated_norm        g = y silu(z); out = g / rms(g over a group) * weight
  gated_norm_grad   its gradients with respect to y, z and the weight
  linear_q8         out[m, n] = sx[m] sw[n] sum_k qx[m, k] qw[n, k], 8-bit integers
  add_project_q8    add_norm with its output in 8 bits, then linear_q8
  gated_project_q8  gated_norm with its output in 8 bits, then linear_q8
  conv_grad         gradients of the depthwise causal convolution

A row v in 8 bits is q = round(v * 127 / max|v|) with scale max|v| / 127; its
columns are padded with zeros to a multiple of 128.  Sizes are those of the
package's workloads: widths 768 / 2048 / 2560 of the 130M, 1.3B and 2.7B
shapes, inner widths 1536 / 4096 / 5120, convolution channels 1792 / 5376, and
10576 = 2 * 5120 + 2 * 128 + 80 columns of the 2.7B shape's first projection.
"""
import math

import torch

own = False

EPS = 1e-5
PAD = 128


def _ssd():
    import state_space_model_amd as ssd
    return ssd


def _dtype(case):
    return torch.float32 if case["io"] == "f32" else torch.bfloat16


def _padded(k):
    return (k + PAD - 1) // PAD * PAD


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decoded token through the norm before a block (130M width): latency only
        dict(name="add_norm_step", op="add_norm", rows=1, d=768, io="bf16", scale=1.0),
        # prefill of 4097 tokens in float32, one past the chunk grid, with a residual scale
        dict(name="add_norm_prefill_f32", op="add_norm", rows=4097, d=768, io="f32", scale=0.5),
        # the batched long prefill (8 x 16384 tokens, 1.3B width): the largest pass
        dict(name="add_norm_long", op="add_norm", rows=131072, d=2048, io="bf16", scale=1.0),
        # a training step's 4096 tokens at the 2.7B width
        dict(name="add_norm_train", op="add_norm_grad", rows=4096, d=2560, io="bf16", scale=1.0),
        # the norm after the scan, 2.7B prefill; the gate is a slice of the projection's rows
        dict(name="gated_norm_prefill", op="gated_norm", rows=4096, d=5120, groups=1, io="bf16",
             zpad=5456),
        # its gradients at the 1.3B inner width, eight norm groups, 8 x 2048 tokens
        dict(name="gated_norm_train", op="gated_norm_grad", rows=16384, d=4096, groups=8,
             io="bf16", zpad=0),
        # float32 training on a ragged 515 tokens of the 130M shape
        dict(name="gated_norm_train_f32", op="gated_norm_grad", rows=515, d=1536, groups=1,
             io="f32", zpad=280),
        # decode, batch 1, 2.7B: norm and first projection, bound by streaming the weights
        dict(name="project_in_step", op="add_project_q8", rows=1, d=2560, n=10576, io="bf16"),
        # decode, batch 64, 2.7B: gated norm and second projection
        dict(name="project_out_batch", op="gated_project_q8", rows=64, d=5120, n=2560, groups=1,
             io="bf16"),
        # prefill, 2.7B: the first projection of 4096 tokens, bound by the matrix cores
        dict(name="linear_prefill", op="linear_q8", rows=4096, d=2560, n=10576, out="bf16"),
        # training the convolution of the 2.7B shape; the scan hands it float32 gradients
        dict(name="conv_train", op="conv_grad", batch=1, t=4096, d=5376, k=4, io="bf16",
             dy="f32", state=False),
        # ragged float32 batch with a carried window and channels off the vector grid
        dict(name="conv_train_f32", op="conv_grad", batch=3, t=1001, d=1793, k=4, io="f32",
             dy="f32", state=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    while True:
        case = _draw(rng)
        if 3072 not in case.values():       # a size of none of the package's workloads
            return case


def _draw(rng):
    op = rng.choice(["add_norm", "add_norm_grad", "gated_norm", "gated_norm_grad", "linear_q8",
                     "add_project_q8", "gated_project_q8", "conv_grad"])
    io = rng.choice(["f32", "bf16"])
    if op in ("add_norm", "add_norm_grad"):
        d = _log_int(rng, 64, 5120)
        if rng.random() < 0.5:
            d = (d + 7) // 8 * 8
        rows = _log_int(rng, 1, min(131072, (1 << 26) // d))
        return dict(op=op, rows=rows, d=d, io=io, scale=rng.choice([1.0, 0.5, 0.25]))
    if op in ("gated_norm", "gated_norm_grad"):
        groups = rng.choice([1, 1, 2, 4, 8])
        width = _log_int(rng, 64, 6144 // groups)
        if rng.random() < 0.5:
            width = (width + 7) // 8 * 8
        d = groups * width
        rows = _log_int(rng, 1, min(65536, (1 << 26) // d))
        zpad = rng.choice([0, rng.randint(1, 400), 8 * rng.randint(1, 700)])
        return dict(op=op, rows=rows, d=d, groups=groups, io=io, zpad=zpad)
    if op == "linear_q8":
        d, n = _log_int(rng, 64, 6144), _log_int(rng, 64, 12000)
        rows = _log_int(rng, 1, min(16384, (1 << 36) // (d * n)))
        return dict(op=op, rows=rows, d=d, n=n, out=io)
    if op in ("add_project_q8", "gated_project_q8"):
        d, n = _log_int(rng, 64, 6144), _log_int(rng, 64, 12000)
        rows = _log_int(rng, 1, min(8192, (1 << 34) // (d * n)))
        case = dict(op=op, rows=rows, d=d, n=n, io="bf16")
        if op == "gated_project_q8":
            groups = rng.choice([1, 2, 4])
            case["d"], case["groups"] = d // groups * groups, groups
        return case
    d = _log_int(rng, 16, 6144)
    if rng.random() < 0.5:
        d = (d + 7) // 8 * 8
    batch = rng.randint(1, 8)
    t = _log_int(rng, 1, min(16384, (1 << 26) // (d * batch)))
    return dict(op=op, batch=batch, t=t, d=d, k=rng.choice([2, 3, 4, 4]), io=io,
                dy=rng.choice(["f32", io]), state=rng.random() < 0.5)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _rows_q8(v):
    """8-bit rows of a float32 matrix, padded, and their scales."""
    amax = v.abs().amax(-1, keepdim=True)
    q = torch.zeros(v.shape[0], _padded(v.shape[1]), dtype=torch.int8, device=v.device)
    q[:, :v.shape[1]] = torch.round(v * (127.0 / amax)).to(torch.int8)
    return q, (amax / 127.0)[:, 0].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)

    op, d = case["op"], case["d"]
    s = {"case": dict(case)}
    if op == "conv_grad":
        io, k = _dtype(case), case["k"]
        bound = 1.0 / math.sqrt(k)
        s["weight"] = (rand(d, k) * 2.0 - 1.0) * bound
        s["bias"] = (rand(d) * 2.0 - 1.0) * bound
        s["x"] = randn(case["batch"], case["t"], d).to(io)
        s["dy"] = randn(case["batch"], case["t"], d).to(
            torch.float32 if case["dy"] == "f32" else io)
        s["state"] = randn(case["batch"], d, k - 1).to(io) if case["state"] else None
        s["dstate_out"] = randn(case["batch"], d, k - 1).to(io) if case["state"] else None
        return s
    rows = case["rows"]
    if op == "linear_q8":
        s["q"], s["qscale"] = _rows_q8(randn(rows, d))
        s["wq"], s["wscale"] = _rows_q8(randn(case["n"], d) / math.sqrt(d))
        return s
    io = _dtype(case)
    s["weight"] = 1.0 + 0.1 * randn(d)
    if op in ("add_norm", "add_norm_grad", "add_project_q8"):
        # the residual stream: channels of unequal size, as training leaves them
        r = randn(rows, d) * (0.5 + 4.0 * rand(d) ** 4)
        if op == "add_norm_grad":
            s["residual_out"] = r
            s["dy"] = randn(rows, d).to(io)
            s["dresidual_out"] = randn(rows, d)
        else:
            s["residual"] = r
            s["x"] = randn(rows, d).to(io)
    else:
        zpad = case.get("zpad", 0)
        s["y"] = randn(rows, d).to(io)
        s["z"] = randn(rows, d + zpad).to(io)[:, :d]
        if op == "gated_norm_grad":
            s["dout"] = randn(rows, d).to(io)
    if op in ("add_project_q8", "gated_project_q8"):
        s["wq"], s["wscale"] = _rows_q8(randn(case["n"], d) / math.sqrt(d))
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    case = state["case"]
    return (_run_own if own else _run_plain)(case["op"], case, state)


def _run_own(op, case, s):
    ssd = _ssd()
    if op == "add_norm":
        return ssd.ssd_add_norm(s["x"], s["weight"], s["residual"], scale=case["scale"], eps=EPS)
    if op == "add_norm_grad":
        return ssd.ssd_add_norm_backward(s["residual_out"], s["weight"], dy=s["dy"],
                                         dresidual_out=s["dresidual_out"], scale=case["scale"],
                                         eps=EPS)
    if op == "gated_norm":
        return ssd.ssd_gated_norm(s["y"], s["z"], s["weight"], groups=case["groups"], eps=EPS)
    if op == "gated_norm_grad":
        return ssd.ssd_gated_norm_backward(s["y"], s["z"], s["weight"], dout=s["dout"],
                                           groups=case["groups"], eps=EPS)
    if op == "linear_q8":
        return ssd.ssd_linear_q8(s["q"], s["qscale"], s["wq"], s["wscale"],
                                 out_dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16)
    if op == "add_project_q8":
        q, qscale, residual = ssd.ssd_add_norm_q8(s["x"], s["weight"], s["residual"], eps=EPS)
        return ssd.ssd_linear_q8(q, qscale, s["wq"], s["wscale"], out_dtype=s["x"].dtype), residual
    if op == "gated_project_q8":
        q, qscale = ssd.ssd_gated_norm_q8(s["y"], s["z"], s["weight"], groups=case["groups"],
                                          eps=EPS)
        return ssd.ssd_linear_q8(q, qscale, s["wq"], s["wscale"], out_dtype=s["y"].dtype)
    return ssd.ssd_conv1d_backward(s["x"], s["weight"], s["bias"], dy=s["dy"], state=s["state"],
                                   dstate_out=s["dstate_out"])


def _norm(v, weight, groups=1):
    """v / rms(v over each of `groups` equal parts of a row) * weight, float32."""
    u = v.reshape(v.shape[0], groups, -1)
    rstd = torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)
    return (u * rstd).reshape(v.shape) * weight


def _silu(z):
    return z / (1.0 + torch.exp(-z))


def _product_q8(q, qscale, wq, wscale, d):
    acc = q[:, :d].float() @ wq[:, :d].float().t()
    return acc * qscale[:, None] * wscale[None, :]


def _quantised(v):
    amax = v.abs().amax(-1, keepdim=True)
    return torch.round(v * (127.0 / amax)), (amax / 127.0)[:, 0]


def _run_plain(op, case, s):
    d = case["d"]
    if op == "add_norm":
        r = s["residual"] + case["scale"] * s["x"].float()
        return _norm(r, s["weight"]).to(s["x"].dtype), r
    if op == "add_norm_grad":
        r, dy = s["residual_out"], s["dy"].float()
        rstd = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
        xhat = r * rstd
        dn = dy * s["weight"]
        dr = s["dresidual_out"] + rstd * (dn - xhat * (dn * xhat).mean(-1, keepdim=True))
        return {"dx": (case["scale"] * dr).to(s["dy"].dtype), "dresidual": dr,
                "dweight": (dy * xhat).sum(0)}
    if op == "gated_norm":
        g = s["y"].float() * _silu(s["z"].float())
        return _norm(g, s["weight"], case["groups"]).to(s["y"].dtype)
    if op == "gated_norm_grad":
        groups = case["groups"]
        y, z, do = s["y"].float(), s["z"].float(), s["dout"].float()
        sg = 1.0 / (1.0 + torch.exp(-z))
        g = y * z * sg
        u = g.reshape(g.shape[0], groups, -1)
        rstd = torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)
        ghat = u * rstd
        dn = (do * s["weight"]).reshape(u.shape)
        dg = (rstd * (dn - ghat * (dn * ghat).mean(-1, keepdim=True))).reshape(g.shape)
        io = s["y"].dtype
        return {"dy": (dg * z * sg).to(io), "dz": (dg * y * sg * (1.0 + z * (1.0 - sg))).to(io),
                "dweight": (do * ghat.reshape(g.shape)).sum(0)}
    if op == "linear_q8":
        out = _product_q8(s["q"], s["qscale"], s["wq"], s["wscale"], d)
        return out if case["out"] == "f32" else out.bfloat16()
    if op == "add_project_q8":
        r = s["residual"] + s["x"].float()
        q, qs = _quantised(_norm(r, s["weight"]))
        return _product_q8(q, qs, s["wq"], s["wscale"], d).to(s["x"].dtype), r
    if op == "gated_project_q8":
        g = s["y"].float() * _silu(s["z"].float())
        q, qs = _quantised(_norm(g, s["weight"], case["groups"]))
        return _product_q8(q, qs, s["wq"], s["wscale"], d).to(s["y"].dtype)
    # conv_grad
    k, t = case["k"], case["t"]
    x, dy, w = s["x"].float(), s["dy"].float(), s["weight"]
    window = (torch.zeros(x.shape[0], k - 1, d, device=x.device) if s["state"] is None
              else s["state"].float().transpose(1, 2))
    xp = torch.cat([window, x], 1)
    zc = s["bias"] + sum(xp[:, i:i + t] * w[:, i] for i in range(k))
    sg = 1.0 / (1.0 + torch.exp(-zc))
    dz = dy * sg * (1.0 + zc * (1.0 - sg))
    dxp = torch.zeros_like(xp)
    for i in range(k):
        dxp[:, i:i + t] += dz * w[:, i]
    if s["dstate_out"] is not None:
        dxp[:, t:] += s["dstate_out"].float().transpose(1, 2)
    return {"dx": dxp[:, k - 1:].to(s["x"].dtype),
            "dweight": torch.stack([(dz * xp[:, i:i + t]).sum((0, 1)) for i in range(k)], -1),
            "dbias": dz.sum((0, 1)),
            "dstate": dxp[:, :k - 1].transpose(1, 2).contiguous().to(s["x"].dtype)}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op, d = case["op"], case["d"]
    if op == "conv_grad":
        e, k = case["batch"] * case["t"] * d, case["k"]
        io = 4 if case["io"] == "f32" else 2
        dy = 4 if case["dy"] == "f32" else io
        window = (3 if case["state"] else 1) * case["batch"] * d * (k - 1) * io
        return {"bytes": e * (2 * io + dy) + 8 * d * (k + 1) + window,
                "flops": e * (6 * k + 12)}
    rows = case["rows"]
    e = rows * d
    if op == "linear_q8":
        out = 4 if case["out"] == "f32" else 2
        return {"bytes": e + 4 * rows + case["n"] * (d + 4) + rows * case["n"] * out,
                "flops": 2 * e * case["n"]}
    io = 4 if case["io"] == "f32" else 2
    if op == "add_norm":
        return {"bytes": e * (2 * io + 8) + 4 * d, "flops": 6 * e}
    if op == "add_norm_grad":
        return {"bytes": e * (2 * io + 12) + 8 * d, "flops": 14 * e}
    if op == "gated_norm":
        return {"bytes": e * 3 * io + 4 * d, "flops": 10 * e}
    if op == "gated_norm_grad":
        return {"bytes": e * 5 * io + 8 * d, "flops": 26 * e}
    weights = case["n"] * (d + 4) + rows * case["n"] * io
    if op == "add_project_q8":
        return {"bytes": e * (io + 8) + 4 * d + weights, "flops": 2 * e * case["n"] + 8 * e}
    return {"bytes": e * 2 * io + 4 * d + weights, "flops": 2 * e * case["n"] + 12 * e}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["d"]
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if op == "conv_grad":
        return _exact_conv(case, s, f)

    def inverse_rms(v, groups):
        ms = v.view(v.shape[0], groups, d // groups).pow(2).sum(-1) * (groups / d)
        return (ms + EPS).pow(-0.5).repeat_interleave(d // groups, 1)

    def eight_bit_product(v):
        step = v.abs().max(1, keepdim=True).values / 127
        return torch.matmul(torch.round(v / step) * step, (f["wq"][:, :d] * f["wscale"][:, None]).T)

    if op == "linear_q8":
        return torch.matmul(f["q"] * f["qscale"][:, None], (f["wq"] * f["wscale"][:, None]).T)
    if op in ("add_norm", "add_project_q8"):
        r = torch.add(f["residual"], f["x"], alpha=case.get("scale", 1.0))
        n = r * inverse_rms(r, 1) * f["weight"]
        return (n if op == "add_norm" else eight_bit_product(n)), r
    if op == "add_norm_grad":
        # n_i = w_i r_i c, c = (sum r^2 / d + eps)^(-1/2), dc/dr_j = -c^3 r_j / d
        r, c = f["residual_out"], inverse_rms(f["residual_out"], 1)
        p = f["dy"] * f["weight"]
        dr = p * c - r * c.pow(3) * ((p * r).sum(1, keepdim=True) / d) + f["dresidual_out"]
        return {"dx": dr * case["scale"], "dresidual": dr, "dweight": (f["dy"] * r * c).sum(0)}
    gate = f["z"] * torch.sigmoid(f["z"])
    v = f["y"] * gate
    c = inverse_rms(v, case["groups"])
    if op == "gated_norm":
        return v * c * f["weight"]
    if op == "gated_project_q8":
        return eight_bit_product(v * c * f["weight"])
    p = f["dout"] * f["weight"]
    share = d // case["groups"]
    dot = (p * v).view(v.shape[0], -1, share).sum(-1).repeat_interleave(share, 1) / share
    dv = p * c - v * c.pow(3) * dot
    # d silu / dz = silu(z) + sigmoid(z) (1 - silu(z))
    return {"dy": dv * gate, "dz": dv * f["y"] * (gate + torch.sigmoid(f["z"]) * (1 - gate)),
            "dweight": (f["dout"] * v * c).sum(0)}


def _exact_conv(case, s, f):
    k, t, d = case["k"], case["t"], case["d"]
    x = f["x"].transpose(1, 2)
    before = f["state"] if s["state"] is not None else x.new_zeros(x.shape[0], d, k - 1)
    taps = torch.cat([before, x], 2).unfold(2, k, 1)             # [batch, channel, token, tap]
    zc = (taps * f["weight"][None, :, None, :]).sum(-1) + f["bias"][None, :, None]
    act = zc * torch.sigmoid(zc)
    dz = f["dy"].transpose(1, 2) * (act + torch.sigmoid(zc) * (1 - act))
    late = torch.nn.functional.pad(dz, (k - 1, k - 1)).unfold(2, k, 1)
    dxp = (late * f["weight"].flip(1)[None, :, None, :]).sum(-1)
    if s["dstate_out"] is not None:
        dxp[:, :, t:] += f["dstate_out"]
    return {"dx": dxp[:, :, k - 1:].transpose(1, 2),
            "dweight": (taps * dz[..., None]).sum((0, 2)), "dbias": dz.sum((0, 2)),
            "dstate": dxp[:, :, :k - 1]}
