"""The gated delta rule and the residual add with dropout: what is measured of them.

A stack may mix its tokens by the gated delta rule where it does not scan them:
the same decay dt, A and the same fixed-size state per head, but a token's write
is what its value differs from what the state already holds for its key.  With
k^ = k / |k|, q^ = scale q / |q| (one group of keys and queries serving several
heads), D = clip(softplus(dt + dt_bias)), a = exp(D A) and b = sigmoid(beta):

  S_t[p, n] = a_t S_{t-1}[p, n] + b_t (v_t[p] - a_t sum_m S_{t-1}[p, m] k^_t[m]) k^_t[n]
  y_t[p]    = sum_n S_t[p, n] q^_t[n]

  delta_scan     y and the final state of a whole sequence
  delta_step     one token, the state updated in place
  delta_grad     gradients of the scan with respect to all of its inputs
  dropout        r' = r + scale / (1 - p) keep x;  y = r' / rms(r') * weight
  dropout_grad   its gradients with respect to x, r and the weight

keep[row, c] holds where word c % 4 of Philox4x32-10 (Salmon, Moraes, Dror and
Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) with the counter
(c // 4, row, offset) and the key seed is at least p 2^32; seed and offset are
inputs.  Sizes are those of the package's workloads (24, 64 and 80 heads of 64
with a state of 128; widths 768, 2048 and 2560), and heads of 128 by 128.
"""
import math

import torch

own = False

CHUNK = 64
NORM_EPS = 1e-6
EPS = 1e-5


def _ssd():
    import state_space_model_amd as ssd
    return ssd


def _dtype(case):
    return torch.float32 if case["io"] == "f32" else torch.bfloat16


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # a short prompt of the 130M shape, one token past half a chunk: latency
        dict(name="delta_scan_short", op="delta_scan", batch=1, t=33, h=24, g=24, p=64, n=128,
             io="bf16", h0=False),
        # a prompt of 4096 tokens at the 2.7B shape, every head with its own key
        dict(name="delta_scan_prefill", op="delta_scan", batch=1, t=4096, h=80, g=80, p=64, n=128,
             io="bf16", h0=False),
        # the batched long prefill at the 1.3B shape, keys shared by eight heads
        dict(name="delta_scan_long", op="delta_scan", batch=8, t=16384, h=64, g=8, p=64, n=128,
             io="bf16", h0=True),
        # a ragged float32 batch continued from a cached state
        dict(name="delta_scan_f32", op="delta_scan", batch=3, t=1001, h=24, g=8, p=64, n=64,
             io="f32", h0=True),
        # decode at the 2.7B shape: one sequence, and 64 of them
        dict(name="delta_step_one", op="delta_step", batch=1, h=80, g=80, p=64, n=128, io="bf16"),
        dict(name="delta_step_batch", op="delta_step", batch=64, h=80, g=80, p=64, n=128,
             io="bf16"),
        # a training step's 4096 tokens, 32 heads of 128 by 128 sharing keys in pairs
        dict(name="delta_train", op="delta_grad", batch=1, t=4096, h=32, g=16, p=128, n=128,
             io="bf16", h0=False),
        # float32 training on ragged sequences of the 130M shape, state gradients included
        dict(name="delta_train_f32", op="delta_grad", batch=2, t=515, h=24, g=24, p=64, n=128,
             io="f32", h0=True),
        # a training step's 4096 tokens at the 2.7B width
        dict(name="dropout_train", op="dropout", rows=4096, d=2560, io="bf16", scale=1.0, p=0.1),
        # 8 x 16384 tokens at the 1.3B width
        dict(name="dropout_long", op="dropout", rows=131072, d=2048, io="bf16", scale=1.0, p=0.1),
        # the gradients of the 2.7B step
        dict(name="dropout_train_grad", op="dropout_grad", rows=4096, d=2560, io="bf16", scale=1.0,
             p=0.1),
        # float32, odd width and rows off the vector grid, a residual scale
        dict(name="dropout_f32_grad", op="dropout_grad", rows=1030, d=769, io="f32", scale=0.5,
             p=0.25),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["delta_scan", "delta_scan", "delta_step", "delta_grad", "delta_grad",
                     "dropout", "dropout_grad"])
    io = rng.choice(["f32", "bf16"])
    if op in ("dropout", "dropout_grad"):
        d = _log_int(rng, 64, 5120)
        if rng.random() < 0.5:
            d = (d + 7) // 8 * 8
        return dict(op=op, rows=_log_int(rng, 1, min(65536, (1 << 26) // d)), d=d, io=io,
                    scale=rng.choice([1.0, 0.5]), p=rng.choice([0.05, 0.1, 0.25, 0.5]))
    g, per = _log_int(rng, 1, 32), rng.choice([1, 1, 2, 4])
    p, n = rng.choice([(64, 128), (64, 64), (128, 128), (8 * rng.randint(2, 16), 8 * rng.randint(2, 16))])
    case = dict(op=op, h=g * per, g=g, p=p, n=n, io=io)
    if op == "delta_step":
        return dict(case, batch=_log_int(rng, 1, max(1, (1 << 26) // (g * per * p * n))))
    batch = rng.randint(1, 4)
    most = (1 << 20) // (batch * g * per) if op == "delta_scan" else (1 << 18) // (batch * g * per)
    return dict(case, batch=batch, t=_log_int(rng, 1, max(1, min(8192, most))),
                h0=rng.random() < 0.5)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda", dtype=torch.float32)

    op, io = case["op"], _dtype(case)
    s = {"case": dict(case)}
    if op in ("dropout", "dropout_grad"):
        rows, d = case["rows"], case["d"]
        s["weight"] = 1.0 + 0.1 * randn(d)
        # seed and offset of the generator, as a training program keeps and advances them
        s["rng"] = torch.randint(0, 1 << 62, (2,), generator=gen, device="cuda", dtype=torch.int64)
        # the residual stream: channels of unequal size, as training leaves them
        r = randn(rows, d) * (0.5 + 4.0 * rand(d) ** 4)
        if op == "dropout":
            s["residual"], s["x"] = r, randn(rows, d).to(io)
        else:
            s["residual_out"], s["dy"], s["dresidual_out"] = r, randn(rows, d).to(io), randn(rows, d)
        return s
    batch, h, g, p, n = (case[k] for k in ("batch", "h", "g", "p", "n"))
    lead = (batch,) if op == "delta_step" else (batch, case["t"])
    # queries, keys and values are slices of the convolution's output, which its
    # activation leaves with a positive mean
    u = randn(*lead, 2 * g * n + h * p, dtype=io)
    u = torch.nn.functional.silu(u, inplace=True)
    s["q"] = u[..., :g * n].unflatten(-1, (g, n))
    s["k"] = u[..., g * n:2 * g * n].unflatten(-1, (g, n))
    s["v"] = u[..., 2 * g * n:].unflatten(-1, (h, p))
    s["dt"] = 0.5 * randn(*lead, h)
    s["beta"] = randn(*lead, h)
    s["dt_bias"] = torch.log(torch.expm1(1e-3 + 0.099 * rand(h)))
    s["A"] = -torch.exp(math.log(16.0) * rand(h))
    if op == "delta_step":
        s["state"] = randn(batch, h, p, n) / math.sqrt(n)
        return s
    s["h0"] = randn(batch, h, p, n) / math.sqrt(n) if case["h0"] else None
    if op == "delta_grad":
        s["dy"] = randn(*lead, h, p).to(io)
        s["dfinal"] = randn(batch, h, p, n) / math.sqrt(n) if case["h0"] else None
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state["case"]["op"], state["case"], state)


def _run_own(op, case, s):
    ssd = _ssd()
    if op == "delta_scan":
        return ssd.ssd_delta_scan(s["q"], s["k"], s["v"], s["dt"], s["A"], s["beta"],
                                  dt_bias=s["dt_bias"], initial_state=s["h0"])
    if op == "delta_step":
        y = ssd.ssd_delta_step(s["state"], s["q"], s["k"], s["v"], s["dt"], s["A"], s["beta"],
                               dt_bias=s["dt_bias"])
        return y, s["state"]
    if op == "delta_grad":
        return ssd.ssd_delta_scan_backward(s["q"], s["k"], s["v"], s["dt"], s["A"], s["beta"],
                                           dt_bias=s["dt_bias"], initial_state=s["h0"],
                                           dy=s["dy"], dfinal_state=s["dfinal"])
    if op == "dropout":
        return ssd.ssd_dropout_add_norm(s["x"], s["weight"], s["residual"], p=case["p"],
                                        rng=s["rng"], scale=case["scale"], eps=EPS)
    return ssd.ssd_dropout_add_norm_backward(s["residual_out"], s["weight"], dy=s["dy"],
                                             dresidual_out=s["dresidual_out"], p=case["p"],
                                             rng=s["rng"], scale=case["scale"], eps=EPS)


def _softplus(z):
    return torch.clamp(z, min=0.0) + torch.log1p(torch.exp(-z.abs()))


def _logistic(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _gates(s):
    """Decay rate D A and write strength, float32."""
    return _softplus(s["dt"] + s["dt_bias"]) * s["A"], _logistic(s["beta"])


def _unit(x):
    """x over its length, and what it was multiplied by."""
    x = x.float()
    r = torch.rsqrt((x * x).sum(-1, keepdim=True) + NORM_EPS)
    return x * r, r


def _spread(x, h):
    """[..., g, n] to the heads [..., h, n]."""
    g = x.shape[-2]
    return x if g == h else x.repeat_interleave(h // g, -2)


def _chunks(x, t):
    """[b, t, h, d] to [chunk, b, h, CHUNK, d], tokens past t zero."""
    nc = (t + CHUNK - 1) // CHUNK
    x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, nc * CHUNK - t))
    return x.unflatten(1, (nc, CHUNK)).permute(1, 0, 3, 2, 4).contiguous()


def _tokens(x, t):
    """[chunk, b, h, CHUNK, d] back to [b, t, h, d]."""
    return x.permute(1, 0, 3, 2, 4).flatten(1, 2)[:, :t]


def _inverse(a):
    """(1 + a)^-1 of strictly lower triangular a: pairs of diagonal blocks of 1, 2, 4 ... joined by
    [[x, 0], [c, z]]^-1 = [[x^-1, 0], [-z^-1 c x^-1, z^-1]]."""
    x = torch.eye(CHUNK, device=a.device).expand_as(a).contiguous()
    size = 1
    while size < CHUNK:
        def block(m, i, j):
            nb = CHUNK // (2 * size)
            m = m.unflatten(-1, (nb, 2, size)).unflatten(-4, (nb, 2, size))
            return m[..., i, :, :, j, :].diagonal(dim1=-4, dim2=-2).movedim(-1, -3)
        joined = -(block(x, 1, 1) @ (block(a, 1, 0) @ block(x, 0, 0)))
        block(x, 1, 0).copy_(joined)
        size *= 2
    return x


def _parts(s, t, h):
    """What both directions need of a sequence, in chunks: q^ and k^ (spread to the heads), the
    sums of the decay from a chunk's start, its factors between tokens, beta and the inverse."""
    g, beta = _gates(s)
    qn, kn = _unit(s["q"])[0], _unit(s["k"])[0]
    q = _chunks(_spread(qn * (qn.shape[-1] ** -0.5), h), t)
    k = _chunks(_spread(kn, h), t)
    v = _chunks(s["v"].float(), t)
    beta = _chunks(beta[..., None], t)
    cum = _chunks(g[..., None], t).double().cumsum(-2)
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=cum.device).tril()
    between = torch.exp(torch.where(lower, cum - cum.mT, -math.inf).float())
    last = cum[..., -1:, :]
    to_end, from_start, whole = ((last - cum).float().exp(), cum.float().exp(), last.float().exp())
    kk = (k @ k.mT) * between
    a = (beta * kk).tril(-1)
    return q, k, v, beta, between, to_end, from_start, whole, kk, _inverse(a)


def _states(k, v, beta, to_end, from_start, whole, inv, h0):
    """The state [.., n, p] before every chunk and after the last, and the writes of its tokens."""
    state = (torch.zeros(*k.shape[1:3], k.shape[-1], v.shape[-1], device=k.device) if h0 is None
             else h0.mT.contiguous())
    before, writes = [], []
    for c in range(k.shape[0]):
        w = inv[c] @ (beta[c] * (v[c] - from_start[c] * (k[c] @ state)))
        before.append(state)
        writes.append(w)
        state = whole[c] * state + k[c].mT @ (to_end[c] * w)
    return torch.stack(before), torch.stack(writes), state


def _run_plain(op, case, s):
    if op == "delta_scan":
        t, h = case["t"], case["h"]
        q, k, v, beta, between, to_end, from_start, whole, _, inv = _parts(s, t, h)
        before, writes, state = _states(k, v, beta, to_end, from_start, whole, inv, s["h0"])
        y = from_start * (q @ before) + ((q @ k.mT) * between) @ writes
        return _tokens(y, t).to(s["v"].dtype).contiguous(), state.mT.contiguous()
    if op == "delta_step":
        g, beta = _gates(s)
        q = _spread(_unit(s["q"])[0] * (case["n"] ** -0.5), case["h"])[..., None, :]
        k = _spread(_unit(s["k"])[0], case["h"])[..., None, :]
        state = torch.exp(g)[..., None, None] * s["state"]
        write = beta[..., None] * (s["v"].float() - (state * k).sum(-1))
        state = state + write[..., None] * k
        s["state"].copy_(state)
        return (state * q).sum(-1).to(s["v"].dtype), s["state"]
    if op == "delta_grad":
        return _plain_grad(case, s)
    return _plain_dropout(op, case, s)


def _plain_grad(case, s):
    t, h, g = case["t"], case["h"], case["g"]
    q, k, v, beta, between, to_end, from_start, whole, kk, inv = _parts(s, t, h)
    before, n, state = _states(k, v, beta, to_end, from_start, whole, inv, s["h0"])
    dy = _chunks(s["dy"].float(), t)
    e = torch.zeros_like(state) if s["dfinal"] is None else s["dfinal"].mT.contiguous()
    intra = ((q @ k.mT) * between).mT @ dy
    e_after, dr, ends = [], [], []
    after = state
    for c in range(k.shape[0] - 1, -1, -1):
        d = inv[c].mT @ (intra[c] + to_end[c] * (k[c] @ e))
        e_after.append(e)
        dr.append(d)
        ends.append((e * after).sum((-1, -2)))
        after = before[c]
        e = (whole[c] * e + (from_start[c] * q[c]).mT @ dy[c]
             - (beta[c] * from_start[c] * k[c]).mT @ d)
    e_after, dr, ends = (torch.stack(x[::-1]) for x in (e_after, dr, ends))
    # gradients of the products q k^T and of the inverse's off-diagonal, over their decay
    dp = (dy @ n.mT) * between
    da = ((dr @ n.mT) * between).tril(-1)
    dq = from_start * (dy @ before.mT) + dp @ k
    z = from_start * (dr @ before.mT) + da @ k
    dk_row = -beta * z
    dk_col = to_end * (n @ e_after.mT) + dp.mT @ q - (beta * da).mT @ k
    dbeta = (dr * v).sum(-1) - (k * z).sum(-1)
    dcum = (q * dq).sum(-1) + (k * (dk_row - dk_col)).sum(-1)
    dcum[..., -1] += ends
    dg = _tokens(dcum.flip(-1).cumsum(-1).flip(-1)[..., None], t)[..., 0]
    b = _logistic(s["beta"])
    out = {"dv": _tokens(beta * dr, t).to(s["v"].dtype).contiguous(),
           "dbeta": _tokens(dbeta[..., None], t)[..., 0] * b * (1.0 - b),
           "dinitial_state": e.mT.contiguous()}
    for name, x, dx, scale in (("dq", s["q"], dq, case["n"] ** -0.5), ("dk", s["k"], dk_row + dk_col, 1.0)):
        u, r = _unit(x)
        du = scale * _tokens(dx, t).unflatten(2, (g, h // g)).sum(3)
        out[name] = (r * (du - u * (u * du).sum(-1, keepdim=True))).to(x.dtype)
    z = s["dt"] + s["dt_bias"]
    ddt = dg * s["A"] * _logistic(z)
    out["ddt"], out["dA"] = ddt, (dg * _softplus(z)).sum((0, 1))
    out["ddt_bias"] = ddt.sum((0, 1))
    return out


def _philox(rng, rows, d):
    """The generator's words [rows, d] as int64."""
    dev = rng.device
    low = 0xFFFFFFFF
    col = torch.arange((d + 3) // 4, device=dev)[None, :].expand(rows, -1)
    row = torch.arange(rows, device=dev)[:, None].expand_as(col)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    x0, x1 = col, row
    x2, x3 = (rng[1] & low).expand_as(col), ((rng[1] >> 32) & low).expand_as(col)

    def high(m, x):
        return (((m >> 16) * x) + (((m & 0xFFFF) * x) >> 16)) >> 16

    for _ in range(10):
        x0, x1, x2, x3 = (high(0xCD9E8D57, x2) ^ x1 ^ k0, (0xCD9E8D57 * x2) & low,
                          high(0xD2511F53, x0) ^ x3 ^ k1, (0xD2511F53 * x0) & low)
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack((x0, x1, x2, x3), -1).flatten(1)[:, :d]


def _plain_dropout(op, case, s):
    p, d = case["p"], case["d"]
    x = s["x"] if op == "dropout" else s["residual_out"]
    keep = _philox(s["rng"], x.shape[0], d) >= round(p * 2.0 ** 32)
    factor = keep * (case["scale"] / (1.0 - p))
    if op == "dropout":
        r = s["residual"] + factor * s["x"].float()
        rstd = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
        return (r * rstd * s["weight"]).to(s["x"].dtype), r
    r, dy = s["residual_out"], s["dy"].float()
    rstd = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    n = r * rstd
    dn = dy * s["weight"]
    dr = s["dresidual_out"] + rstd * (dn - n * (dn * n).mean(-1, keepdim=True))
    return {"dx": (factor * dr).to(s["dy"].dtype), "dresidual": dr, "dweight": (dy * n).sum(0)}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op, io = case["op"], 4 if case["io"] == "f32" else 2
    if op in ("dropout", "dropout_grad"):
        e = case["rows"] * case["d"]
        if op == "dropout":
            return {"bytes": e * (2 * io + 8) + 4 * case["d"] + 16, "flops": 8 * e}
        return {"bytes": e * (2 * io + 12) + 8 * case["d"] + 16, "flops": 16 * e}
    batch, h, g, p, n = (case[k] for k in ("batch", "h", "g", "p", "n"))
    state = batch * h * p * n
    tokens = batch * case.get("t", 1)
    qkv = tokens * (2 * g * n + h * p) * io
    gates = 8 * tokens * h + 8 * h
    if op == "delta_step":
        return {"bytes": qkv + gates + tokens * h * p * io + 8 * state, "flops": 7 * state}
    if op == "delta_scan":
        return {"bytes": qkv + gates + tokens * h * p * io + 4 * state * (2 if case["h0"] else 1),
                "flops": 6 * tokens * h * p * n}
    return {"bytes": 2 * (qkv + gates) + tokens * h * p * io + 4 * state * (3 if case["h0"] else 1),
            "flops": 16 * tokens * h * p * n}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] in ("dropout", "dropout_grad"):
        return _exact_dropout(case, prepare(case, seed))
    # token by token: what would take too long, or whose states would not fit
    per = 16.0 * case["batch"] * case["h"] * case["p"] * case["n"]
    t = case.get("t", 1)
    if t * max(per * 2.5e-12, 1.5e-4) > 12.0 or (case["op"] == "delta_grad" and t * per > 6e10):
        return None
    s = prepare(case, seed)
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    rate = torch.nn.functional.softplus(f["dt"] + f["dt_bias"], threshold=1e6)
    a, b = torch.exp(rate * f["A"]), torch.sigmoid(f["beta"])
    per_group = case["h"] // case["g"]
    heads = lambda x: x.repeat_interleave(per_group, -2)    # noqa: E731
    size = {x: (f[x].pow(2).sum(-1, keepdim=True) + NORM_EPS).sqrt() for x in ("q", "k")}
    q = heads(f["q"] / size["q"]) / math.sqrt(case["n"])
    k = heads(f["k"] / size["k"])
    if case["op"] == "delta_step":
        old = f["state"] * a[..., None, None]
        new = old + torch.einsum("bhp,bhn->bhpn", b[..., None] * (f["v"] - (old @ k[..., None])[..., 0]), k)
        return (new @ q[..., None])[..., 0], new
    state = f.get("h0")
    if state is None:
        state = f["v"].new_zeros(case["batch"], case["h"], case["p"], case["n"])
    ys, kept = [], []
    for i in range(t):
        if case["op"] == "delta_grad":
            kept.append(state)
        state = state * a[:, i, :, None, None]
        miss = f["v"][:, i] - (state @ k[:, i, :, :, None])[..., 0]
        state = state + (b[:, i, :, None] * miss)[..., None] * k[:, i, :, None, :]
        if case["op"] == "delta_scan":
            ys.append((state @ q[:, i, :, :, None])[..., 0])
    if case["op"] == "delta_scan":
        return torch.stack(ys, 1), state
    return _exact_grad(case, f, rate, a, b, q, k, size, kept)


def _exact_grad(case, f, rate, a, b, q, k, size, kept):
    """The recurrence's adjoint, token by token from the last: d is the gradient of the state."""
    d = f.get("dfinal")
    if d is None:
        d = torch.zeros_like(kept[0])
    dq, dk, dv, da, db = (torch.empty_like(x) for x in (q, k, f["v"], a, b))
    for i in range(case["t"] - 1, -1, -1):
        old = kept[i] * a[:, i, :, None, None]
        ki, bi, dyi = k[:, i], b[:, i, :, None], f["dy"][:, i]
        miss = f["v"][:, i] - (old @ ki[..., None])[..., 0]
        new = old + (bi * miss)[..., None] * ki[..., None, :]
        dq[:, i] = (new.mT @ dyi[..., None])[..., 0]
        d = d + dyi[..., None] * q[:, i][..., None, :]
        dwrite = (d @ ki[..., None])[..., 0]
        db[:, i] = (dwrite * miss).sum(-1)
        dv[:, i] = bi * dwrite
        dk[:, i] = (d.mT @ (bi * miss)[..., None])[..., 0] - (old.mT @ dv[:, i][..., None])[..., 0]
        d = d - dv[:, i][..., None] * ki[..., None, :]
        da[:, i] = (d * kept[i]).sum((-1, -2))
        d = d * a[:, i, :, None, None]
    drate = da * a * f["A"]
    ddt = drate * torch.sigmoid(f["dt"] + f["dt_bias"])
    out = {"dv": dv, "dbeta": db * b * (1 - b), "dinitial_state": d, "ddt": ddt,
           "dA": (da * a * rate).sum((0, 1)), "ddt_bias": ddt.sum((0, 1))}
    for name, dx, scale in (("q", dq, 1 / math.sqrt(case["n"])), ("k", dk, 1.0)):
        du = scale * dx.reshape(*dx.shape[:2], case["g"], -1, case["n"]).sum(3)
        x, length = f[name], size[name]
        out["d" + name] = du / length - x * ((x * du).sum(-1, keepdim=True) / length ** 3)
    return out


def _exact_dropout(case, s):
    rows, d, p = case["rows"], case["d"], case["p"]
    # the generator on 16-bit halves: a product of two words is four of them with carries
    m16 = 0xFFFF

    def product(m, x):
        ml, mh, xl, xh = m & m16, m >> 16, x & m16, x >> 16
        ll = ml * xl
        mid = mh * xl + (ll >> 16)
        other = ml * xh + (mid & m16)
        return mh * xh + (mid >> 16) + (other >> 16), ((other & m16) << 16) | (ll & m16)

    seed, offset = (int(v) for v in s["rng"].tolist())
    word = lambda v, i: (v >> (32 * i)) & 0xFFFFFFFF     # noqa: E731
    quads = (d + 3) // 4
    at = torch.arange(rows * quads, device="cuda")
    c = [at % quads, at // quads, torch.full_like(at, word(offset, 0)),
         torch.full_like(at, word(offset, 1))]
    for i in range(10):
        keys = [(word(seed, j) + i * w) % (1 << 32) for j, w in ((0, 0x9E3779B9), (1, 0xBB67AE85))]
        (h0, l0), (h1, l1) = product(0xD2511F53, c[0]), product(0xCD9E8D57, c[2])
        c = [h1 ^ c[1] ^ keys[0], l1, h0 ^ c[3] ^ keys[1], l0]
    drop = (torch.stack(c, 1).view(rows, 4 * quads)[:, :d] < int(math.floor(p * 2 ** 32 + 0.5)))
    del at, c
    w = s["weight"].double()
    gain = case["scale"] / (1 - p)
    if case["op"] == "dropout":
        r = s["residual"].double() + (s["x"].double() * gain).masked_fill_(drop, 0.0)
        return r * ((r ** 2).sum(1, keepdim=True) / d + EPS).pow(-0.5) * w, r
    r, dy = s["residual_out"].double(), s["dy"].double()
    c = ((r ** 2).sum(1, keepdim=True) / d + EPS).pow(-0.5)
    dn = dy * w
    dr = dn * c - r * c ** 3 * ((dn * r).sum(1, keepdim=True) / d) + s["dresidual_out"].double()
    return {"dx": (dr * gain).masked_fill(drop, 0.0), "dresidual": dr, "dweight": (dy * r * c).sum(0)}
