"""Inputs and bars of the gated delta rule's tests."""
import math

import numpy as np
import torch

from oracle import delta

U = 2.0 ** -24                              # float32: half a step, relative
IO_U = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def make(seed, Bt, T, H, G, P, N, io=torch.float32, h0=True, bias=True, pad=0, spread=1.0):
    """CPU inputs; q, k, v are slices of one tensor with `pad` unused columns between them."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)     # noqa: E731
    width = 2 * G * N + H * P + 2 * pad
    u = torch.nn.functional.silu(spread * r(Bt, T, width)).to(io)
    x = {"q": u[..., :G * N].unflatten(-1, (G, N)),
         "k": u[..., G * N + pad:2 * G * N + pad].unflatten(-1, (G, N)),
         "v": u[..., 2 * G * N + 2 * pad:].unflatten(-1, (H, P)),
         "dt": 0.5 * r(Bt, T, H), "beta": r(Bt, T, H),
         "A": -torch.exp(torch.rand(H, generator=g) * math.log(16.0)),
         "dt_bias": torch.log(torch.expm1(1e-3 + 0.099 * torch.rand(H, generator=g))) if bias else None,
         "h0": r(Bt, H, P, N) / math.sqrt(N) if h0 else None}
    return x, u


def on_device(x, u):
    """The same on the GPU, q, k, v still slices of one tensor."""
    d = {n: None if t is None else t.cuda() for n, t in x.items() if n not in "qkv"}
    ud = u.cuda()
    for n in "qkv":
        t = x[n]
        d[n] = ud.as_strided(t.shape, t.stride(), t.storage_offset())
    return d


def state_bar(states, T, N):
    """A state is a sum of T decayed writes, a write a dot product of N terms (of a chunk's 64 more by
    the chunked form): T + N + 64 roundings of magnitudes that the largest row bounds, since a row's
    length grows by writes alone.  They are independent (their sum grows with the root), and the
    largest of some thousand sums is under 4 of its deviations; 2 for the products chained."""
    row = max(float(s.square().sum(-1).max().sqrt()) for s in states)
    return 8 * math.sqrt(T + N + 64) * U * max(row, 1e-30)


def y_bar(y, states, T, N, io, scale):
    """The state's bar through a dot product with q^ (of length `scale`); a bfloat16 y from two planes
    of each operand (2^-15 of the magnitudes between them) and its rounding."""
    bar = state_bar(states, T, N) * scale
    if io == torch.bfloat16:
        bar += 2.0 ** -14 * scale * max(float(s.square().sum(-1).max().sqrt()) for s in states)
    return bar + IO_U[io] * 1.01 * y.abs().numpy()


def length(ts, dims):
    """The greatest length of the vectors that `dims` dimensions make up."""
    return max((float(t.double().flatten(-dims).square().sum(-1).max().sqrt()) for t in ts), default=0.0)


def grad_bars(x, dy, ref, states, dstates, scale, norm=True):
    """Bars of the gradients.  Each is a sum of products of states S, their gradients dS, values and
    dy, and is formed from sums of n = T + N + P + 64 terms at most, whose roundings add as in
    state_bar; the magnitudes are bounded by lengths (a write by |v| + |S|).  The gradient of a
    decay sums 64 tokens' terms, those of A and dt_bias those of all tokens."""
    io = x["v"].dtype
    Bt, T, H, P = x["v"].shape
    G, N = x["q"].shape[2:]
    e = 8 * math.sqrt(T + N + P + 64) * U
    S, dS, V, dY = length(states, 2), length(dstates, 2), length([x["v"]], 1), length([dy], 1)
    least = lambda t: float(t.double().square().sum(-1).min().sqrt()) if norm else 1.0  # noqa: E731
    most = lambda t: 1.0 if norm else length([t], 1)                                     # noqa: E731
    kl, ql = most(x["k"]), most(x["q"]) * scale
    write = V + S * kl
    per, rate = H // G, float(ref["rates"].abs().max())
    token = dS * write * kl + dY * S * ql + dS * S
    dg = e * 8 * 3 * token
    slope = float(x["A"].abs().max())
    rounded = lambda n: IO_U[io] * 1.01 * ref[n].abs().numpy() if io != torch.float32 else 0.0  # noqa: E731
    return {"dq": e * per * dY * S * scale / least(x["q"]) + rounded("dq"),
            "dk": e * per * 3 * dS * (write + S) / least(x["k"]) + rounded("dk"),
            "dv": e * dS * kl + rounded("dv"), "dbeta": e * 3 * dS * kl * (write + S),
            "ddt": dg * slope, "dA": dg * rate * math.sqrt(Bt * T), "ddt_bias": dg * slope * math.sqrt(Bt * T),
            "dinitial_state": e * dS}


def oracle_of(x, **options):
    return delta.scan(**{n: delta.f64(t) for n, t in x.items()}, **options)


def close(got, want, bar, what):
    got, want = delta.f64(got).numpy(), want.numpy()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = np.abs(got - want)
    worst = float((off / np.maximum(np.broadcast_to(bar, off.shape), 1e-300)).max()) if off.size else 0.0
    print(f"{what}: {worst:.3f} of its bar, largest error {float(off.max()) if off.size else 0:.2e}")
    assert worst <= 1.0, (what, worst)
