"""Bars of the gated delta rule's gradients, element by element, from the terms that each is a sum of.

Every quantity of the chunked form is computed in float64 next to a magnitude M: of an input its
absolute value, of a sum of products |sum| + sqrt(sum of M(x)^2 M(y)^2).  Rounded to float32, a sum
of n products is off by n roundings of its partial sums, which M bounds, and by its factors' own
errors: they are independent, so both add as roots of sums of squares.  e = 8 sqrt(n) U (4
deviations, for the largest of some thousand; 2 for the products chained) times M bounds the error,
n = T + N + P + 64 the longest sum's terms.  The states that enter chunks and their gradients have
a row's root mean square as the least magnitude of its elements, which are sums over the past."""
import math

import torch

from delta_cases import IO_U, U
from oracle import delta

C = 64
# A float32 factor below 2^-126 may be held as 0 (a write strength of e^-120 = 2^-173 is), which leaves
# out at most 2^-126 times the other factors: the tests' inputs keep those below 2^6.
TINY = 2.0 ** -120


class Sum:
    """A value and its magnitude."""

    def __init__(self, v, m=None):
        self.v, self.m = v, v.abs() if m is None else m

    def __matmul__(self, o):
        v = self.v @ o.v
        return Sum(v, v.abs() + torch.sqrt(self.m.square() @ o.m.square()))

    def __add__(self, o):
        return Sum(self.v + o.v, self.m + o.m)

    def __sub__(self, o):
        return Sum(self.v - o.v, self.m + o.m)

    def __neg__(self):
        return Sum(-self.v, self.m)

    def __mul__(self, f):        # by an exact factor, or another quantity
        return Sum(self.v * f.v, self.m * f.m) if isinstance(f, Sum) else Sum(self.v * f, self.m * f.abs())

    def __getitem__(self, at):
        return Sum(self.v[at], self.m[at])

    def map(self, f):            # of what moves elements alone
        return Sum(f(self.v), f(self.m))

    def sum(self, dim, keepdim=False):
        v = self.v.sum(dim, keepdim=keepdim)
        return Sum(v, v.abs() + torch.sqrt(self.m.square().sum(dim, keepdim=keepdim)))

    @property
    def mT(self):
        return self.map(lambda t: t.mT)


def rows(t):
    return Sum(t, t.abs() + t.square().mean(-1, keepdim=True).sqrt())


def join(qs, f, dim):
    return Sum(f([q.v for q in qs], dim), f([q.m for q in qs], dim))


def reference(x, dy, dfinal, softplus=True, limit=(0.0, math.inf), sigmoid=True, norm=True, eps=1e-6, scale=None):
    """The float64 gradients {name: value} by automatic derivatives, and {name: [a Sum for each term]} of
    the chunked form, which add up to them."""
    Bt, T, H, P = x["v"].shape
    G, N = x["q"].shape[2:]
    scale = 1.0 / math.sqrt(N) if scale is None else scale
    f = {n: delta.f64(t) for n, t in x.items()}
    if f["h0"] is None:
        f["h0"] = torch.zeros(Bt, H, P, N, dtype=torch.float64)
    dy, last = delta.f64(dy), torch.zeros_like(f["h0"]) if dfinal is None else delta.f64(dfinal)
    opts = dict(softplus=softplus, limit=limit, sigmoid=sigmoid, norm=norm, eps=eps, scale=scale)
    grads, states, dstates = delta.gradients(f, dy, delta.f64(dfinal), **opts)
    grads["dinitial_state"] = grads.pop("dh0")
    grads.setdefault("ddt_bias", grads["ddt"].sum((0, 1)))

    spread = lambda t: t.repeat_interleave(H // G, 2).transpose(1, 2)        # noqa: E731  [Bt,H,T,N]
    rq = scale * ((f["q"].square().sum(-1, keepdim=True) + eps).rsqrt() if norm else torch.ones(Bt, T, G, 1, dtype=torch.float64))
    rk = (f["k"].square().sum(-1, keepdim=True) + eps).rsqrt() if norm else torch.ones(Bt, T, G, 1, dtype=torch.float64)
    q, k = spread(f["q"] * rq), spread(f["k"] * rk)
    v, dY = f["v"].transpose(1, 2), dy.transpose(1, 2)
    z = f["dt"] if f["dt_bias"] is None else f["dt"] + f["dt_bias"]
    rate = delta.rates(f["dt"], f["dt_bias"], softplus, limit)
    pre = delta.rates(f["dt"], f["dt_bias"], softplus, (-math.inf, math.inf))
    slope = torch.where((pre < limit[0]) | (pre > limit[1]), 0.0, f["A"]) * (torch.sigmoid(z) if softplus else 1.0)
    g = (rate * f["A"]).clamp(min=-1e5).transpose(1, 2)                      # logarithms, e^-1e5 is 0
    b = (torch.sigmoid(f["beta"]) if sigmoid else f["beta"]).transpose(1, 2)
    db = torch.sigmoid(f["beta"]) * torch.sigmoid(-f["beta"]) if sigmoid else torch.ones_like(f["beta"])

    terms = {n: [[] for _ in range(parts)] for n, parts in
             (("dq", 2), ("dk", 5), ("dv", 2), ("dbeta", 2), ("ddt", 4))}
    for c in range((T + C - 1) // C):
        at = slice(c * C, min(T, c * C + C))
        n = at.stop - at.start
        cum = g[:, :, at].cumsum(-1)
        D = torch.exp((cum[..., :, None] - cum[..., None, :]).clamp(max=0.0)).tril()
        gam, eta = torch.exp(cum)[..., None], torch.exp(cum[..., -1:] - cum)[..., None]
        whole = gam[..., -1:, :]
        bc = b[:, :, at, None]
        K, Qu, V, Y = Sum(k[:, :, at]), Sum(q[:, :, at]), Sum(v[:, :, at]), Sum(dY[:, :, at])
        S = rows(states[at.start])
        E = rows(last if at.stop == T else dstates[at.stop] - dY[:, :, at.stop - 1, :, None] * q[:, :, at.stop - 1, None])
        KK, QK = K @ K.mT, Qu @ K.mT
        L = KK * (bc * D.tril(-1))
        t = torch.linalg.solve_triangular(torch.eye(n, dtype=torch.float64) + L.v,
                                          torch.eye(n, dtype=torch.float64).expand(Bt, H, n, n), upper=False)
        Ti = Sum(t, t.abs() + torch.sqrt(t.square() @ L.m.square() @ t.square()))
        W = Ti @ ((V - (K @ S.mT) * gam) * bc)
        dW = [(QK * D).mT @ Y, (K @ E.mT) * eta]
        dRs = [Ti.mT @ p for p in dW]
        dR = dRs[0] + dRs[1]
        dP, dL = (Y @ W.mT) * D, (dR @ W.mT) * D.tril(-1)
        YS, RS, WE = (Y @ S) * gam, (dR @ S) * gam, (W @ E) * eta
        Z = [RS, dL @ K]
        terms["dq"][0].append(YS)
        terms["dq"][1].append(dP @ K)
        for i, p in enumerate((WE, dP.mT @ Qu, -(dL.mT @ (K * bc)), Z[0] * -bc, Z[1] * -bc)):
            terms["dk"][i].append(p)
        for i, p in enumerate(dRs):
            terms["dv"][i].append(p * bc)
        terms["dbeta"][0].append((dR * V).sum(-1))
        terms["dbeta"][1].append(-(K * (Z[0] + Z[1])).sum(-1))
        # of the decays: pairs across a token, later reads, earlier writes, what passes through
        pair = (dP * QK - dL * (KK * bc)) * torch.ones(n, n).tril(-1)
        read = (Qu * YS).sum(-1) - (K * RS).sum(-1) * bc[..., 0]
        wrote = (K * WE).sum(-1)
        parts = ([pair[..., i:, :i].sum((-1, -2)) for i in range(n)], [read[..., i:].sum(-1) for i in range(n)],
                 [wrote[..., :i].sum(-1) for i in range(n)], [(E * S).sum((-1, -2)) * whole[..., 0, 0]] * n)
        for i, p in enumerate(parts):
            terms["ddt"][i].append(join(p, torch.stack, -1))
        if c == 0:
            terms["dinitial_state"] = [E * whole, (Y * gam).mT @ Qu, -((dR * (bc * gam)).mT @ K)]

    first = terms.pop("dinitial_state")
    terms = {n: [join(p, torch.cat, 2).map(lambda t: t.transpose(1, 2)) for p in parts] for n, parts in terms.items()}
    terms["dinitial_state"] = first

    def through_norm(parts, x, r):
        """Sums over a group's heads, then r (g - u (u.g)) with u = x / |x|, of each term."""
        sums = [p.map(lambda t: t.unflatten(2, (G, H // G))).sum(3) * r for p in parts]
        if not norm:
            return sums
        u = x * (x.square().sum(-1, keepdim=True) + eps).rsqrt()
        return [p - (p * u).sum(-1, keepdim=True) * u for p in sums]

    terms["dq"] = through_norm(terms["dq"], f["q"], rq)
    terms["dk"] = through_norm(terms["dk"], f["k"], rk)
    # automatic derivatives form the logistic's slope as b (1 - b), which cancels where b is close to
    # 1 (2^-53 of the rest of the product): here it is the product of both logistics
    strength = sum(p.m for p in terms["dbeta"])
    terms["dbeta"] = [p * db for p in terms["dbeta"]]
    exact = sum(p.v for p in terms["dbeta"])
    assert bool(((exact - grads["dbeta"]).abs() <= 2.0 ** -50 * strength + 1e-12 * exact.abs()).all())
    grads["dbeta"] = exact
    dg = terms["ddt"]
    terms["ddt"] = [p * slope for p in dg]
    terms["dA"] = [(p * rate).sum((0, 1)) for p in dg]
    terms["ddt_bias"] = [p.sum((0, 1)) for p in terms["ddt"]]
    return grads, terms


def bars(x, grads, terms):
    """{gradient: bar of every element}."""
    Bt, T, H, P = x["v"].shape
    N, io = x["q"].shape[-1], x["v"].dtype
    e = 8 * math.sqrt(T + N + P + 64) * U
    out = {}
    for n, parts in terms.items():
        out[n] = e * sum(p.m for p in parts) + TINY
        if n in ("dq", "dk", "dv") and io != torch.float32:
            out[n] = out[n] + IO_U[io] * 1.01 * grads[n].abs()
    return out
