"""The gated delta rule in float64 (torch on the CPU), token by token from its
definition: test infrastructure.  Every operation is differentiable, so that
gradients come from automatic differentiation of the recurrence, not from the
chunked formulas that the library uses."""
from __future__ import annotations

import math

import torch


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64)


def rates(dt, dt_bias, softplus=True, limit=(0.0, math.inf)):
    z = dt if dt_bias is None else dt + dt_bias
    if softplus:
        z = torch.logaddexp(z, torch.zeros_like(z))
    return torch.clamp(z, *limit)


def unit(x, eps):
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + eps)


def scan(q, k, v, dt, A, beta, dt_bias=None, *, softplus=True, limit=(0.0, math.inf), sigmoid=True,
         norm=True, eps=1e-6, scale=None, h0=None):
    """(y [Bt,T,H,P], states [T+1] of [Bt,H,P,N]) of float64 inputs."""
    Bt, T, H, P = v.shape
    G, N = q.shape[-2:]
    scale = 1.0 / math.sqrt(N) if scale is None else scale
    if norm:
        q, k = unit(q, eps), unit(k, eps)
    q, k = (x.repeat_interleave(H // G, -2) for x in (q * scale, k))
    a = torch.exp(rates(dt, dt_bias, softplus, limit) * A)
    b = torch.sigmoid(beta) if sigmoid else beta
    state = torch.zeros(Bt, H, P, N, dtype=torch.float64) if h0 is None else h0
    ys, states = [], [state]
    for t in range(T):
        kt = k[:, t, :, None, :]
        state = a[:, t, :, None, None] * state
        write = b[:, t, :, None] * (v[:, t] - (state * kt).sum(-1))
        state = state + write[..., None] * kt
        ys.append((state * q[:, t, :, None, :]).sum(-1))
        states.append(state)
    y = torch.stack(ys, 1) if T else torch.zeros(Bt, 0, H, P, dtype=torch.float64)
    return y, states


def gradients(inputs, dy, dfinal=None, **options):
    """Gradients of sum(dy y) + sum(dfinal final) with respect to every float64
    input of the dict `inputs` (q, k, v, dt, A, beta, and dt_bias, h0 if there),
    and the states and their gradients."""
    leaves = {n: t.clone().requires_grad_(True) for n, t in inputs.items() if t is not None}
    y, states = scan(**leaves, **options)
    loss = (y * dy).sum()
    if dfinal is not None:
        loss = loss + (states[-1] * dfinal).sum()
    kept = [s for s in states if s.requires_grad]
    got = torch.autograd.grad(loss, list(leaves.values()) + kept, allow_unused=True)
    grads = {"d" + n: torch.zeros_like(x) if g is None else g
             for (n, x), g in zip(leaves.items(), got)}
    return grads, [s.detach() for s in states], [g for g in got[len(leaves):] if g is not None]
