"""The operators between two scans in float64 (numpy): test infrastructure.

The norms, their gradients and those of the depthwise convolution, written from
their definitions.  Gradients come from the chain rule term by term (Jacobian
products formed directly), not from the fused expressions the library uses.
"""
from __future__ import annotations

import numpy as np


def f64(t):
    """A tensor's exact float64 values."""
    if hasattr(t, "detach"):
        import torch
        return t.detach().to("cpu", torch.float64).numpy()
    return np.asarray(t, np.float64)


def logistic(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def silu(z):
    return z * logistic(z)


def silu_slope(z):
    s = logistic(z)
    return s + z * s * (1.0 - s)


def _parts(v, groups):
    return v.reshape(*v.shape[:-1], groups, v.shape[-1] // groups)


def norm(v, weight, eps, groups=1):
    u = _parts(v, groups)
    c = 1.0 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    return (u * c).reshape(v.shape) * weight


def norm_backward(v, weight, eps, dout, groups=1):
    """(dv, dweight): with n = v c, dn = dout * weight, dv = c dn + v dc,
    dc = sum(dn v) * dc/dv, dc/dv_j = -c^3 v_j / width."""
    u, dn = _parts(v, groups), _parts(dout * weight, groups)
    width = u.shape[-1]
    c = 1.0 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    dc = (dn * u).sum(-1, keepdims=True)
    dv = c * dn + dc * (-(c ** 3) * u / width)
    n = (u * c).reshape(v.shape)
    return dv.reshape(v.shape), (dout * n).reshape(-1, v.shape[-1]).sum(0)


def add_norm(x, weight, residual, scale, eps):
    r = scale * x + (0.0 if residual is None else residual)
    return norm(r, weight, eps), r


def add_norm_backward(r, weight, dy, dr_out, scale, eps):
    dv, dw = norm_backward(r, weight, eps, dy)
    dr = dv + (0.0 if dr_out is None else dr_out)
    return {"dx": scale * dr, "dresidual": dr, "dweight": dw}


def gated_norm(y, z, weight, eps, groups=1):
    return norm(y * silu(z), weight, eps, groups)


def gated_norm_backward(y, z, weight, dout, eps, groups=1):
    dg, dw = norm_backward(y * silu(z), weight, eps, dout, groups)
    return {"dy": dg * silu(z), "dz": dg * y * silu_slope(z), "dweight": dw}


def conv1d_backward(x, weight, bias, dy, state=None, dstate_out=None, silu_on=True):
    """Gradients of the causal convolution, token by token over all taps."""
    Bt, T, D = x.shape
    K = weight.shape[1]
    xp = np.zeros((Bt, T + K - 1, D))
    if state is not None:
        xp[:, :K - 1] = state.transpose(0, 2, 1)
    xp[:, K - 1:] = x
    z = np.zeros((Bt, T, D)) + (0.0 if bias is None else bias)
    for i in range(K):
        z += weight[:, i] * xp[:, i:i + T]
    dz = dy * (silu_slope(z) if silu_on else 1.0)
    dxp = np.zeros_like(xp)
    dw = np.zeros_like(weight)
    for i in range(K):
        dxp[:, i:i + T] += weight[:, i] * dz
        dw[:, i] = (dz * xp[:, i:i + T]).sum((0, 1))
    if dstate_out is not None:
        dxp[:, T:] += dstate_out.transpose(0, 2, 1)
    return {"dx": dxp[:, K - 1:], "dweight": dw, "dbias": dz.sum((0, 1)),
            "dstate": dxp[:, :K - 1].transpose(0, 2, 1), "dz": dz, "xp": xp, "z": z}
