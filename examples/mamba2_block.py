"""One Mamba-2 block on the library's operators, trained and served.

    residual add + norm -> first projection -> convolution -> scan ->
    gated norm -> second projection

Training keeps the projections in the io type (plain matrix products) and runs
the whole block forward and backward; serving keeps them in 8 bits, with a
scale per output channel laid out once and a scale per token from the norms
that feed them, over a prompt and then token by token from the cached window
and state.

    python examples/mamba2_block.py        times both at the 2.7B layer shape

Weights are random: the example shows how the operators are called together.
Source: "Compiler-First State Space Duality and Portable O(1) Autoregressive
Caching", Implementation choices and O(1) cache.
"""
from __future__ import annotations

import math
import os
import sys
from dataclasses import dataclass

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import state_space_model_amd as ssd  # noqa: E402


@dataclass(frozen=True)
class Shape:
    """Sizes of a block: `width` of the residual stream, `heads` of `headdim`
    channels, `groups` of B/C and of the gated norm, state size `dstate`."""
    width: int
    heads: int
    headdim: int
    dstate: int
    groups: int = 1
    taps: int = 4
    chunk: int = 256

    @property
    def inner(self):
        return self.heads * self.headdim

    @property
    def channels(self):                     # of the convolution: x, B and C
        return self.inner + 2 * self.groups * self.dstate

    @property
    def projected(self):                    # gate, convolution channels, dt
        return self.inner + self.channels + self.heads


def make_block(s: Shape, io: torch.dtype, seed: int = 0, device="cuda") -> dict:
    """Random parameters of one block: projections in `io`, the rest float32."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *shape: torch.randn(*shape, generator=g)
    u = lambda *shape: torch.rand(*shape, generator=g)
    p = {"norm": 1 + 0.1 * n(s.width), "w_in": n(s.projected, s.width) / math.sqrt(s.width),
         "conv_w": u(s.channels, s.taps) - 0.5, "conv_b": u(s.channels) - 0.5,
         "A": -torch.exp(u(s.heads) * math.log(16.0)), "D": n(s.heads),
         "dt_bias": torch.log(torch.expm1(u(s.heads) * 0.1 + 1e-3)),
         "gate_norm": 1 + 0.1 * n(s.inner),
         "w_out": n(s.width, s.inner) / math.sqrt(s.inner)}
    return {k: v.to(device, io if k.startswith("w_") else torch.float32) for k, v in p.items()}


def split_projection(s: Shape, zxd: torch.Tensor):
    """The gate (a slice, read where it lies), the convolution's input and dt."""
    z, xbc, dt = zxd.split([s.inner, s.channels, s.heads], -1)
    return z, xbc.contiguous(), dt.float().contiguous()


def split_channels(s: Shape, xbc: torch.Tensor):
    """x [..., H, P], B and C [..., G, N] of the convolution's output."""
    gn = s.groups * s.dstate
    x, B, C = xbc.split([s.inner, gn, gn], -1)
    lead = xbc.shape[:-1]
    return (x.reshape(*lead, s.heads, s.headdim), B.reshape(*lead, s.groups, s.dstate),
            C.reshape(*lead, s.groups, s.dstate))


# --------------------------------------------------------------------------
# training
# --------------------------------------------------------------------------
def train_forward(s: Shape, p: dict, x: torch.Tensor, residual=None):
    """x [Bt,T,width]: (the block's output, the residual stream, what the
    backward pass reads)."""
    h, residual = ssd.ssd_add_norm(x, p["norm"], residual)
    z_xbc_dt = torch.matmul(h, p["w_in"].t())
    z, xbc, dt = split_projection(s, z_xbc_dt)
    conv, _ = ssd.ssd_conv1d(xbc, p["conv_w"], p["conv_b"], return_state=False)
    xs, B, C = (t.contiguous() for t in split_channels(s, conv))
    y, _ = ssd.ssd_chunk_scan(xs, dt, p["A"], B, C, p["D"], chunk=s.chunk, dt_bias=p["dt_bias"],
                              return_final_state=False)
    y = y.view(*x.shape[:2], s.inner)
    g = ssd.ssd_gated_norm(y, z, p["gate_norm"], groups=s.groups)
    out = torch.matmul(g, p["w_out"].t())
    return out, residual, (h, residual, z_xbc_dt, xbc, dt, xs, B, C, y, g)


def train_backward(s: Shape, p: dict, saved, dout: torch.Tensor, dresidual=None):
    """Gradients of train_forward for sum(dout * out) + sum(dresidual *
    residual): (dx, the incoming residual's, a dict of the parameters')."""
    h, residual, z_xbc_dt, xbc, dt, xs, B, C, y, g = saved
    z = z_xbc_dt[..., :s.inner]
    flat = lambda t: t.reshape(-1, t.shape[-1])
    d = {"w_out": flat(dout).t() @ flat(g)}
    # gate, convolution channels and dt of the projection's gradient, side by side
    dproj = torch.empty_like(z_xbc_dt)
    gn = ssd.ssd_gated_norm_backward(y, z, p["gate_norm"], dout=torch.matmul(dout, p["w_out"]),
                                     groups=s.groups, grads={"dz": dproj[..., :s.inner]})
    d["gate_norm"] = gn["dweight"]
    sc = ssd.ssd_chunk_scan_backward(xs, dt, p["A"], B, C, p["D"], dy=gn["dy"].view_as(xs),
                                     chunk=s.chunk, dt_bias=p["dt_bias"])
    d["A"], d["D"], d["dt_bias"] = sc["dA"], sc["dD"], sc["ddt_bias"]
    dconv = torch.cat([sc[k].flatten(2) for k in ("dx", "dB", "dC")], -1)     # float32
    cv = ssd.ssd_conv1d_backward(xbc, p["conv_w"], p["conv_b"], dy=dconv)
    d["conv_w"], d["conv_b"] = cv["dweight"], cv["dbias"]
    dproj[..., s.inner:s.inner + s.channels] = cv["dx"]
    dproj[..., s.inner + s.channels:] = sc["ddt"]
    d["w_in"] = flat(dproj).t() @ flat(h)
    an = ssd.ssd_add_norm_backward(residual, p["norm"], dy=torch.matmul(dproj, p["w_in"]),
                                   dresidual_out=dresidual)
    d["norm"] = an["dweight"]
    return an["dx"], an["dresidual"], d


# --------------------------------------------------------------------------
# serving
# --------------------------------------------------------------------------
def quantise_block(p: dict) -> dict:
    """The block's parameters with its projections in 8 bits."""
    q = {k: v for k, v in p.items() if not k.startswith("w_")}
    q["w_in"] = ssd.ssd_quantize_q8(p["w_in"])
    q["w_out"] = ssd.ssd_quantize_q8(p["w_out"])
    return q


def serve_prompt(s: Shape, q: dict, x: torch.Tensor, residual=None):
    """x [Bt,T,width]: (output, residual stream, cache) after a whole prompt."""
    h, hs, residual = ssd.ssd_add_norm_q8(x, q["norm"], residual)
    z, xbc, dt = split_projection(s, ssd.ssd_linear_q8(h, hs, *q["w_in"], out_dtype=x.dtype))
    conv, window = ssd.ssd_conv1d(xbc, q["conv_w"], q["conv_b"])
    xs, B, C = (t.contiguous() for t in split_channels(s, conv))
    y, state = ssd.ssd_chunk_scan(xs, dt, q["A"], B, C, q["D"], chunk=s.chunk, dt_bias=q["dt_bias"])
    g, gs = ssd.ssd_gated_norm_q8(y.view(*x.shape[:2], s.inner), z, q["gate_norm"], groups=s.groups)
    return ssd.ssd_linear_q8(g, gs, *q["w_out"], out_dtype=x.dtype), residual, (window, state)


def serve_token(s: Shape, q: dict, x: torch.Tensor, residual, cache):
    """x [Bt,width]: (output, residual stream); the cache is updated in place."""
    window, state = cache
    h, hs, residual = ssd.ssd_add_norm_q8(x, q["norm"], residual)
    z, xbc, dt = split_projection(s, ssd.ssd_linear_q8(h, hs, *q["w_in"], out_dtype=x.dtype))
    xs, B, C = split_channels(s, ssd.ssd_conv1d_step(window, xbc, q["conv_w"], q["conv_b"]))
    y = ssd.ssd_step(state, xs.contiguous(), dt, q["A"], B.contiguous(), C.contiguous(), q["D"],
                     dt_bias=q["dt_bias"])
    g, gs = ssd.ssd_gated_norm_q8(y.view(x.shape[0], s.inner), z, q["gate_norm"], groups=s.groups)
    return ssd.ssd_linear_q8(g, gs, *q["w_out"], out_dtype=x.dtype), residual


def main():
    s = Shape(width=2560, heads=80, headdim=64, dstate=128)
    io = torch.bfloat16
    p = make_block(s, io)
    q = quantise_block(p)
    x = torch.randn(1, 4096, s.width, device="cuda").to(io)
    r = torch.randn(1, 4096, s.width, device="cuda")

    def timed(name, f, reps=20):
        f()
        torch.cuda.synchronize()
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        for _ in range(reps):
            f()
        e1.record()
        torch.cuda.synchronize()
        print(f"{name}: {e0.elapsed_time(e1) / reps * 1e3:.1f} us", flush=True)

    def step():
        out, res, saved = train_forward(s, p, x, r)
        train_backward(s, p, saved, out, res)

    timed("train, 4096 tokens, forward", lambda: train_forward(s, p, x, r))
    timed("train, 4096 tokens, forward and backward", step)
    timed("serve, prompt of 4096 tokens", lambda: serve_prompt(s, q, x, r))
    for batch in (1, 64):
        _, _, cache = serve_prompt(s, q, x[:, :64].expand(batch, 64, s.width).contiguous())
        xt, rt = x[0, :batch].contiguous(), r[0, :batch].contiguous()
        graph = torch.cuda.CUDAGraph()
        serve_token(s, q, xt, rt, cache)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            serve_token(s, q, xt, rt, cache)
        timed(f"serve, one token, batch {batch} (graph)", graph.replay, 200)


if __name__ == "__main__":
    main()
