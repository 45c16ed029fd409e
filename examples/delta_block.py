"""One block of the gated delta rule on the library's operators, trained and served.

    dropout, residual add + norm -> first projection -> convolution ->
    gated delta rule -> gated norm -> second projection

The convolution's output holds queries, keys and values side by side; the scan
reads them where they lie, and its gradients are written back the same way.
Dropout's mask is drawn again in the backward pass from a seed and an offset that
live on the device: a captured step advances them itself.  Serving runs a prompt
and then single tokens from the cached window and state.

    python examples/delta_block.py         times both at 2.7B layer sizes

Weights are random: the example shows how the operators are called together.
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
    values, `groups` of queries and keys of `dstate`."""
    width: int
    heads: int
    headdim: int
    dstate: int
    groups: int
    taps: int = 4
    dropout: float = 0.1

    @property
    def inner(self):
        return self.heads * self.headdim

    @property
    def keys(self):
        return self.groups * self.dstate

    @property
    def channels(self):                     # of the convolution: q, k and v
        return 2 * self.keys + self.inner

    @property
    def projected(self):                    # gate, convolution channels, decay, write strength
        return self.inner + self.channels + 2 * self.heads


def make_block(s: Shape, io: torch.dtype, seed: int = 0, device="cuda") -> dict:
    """Random parameters of one block: projections in `io`, the rest float32."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *shape: torch.randn(*shape, generator=g)
    u = lambda *shape: torch.rand(*shape, generator=g)
    p = {"norm": 1 + 0.1 * n(s.width), "w_in": n(s.projected, s.width) / math.sqrt(s.width),
         "conv_w": u(s.channels, s.taps) - 0.5, "conv_b": u(s.channels) - 0.5,
         "A": -torch.exp(u(s.heads) * math.log(16.0)),
         "dt_bias": torch.log(torch.expm1(u(s.heads) * 0.1 + 1e-3)),
         "gate_norm": 1 + 0.1 * n(s.inner),
         "w_out": n(s.width, s.inner) / math.sqrt(s.inner)}
    return {k: v.to(device, io if k.startswith("w_") else torch.float32) for k, v in p.items()}


def split_projection(s: Shape, proj: torch.Tensor):
    """The gate (a slice, read where it lies), the convolution's input, decay and write strength."""
    z, qkv, dt, beta = proj.split([s.inner, s.channels, s.heads, s.heads], -1)
    return z, qkv.contiguous(), dt.float().contiguous(), beta.float().contiguous()


def split_channels(s: Shape, qkv: torch.Tensor):
    """q and k [..., G, N], v [..., H, P]: slices of the convolution's output."""
    q, k, v = qkv.split([s.keys, s.keys, s.inner], -1)
    return (q.unflatten(-1, (s.groups, s.dstate)), k.unflatten(-1, (s.groups, s.dstate)),
            v.unflatten(-1, (s.heads, s.headdim)))


# --------------------------------------------------------------------------
# training
# --------------------------------------------------------------------------
def train_forward(s: Shape, p: dict, x: torch.Tensor, residual, rng: torch.Tensor):
    """x [Bt,T,width], rng [2] int64 (seed, offset): (the block's output, the
    residual stream, what the backward pass reads)."""
    h, residual = ssd.ssd_dropout_add_norm(x, p["norm"], residual, p=s.dropout, rng=rng)
    proj = torch.matmul(h, p["w_in"].t())
    z, qkv, dt, beta = split_projection(s, proj)
    conv, _ = ssd.ssd_conv1d(qkv, p["conv_w"], p["conv_b"], return_state=False)
    y, _ = ssd.ssd_delta_scan(*split_channels(s, conv), dt, p["A"], beta, dt_bias=p["dt_bias"],
                              return_final_state=False)
    y = y.flatten(2)
    g = ssd.ssd_gated_norm(y, z, p["gate_norm"], groups=s.heads)
    out = torch.matmul(g, p["w_out"].t())
    return out, residual, (h, residual, proj, qkv, dt, beta, conv, y, g, rng.clone())


def train_backward(s: Shape, p: dict, saved, dout: torch.Tensor, dresidual=None):
    """Gradients of train_forward for sum(dout * out) + sum(dresidual *
    residual): (dx, the incoming residual's, a dict of the parameters')."""
    h, residual, proj, qkv, dt, beta, conv, y, g, rng = saved
    z = proj[..., :s.inner]
    flat = lambda t: t.reshape(-1, t.shape[-1])
    d = {"w_out": flat(dout).t() @ flat(g)}
    # gate, convolution channels, decay and write strength of the projection's gradient, side by side
    dproj = torch.empty_like(proj)
    gn = ssd.ssd_gated_norm_backward(y, z, p["gate_norm"], dout=torch.matmul(dout, p["w_out"]),
                                     groups=s.heads, grads={"dz": dproj[..., :s.inner]})
    d["gate_norm"] = gn["dweight"]
    q, k, v = split_channels(s, conv)
    dconv = torch.empty_like(conv)
    sc = ssd.ssd_delta_scan_backward(q, k, v, dt, p["A"], beta, dt_bias=p["dt_bias"], dy=gn["dy"].view_as(v),
                                     grads=dict(zip(("dq", "dk", "dv"), split_channels(s, dconv))))
    d["A"], d["dt_bias"] = sc["dA"], sc["ddt_bias"]
    cv = ssd.ssd_conv1d_backward(qkv, p["conv_w"], p["conv_b"], dy=dconv)
    d["conv_w"], d["conv_b"] = cv["dweight"], cv["dbias"]
    rest = dproj[..., s.inner:]
    rest[..., :s.channels] = cv["dx"]
    rest[..., s.channels:s.channels + s.heads] = sc["ddt"]
    rest[..., s.channels + s.heads:] = sc["dbeta"]
    d["w_in"] = flat(dproj).t() @ flat(h)
    an = ssd.ssd_dropout_add_norm_backward(residual, p["norm"], dy=torch.matmul(dproj, p["w_in"]),
                                           p=s.dropout, rng=rng, dresidual_out=dresidual)
    d["norm"] = an["dweight"]
    return an["dx"], an["dresidual"], d


# --------------------------------------------------------------------------
# serving
# --------------------------------------------------------------------------
def serve_prompt(s: Shape, p: dict, x: torch.Tensor, residual=None, lengths=None):
    """x [Bt,T,width]: (output, residual stream, cache) after a whole prompt.
    `lengths` [Bt]: rows that end earlier; their padding changes no state."""
    h, residual = ssd.ssd_add_norm(x, p["norm"], residual)
    z, qkv, dt, beta = split_projection(s, torch.matmul(h, p["w_in"].t()))
    conv, window = ssd.ssd_conv1d(qkv, p["conv_w"], p["conv_b"])
    if lengths is not None:
        past = torch.arange(x.shape[1], device=x.device) >= lengths[:, None]
        dt.masked_fill_(past[..., None], -math.inf)      # no decay and no write
        beta.masked_fill_(past[..., None], -math.inf)
        at = lengths[:, None] - torch.arange(s.taps - 1, 0, -1, device=x.device)
        last = qkv.gather(1, at.clamp(min=0)[..., None].expand(-1, -1, s.channels))
        window = torch.where((at >= 0)[..., None], last, 0).transpose(1, 2).contiguous()
    y, state = ssd.ssd_delta_scan(*split_channels(s, conv), dt, p["A"], beta, dt_bias=p["dt_bias"])
    g = ssd.ssd_gated_norm(y.flatten(2), z, p["gate_norm"], groups=s.heads)
    return torch.matmul(g, p["w_out"].t()), residual, (window, state)


def serve_token(s: Shape, p: dict, x: torch.Tensor, residual, cache):
    """x [Bt,width]: (output, residual stream); the cache is updated in place."""
    window, state = cache
    h, residual = ssd.ssd_add_norm(x, p["norm"], residual)
    z, qkv, dt, beta = split_projection(s, torch.matmul(h, p["w_in"].t()))
    conv = ssd.ssd_conv1d_step(window, qkv, p["conv_w"], p["conv_b"])
    y = ssd.ssd_delta_step(state, *split_channels(s, conv), dt, p["A"], beta, dt_bias=p["dt_bias"])
    g = ssd.ssd_gated_norm(y.flatten(1), z, p["gate_norm"], groups=s.heads)
    return torch.matmul(g, p["w_out"].t()), residual


def main():
    s = Shape(width=2560, heads=80, headdim=64, dstate=128, groups=80)
    io = torch.bfloat16
    p = make_block(s, io)
    x = torch.randn(1, 4096, s.width, device="cuda").to(io)
    r = torch.randn(1, 4096, s.width, device="cuda")
    rng = torch.tensor([1, 0], device="cuda")

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
        out, res, saved = train_forward(s, p, x, r, rng)
        rng[1] += 1
        train_backward(s, p, saved, out, res)

    timed("train, 4096 tokens, forward", lambda: train_forward(s, p, x, r, rng))
    timed("train, 4096 tokens, forward and backward", step)
    timed("serve, prompt of 4096 tokens", lambda: serve_prompt(s, p, x, r))
    for batch in (1, 64):
        _, _, cache = serve_prompt(s, p, x[:, :64].expand(batch, 64, s.width).contiguous())
        xt, rt = x[0, :batch].contiguous(), r[0, :batch].contiguous()
        graph = torch.cuda.CUDAGraph()
        serve_token(s, p, xt, rt, cache)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            serve_token(s, p, xt, rt, cache)
        timed(f"serve, one token, batch {batch} (graph)", graph.replay, 200)


if __name__ == "__main__":
    main()
