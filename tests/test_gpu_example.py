"""The example block: its training gradients against automatic derivatives of
the same block in float64, its 8-bit serving path against the unquantised
forward, and a prompt continued token by token against the longer prompt."""
import os
import sys

import pytest
import torch

from gpu_util import TOL, announce, need_gpu

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def reference_block(s, p, x, residual):
    """The block token by token in float64 (torch, differentiable)."""
    def norm(v, w, groups=1):
        u = v.reshape(*v.shape[:-1], groups, -1)
        return (u / torch.sqrt((u * u).mean(-1, keepdim=True) + 1e-5)).reshape(v.shape) * w

    residual = residual + x
    proj = norm(residual, p["norm"]) @ p["w_in"].t()
    z, xbc, dt = proj.split([s.inner, s.channels, s.heads], -1)
    pad = torch.cat([torch.zeros(x.shape[0], s.taps - 1, s.channels, dtype=x.dtype), xbc], 1)
    T = x.shape[1]
    conv = p["conv_b"] + sum(pad[:, i:i + T] * p["conv_w"][:, i] for i in range(s.taps))
    conv = conv * torch.sigmoid(conv)
    gn = s.groups * s.dstate
    xs, B, C = conv.split([s.inner, gn, gn], -1)
    xs = xs.reshape(*x.shape[:2], s.heads, s.headdim)
    per = s.heads // s.groups
    B = B.reshape(*x.shape[:2], s.groups, s.dstate).repeat_interleave(per, 2)
    C = C.reshape(*x.shape[:2], s.groups, s.dstate).repeat_interleave(per, 2)
    d = torch.nn.functional.softplus(dt + p["dt_bias"]).clamp(1e-4, 0.5)
    h = torch.zeros(x.shape[0], s.heads, s.headdim, s.dstate, dtype=x.dtype)
    ys = []
    for t in range(T):
        h = (torch.exp(d[:, t] * p["A"])[..., None, None] * h
             + (d[:, t, :, None] * xs[:, t])[..., None] * B[:, t, :, None, :])
        ys.append((h * C[:, t, :, None, :]).sum(-1) + p["D"][:, None] * xs[:, t])
    y = torch.stack(ys, 1).reshape(*x.shape[:2], s.inner)
    g = norm(y * z * torch.sigmoid(z), p["gate_norm"], s.groups)
    return g @ p["w_out"].t(), residual


def rel(got, ref):
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    return float((got - ref).norm() / ref.norm())


@pytest.mark.parametrize("groups", [1, 2])
def test_training_gradients(groups):
    """float32, every gradient within the float32 bar of the scan's own tests."""
    need_gpu()
    import mamba2_block as mb
    s = mb.Shape(width=40, heads=4, headdim=16, dstate=32, groups=groups, chunk=32)
    announce(f"example training gradients, {groups} groups")
    p = mb.make_block(s, torch.float32, seed=groups)
    g = torch.Generator().manual_seed(3)
    x, r, dout, dres = (torch.randn(2, 45, s.width, generator=g) for _ in range(4))
    ref_p = {k: v.double().cpu().requires_grad_() for k, v in p.items()}
    rx, rr = x.double().requires_grad_(), r.double().requires_grad_()
    ref_out, ref_res = reference_block(s, ref_p, rx, rr)
    ((ref_out * dout).sum() + (ref_res * dres).sum()).backward()

    out, res, saved = mb.train_forward(s, p, x.cuda(), r.cuda())
    dx, dr, d = mb.train_backward(s, p, saved, dout.cuda(), dres.cuda())
    assert rel(out, ref_out) <= TOL["f32"] and rel(res, ref_res) <= TOL["f32"]
    assert rel(dx, rx.grad) <= TOL["f32"] and rel(dr, rr.grad) <= TOL["f32"]
    for k in ref_p:
        assert rel(d[k], ref_p[k].grad) <= TOL["f32"], k


def test_serving_in_8_bits():
    """Two products with both operands rounded to 127 steps of their row's
    largest value: for normal values (largest near 3.5 to 4 deviations) each
    operand carries about 4 / 127 / sqrt(12) = 0.9% and each product 1.3%, so
    the block's output stays within 5% of the unquantised one."""
    need_gpu()
    import mamba2_block as mb
    s = mb.Shape(width=256, heads=8, headdim=64, dstate=128, chunk=64)
    announce("example serving in 8 bits")
    p = mb.make_block(s, torch.bfloat16, seed=5)
    q = mb.quantise_block(p)
    g = torch.Generator().manual_seed(6)
    x = torch.randn(3, 131, s.width, generator=g).bfloat16().cuda()
    r = torch.randn(3, 131, s.width, generator=g).cuda()
    plain, _, _ = mb.train_forward(s, p, x, r)
    out, res, cache = mb.serve_prompt(s, q, x, r)
    assert rel(out, plain) <= 5e-2
    # 128 tokens at once, then three one by one
    first, _, (window, state) = mb.serve_prompt(s, q, x[:, :128].contiguous(), r[:, :128].contiguous())
    assert torch.equal(first, out[:, :128])
    for t in range(128, 131):
        o, rt = mb.serve_token(s, q, x[:, t].contiguous(), r[:, t].contiguous(), (window, state))
        assert rel(o, out[:, t]) <= TOL["bf16"] and torch.equal(rt, res[:, t])
    assert torch.equal(window, cache[0]) and rel(state, cache[1]) <= TOL["bf16"]
