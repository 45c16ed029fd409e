"""The example block of the gated delta rule: its training gradients against
automatic derivatives of the same block in float64, under the mask that the
dropout's oracle draws; a captured training step that advances its own offset; a
padded prompt continued token by token against the longer prompt."""
import os
import sys

import pytest
import torch

from gpu_util import TOL, announce, need_gpu
from oracle import delta, dropout

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def reference_block(s, p, x, residual, keep):
    """The block token by token in float64 (torch, differentiable)."""
    def norm(v, w, groups=1):
        u = v.reshape(*v.shape[:-1], groups, -1)
        return (u / torch.sqrt((u * u).mean(-1, keepdim=True) + 1e-5)).reshape(v.shape) * w

    residual = residual + x * keep / (1 - s.dropout)
    proj = norm(residual, p["norm"]) @ p["w_in"].t()
    z, qkv, dt, beta = proj.split([s.inner, s.channels, s.heads, s.heads], -1)
    pad = torch.cat([torch.zeros(x.shape[0], s.taps - 1, s.channels, dtype=x.dtype), qkv], 1)
    T = x.shape[1]
    conv = p["conv_b"] + sum(pad[:, i:i + T] * p["conv_w"][:, i] for i in range(s.taps))
    conv = conv * torch.sigmoid(conv)
    q, k, v = conv.split([s.keys, s.keys, s.inner], -1)
    split = lambda t, n: t.unflatten(-1, (n, -1))
    y, _ = delta.scan(split(q, s.groups), split(k, s.groups), split(v, s.heads), dt, p["A"], beta, p["dt_bias"])
    y = y.flatten(2)
    g = norm(y * z * torch.sigmoid(z), p["gate_norm"], s.heads)
    return g @ p["w_out"].t(), residual


def rel(got, ref):
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    return float((got - ref).norm() / ref.norm())


def mask(s, x, rng):
    seed, offset = (int(v) for v in rng.cpu())
    keep = dropout.kept(x.shape[0] * x.shape[1], s.width, s.dropout, seed, offset)
    return torch.as_tensor(keep, dtype=torch.float64).view(x.shape)


@pytest.mark.parametrize("heads,groups", [(4, 4), (6, 2)])
def test_training_gradients(heads, groups):
    """float32, every gradient within the float32 bar of the scan's own tests."""
    need_gpu()
    import delta_block as db
    s = db.Shape(width=40, heads=heads, headdim=16, dstate=32, groups=groups)
    announce(f"delta block training gradients, {heads} heads of {groups} groups")
    p = db.make_block(s, torch.float32, seed=groups)
    g = torch.Generator().manual_seed(3)
    x, r, dout, dres = (torch.randn(2, 85, s.width, generator=g) for _ in range(4))
    rng = torch.tensor([11, 1 << 33], device="cuda")
    ref_p = {k: v.double().cpu().requires_grad_() for k, v in p.items()}
    rx, rr = x.double().requires_grad_(), r.double().requires_grad_()
    ref_out, ref_res = reference_block(s, ref_p, rx, rr, mask(s, x, rng))
    ((ref_out * dout).sum() + (ref_res * dres).sum()).backward()

    out, res, saved = db.train_forward(s, p, x.cuda(), r.cuda(), rng)
    dx, dr, d = db.train_backward(s, p, saved, dout.cuda(), dres.cuda())
    assert rel(out, ref_out) <= TOL["f32"] and rel(res, ref_res) <= TOL["f32"]
    assert rel(dx, rx.grad) <= TOL["f32"] and rel(dr, rr.grad) <= TOL["f32"]
    for k in ref_p:
        assert rel(d[k], ref_p[k].grad) <= TOL["f32"], k


def test_captured_step():
    """A training step in a graph that advances the offset: every replay is the eager step at its
    offset, to the bit, with eager steps between."""
    need_gpu()
    import delta_block as db
    s = db.Shape(width=64, heads=4, headdim=64, dstate=128, groups=2)
    announce("delta block, captured step")
    p = db.make_block(s, torch.bfloat16, seed=8)
    g = torch.Generator().manual_seed(9)
    x, dout = (torch.randn(2, 70, s.width, generator=g).bfloat16().cuda() for _ in range(2))
    r, dres = (torch.randn(2, 70, s.width, generator=g).cuda() for _ in range(2))

    def step(rng):
        out, res, saved = db.train_forward(s, p, x, r, rng)
        rng[1] += 1
        dx, dr, d = db.train_backward(s, p, saved, dout, dres)
        return [out, res, dx, dr] + [d[k] for k in sorted(d)]

    rng = torch.tensor([5, 40], device="cuda")
    step(rng)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(rng)
    start = int(rng[1])
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert int(rng[1]) == start + i + 1
        for a, b in zip(got, step(torch.tensor([5, start + i], device="cuda"))):
            assert torch.equal(a, b), i
    assert not torch.equal(step(torch.tensor([5, 1], device="cuda"))[1], got[1])


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_serving(io):
    """Rows of different lengths in one padded prompt, each continued by three tokens from its cache."""
    need_gpu()
    import delta_block as db
    s = db.Shape(width=256, heads=8, headdim=64, dstate=128, groups=4)
    announce(f"delta block serving {io}")
    p = db.make_block(s, io, seed=5)
    g = torch.Generator().manual_seed(6)
    x = torch.randn(3, 134, s.width, generator=g).to(io).cuda()
    r = torch.randn(3, 134, s.width, generator=g).cuda()
    lengths = torch.tensor([131, 2, 70], device="cuda")
    tol = TOL["f32" if io == torch.float32 else "bf16"]
    _, _, cache = db.serve_prompt(s, p, x[:, :131].contiguous(), r[:, :131].contiguous(), lengths)
    rows = torch.arange(3, device="cuda")
    outs = [db.serve_token(s, p, x[rows, lengths + t].contiguous(), r[rows, lengths + t].contiguous(), cache)[0]
            for t in range(3)]
    for b in range(3):
        n = int(lengths[b])
        whole, _, (window, state) = db.serve_prompt(s, p, x[b:b + 1, :n + 3].contiguous(), r[b:b + 1, :n + 3].contiguous())
        for t in range(3):
            assert rel(outs[t][b], whole[0, n + t]) <= tol, (b, t)
        assert rel(cache[1][b], state[0]) <= tol and rel(cache[0][b], window[0]) <= tol, b
