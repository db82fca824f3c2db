"""The feed-forward block and linear attention in a run together, as the example network
uses them: next to rotary positions, gated norms and 8-bit checkpoints."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    import __graft_entry__
    __graft_entry__.build()
    import predict_gaussians
    return predict_gaussians


def _plain(net, w, pixels):
    """The same network in fp32 torch, differentiable in its weights."""
    T, H, F = net.T, net.H, net.F
    of = torch.arange(T, device="cuda") // (T // net.V)

    def norm(x):
        return x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-6)

    def rope(x):
        y, at = [], 0
        for a, d in enumerate(net.rope.dims):
            f = 10000.0 ** (-torch.arange(0, d, 2, device="cuda") / d)
            ang = (net.positions[:, a, None].float() * f)[:, None]
            u, v = x[..., at:at + d // 2], x[..., at + d // 2:at + d]
            y += [u * ang.cos() - v * ang.sin(), u * ang.sin() + v * ang.cos()]
            at += d
        return torch.cat(y, -1)

    def attend(q, k, v):
        q, k, v = (t.transpose(0, 1) for t in (q, k, v))
        s = q @ k.transpose(1, 2) / 8.0
        if not net.linear:
            return (torch.softmax(s, -1) @ v).transpose(0, 1).flatten(1)
        gap = torch.arange(T, device="cuda")[:, None] - torch.arange(T, device="cuda")
        d = torch.where(gap >= 0, torch.exp(net.log_decay[:, None, None] * gap.clamp(min=0)), 0.0)
        return ((s * d) @ v).transpose(0, 1).flatten(1)

    def join(x, block, j):
        if block is not None:
            x = x + w["scale%d" % j] * w["gate%d" % j][of] * (w["post%d" % j] * norm(block))
        return x, norm(x) * w["pre%d" % j]

    x, y = join(pixels.float() @ w["embed"].t(), None, 0)
    for b in range(net.blocks):
        q, k, v = (y @ w["qkv%d" % b].t()).view(T, 3, H, 64).unbind(1)
        x, y = join(x, attend(rope(q), rope(k), v) @ w["out%d" % b].t(), 2 * b + 1)
        gu = y @ w["up%d" % b].t()
        h = torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]
        x, y = join(x, h @ w["down%d" % b].t(), 2 * b + 2)
    return y @ w["head"].t()


@pytest.mark.parametrize("linear,fused", [(True, False), (False, True), (True, True)])
def test_network_matches_plain_torch(ex, linear, fused):
    """Outputs within bf16's roundings (2^-9 at each of about 20 roundings, added
    in quadrature and amplified by a few: 5 %), gradients within those and the
    checkpoints' (a step of at most 1/63.5 of a group's largest value: 1 to 2 %
    each)."""
    net = ex.Network(2, 13, 11, width=128, blocks=2, per_token=1, seed=3, linear=linear, fused=fused)
    g = torch.Generator(device="cuda").manual_seed(4)
    pixels = torch.randn(net.T, 768, generator=g, device="cuda").to(torch.bfloat16)
    for name, v in net.w.items():
        if v.dim() == 1 or name.startswith("gate"):
            v += 0.1 * torch.randn(v.shape, generator=g, device="cuda")
    out = net.forward(pixels)
    w = {k: v.clone().requires_grad_(True) for k, v in net.w.items()}
    want = _plain(net, w, pixels)
    assert (out - want).norm() <= 0.05 * want.norm()
    dout = torch.randn(out.shape, generator=g, device="cuda")
    grads = net.backward(dout)
    want.backward(dout)
    assert set(grads) == set(w)
    for name in w:
        err = (grads[name] - w[name].grad).norm() / w[name].grad.norm()
        assert err <= 0.1, (name, float(err))
    ex.gs.gs_linear_attn_status()
    if fused:
        assert ex.gs.gs_workspace_status(net.ffn_ws) == ex.gs.GS_OK


def test_the_example_trains_with_both(ex):
    import numpy as np

    import scenes
    cams = [scenes.camera(np.eye(3), [-0.2 * v, 0, 0], 96, 96, 48, 48, 96, 96) for v in range(2)]
    tr = ex.Trainer(ex.smooth_images(2, 96), cams, width=128, blocks=1, per_token=1, linear=True, fused=True)
    before = {k: v.clone() for k, v in tr.net.w.items()}
    assert all(np.isfinite(float(tr.step())) for _ in range(3))
    assert all(torch.isfinite(v).all() and not torch.equal(v, before[k]) for k, v in tr.net.w.items())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_a_prompt_and_then_single_tokens(ex, dt):
    """One stream's block: the chunked form over the first tokens leaves the state that the
    single tokens go on from; the feed-forward block takes many rows and then one.  Both
    agree with the chunked forms over all tokens (whose own errors are half of the bound)."""
    gs = ex.gs
    g = torch.Generator(device="cuda").manual_seed(1)
    T, P, H, D, C, F = 150, 141, 4, 64, 256, 320
    q, k, v = (torch.randn(T, H, D, generator=g, device="cuda").to(dt) for _ in range(3))
    w = (torch.randn(2 * F, C, generator=g, device="cuda") / 16).to(dt)
    a = -torch.exp2(-2.0 * torch.arange(1, H + 1, device="cuda"))
    ws = torch.empty(gs.gs_linear_attn_workspace_bytes(T, H, H, D, D), dtype=torch.uint8, device="cuda")
    fws = torch.zeros(gs.gs_ffn_workspace_bytes(T, C, F), dtype=torch.uint8, device="cuda")

    def block(attend, n):
        x = torch.empty(n, H, D, dtype=dt, device="cuda")
        attend(x)
        h = torch.empty(n, F, dtype=dt, device="cuda")
        gs.gs_ffn_fwd(x.flatten(1), w, h, fws)
        return x, h

    whole_s, s = torch.empty(1, H, D, D, device="cuda"), torch.empty(1, H, D, D, device="cuda")
    x, h = block(lambda o: gs.gs_linear_attn_fwd(q, k, v, a, o, state_out=whole_s, workspace=ws), T)
    xs, hs = block(lambda o: gs.gs_linear_attn_fwd(q[:P], k[:P], v[:P], a, o, state_out=s, workspace=ws), P)
    assert torch.equal(xs, x[:P]) and torch.equal(hs, h[:P])  # a chunk's results do not depend on what follows
    eps = torch.finfo(dt).eps
    for t in range(P, T):
        xt, ht = block(lambda o: gs.gs_linear_attn_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], a, s, o), 1)
        assert (xt - x[t:t + 1]).float().norm() <= 3 * eps * x[t:t + 1].float().norm()
        assert (ht - h[t:t + 1]).float().norm() <= 8 * eps * h[t:t + 1].float().norm()
    assert (s - whole_s).norm() <= 1e-5 * whole_s.norm()
