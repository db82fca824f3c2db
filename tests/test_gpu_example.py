"""The example network: its operators together, against plain torch."""
import os
import sys

import numpy as np
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
    T, C, H, F = net.T, net.C, net.H, net.F
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

    def join(x, block, j):
        if block is not None:
            x = x + w["scale%d" % j] * w["gate%d" % j][of] * (w["post%d" % j] * norm(block))
        return x, norm(x) * w["pre%d" % j]

    x, y = join(pixels.float() @ w["embed"].t(), None, 0)
    for b in range(net.blocks):
        q, k, v = (y @ w["qkv%d" % b].t()).view(T, 3, H, 64).unbind(1)
        q, k, v = (t.transpose(0, 1) for t in (rope(q), rope(k), v))
        a = (torch.softmax(q @ k.transpose(1, 2) / 8.0, -1) @ v).transpose(0, 1).flatten(1)
        x, y = join(x, a @ w["out%d" % b].t(), 2 * b + 1)
        gu = y @ w["up%d" % b].t()
        h = torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]
        x, y = join(x, h @ w["down%d" % b].t(), 2 * b + 2)
    return y @ w["head"].t()


def test_network_matches_plain_torch(ex):
    """Outputs within bf16's roundings (2^-9 at each of about 20 roundings, added
    in quadrature and amplified by a few: 5 %), gradients within those and the
    checkpoints' (a step of at most 1/63.5 of a group's largest value: 1 to 2 %
    each)."""
    net = ex.Network(2, 6, 5, width=128, blocks=2, per_token=1, seed=3)
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


def test_training_through_the_renderer(ex):
    import scenes
    cams = [scenes.camera(np.eye(3), [-0.2 * v, 0, 0], 96, 96, 48, 48, 96, 96) for v in range(2)]
    tr = ex.Trainer(ex.smooth_images(2, 96), cams, width=128, blocks=1, per_token=1)
    losses = [float(tr.step()) for _ in range(12)]
    assert all(np.isfinite(losses)) and losses[-1] < 0.8 * losses[0], losses
    assert ex.gs.gs_workspace_status(tr.net.wgrad_ws) == ex.gs.GS_OK
