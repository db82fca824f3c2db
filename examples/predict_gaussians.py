"""A network that predicts Gaussians from views, trained through the renderer.

Every 16x16 pixel tile of the input views is a token.  A few blocks (attention
with rotary positions in view, row and column; a gated unit) turn the tokens
into the 59 parameters of `per_token` Gaussians each; the training step renders
those and gives the gradient of the 59 parameters, which goes back through the
network.  Attention's products and the linear layers are torch products; what
passes over all tokens in between is the library's:

  gs_gated_norm_fwd/bwd   joins every two blocks: norm after, gate, residual
                          scale, sum, norm before; writes the next layer's
                          input and its 8-bit checkpoint in one pass
  gs_rope                 queries and keys, in place, and their gradients
  gs_glu_fwd/bwd          the gated unit, whose inputs are kept in 8 bits only
  gs_act8_wgrad           every weight gradient, from the 8-bit checkpoints

so that between the two directions a block keeps bytes, not 16-bit activations
(the residual stream and the block outputs stay as they are).

  python examples/predict_gaussians.py [--steps 20]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gaussian_splatting_differentiable_gs_gb300 as gs  # noqa: E402
import scenes  # noqa: E402

DT = torch.bfloat16


class Kept:
    """An 8-bit checkpoint's arrays and how many channels it has."""

    def __init__(self, tokens, channels):
        self.q, self.e = gs.act8_empty(tokens, channels)


class Network:
    """width = heads * 64; `groups`: the views, each with its own gates."""

    def __init__(self, views, rows, cols, width=256, blocks=2, per_token=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.C, self.F, self.V = views * rows * cols, width, 2 * width, views
        self.H, self.blocks, self.per_token = width // 64, blocks, per_token
        t = torch.arange(self.T, device="cuda")
        self.positions = torch.stack([t // (rows * cols), t % (rows * cols) // cols, t % cols],
                                     1).to(torch.int32).contiguous()
        self.rope = gs.Rope((16, 24, 24))
        self.offsets = torch.arange(0, self.T + 1, rows * cols, dtype=torch.int32, device="cuda")

        def lin(n, k, scale=1.0):
            return torch.randn(n, k, generator=g, device="cuda") * (scale / k ** 0.5)

        C, F = self.C, self.F
        self.w = {"embed": lin(C, 3 * 256), "head": lin(gs.NPARAM * per_token, C, 0.2)}
        for b in range(blocks):
            self.w.update({"qkv%d" % b: lin(3 * C, C), "out%d" % b: lin(C, C),
                           "up%d" % b: lin(2 * F, C), "down%d" % b: lin(C, F)})
        for j in range(2 * blocks + 1):  # the joins: before the first block, between, after the last
            self.w["pre%d" % j] = torch.ones(C, device="cuda")
            if j:
                self.w["post%d" % j] = torch.ones(C, device="cuda")
                self.w["scale%d" % j] = torch.full((C,), 0.5, device="cuda")
                self.w["gate%d" % j] = torch.ones(views, C, device="cuda")
        self.norm_ws = torch.empty(gs.gs_gated_norm_workspace_bytes(C, views), dtype=torch.uint8,
                                   device="cuda")
        room = max(gs.gs_act8_wgrad_workspace_bytes(self.T, w.shape[0], w.shape[1], dt)
                   for w in self.w.values() if w.dim() == 2 for dt in (DT, torch.float32))
        self.wgrad_ws = torch.zeros(room, dtype=torch.uint8, device="cuda")

    # ---- pieces ------------------------------------------------------------
    def _mat(self, c, dt=DT):
        return torch.empty(self.T, c, dtype=dt, device="cuda")

    def _linear(self, x, name):
        return x @ self.w[name].to(DT).t()

    def _linear_back(self, dy, kept, name, grads, need_dx=True):
        """The weight's gradient from the checkpoint of the layer's input; the input's."""
        w = self.w[name]
        grads[name] = torch.empty_like(w)
        gs.gs_act8_wgrad(dy, kept.q, kept.e, grads[name], self.wgrad_ws)
        return dy.to(DT) @ w.to(DT) if need_dx else None

    def _gate(self, j):
        return self.w["gate%d" % j].to(DT)

    def _join(self, x, block, j):
        """x' and the next layer's input y, with y's checkpoint."""
        y, stats, kept = self._mat(self.C), self._mat(4, torch.float32), Kept(self.T, self.C)
        if block is None:
            gs.gs_gated_norm_fwd(x, None, None, y, stats, w_pre=self.w["pre%d" % j], y_q=kept.q, y_e=kept.e)
            return x, y, (x, None, stats, kept)
        xo = self._mat(self.C)
        gs.gs_gated_norm_fwd(x, block, xo, y, stats, w_pre=self.w["pre%d" % j],
                             w_post=self.w["post%d" % j], gate=self._gate(j),
                             group_offsets=self.offsets, res_scale=self.w["scale%d" % j],
                             y_q=kept.q, y_e=kept.e)
        return xo, y, (xo, block, stats, kept)

    def _join_back(self, dx, dy, saved, j, grads):
        """(gradient of x, of the block before)."""
        xo, block, stats, _ = saved
        new = lambda n: torch.empty_like(self.w[n + str(j)])  # noqa: E731
        dxi = self._mat(self.C)
        grads["pre%d" % j] = new("pre")
        if block is None:
            gs.gs_gated_norm_bwd(xo, None, stats, dx, dy, dxi, None, w_pre=self.w["pre%d" % j],
                                 dw_pre=grads["pre%d" % j], workspace=self.norm_ws)
            return dxi, None
        db = self._mat(self.C)
        for n in ("post", "scale", "gate"):
            grads[n + str(j)] = new(n)
        gs.gs_gated_norm_bwd(xo, block, stats, dx, dy, dxi, db, w_pre=self.w["pre%d" % j],
                             w_post=self.w["post%d" % j], gate=self._gate(j),
                             group_offsets=self.offsets, res_scale=self.w["scale%d" % j],
                             dw_pre=grads["pre%d" % j], dw_post=grads["post%d" % j],
                             dgate=grads["gate%d" % j], dres_scale=grads["scale%d" % j],
                             workspace=self.norm_ws)
        return dxi, db

    @staticmethod
    def _attend(qkv):
        q, k, v = (t.transpose(0, 1) for t in qkv.unbind(1))  # [heads, tokens, 64]
        p = torch.softmax((q @ k.transpose(1, 2)).float() / 8.0, -1).to(DT)
        return (p @ v).transpose(0, 1).flatten(1)

    # ---- both directions -----------------------------------------------------
    def forward(self, pixels):
        """pixels [tokens, 768] -> the head's output [tokens, 59 * per_token] (fp32)."""
        self.saved, T, H = [], self.T, self.H
        kept = Kept(T, pixels.shape[1])
        gs.gs_act8_encode(pixels, kept.q, kept.e)
        self.saved.append(kept)
        x, y, s = self._join(self._linear(pixels, "embed"), None, 0)
        for b in range(self.blocks):
            self.saved.append(s)
            qkv = self._linear(y, "qkv%d" % b).view(T, 3, H, 64)
            gs.gs_rope(self.rope, self.positions, qkv[:, 0], qkv[:, 1])
            a = self._attend(qkv)
            kept = Kept(T, self.C)
            gs.gs_act8_encode(a, kept.q, kept.e)
            self.saved.append((qkv, kept))
            x, y, s = self._join(x, self._linear(a, "out%d" % b), 2 * b + 1)
            self.saved.append(s)
            gu, h = self._linear(y, "up%d" % b), self._mat(self.F)
            g8, u8 = Kept(T, self.F), Kept(T, self.F)
            gs.gs_glu_fwd(gu[:, :self.F], gu[:, self.F:], h, g8.q, g8.e, u8.q, u8.e)
            self.saved.append((g8, u8))
            x, y, s = self._join(x, self._linear(h, "down%d" % b), 2 * b + 2)
        self.saved.append(s)
        return self._linear(y, "head").float()

    def backward(self, dout):
        """Weight gradients from that of the head's output [tokens, 59 * per_token] (fp32)."""
        grads, saved, T = {}, list(self.saved), self.T
        s = saved.pop()
        dy = self._linear_back(dout, s[3], "head", grads)
        dx = None
        for b in reversed(range(self.blocks)):
            dx, db = self._join_back(dx, dy, s, 2 * b + 2, grads)
            g8, u8 = saved.pop()
            h8, dgu = Kept(T, self.F), self._mat(2 * self.F)
            gs.gs_glu_bwd(g8.q, g8.e, u8.q, u8.e, db @ self.w["down%d" % b].to(DT),
                          dgu[:, :self.F], dgu[:, self.F:], h8.q, h8.e)
            self._linear_back(db, h8, "down%d" % b, grads, need_dx=False)
            s = saved.pop()
            dy = self._linear_back(dgu, s[3], "up%d" % b, grads)
            dx, db = self._join_back(dx, dy, s, 2 * b + 1, grads)
            qkv, kept = saved.pop()
            da = self._linear_back(db, kept, "out%d" % b, grads)
            qkv = qkv.detach().requires_grad_(True)
            with torch.enable_grad():
                dqkv, = torch.autograd.grad(self._attend(qkv), qkv, da)
            gs.gs_rope(self.rope, self.positions, dqkv[:, 0], dqkv[:, 1], inverse=True)
            s = saved.pop()
            dy = self._linear_back(dqkv.reshape(T, 3 * self.C), s[3], "qkv%d" % b, grads)
        dx, _ = self._join_back(dx, dy, s, 0, grads)
        self._linear_back(dx, saved.pop(), "embed", grads, need_dx=False)
        return grads


def tiles_of(images):
    """[views, 3, H, W] -> tokens [views * (H/16) * (W/16), 768], bf16."""
    V, _, H, W = images.shape
    t = images.view(V, 3, H // 16, 16, W // 16, 16).permute(0, 2, 4, 1, 3, 5)
    return (t.reshape(-1, 768) - 0.5).to(DT).contiguous()


class Trainer:
    """Network and renderer: one step renders the predicted Gaussians into the
    input views and takes the L1 loss's gradient back to the weights."""

    def __init__(self, images, cams, lr=2e-3, **kw):
        V, _, H, W = images.shape
        self.net = Network(V, H // 16, W // 16, **kw)
        self.pixels = tiles_of(images)
        n = self.net.T * self.net.per_token
        self.base = self._base(cams, H, W, n)
        self.render = gs.TrainStep(self.base.clone(), cams, images, fused=True)
        self.spread = torch.full((gs.NPARAM, 1), 0.1, device="cuda")  # of each parameter per unit of output
        self.opt = torch.optim.Adam([w.requires_grad_(False) for w in self.net.w.values()], lr=lr)

    def _base(self, cams, H, W, n):
        """Gaussians on their tile's ray, four units from the camera."""
        base = torch.zeros(gs.NPARAM, n, device="cuda")
        rows, cols = H // 16, W // 16
        i = torch.arange(n, device="cuda") // self.net.per_token
        u, v = (i % cols) * 16.0 + 8, (i % (rows * cols) // cols) * 16.0 + 8
        for c, cam in enumerate(cams):
            of = i // (rows * cols) == c
            p = torch.stack([(u - cam["cx"]) / cam["fx"], (v - cam["cy"]) / cam["fy"], torch.ones_like(u)]) * 4
            R = torch.as_tensor(np.asarray(cam["R"], dtype=np.float32).reshape(3, 3), device="cuda")
            t = torch.as_tensor(np.asarray(cam["t"], dtype=np.float32).reshape(3, 1), device="cuda")
            base[:3] = torch.where(of, R.t() @ (p - t), base[:3])
        base[3:6], base[6] = float(np.log(4 * 8 / cams[0]["fx"])), 1.0
        return base

    def step(self):
        out = self.net.forward(self.pixels)
        delta = out.view(-1, gs.NPARAM).t()
        self.render.params.copy_(self.base + self.spread * delta)
        r = self.render
        r.project()
        r.bin_and_sort()
        r.rasterize_fused()
        r.project_bwd()
        grads = self.net.backward((r.grad * self.spread).t().contiguous().view(self.net.T, -1))
        for name, w in self.net.w.items():
            w.grad = grads[name]
        self.opt.step()
        return r.loss


def smooth_images(views, size, seed=0):
    """Smooth colour fields in [0, 1], as stand-ins for photographs."""
    g = torch.Generator().manual_seed(seed)
    x = torch.rand(views, 3, 6, 6, generator=g)
    return torch.nn.functional.interpolate(x, size=(size, size), mode="bicubic", align_corners=True).clamp(0, 1).cuda()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--size", type=int, default=256)
    a = ap.parse_args()
    cams = [scenes.camera(np.eye(3), [-0.2 * v, 0, 0], a.size, a.size, a.size / 2, a.size / 2, a.size, a.size)
            for v in range(2)]
    tr = Trainer(smooth_images(len(cams), a.size), cams)
    for i in range(a.steps):
        loss = tr.step()
        print("step %d  loss %.5f" % (i, loss.item()))
    assert gs.gs_workspace_status(tr.net.wgrad_ws) == gs.GS_OK


if __name__ == "__main__":
    main()
