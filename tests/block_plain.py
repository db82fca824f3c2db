"""Plain 64-bit forms of the gated feed-forward block and of linear attention with
decays (CPU tensors), which the GPU tests compare the library with.  They share no code
with it."""
import torch

import net_plain


def ffn(x, w, act):
    """(h, gate, up) of x [T, C] and w [2F, C]; differentiable."""
    F = w.shape[0] // 2
    gate, up = x @ w[:F].t(), x @ w[F:].t()
    return net_plain.act(gate, act) * up, gate, up


def act_both(v, name):
    """The function and its derivative."""
    v = v.detach().requires_grad_(True)
    f = net_plain.act(v, name)
    df, = torch.autograd.grad(f.sum(), v)
    return f.detach(), df


def attn(q, k, v, log_decay, offsets, state, scale):
    """(out, last states), token after token; differentiable.  Heads are shared, groups
    may be empty; rows outside the groups are zeros."""
    T, H, D = q.shape
    rep = H // k.shape[1]
    k, v = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    d = torch.exp(log_decay.double())[:, None, None]
    rows, last = [torch.zeros(H, v.shape[2], dtype=torch.float64)] * T, []
    for g in range(len(offsets) - 1):
        S = state[g] if state is not None else torch.zeros(H, D, v.shape[2], dtype=torch.float64)
        for t in range(int(offsets[g]), int(offsets[g + 1])):
            S = d * S + k[t][:, :, None] * v[t][:, None, :]
            rows[t] = scale * (q[t][:, None, :] @ S)[:, 0]
        last.append(S)
    out = torch.stack(rows) if rows else torch.zeros(0, H, v.shape[2], dtype=torch.float64)
    return out, torch.stack(last)
