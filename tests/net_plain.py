"""Plain 64-bit forms of the network operators (CPU tensors), which the GPU
tests compare the library with.  They share no code with it."""
import math

import torch

GROUP = 32


def rope(x, pos, dims, base, scale, interleaved, inverse):
    """x [T, H, D], pos [T, A]; every pair turned by pos * scale * base^(-2j/d)."""
    x = x.double()
    y = x.clone()
    at = 0
    for a, d in enumerate(dims):
        for j in range(d // 2):
            ang = pos[:, a].double() * (scale[a] * base[a] ** (-2.0 * j / d))
            c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
            if inverse:
                s = -s
            i0, i1 = (at + 2 * j, at + 2 * j + 1) if interleaved else (at + j, at + j + d // 2)
            u, v = x[..., i0], x[..., i1]
            y[..., i0], y[..., i1] = u * c - v * s, u * s + v * c
        at += d
    return y


def group_of(tokens, offsets, groups):
    out = torch.zeros(tokens, dtype=torch.long)
    if offsets is not None:
        for g in range(groups):
            out[int(offsets[g]):int(offsets[g + 1])] = g
    return out


def moments(v, center, eps):
    mean = v.mean(1) if center else torch.zeros(v.shape[0], dtype=v.dtype)
    var = ((v - mean[:, None]) ** 2).mean(1)
    return mean, 1.0 / torch.sqrt(var + eps)


def norm_fwd(x, block, w_pre, w_post, gate, offsets, scale, post, center, eps):
    """(x', y, stats [T, 4]) in 64 bits; differentiable in every argument."""
    T = x.shape[0]
    zero = torch.zeros(T, dtype=torch.float64)
    mb = rb = zero
    xo = x
    if block is not None:
        u = block
        if post:
            mb, rb = moments(block, center, eps)
            u = (block - mb[:, None]) * rb[:, None]
            if w_post is not None:
                u = u * w_post
        if scale is not None:
            u = u * scale
        if gate is not None:
            u = u * gate[group_of(T, offsets, gate.shape[0])]
        xo = x + u
    m, r = moments(xo, center, eps)
    y = (xo - m[:, None]) * r[:, None]
    if w_pre is not None:
        y = y * w_pre
    return xo, y, torch.stack([mb, rb, m, r], 1)


def encode(x):
    """(q, e) of x [T, C] (any float type), value by value from the definition."""
    T, C = x.shape
    ld = -(-C // GROUP) * GROUP
    q = torch.zeros(T, ld, dtype=torch.int8)
    e = torch.zeros(T, ld // GROUP, dtype=torch.uint8)
    xd = x.double()
    for t in range(T):
        for g in range(ld // GROUP):
            v = xd[t, g * GROUP:min(C, (g + 1) * GROUP)]
            if not torch.isfinite(v).all():
                e[t, g] = 255
                continue
            big = float(v.abs().max())
            k = -126
            if big > 0:
                m, p = math.frexp(big / 127.0)
                k = max(k, p - 1 if m == 0.5 else p)
            e[t, g] = k + 127
            q[t, g * GROUP:g * GROUP + len(v)] = torch.round(v * 2.0 ** -k).to(torch.int8)
    return q, e


def decode(q, e, C):
    step = torch.exp2(e.double() - 127)
    step = torch.where(e == 255, torch.full_like(step, math.nan), step)
    return (q.double().view(q.shape[0], -1, GROUP) * step[..., None]).flatten(1)[:, :C]


def act(v, name):
    if name == "silu":
        return v / (1 + torch.exp(-v))
    return v * 0.5 * (1 + torch.erf(v / math.sqrt(2.0)))
