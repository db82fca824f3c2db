"""The network operators on the GPU against their plain 64-bit forms.

Tolerances come from the arithmetic: a result computed in fp32 from exact
inputs carries a few roundings (u = 2^-24 each) of its terms' magnitude, a sum
of n terms at most n u of the sum of magnitudes (n = the longest chain of
additions), and the stored type adds half a unit in its last place."""
import pytest
import torch

import net_plain as plain

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -24, torch.float32: 1e-38}  # subnormal step


@pytest.fixture(scope="module")
def gs():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_splatting_differentiable_gs_gb300 as gs
    return gs


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _cuda(t, pad=0, offset=0):
    """The tensor on the GPU as a slice of a wider one: rows `pad` elements
    further apart, starting `offset` elements in."""
    if t is None:
        return None
    if not pad and not offset:
        return t.cuda()
    w = t.shape[-1] + pad
    flat = torch.full((t[..., 0].numel() * w + offset + 1,), 7.0, dtype=torch.float32).to(t.dtype).cuda()
    v = flat[offset:offset + t[..., 0].numel() * w].view(*t.shape[:-1], w)[..., :t.shape[-1]]
    v.copy_(t)
    return v


def _close(got, want, bound, what):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, what
    err = (got - want).abs()
    over = err > bound
    assert not over.any() and not torch.isnan(got).any(), (
        what, int(over.sum()), float((err - bound).max()), float(err.max()))


# --------------------------------------------------------------------------
# rotary positions


def _rope_bound(want, x, dims, interleaved, dt):
    # |error| <= (|u| + |v|) * (angle: pi 2^-25 rounding + 2 ulp of the sine + 3 roundings)
    mag = x.double().abs()
    pair = mag.clone()
    at = 0
    for d in dims:
        for j in range(d // 2):
            a, b = (at + 2 * j, at + 2 * j + 1) if interleaved else (at + j, at + j + d // 2)
            s = mag[..., a] + mag[..., b]
            pair[..., a] = pair[..., b] = s
        at += d
    return pair * 10 * U + want.abs() * EPS[dt] + TINY[dt]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,hq,hk,D,dims,inter,pad", [
    (1, 1, 0, 64, (64,), False, 0),
    (1, 8, 2, 64, (16, 24, 24), False, 0),
    (257, 3, 1, 64, (32, 32), True, 0),
    (100, 5, 5, 80, (20, 26, 26), True, 0),
    (100, 5, 5, 80, (20, 26, 26), False, 3),      # odd strides: single channels
    (33, 2, 2, 72, (12, 12, 12, 12), False, 8),
    (65, 7, 1, 128, (32, 48, 48), False, 64),
    (19, 2, 1, 11, (4, 2), False, 0),             # an odd head
    (19, 2, 1, 11, (4, 2), True, 0),
    (10, 40, 40, 256, (256,), True, 0),
    (50, 1, 1, 34, (0, 2, 30), False, 0),         # an axis without channels
])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(gs, dt, T, hq, hk, D, dims, inter, pad, inverse):
    g = _gen(T + D)
    base = [10000.0, 100.0, 500.0, 10.0][:len(dims)]
    scale = [1.0, 0.5, 2.0, -1.0][:len(dims)]
    pos = torch.randint(-50, 5000, (T, len(dims)), generator=g, dtype=torch.int32)
    q = torch.randn(T, hq, D, generator=g).to(dt)
    k = torch.randn(T, hk, D, generator=g).to(dt)
    rope = gs.Rope(dims, base=base, scale=scale, interleaved=inter)
    qc, kc = _cuda(q, pad), _cuda(k, pad) if hk else None
    qo, ko = torch.full_like(qc, 9.0), torch.full_like(kc, 9.0) if hk else None
    gs.gs_rope(rope, pos.cuda(), qc, kc, q_out=qo, k_out=ko, inverse=inverse)
    for got, x in ((qo, q), (ko, k)):
        if got is not None:
            want = plain.rope(x, pos, dims, base, scale, inter, inverse)
            _close(got, want, _rope_bound(want, x, dims, inter, dt), "rope")
    # in place: the same bits
    gs.gs_rope(rope, pos.cuda(), qc, kc, inverse=inverse)
    assert torch.equal(qc, qo) and (kc is None or torch.equal(kc, ko))


def test_rope_positions_far_away(gs):
    """Positions beyond 2^24, where a 32-bit product would have lost the angle."""
    pos = torch.tensor([[2 ** 31 - 1], [-2 ** 31], [123456789], [0]], dtype=torch.int32)
    x = torch.randn(4, 2, 32, generator=_gen(1))
    got = torch.empty(4, 2, 32, device="cuda")
    gs.gs_rope(gs.Rope([32]), pos.cuda(), x.cuda(), q_out=got)
    want = plain.rope(x, pos, (32,), [1e4], [1.0], False, False)
    # the 64-bit frequency itself is a double's: 2^-53 of a turn times 2^31
    _close(got, want, _rope_bound(want, x, (32,), False, torch.float32) + 2.0 ** -18, "far")


def test_rope_inverse_is_the_transpose(gs):
    """<R x, y> = <x, R^T y>: the inverse is the gradient."""
    g = _gen(2)
    x, y = (torch.randn(40, 3, 64, generator=g).cuda() for _ in range(2))
    pos = torch.randint(0, 200, (40, 3), generator=g, dtype=torch.int32).cuda()
    rope = gs.Rope((16, 24, 24))
    rx, ry = torch.empty_like(x), torch.empty_like(y)
    gs.gs_rope(rope, pos, x, q_out=rx)
    gs.gs_rope(rope, pos, y, q_out=ry, inverse=True)
    a, b = (rx.double() * y.double()).sum(), (x.double() * ry.double()).sum()
    assert abs(a - b) <= 20 * U * (x.double().abs() * y.double().abs()).sum()


def test_rope_keeps_nan_and_inf_to_their_pairs(gs):
    x = torch.ones(2, 2, 16)
    x[0, 1, 3] = float("nan")
    x[1, 0, 5] = float("inf")
    out = torch.empty(2, 2, 16, device="cuda")
    pos = torch.full((2, 1), 3, dtype=torch.int32).cuda()
    gs.gs_rope(gs.Rope([16]), pos, x.cuda(), q_out=out)
    bad = ~torch.isfinite(out.cpu())
    want = torch.zeros_like(bad)
    want[0, 1, 3] = want[0, 1, 11] = want[1, 0, 5] = want[1, 0, 13] = True
    assert torch.equal(bad, want)


# --------------------------------------------------------------------------
# gated norms

NORM_CASES = [
    # tokens, channels, groups (0: no gate), center, post, scale, pad, offset
    (1, 1, 1, False, True, True, 0, 0),
    (1, 8, 0, True, True, False, 0, 0),
    (5, 33, 2, True, True, True, 0, 0),
    (7, 64, 3, False, False, True, 8, 0),
    (300, 256, 4, False, True, True, 0, 0),
    (310, 384, 5, True, True, True, 16, 0),
    (37, 1000, 1, False, True, False, 0, 0),
    (37, 1001, 3, True, True, True, 1, 3),
    (9, 1032, 2, False, True, True, 8, 0),
    (3, 2048, 3, True, False, True, 0, 0),
    (611, 520, 7, False, True, True, 0, 0),
    (2, 4097, 2, True, True, True, 0, 0),
    (3, 8192, 1, False, True, True, 0, 0),
]
NORM_TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
              (torch.float16, torch.float16), (torch.float16, torch.float32),
              (torch.float32, torch.float32)]


def _offsets(T, G, g):
    if not G:
        return None
    cuts = torch.randint(0, T + 1, (G - 1,), generator=g).sort().values
    if G > 2:
        cuts[1] = cuts[0]  # an empty group
    return torch.cat([torch.tensor([0]), cuts, torch.tensor([T])]).to(torch.int32)


def _norm_inputs(T, Cn, G, scale, post, dt, rt):
    g = _gen(T * 7 + Cn)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(x=r(T, Cn).to(rt), block=(2 * r(T, Cn) + 0.5).to(dt), w_pre=1 + 0.2 * r(Cn),
             w_post=1 + 0.2 * r(Cn) if post else None, scale=0.5 + 0.2 * r(Cn) if scale else None,
             gate=r(G, Cn).to(dt) if G else None, offsets=_offsets(T, G, g))
    return d, g


def _dbl(t, grad=False):
    return None if t is None else t.double().requires_grad_(grad)


def _stat_bounds(v, center, eps):
    """Bounds of the fp32 statistics of rows v (64 bits): (mean, deviation's
    relative error).  Chains: at most 32 values a lane, 5 shuffles, 16 warps."""
    chain = 56 * U
    mean_err = chain * v.abs().mean(1, keepdim=True) if center else torch.zeros_like(v[:, :1])
    m, r = plain.moments(v, center, eps)
    rel = chain + 4 * U + mean_err * r[:, None]
    return mean_err, rel, m, r


@pytest.mark.parametrize("dt,rt", NORM_TYPES)
@pytest.mark.parametrize("T,Cn,G,center,post,scale,pad,offset", NORM_CASES)
def test_norm_forward(gs, dt, rt, T, Cn, G, center, post, scale, pad, offset):
    eps = 1e-5
    d, _ = _norm_inputs(T, Cn, G, scale, post, dt, rt)
    xo, y, st = plain.norm_fwd(_dbl(d["x"]), _dbl(d["block"]), _dbl(d["w_pre"]), _dbl(d["w_post"]),
                               _dbl(d["gate"]), d["offsets"], _dbl(d["scale"]), post, center, eps)
    out = {k: _cuda(torch.zeros(T, Cn, dtype=t), pad, offset) for k, t in (("xo", rt), ("y", dt))}
    stats = torch.empty(T, 4, device="cuda")
    y_q, y_e = gs.act8_empty(T, Cn)
    kw = dict(w_pre=d["w_pre"].cuda(), w_post=_cuda(d["w_post"]), gate=_cuda(d["gate"]),
              group_offsets=_cuda(d["offsets"]), res_scale=_cuda(d["scale"]), post=post,
              center=center, eps=eps)
    gs.gs_gated_norm_fwd(_cuda(d["x"], pad, offset), _cuda(d["block"], pad, offset), out["xo"],
                         out["y"], stats, y_q=y_q, y_e=y_e, **kw)
    # x' carries the relative error of the block's normalised value
    u = xo - d["x"].double()
    b = d["block"].double()
    k = (u / torch.where(b == 0, torch.ones_like(b), b)).abs()
    xo_err = 8 * U * (u.abs() + xo.abs())
    if post:
        mean_err, rel, m, r = _stat_bounds(b, center, eps)
        w = torch.ones(Cn, dtype=torch.float64) if d["w_post"] is None else d["w_post"].double()
        k = w.abs() * r[:, None]
        if d["scale"] is not None:
            k = k * d["scale"].double().abs()
        if d["gate"] is not None:
            k = k * d["gate"].double().abs()[plain.group_of(T, d["offsets"], G)]
        xo_err = xo_err + u.abs() * rel + k * (mean_err + U * b.abs())
    _close(out["xo"], xo, xo_err + EPS[rt] * xo.abs() + TINY[rt], "x'")
    mean_err, rel, m, r = _stat_bounds(xo, center, eps)
    w = d["w_pre"].double().abs() * r[:, None]
    worst = xo_err.amax(1, keepdim=True)
    rel = rel + worst * r[:, None] * 2
    mean_err = mean_err + worst
    y_err = y.abs() * (rel + 8 * U) + w * (mean_err + xo_err + U * xo.abs())
    _close(out["y"], y, y_err + EPS[dt] * y.abs() + TINY[dt], "y")
    want = st.clone()
    bound = torch.cat([*(2 * [torch.zeros(T, 1, dtype=torch.float64)]), mean_err, rel * r[:, None]], 1)
    if post:
        me, re_, _, rb = _stat_bounds(b, center, eps)
        bound[:, :2] = torch.cat([me, re_ * rb[:, None]], 1)
    _close(stats, want, bound + 2 * U * want.abs(), "stats")
    # the checkpoint is that of y as stored, byte for byte
    wq, we = plain.encode(out["y"].cpu())
    assert torch.equal(y_q.cpu(), wq) and torch.equal(y_e.cpu(), we)
    # the sum alone, and in place, gives the same x'
    x2 = _cuda(d["x"], pad, offset)
    if not pad:
        x2 = x2.clone()
    gs.gs_gated_norm_fwd(x2, _cuda(d["block"], pad, offset), x2, None, torch.empty_like(stats), **kw)
    assert torch.equal(x2, out["xo"])
    # without a block: the norm before alone
    y2 = torch.empty(T, Cn, dtype=dt, device="cuda")
    gs.gs_gated_norm_fwd(out["xo"], None, None, y2, stats, w_pre=kw["w_pre"], center=center, eps=eps)
    xr = out["xo"].double().cpu()
    _, want2, _ = plain.norm_fwd(xr, None, _dbl(d["w_pre"]), None, None, None, None, False, center, eps)
    mean_err, rel, _, r = _stat_bounds(xr, center, eps)
    w = d["w_pre"].double().abs() * r[:, None]
    _close(y2, want2, want2.abs() * (rel + 8 * U + EPS[dt]) + w * (mean_err + U * xr.abs()) + TINY[dt],
           "norm alone")


@pytest.mark.parametrize("dt,rt", NORM_TYPES)
@pytest.mark.parametrize("T,Cn,G,center,post,scale,pad,offset", NORM_CASES)
def test_norm_backward(gs, dt, rt, T, Cn, G, center, post, scale, pad, offset):
    eps = 1e-3  # one channel has no spread: its deviation is eps alone
    d, g = _norm_inputs(T, Cn, G, scale, post, dt, rt)
    dxo = torch.randn(T, Cn, generator=g).to(rt)
    dy = torch.randn(T, Cn, generator=g).to(dt)
    leaf = {k: _dbl(v, True) if isinstance(v, torch.Tensor) and k != "offsets" else v
            for k, v in d.items()}
    # d["x"] is x': the gradient of the sum's own inputs follows by hand
    _, y, st = plain.norm_fwd(leaf["x"], None, leaf["w_pre"], None, None, None, None, False, center,
                              eps)
    dn, dwp = torch.autograd.grad(y, (leaf["x"], leaf["w_pre"]), dy.double())
    dd = dn + dxo.double()
    zero = torch.zeros(T, Cn, dtype=torch.float64)
    u, _, st_b = plain.norm_fwd(zero, leaf["block"], None, leaf["w_post"], leaf["gate"], d["offsets"],
                                leaf["scale"], post, center, eps)
    names = [k for k in ("block", "w_post", "gate", "scale") if leaf[k] is not None]
    grads = dict(zip(names, torch.autograd.grad(u, [leaf[k] for k in names], dd)))
    stats = torch.cat([st_b[:, :2], st[:, 2:]], 1).detach().float().cuda()

    out = {k: _cuda(torch.zeros(T, Cn, dtype=t), pad, offset) for k, t in (("dx", rt), ("db", dt))}
    f = lambda t: None if t is None else torch.full(t.shape, 5.0, device="cuda")  # noqa: E731
    sums = dict(dw_pre=f(d["w_pre"]), dw_post=f(d["w_post"]), dgate=f(d["gate"]),
                dres_scale=f(d["scale"]))
    ws = torch.empty(gs.gs_gated_norm_workspace_bytes(Cn, max(G, 1)), dtype=torch.uint8, device="cuda")
    kw = dict(w_pre=d["w_pre"].cuda(), w_post=_cuda(d["w_post"]), gate=_cuda(d["gate"]),
              group_offsets=_cuda(d["offsets"]), res_scale=_cuda(d["scale"]), workspace=ws,
              post=post, center=center)
    args = (_cuda(d["x"], pad, offset), _cuda(d["block"], pad, offset), stats,
            _cuda(dxo, pad, offset), _cuda(dy, pad, offset))
    gs.gs_gated_norm_bwd(*args, out["dx"], out["db"], **sums, **kw)

    # terms of d: h r, n mean(h n) r, mean(h) r; statistics rounded to fp32
    r = st[:, 3:4].detach()
    n = (d["x"].double() - st[:, 2:3].detach()) * r
    nx = n.abs() + d["x"].double().abs() * r  # cancellation of x - mean in fp32
    h = (dy.double() * d["w_pre"].double()).abs()
    mag = r * (h + nx * (h * nx).mean(1, keepdim=True) + h.mean(1, keepdim=True))
    tol = 64 * U  # a chain of <= 16 values, 5 shuffles, 16 warps and the formula's roundings
    d_err = tol * (mag + dxo.double().abs())
    _close(out["dx"], dd, d_err + EPS[rt] * dd.abs() + TINY[rt], "dx")
    m = b = d["block"].double()
    rb = torch.ones(T, 1, dtype=torch.float64)
    if post:
        rb = st_b[:, 1:2].detach()
        m = (b - st_b[:, 0:1].detach()) * rb
    mx = m.abs() + (b.abs() * rb if post else 0)
    k = torch.ones(T, Cn, dtype=torch.float64)
    if d["gate"] is not None:
        k = k * d["gate"].double().abs()[plain.group_of(T, d["offsets"], G)]
    s = 1 if d["scale"] is None else d["scale"].double().abs()
    w = 1 if d["w_post"] is None else d["w_post"].double().abs()
    dm = (mag + dxo.double().abs())       # magnitudes of d's terms
    e = dm * k * s * w
    db_mag = rb * (e + mx * (e * mx).mean(1, keepdim=True) + e.mean(1, keepdim=True)) if post else e
    _close(out["db"], grads["block"], 2 * tol * db_mag + EPS[dt] * grads["block"].abs() + TINY[dt], "dblock")
    # sums over tokens: <= 304 row ranges, joined by 32 lanes of 10 each, teams, groups
    chain = (T / 304 + 64) * U + 2 * tol
    _close(sums["dw_pre"], dwp, chain * (dy.double().abs() * nx).sum(0) + 1e-30, "dw_pre")
    if post:
        _close(sums["dw_post"], grads["w_post"], chain * (dm * k * s * mx).sum(0) + 1e-30, "dw_post")
    if scale:
        _close(sums["dres_scale"], grads["scale"], chain * (dm * k * w * mx).sum(0) + 1e-30, "dscale")
    if G:
        of = (plain.group_of(T, d["offsets"], G)[None] == torch.arange(G)[:, None]).double()
        _close(sums["dgate"], grads["gate"], chain * (of @ (dm * mx * s * w)) + 1e-30, "dgate")
    # fixed order: the same bits again; gradients in place of their inputs too
    again = {k_: f(v) for k_, v in sums.items()}
    x2, y2 = args[3].clone() if not pad else args[3], args[4].clone() if not pad else args[4]
    gs.gs_gated_norm_bwd(args[0], args[1], stats, x2, y2, x2, y2, **again, **kw)
    assert torch.equal(x2, out["dx"]) and torch.equal(y2, out["db"])
    assert all(v is None or torch.equal(v, again[k_]) for k_, v in sums.items())


def test_norm_backward_parts(gs):
    """Without dy, without dx_out, without a block; gradients of either part add up."""
    T, Cn = 50, 96
    d, g = _norm_inputs(T, Cn, 2, True, True, torch.float32, torch.float32)
    c = {k: _cuda(v) for k, v in d.items()}
    dxo, dy = torch.randn(T, Cn, generator=g).cuda(), torch.randn(T, Cn, generator=g).cuda()
    xo, y, stats = (torch.empty(T, Cn, device="cuda"), torch.empty(T, Cn, device="cuda"),
                    torch.empty(T, 4, device="cuda"))
    kw = dict(w_pre=c["w_pre"], w_post=c["w_post"], gate=c["gate"], group_offsets=c["offsets"],
              res_scale=c["scale"])
    gs.gs_gated_norm_fwd(c["x"], c["block"], xo, y, stats, **kw)
    ws = torch.empty(gs.gs_gated_norm_workspace_bytes(Cn, 2), dtype=torch.uint8, device="cuda")

    def bwd(a, b, block=True):
        o = [torch.full((T, Cn), 3.0, device="cuda") for _ in range(2)]
        s = [torch.full((Cn,), 3.0, device="cuda") for _ in range(3)] + [torch.full((2, Cn), 3.0, device="cuda")]
        extra = kw if block else dict(w_pre=c["w_pre"])
        gs.gs_gated_norm_bwd(xo, c["block"] if block else None, stats, a, b, o[0],
                             o[1] if block else None, dw_pre=s[0], dw_post=s[1], dres_scale=s[2],
                             dgate=s[3] if block else None, workspace=ws, **extra)
        return o + s

    both, only_x, only_y = bwd(dxo, dy), bwd(dxo, None), bwd(None, dy)
    for a, b, c2 in zip(both, only_x, only_y):
        scale = (b.abs() + c2.abs()).max().double()
        assert ((a.double() - b.double() - c2.double()).abs() <= 2e-5 * scale).all()
    assert torch.equal(only_x[0], dxo) and not only_x[2].any()
    alone = bwd(None, dy, block=False)
    assert torch.equal(alone[0], only_y[0]) and torch.equal(alone[2], only_y[2])
    assert not alone[3].any() and not alone[4].any()


def test_norm_gradient_against_differences(gs):
    """Directional derivatives of the library's own forward in fp32: central
    differences with step h err by O(h^2) and by roundings of about
    sqrt(N) u |y| / h."""
    T, Cn, G = 24, 64, 3
    d, g = _norm_inputs(T, Cn, G, True, True, torch.float32, torch.float32)
    c = {k: _cuda(v) for k, v in d.items()}
    ry, rx = (torch.randn(T, Cn, generator=g).cuda() for _ in range(2))
    for center in (False, True):
        def fwd(v):
            xo, y, st = (torch.empty(T, Cn, device="cuda"), torch.empty(T, Cn, device="cuda"),
                         torch.empty(T, 4, device="cuda"))
            gs.gs_gated_norm_fwd(v["x"], v["block"], xo, y, st, w_pre=v["w_pre"], w_post=v["w_post"],
                                 gate=v["gate"], group_offsets=c["offsets"], res_scale=v["scale"],
                                 center=center)
            return xo, y, st

        def loss(v):
            xo, y, _ = fwd(v)
            return float((xo.double() * rx).sum() + (y.double() * ry).sum())

        xo, y, st = fwd(c)
        ws = torch.empty(gs.gs_gated_norm_workspace_bytes(Cn, G), dtype=torch.uint8, device="cuda")
        grad = {k: torch.empty_like(c[k]) for k in ("x", "block", "w_pre", "w_post", "gate", "scale")}
        gs.gs_gated_norm_bwd(xo, c["block"], st, rx, ry, grad["x"], grad["block"], w_pre=c["w_pre"],
                             w_post=c["w_post"], gate=c["gate"], group_offsets=c["offsets"],
                             res_scale=c["scale"], dw_pre=grad["w_pre"], dw_post=grad["w_post"],
                             dgate=grad["gate"], dres_scale=grad["scale"], workspace=ws, center=center)
        for name, gr in grad.items():
            v = torch.randn(gr.shape, generator=g).cuda()
            h = 2e-3
            hi, lo = dict(c), dict(c)
            hi[name], lo[name] = c[name] + h * v, c[name] - h * v
            # the step that was really taken, after rounding
            num = loss(hi) - loss(lo)
            want = float((gr.double() * (hi[name].double() - lo[name].double())).sum())
            noise = 40 * U * (T * Cn) ** 0.5 * 4
            curve = 2 * h ** 3 * float(v.abs().max()) ** 3 * (T * Cn) ** 0.5
            assert abs(num - want) <= noise + curve + 1e-4 * abs(want), (name, num, want)


def test_norm_rows_do_not_mix(gs):
    """NaN and infinity in a row stay there; a row of zeros gives zeros."""
    T, Cn = 9, 200
    x, b = torch.randn(T, Cn, generator=_gen(5)), torch.randn(T, Cn, generator=_gen(6))
    x[2, 7], b[4, 100] = float("nan"), float("inf")
    x[6], b[6] = 0, 0
    xo, y, st = torch.empty(T, Cn).cuda(), torch.empty(T, Cn).cuda(), torch.empty(T, 4).cuda()
    y_q, y_e = gs.act8_empty(T, Cn)
    gs.gs_gated_norm_fwd(x.cuda(), b.cuda(), xo, y, st, y_q=y_q, y_e=y_e)
    fine = torch.isfinite(y.cpu()).all(1)
    assert fine.tolist() == [i not in (2, 4) for i in range(T)]
    assert not y[6].any() and not xo[6].any()
    assert (y_e[2] == 255).all() and not y_q[2].any() and (y_e[6] == 1).all()


def test_norm_without_tokens(gs):
    Cn, G = 40, 3
    e = lambda: torch.empty(0, Cn, device="cuda")  # noqa: E731
    sums = [torch.full((Cn,), 2.0, device="cuda") for _ in range(3)] + [torch.full((G, Cn), 2.0, device="cuda")]
    ws = torch.empty(gs.gs_gated_norm_workspace_bytes(Cn, G), dtype=torch.uint8, device="cuda")
    w = torch.ones(Cn, device="cuda")
    gate, off = torch.ones(G, Cn, device="cuda"), torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    st = torch.empty(0, 4, device="cuda")
    gs.gs_gated_norm_fwd(e(), e(), e(), e(), st, gate=gate, group_offsets=off)
    gs.gs_gated_norm_bwd(e(), e(), st, e(), e(), e(), e(), w_post=w, res_scale=w, gate=gate,
                         group_offsets=off, dw_pre=sums[0], dw_post=sums[1], dres_scale=sums[2],
                         dgate=sums[3], workspace=ws)
    assert not any(s.any() for s in sums)


# --------------------------------------------------------------------------
# 8-bit checkpoints


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,Cn,pad,offset", [(1, 1, 0, 0), (1, 31, 0, 0), (3, 32, 0, 0), (3, 33, 0, 0),
                                             (2, 8, 0, 0), (5, 64, 8, 0), (17, 72, 0, 0),
                                             (200, 264, 3, 1), (4, 2100, 0, 0)])
def test_act8_encode_decode(gs, dt, T, Cn, pad, offset):
    g = _gen(Cn)
    x = torch.randn(T, Cn, generator=g) * torch.exp2(torch.randint(-12, 12, (T, 1), generator=g).float())
    x = x.to(dt)
    q, e = gs.act8_empty(T, Cn)
    q.fill_(77), e.fill_(77)
    gs.gs_act8_encode(_cuda(x, pad, offset), q, e)
    wq, we = plain.encode(x)
    assert torch.equal(e.cpu(), we) and torch.equal(q.cpu(), wq)
    for out_t in (torch.float32, torch.bfloat16, torch.float16):
        back = _cuda(torch.zeros(T, Cn, dtype=out_t), pad, offset)
        gs.gs_act8_decode(q, e, back)
        want = plain.decode(wq, we, Cn)
        if out_t == torch.float16:
            assert torch.equal(back.cpu(), want.float().half())
        else:
            assert torch.equal(back.double().cpu(), want)  # exact in both


def test_act8_edges(gs):
    big = torch.finfo(torch.float32).max
    rows = [[0.0] * 32, [127.0] + [0.5] * 31, [127.00001] + [63.5] * 31, [1e-40] * 32, [big, -big] * 16,
            [float("inf")] + [1.0] * 31, [float("nan")] + [1.0] * 31, [-127 * 2.0 ** -126] * 32,
            [127 * 2.0 ** -127, 2.0 ** -127] * 16, [0.5, 1.5, 2.5, -0.5, -1.5, 127.0] + [0.0] * 26,
            [-1.984375] * 32, [1.9843751] * 32]
    x = torch.tensor(rows)
    q, e = gs.act8_empty(len(rows), 32)
    gs.gs_act8_encode(x.cuda(), q, e)
    wq, we = plain.encode(x)
    assert torch.equal(e.cpu(), we) and torch.equal(q.cpu(), wq)
    back = torch.empty_like(x).cuda()
    gs.gs_act8_decode(q, e, back)
    assert torch.equal(torch.isnan(back.cpu()).all(1), ~torch.isfinite(x).all(1))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("T,Cn,pad", [(1, 1, 0), (3, 40, 0), (129, 264, 8), (20, 77, 0), (5, 96, 3)])
def test_glu(gs, dt, act, gated, T, Cn, pad):
    g = _gen(T + Cn)
    gate, up = (3 * torch.randn(T, Cn, generator=g)).to(dt), torch.randn(T, Cn, generator=g).to(dt)
    dh = torch.randn(T, Cn, generator=g).to(dt)
    h = _cuda(torch.zeros(T, Cn, dtype=dt), pad)
    g8, u8, h8 = gs.act8_empty(T, Cn), gs.act8_empty(T, Cn), gs.act8_empty(T, Cn)
    gs.gs_glu_fwd(_cuda(gate, pad), _cuda(up, pad) if gated else None, h, *g8,
                  *(u8 if gated else (None, None)), act=act)
    one = torch.ones(T, Cn, dtype=torch.float64)
    f = plain.act(gate.double(), act)
    want = f * (up.double() if gated else one)
    # act: the argument times 2 u inside the exponential or error function, then
    # a few roundings; the tail of gelu loses 1 + erf: an absolute 4 u |gate up|
    mag = (gate.double().abs() * (up.double().abs() if gated else one))
    slack = (8 + 4 * gate.double().abs()) * U
    _close(h, want, want.abs() * (slack + EPS[dt]) + 4 * U * mag + TINY[dt], "h")
    for got, x in ((g8, gate),) + (((u8, up),) if gated else ()):
        wq, we = plain.encode(x)
        assert torch.equal(got[0].cpu(), wq) and torch.equal(got[1].cpu(), we)
    # backward, at the checkpoint's values
    gv = plain.decode(*plain.encode(gate), Cn).requires_grad_(True)
    uv = plain.decode(*plain.encode(up), Cn).requires_grad_(True)
    hv = plain.act(gv, act) * (uv if gated else one)
    dg, *du = torch.autograd.grad(hv, (gv, uv) if gated else (gv,), dh.double())
    ug = uv.detach().abs() if gated else one
    dgate, dup = (_cuda(torch.zeros(T, Cn, dtype=dt), pad) for _ in range(2))
    gs.gs_glu_bwd(*g8, *(u8 if gated else (None, None)), _cuda(dh, pad), dgate,
                  dup if gated else None, *h8, act=act)
    a = gv.detach().abs()
    # |act'| <= 1.2 and its parts (s, v s (1 - s); Phi, v phi) are of that size
    _close(dgate, dg, (12 + 6 * a) * U * 2 * dh.double().abs() * ug + EPS[dt] * dg.abs() + TINY[dt], "dgate")
    if gated:
        _close(dup, du[0], (8 + 4 * a) * U * dh.double().abs() * (a + 1) + EPS[dt] * du[0].abs() + TINY[dt], "dup")
    # h's checkpoint: within half a step, up to the error of h itself
    back = torch.empty(T, Cn, device="cuda")
    gs.gs_act8_decode(*h8, back)
    step = torch.exp2(h8[1].cpu().double() - 127).repeat_interleave(32, 1)[:, :Cn]
    _close(back, hv.detach(), 0.5 * step + (8 + 4 * a) * U * (a * ug + 1e-30), "h8")
    # in place of dh
    d2 = dh.cuda()
    gs.gs_glu_bwd(*g8, *(u8 if gated else (None, None)), d2, d2, dup if gated else None, act=act)
    assert torch.equal(d2, dgate)


@pytest.mark.parametrize("dt", [torch.float16, torch.float32])
@pytest.mark.parametrize("Cn", [1, 2, 3, 5, 7, 8, 9, 15, 16, 17, 23, 31, 33, 250, 263, 520])
@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (1, 1), (3, 2), (5, 6), (8, 8), (7, 9)])
def test_rows_at_any_alignment(gs, dt, Cn, offset, pad):
    """Every alignment of a row: the same bits as from aligned rows, and nothing
    but the rows is written."""
    T = 37
    g = _gen(Cn)
    gate, up, dh = (torch.randn(T, Cn, generator=g).to(dt) for _ in range(3))
    wide = -(-Cn // 32) * 32

    def aligned(x):
        v = torch.zeros(T, wide, dtype=dt, device="cuda")
        v[:, :Cn] = x
        return v

    def room():
        w = Cn + pad
        flat = torch.full((T * w + offset + 40,), 7.0, dtype=dt, device="cuda")
        return flat, flat[offset:offset + T * w].view(T, w)[:, :Cn]

    def untouched(flat):
        w = Cn + pad
        keep = torch.ones_like(flat, dtype=torch.bool)
        keep[offset:offset + T * w].view(T, w)[:, :Cn] = False
        return bool((flat[keep] == 7.0).all())

    ref = [torch.empty(T, wide, dtype=dt, device="cuda") for _ in range(3)]
    r8 = gs.act8_empty(T, wide), gs.act8_empty(T, wide)
    gs.gs_glu_fwd(aligned(gate), aligned(up), ref[0], *r8[0], *r8[1], act="gelu")
    gs.gs_glu_bwd(*r8[0], *r8[1], aligned(dh), ref[1], ref[2], act="gelu")
    k8 = gs.act8_empty(T, Cn), gs.act8_empty(T, Cn)
    bufs = [room() for _ in range(4)]
    args = [room() for _ in range(3)]
    for (_, v), x in zip(args, (gate, up, dh)):
        v.copy_(x)
    gs.gs_glu_fwd(args[0][1], args[1][1], bufs[0][1], *k8[0], *k8[1], act="gelu")
    gs.gs_glu_bwd(*k8[0], *k8[1], args[2][1], bufs[1][1], bufs[2][1], act="gelu")
    assert all(torch.equal(a, b) for x, y in zip(k8, r8) for a, b in zip(x, y))
    for (flat, v), want in zip(bufs, ref):
        assert torch.equal(v, want[:, :Cn]) and untouched(flat)
    flat, v = bufs[3]
    gs.gs_act8_decode(*k8[0], v)
    assert torch.equal(v.double().cpu(), plain.decode(*[z.cpu() for z in k8[0]], Cn).to(dt).double())
    assert untouched(flat)
    # norms: the same bits at every alignment that is not a multiple of 16 bytes
    # (rows on such multiples are summed in another order)
    size = gate.element_size()
    if offset * size % 16 == 0 and (Cn + pad) * size % 16 == 0 and Cn * size % 16 == 0:
        return
    st, xo, y = torch.empty(T, 4, device="cuda"), room(), room()
    gs.gs_gated_norm_fwd(args[0][1], args[1][1], xo[1], y[1], st)
    st2, want = torch.empty(T, 4, device="cuda"), [_cuda(torch.zeros(T, Cn, dtype=dt), 1, 1) for _ in range(2)]
    gs.gs_gated_norm_fwd(_cuda(gate, 1, 1), _cuda(up, 1, 1), *want, st2)
    assert torch.equal(xo[1], want[0]) and torch.equal(y[1], want[1]) and torch.equal(st, st2)
    assert untouched(xo[0]) and untouched(y[0])


def test_glu_gradient_against_differences(gs):
    """dgate and dup against central differences of the library's forward at
    the checkpoint's values."""
    T, Cn, h = 16, 64, 1e-2
    g = _gen(9)
    gate, up, dh = (torch.randn(T, Cn, generator=g).cuda() for _ in range(3))
    for act in ("silu", "gelu"):
        g8, u8 = gs.act8_empty(T, Cn), gs.act8_empty(T, Cn)
        o = torch.empty_like(gate)
        gs.gs_glu_fwd(gate, up, o, *g8, *u8, act=act)
        gv, uv = torch.empty_like(gate), torch.empty_like(up)
        gs.gs_act8_decode(*g8, gv)
        gs.gs_act8_decode(*u8, uv)
        dg, du = torch.empty_like(gate), torch.empty_like(gate)
        gs.gs_glu_bwd(*g8, *u8, dh, dg, du, act=act)

        def at(a, b):
            out = torch.empty_like(a)
            gs.gs_glu_fwd(a, b, out, act=act)
            return out.double()

        num = (at(gv + h, uv) - at(gv - h, uv)) / (2 * h) * dh
        # third derivative of act is below 2; roundings 8 u |h| / step
        tol = (h * h / 3 + 16 * U * (gv.abs() + 1) / h) * (uv * dh).abs().double() + 1e-6
        assert ((num - dg.double()).abs() <= tol).all()
        num = (at(gv, uv + h) - at(gv, uv - h)) / (2 * h) * dh
        tol = (16 * U * (uv.abs() + 1) * (gv.abs() + 1) / h) * dh.abs().double() + 1e-6
        assert ((num - du.double()).abs() <= tol).all()


WGRAD = [(0, 8, 32), (1, 1, 1), (1, 59, 64), (63, 64, 32), (64, 128, 128), (65, 130, 100), (200, 59, 257),
         (1000, 256, 256), (129, 1, 1000), (513, 300, 33), (4100, 136, 520), (777, 520, 1032)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("out_t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,N,K", WGRAD)
def test_wgrad(gs, dt, out_t, T, N, K):
    g = _gen(T + 3 * N + 7 * K)
    dy = torch.randn(T, N, generator=g).to(dt)
    x = torch.randn(T, K, generator=g) * torch.exp2(torch.randint(-6, 6, (T, 1), generator=g).float())
    ws = torch.zeros(gs.gs_act8_wgrad_workspace_bytes(T, N, K, dt), dtype=torch.uint8, device="cuda")
    q, e = gs.act8_empty(T, K)
    gs.gs_act8_encode(x.cuda(), q, e)
    xv = torch.empty(T, K, device="cuda")
    gs.gs_act8_decode(q, e, xv)
    xv = xv.double().cpu()
    want, mag = dy.double().t() @ xv, dy.double().abs().t() @ xv.abs()
    bound = (T / 8 + 32) * U * 2 * mag + EPS[out_t] * want.abs() + 1e-30
    for pad, offset in ((0, 0), (8, 0), (3, 1)):
        dw = torch.full((N, K), 3.0, device="cuda").to(out_t)
        gs.gs_act8_wgrad(_cuda(dy, pad, offset) if T else dy.cuda(), q, e, dw, ws)
        _close(dw, want, bound, "dw pad %d" % pad)
        assert gs.gs_workspace_status(ws) == gs.GS_OK
    again = torch.empty_like(dw)
    gs.gs_act8_wgrad(dy.cuda(), q, e, again, ws)
    first = again.clone()
    gs.gs_act8_wgrad(dy.cuda(), q, e, again, ws)
    assert torch.equal(first, again)  # a fixed order of summation
    # added to what is there, into rows further apart
    base = torch.randn(N, K + 5, generator=g).to(out_t)
    acc = base.cuda()
    gs.gs_act8_wgrad(dy.cuda(), q, e, acc[:, :K], ws, accumulate=True)
    want2 = want + base[:, :K].double()
    _close(acc[:, :K], want2, bound + (2 * U + EPS[out_t]) * (want2.abs() + base[:, :K].double().abs()), "acc")
    assert torch.equal(acc[:, K:].cpu(), base[:, K:])


def test_wgrad_not_a_number_stays_in_its_channels(gs):
    T, N, K = 100, 70, 96
    x, dy = torch.randn(T, K, generator=_gen(1)), torch.randn(T, N, generator=_gen(2))
    x[17, 40] = float("nan")
    dy[30, 5] = float("inf")
    q, e = gs.act8_empty(T, K)
    gs.gs_act8_encode(x.cuda(), q, e)
    for dt in (torch.bfloat16, torch.float32):
        ws = torch.zeros(gs.gs_act8_wgrad_workspace_bytes(T, N, K, dt), dtype=torch.uint8, device="cuda")
        dw = torch.empty(N, K, device="cuda")
        gs.gs_act8_wgrad(dy.to(dt).cuda(), q, e, dw, ws)
        bad = ~torch.isfinite(dw.cpu())
        want = torch.zeros(N, K, dtype=torch.bool)
        want[:, 32:64] = True
        want[5] = True
        assert torch.equal(bad, want)


def test_wgrad_uses_every_bit_of_a_wide_gradient(gs):
    """fp32 and fp16 gradients enter the product whole: one token, so that no sum hides it."""
    for dt in (torch.float16, torch.float32):
        dy = torch.randn(1, 200, generator=_gen(4)).to(dt)
        x = torch.ones(1, 64)
        q, e = gs.act8_empty(1, 64)
        gs.gs_act8_encode(x.cuda(), q, e)
        ws = torch.zeros(gs.gs_act8_wgrad_workspace_bytes(1, 200, 64, dt), dtype=torch.uint8, device="cuda")
        dw = torch.empty(200, 64, device="cuda")
        gs.gs_act8_wgrad(dy.cuda(), q, e, dw, ws)
        want = dy.double().t().expand(200, 64)
        _close(dw, want, 2 * U * want.abs(), "bits")


# --------------------------------------------------------------------------
# streams, graphs, refusals


def test_net_calls_run_on_the_given_stream_and_in_a_graph(gs):
    T, Cn = 512, 256
    g = _gen(3)
    x, b = torch.randn(T, Cn, generator=g).cuda().bfloat16(), torch.randn(T, Cn, generator=g).cuda().bfloat16()
    pos = torch.randint(0, 99, (T, 2), generator=g, dtype=torch.int32).cuda()
    rope = gs.Rope((32, 32))
    ws = torch.zeros(gs.gs_act8_wgrad_workspace_bytes(T, Cn, Cn), dtype=torch.uint8, device="cuda")

    def chain(stream=None):
        o = dict(xo=torch.empty_like(x), y=torch.empty_like(x), st=torch.empty(T, 4, device="cuda"),
                 dw=torch.empty(Cn, Cn, device="cuda"), q=torch.empty(T, 4, 64, dtype=x.dtype, device="cuda"))
        ck = gs.act8_empty(T, Cn)
        return o, ck, lambda s: (
            gs.gs_gated_norm_fwd(x, b, o["xo"], o["y"], o["st"], y_q=ck[0], y_e=ck[1], stream=s),
            gs.gs_rope(rope, pos, o["y"].view(T, 4, 64), q_out=o["q"], stream=s),
            gs.gs_act8_wgrad(o["q"].view(T, Cn), *ck, o["dw"], ws, stream=s))

    ref, _, run = chain()
    run(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, _, run = chain()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(20_000_000)  # the default stream is busy meanwhile
    run(side)
    side.synchronize()
    assert all(torch.equal(got[k], ref[k]) for k in ref)
    torch.cuda.synchronize()
    rec, _, run = chain()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(None)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(rec[k], ref[k]) for k in ref)


def test_net_wrappers_refuse(gs):
    T, Cn = 4, 64
    x = torch.zeros(T, Cn, device="cuda")
    q, e = gs.act8_empty(T, Cn)
    st = torch.empty(T, 4, device="cuda")
    bad = [
        lambda: gs.gs_act8_encode(x.t(), q, e),                                  # columns, not rows
        lambda: gs.gs_act8_encode(x.double(), q, e),
        lambda: gs.gs_act8_encode(x, q[:, :32], e),
        lambda: gs.gs_act8_encode(x, q, e[:, :1]),
        lambda: gs.gs_act8_encode(x[0], q, e),
        lambda: gs.gs_act8_decode(q, e, x[:, :31]),
        lambda: gs.gs_gated_norm_fwd(x, x.half(), x, x.bfloat16(), st),          # two types
        lambda: gs.gs_gated_norm_fwd(x, x, x[:2], x, st),
        lambda: gs.gs_gated_norm_fwd(x, x, x, x, st[:2]),
        lambda: gs.gs_gated_norm_fwd(x, x, x, x, st, w_pre=torch.ones(5, device="cuda")),
        lambda: gs.gs_gated_norm_fwd(x, x, x, x, st, gate=torch.ones(2, Cn, device="cuda")),
        lambda: gs.gs_gated_norm_fwd(x, x, x, x, st, group_offsets=torch.zeros(2, dtype=torch.int32, device="cuda")),
        lambda: gs.gs_gated_norm_fwd(x, None, None, None, st),
        lambda: gs.gs_gated_norm_fwd(x, x, x, x, st, y_q=q),
        lambda: gs.gs_glu_fwd(x, x[:, :8], x),
        lambda: gs.gs_glu_bwd(q, e, q, e, x, x[:2], x),
        lambda: gs.gs_act8_wgrad(x, q, e, torch.empty(5, Cn, device="cuda"), q.view(torch.uint8).view(-1)),
        lambda: gs.gs_act8_wgrad(x, q, e, torch.empty(Cn, Cn, device="cuda").half(), q.view(torch.uint8).view(-1)),
        lambda: gs.gs_rope(gs.Rope([64]), torch.zeros(T, 2, dtype=torch.int32, device="cuda"), x[:, None]),
        lambda: gs.gs_rope(gs.Rope([64]), torch.zeros(T, 1, device="cuda"), x[:, None]),
        lambda: gs.gs_rope(gs.Rope([64]), torch.zeros(T, 1, dtype=torch.int32, device="cuda"), x),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail("call %d was accepted" % i)
    with pytest.raises(gs.GSError, match="invalid argument"):                    # a wider head than 64
        gs.gs_rope(gs.Rope([66]), torch.zeros(T, 1, dtype=torch.int32, device="cuda"), x[:, None])
    with pytest.raises(gs.GSError, match="invalid argument"):                    # a gradient with no gate
        gs.gs_gated_norm_bwd(x, x, st, x, x, x, x, dgate=torch.empty(1, Cn, device="cuda"),
                             workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    with pytest.raises(KeyError):
        gs.gs_glu_fwd(x, x, x, act="relu")
