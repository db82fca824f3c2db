"""The network operators over sizes that reach the kernels' steady state: rings that
wrap, blocks and teams that go from row to row, tiles that one pair of SMs sums whole
before it takes its share of the others.  Compared with 64-bit torch on the GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -24, torch.float32: 1e-38}


@pytest.fixture(scope="module")
def gs():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_splatting_differentiable_gs_gb300 as gs
    return gs


def _rand(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def _rows(t, pad, offset):
    """A copy of a matrix whose rows are `pad` elements further apart, `offset` in."""
    T, C = t.shape
    flat = torch.full((T * (C + pad) + offset,), 7.0, device="cuda").to(t.dtype)
    v = flat[offset:].view(T, C + pad)[:, :C]
    v.copy_(t)
    return v


def _close(got, want, bound, what):
    got = got.double()
    err = (got - want).abs()
    assert not torch.isnan(got).any() and (err <= bound).all(), (what, float((err - bound).max()))


def _ckpt(x):
    """The checkpoint of x from the definition: (q, e, values), on the GPU."""
    T, C = x.shape
    ld = -(-C // 32) * 32
    v = torch.nn.functional.pad(x.double(), (0, ld - C)).view(T, -1, 32)
    big = v.abs().amax(2)
    m, k = torch.frexp(big / 127)
    k = torch.where(big > 0, (k - (m == 0.5).int()).clamp(min=-126), -126)
    step = ((k.long() + 1023) << 52).view(torch.float64)  # 2^k to the last bit
    q = (v / step[..., None]).round()
    return q.flatten(1).to(torch.int8), (k + 127).to(torch.uint8), (q * step[..., None]).flatten(1)[:, :C]


# -- rotary positions ------------------------------------------------------


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,hq,hk,D,dims,inter,pad", [
    (20011, 8, 2, 64, (16, 24, 24), False, 0),
    (40000, 3, 3, 80, (20, 26, 26), True, 0),
    (25000, 2, 1, 31, (6, 10), False, 1),      # odd strides
    (70000, 1, 0, 8, (8,), True, 0),
])
def test_rope_blocks_walk_over_the_tokens(gs, dt, T, hq, hk, D, dims, inter, pad):
    r = _rand(T)
    pos = torch.randint(0, 300, (T, len(dims)), device="cuda", dtype=torch.int32,
                        generator=torch.Generator(device="cuda").manual_seed(T))
    rope = gs.Rope(dims, interleaved=inter)
    sets = []
    for h in (hq, hk):
        sets.append(_rows(r(T, h * D).to(dt), pad, pad).unflatten(1, (h, D)) if h else None)
    out = [torch.empty(T, x.shape[1], D, dtype=dt, device="cuda") if x is not None else None for x in sets]
    gs.gs_rope(rope, pos, sets[0], sets[1], q_out=out[0], k_out=out[1])
    for got, x in zip(out, sets):
        if x is None:
            continue
        want, mag, at = x.double().clone(), x.double().abs(), 0
        pair = mag.clone()
        for a, d in enumerate(dims):
            f = 10000.0 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
            ang = (pos[:, a, None].double() * f)[:, None]
            i0 = slice(at, at + d, 2) if inter else slice(at, at + d // 2)
            i1 = slice(at + 1, at + d, 2) if inter else slice(at + d // 2, at + d)
            u, v = x[..., i0].double(), x[..., i1].double()
            want[..., i0], want[..., i1] = u * ang.cos() - v * ang.sin(), u * ang.sin() + v * ang.cos()
            pair[..., i0] = pair[..., i1] = mag[..., i0] + mag[..., i1]
            at += d
        # the angle (pi 2^-25), two ulp of the sine, three roundings; the stored type
        _close(got, want, pair * 10 * U + want.abs() * EPS[dt] + TINY[dt], "rope")


# -- gated norms -------------------------------------------------------------


def _norm(v, center, eps):
    mean = v.mean(1, keepdim=True) if center else torch.zeros_like(v[:, :1])
    return mean, ((v - mean) ** 2).mean(1, keepdim=True).add(eps).rsqrt()


@pytest.mark.parametrize("dt,rt", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32),
                                   (torch.float32, torch.float32)])
@pytest.mark.parametrize("T,C,G,center,pad,offset", [
    (6500, 256, 7, False, 0, 0),      # sixteen teams of a warp, ragged groups
    (9001, 96, 3, True, 0, 0),
    (6100, 1000, 5, True, 8, 0),
    (6007, 517, 4, False, 0, 0),      # rows that start anywhere
    (7001, 130, 9, True, 3, 1),
    (2500, 4104, 2, False, 0, 0),     # teams of several warps
    (1500, 4099, 3, True, 0, 0),
])
def test_norms_over_many_rows(gs, dt, rt, T, C, G, center, pad, offset):
    eps, r = 1e-5, _rand(T + C)
    x, block, dxo, dy = r(T, C).to(rt), (2 * r(T, C) + 0.5).to(dt), r(T, C).to(rt), r(T, C).to(dt)
    w_pre, w_post, scale, gate = 1 + 0.2 * r(C), 1 + 0.2 * r(C), 0.5 + 0.2 * r(C), r(G, C).to(dt)
    cuts = torch.randint(0, T + 1, (G - 1,), generator=torch.Generator().manual_seed(C)).sort().values
    if G > 2:
        cuts[1] = cuts[0]
    off = torch.cat([torch.tensor([0]), cuts, torch.tensor([T])]).to(torch.int32).cuda()
    of = torch.repeat_interleave(torch.arange(G, device="cuda"), (off[1:] - off[:-1]).long())
    kw = dict(w_pre=w_pre, w_post=w_post, gate=gate, group_offsets=off, res_scale=scale, center=center)
    rows = lambda t: _rows(t, pad, offset)  # noqa: E731
    xo, y, st = rows(torch.zeros_like(x)), rows(torch.zeros_like(block)), torch.empty(T, 4, device="cuda")
    y_q, y_e = gs.act8_empty(T, C)
    gs.gs_gated_norm_fwd(rows(x), rows(block), xo, y, st, y_q=y_q, y_e=y_e, eps=eps, **kw)
    b = block.double()
    mb, rb = _norm(b, center, eps)
    k = w_post.double() * scale.double() * gate.double()[of]
    m = (b - mb) * rb
    want = x.double() + k * m
    # statistics: chains of 32 values a lane, 5 shuffles, 16 warps; then a few roundings.
    # A mean is off by chain times the mean magnitude; 1 / deviation, relatively, by the
    # chain, 4 u and what the mean and the values are off by.
    chain, size = 64 * U, lambda v: v.abs().mean(1, keepdim=True)  # noqa: E731
    b_err = chain * size(b)
    m_err = rb * (b_err + U * b.abs()) + m.abs() * (chain + 8 * U + rb * b_err)
    xo_err = 8 * U * ((k * m).abs() + want.abs()) + k.abs() * m_err
    _close(xo, want, xo_err + EPS[rt] * want.abs() + TINY[rt], "x'")
    mean, rstd = _norm(want, center, eps)
    n, worst, x_err = (want - mean) * rstd, xo_err.amax(1, keepdim=True), chain * size(want)
    n_err = rstd * (xo_err + worst + x_err + U * want.abs()) + n.abs() * (
        chain + 8 * U + rstd * (2 * worst + x_err))
    wy = w_pre.double() * n
    _close(y, wy, w_pre.double().abs() * n_err + (8 * U + EPS[dt]) * wy.abs() + TINY[dt], "y")
    q, e, _ = _ckpt(y)
    assert torch.equal(y_q, q) and torch.equal(y_e, e)

    # backward, from the values that the forward left
    out = dict(dw_pre=torch.empty(C, device="cuda"), dw_post=torch.empty(C, device="cuda"),
               dres_scale=torch.empty(C, device="cuda"), dgate=torch.empty(G, C, device="cuda"))
    ws = torch.empty(gs.gs_gated_norm_workspace_bytes(C, G), dtype=torch.uint8, device="cuda")
    dx, db = rows(torch.zeros_like(x)), rows(torch.zeros_like(block))
    args = (xo, rows(block), st, rows(dxo), rows(dy))
    gs.gs_gated_norm_bwd(*args, dx, db, workspace=ws, **kw, **out)
    s = st.double()
    n = (xo.double() - s[:, 2:3]) * s[:, 3:4]
    m = (b - s[:, 0:1]) * s[:, 1:2]
    h = dy.double() * w_pre.double()
    mean = lambda v: v.mean(1, keepdim=True)  # noqa: E731
    c = 1.0 if center else 0.0
    d = dxo.double() + s[:, 3:4] * (h - n * mean(h * n) - c * mean(h))
    nx = n.abs() + xo.double().abs() * s[:, 3:4]
    mag = s[:, 3:4] * (h.abs() + nx * mean(h.abs() * nx) + mean(h.abs())) + dxo.double().abs()
    _close(dx, d, chain * mag + EPS[rt] * d.abs() + TINY[rt], "dx")
    dk = d * k
    want = s[:, 1:2] * (dk - m * mean(dk * m) - c * mean(dk))
    mx, km = m.abs() + b.abs() * s[:, 1:2], mag * k.abs()
    big = s[:, 1:2] * (km + mx * mean(km * mx) + mean(km))
    _close(db, want, 2 * chain * big + EPS[dt] * want.abs() + TINY[dt], "dblock")
    # sums: a range's rows in turn (T / 152 and one), teams, 304 ranges over 32 lanes, groups
    add = (T / 152 + 128) * U + 2 * chain
    one = torch.zeros(T, G, dtype=torch.float64, device="cuda")
    one[torch.arange(T, device="cuda"), of] = 1.0
    g, wp, sc = gate.double()[of], w_post.double(), scale.double()
    for name, terms, size in (("dw_pre", dy.double() * n, dy.double().abs() * nx),
                              ("dw_post", d * m * g * sc, mag * mx * (g * sc).abs()),
                              ("dres_scale", d * m * g * wp, mag * mx * (g * wp).abs())):
        _close(out[name], terms.sum(0), add * size.sum(0) + 1e-30, name)
    _close(out["dgate"], one.t() @ (d * m * sc * wp), add * (one.t() @ (mag * mx * (sc * wp).abs())) + 1e-30, "dgate")
    again = {name: torch.empty_like(v) for name, v in out.items()}
    dx2, db2 = rows(torch.zeros_like(x)), rows(torch.zeros_like(block))
    gs.gs_gated_norm_bwd(*args, dx2, db2, workspace=ws, **kw, **again)
    assert torch.equal(dx, dx2) and torch.equal(db, db2)
    assert all(torch.equal(out[name], again[name]) for name in out)


# -- 8-bit checkpoints -------------------------------------------------------


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,C,pad,offset", [(5000, 256, 0, 0), (9000, 40, 8, 0), (3500, 301, 0, 0),
                                            (4001, 83, 2, 3), (20000, 7, 0, 1), (3000, 1361, 0, 0)])
def test_checkpoints_and_gated_units_over_many_rows(gs, dt, T, C, pad, offset):
    r = _rand(T + C)
    gate, up, dh = (2 * r(T, C)).to(dt), r(T, C).to(dt), r(T, C).to(dt)
    (gq, ge, gv), (uq, ue, uv) = _ckpt(gate), _ckpt(up)
    rows = lambda t: _rows(t, pad, offset)  # noqa: E731
    q, e = gs.act8_empty(T, C)
    gs.gs_act8_encode(rows(gate), q, e)
    assert torch.equal(q, gq) and torch.equal(e, ge)
    back = rows(torch.zeros_like(gate))
    gs.gs_act8_decode(q, e, back)
    assert torch.equal(back.double(), gv.to(dt).double())
    h = rows(torch.zeros_like(gate))
    g8, u8, h8 = (gs.act8_empty(T, C) for _ in range(3))
    dg, du = rows(torch.zeros_like(gate)), rows(torch.zeros_like(gate))
    gs.gs_glu_fwd(rows(gate), rows(up), h, *g8, *u8)
    gs.gs_glu_bwd(*g8, *u8, rows(dh), dg, du, *h8)
    assert torch.equal(g8[0], gq) and torch.equal(g8[1], ge) and torch.equal(u8[0], uq) and torch.equal(u8[1], ue)
    a = gate.double()
    want = a * torch.sigmoid(a) * up.double()
    _close(h, want, want.abs() * ((8 + 4 * a.abs()) * U + EPS[dt]) + 4 * U * (a * up.double()).abs() + TINY[dt], "h")
    s = torch.sigmoid(gv)
    f, df = gv * s, s * (1 + gv * (1 - s))
    g, mag = dh.double(), gv.abs()
    want = g * uv * df
    _close(dg, want, (12 + 6 * mag) * 2 * U * (g * uv).abs() + EPS[dt] * want.abs() + TINY[dt], "dgate")
    want = g * f
    _close(du, want, (8 + 4 * mag) * U * g.abs() * (mag + 1) + EPS[dt] * want.abs() + TINY[dt], "dup")
    hv = torch.empty(T, C, device="cuda")
    gs.gs_act8_decode(*h8, hv)
    step = torch.exp2(h8[1].double() - 127).repeat_interleave(32, 1)[:, :C]
    _close(hv, f * uv, 0.5 * step + (8 + 4 * mag) * U * (mag * uv.abs() + 1e-30), "h8")


# -- weight gradient ---------------------------------------------------------


@pytest.mark.parametrize("dt,out_t", [(torch.bfloat16, torch.float32), (torch.float16, torch.bfloat16),
                                      (torch.float32, torch.float32)])
@pytest.mark.parametrize("T,N,K", [
    (1100, 2600, 2050),      # 99 tiles: whole ones first, then shares of the rest
    (70, 5200, 1900),        # two steps a tile, two whole tiles each
    (9000, 5120, 1024),      # 80 tiles of 141 steps: rings wrap many times, runs end within a tile
    (40000, 256, 256),       # one tile, dealt out
    (30001, 300, 90),
])
def test_wgrad_steady_state(gs, dt, out_t, T, N, K):
    r = _rand(T + N)
    dy = r(T, N).to(dt)
    q, e, x = _ckpt(r(T, K) * torch.exp2(torch.randint(-6, 6, (T, 1), device="cuda").float()))
    ws = torch.zeros(gs.gs_act8_wgrad_workspace_bytes(T, N, K, dt), dtype=torch.uint8, device="cuda")
    dw = torch.full((N, K), 3.0, device="cuda").to(out_t)
    gs.gs_act8_wgrad(dy, q, e, dw, ws)
    want = dy.double().t() @ x
    mag = dy.double().abs().t() @ x.abs()
    # runs of 32 steps of 64 tokens cut at every 16 (128 cuts of 2^-23), then runs and shares
    bound = (2 * 128 + T / 2048 + 80) * U * mag + EPS[out_t] * want.abs() + 1e-30
    _close(dw, want, bound, "dw")
    again = torch.empty_like(dw)
    gs.gs_act8_wgrad(dy, q, e, again, ws)
    assert torch.equal(dw, again)
    base = r(N, K).to(out_t)
    acc = base.clone()
    gs.gs_act8_wgrad(dy, q, e, acc, ws, accumulate=True)
    total = want + base.double()
    _close(acc, total, bound + (2 * U + EPS[out_t]) * (total.abs() + base.double().abs()), "added")
    assert gs.gs_workspace_status(ws) == gs.GS_OK
