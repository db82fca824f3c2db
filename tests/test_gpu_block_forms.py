"""The feed-forward block and linear attention where such kernels go wrong: extreme values,
groups beside broken ones, other streams, captured graphs, repeated calls, arrays past 2^31
elements, waits that run out, gradients against differences."""
import ctypes as C

import pytest
import torch

import block_plain as plain

pytestmark = pytest.mark.gpu
EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def gs():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_splatting_differentiable_gs_gb300 as gs
    return gs


def _rand(*shape, seed=0, std=1.0, dt=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)


def _attn_ws(gs, *a):
    return torch.empty(gs.gs_linear_attn_workspace_bytes(*a), dtype=torch.uint8, device="cuda")


def _ffn_ws(gs, *a):
    return torch.zeros(gs.gs_ffn_workspace_bytes(*a), dtype=torch.uint8, device="cuda")


# --------------------------------------------------------------------------
# values


@pytest.mark.parametrize("dt,size,vsize", [
    (torch.float16, 1.0, 300.0),       # states past fp16's range (about 300 * 40 tokens' keys)
    (torch.float16, 2.0 ** -12, 1.0),  # keys whose terms are below it
    (torch.bfloat16, 2.0 ** -60, 2.0 ** 40),
    (torch.bfloat16, 2.0 ** 40, 2.0 ** -60),
])
def test_attention_at_other_scales(gs, dt, size, vsize):
    """Keys and values scaled: outputs and states scale with them, exactly for powers of two
    as long as nothing leaves the type's range.  300 is none: its products with fp16 values
    are rounded once more, by up to 2^-11 of each value, and so are keys below 2^-14: the sums
    of both are off by 2^-11 of their terms at most, at random signs 2^-11 of their norm."""
    T, H, D = 300, 2, 64
    q, k, v = (_rand(T, H, D, seed=i, dt=dt) for i in range(3))
    k = k.clamp(min=-4, max=4)
    a = torch.tensor([0.0, -0.02], device="cuda")
    ws = _attn_ws(gs, T, H, H, D, D)

    def run(k, v, scale):
        o, s = torch.empty_like(q), torch.empty(1, H, D, D, device="cuda")
        gs.gs_linear_attn_fwd(q, k, v, a, o, state_out=s, scale=scale, workspace=ws)
        return o.double(), s.double()

    # (a smaller query keeps the products of q and k in fp16's range, and the outputs)
    want_o, want_s = run(k, v, 0.125)
    o, s = run((k.float() * size).to(dt), (v.float() * vsize).to(dt), 0.125 / vsize / size)
    rel = 2.0 ** -11 if dt is torch.float16 else 0.0
    assert (s / size / vsize - want_s).norm() <= (2e-6 + rel) * want_s.norm()
    assert (o - want_o).norm() <= (2 * EPS[dt] + rel) * want_o.norm()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_broken_group_leaves_the_others_alone(gs, bad):
    T, H, D = 400, 2, 64
    q, k, v, do = (_rand(T, H, D, seed=i) for i in range(4))
    off = torch.tensor([0, 130, 131, 300, 400], dtype=torch.int32, device="cuda")
    a = torch.tensor([-0.1, 0.0], device="cuda")
    ws = _attn_ws(gs, T, H, H, D, D, 4)

    def run():
        out = [torch.zeros_like(q) for _ in range(4)]
        s, ds = (torch.zeros(4, H, D, D, device="cuda") for _ in range(2))
        gs.gs_linear_attn_fwd(q, k, v, a, out[0], group_offsets=off, state_out=s, workspace=ws)
        gs.gs_linear_attn_bwd(q, k, v, a, do, *out[1:], group_offsets=off, dstate=ds, workspace=ws)
        return out, s, ds

    out, s, ds = run()
    for t in (q, k, v, do):
        t[200, 1, 3] = bad
    new, ns, nds = run()
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[131:300] = False
    for x, y in zip(out, new):
        assert torch.equal(x[keep], y[keep]) and torch.equal(x[:, 0], y[:, 0])
        assert not torch.isfinite(y[131:300, 1]).all()
    for x, y in ((s, ns), (ds, nds)):
        assert torch.equal(x[[0, 1, 3]], y[[0, 1, 3]]) and torch.equal(x[:, 0], y[:, 0])


def test_a_broken_row_of_the_block_stays_one(gs):
    T, Ch, F = 300, 96, 160
    x, w, dh = _rand(T, Ch), _rand(2 * F, Ch, seed=1, std=0.1), _rand(T, F, seed=2)
    ws = _ffn_ws(gs, T, Ch, F)

    def run():
        h, dx = torch.empty(T, F, dtype=x.dtype, device="cuda"), torch.empty_like(x)
        gs.gs_ffn_fwd(x, w, h, ws)
        gs.gs_ffn_bwd(x, w, dh, dx, None, ws)
        return h, dx

    before = run()
    x[77, 5], dh[78, 9] = float("nan"), float("inf")
    for y, z, rows in zip(before, run(), ((77,), (77, 78))):
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[list(rows)] = False
        assert torch.equal(y[keep], z[keep]) and not torch.isfinite(z[list(rows)]).all(1).any()


# --------------------------------------------------------------------------
# calls


def test_accumulated_and_missing_gradients(gs):
    T, Ch, F = 700, 200, 136
    x, w, dh = _rand(T, Ch), _rand(2 * F, Ch, seed=1, std=0.1), _rand(T, F, seed=2)
    ws = _ffn_ws(gs, T, Ch, F)
    dx, dw = torch.empty_like(x), torch.empty(2 * F, Ch, device="cuda")
    gs.gs_ffn_bwd(x, w, dh, dx, dw, ws)
    one, two = torch.empty_like(x), torch.empty_like(dw)
    gs.gs_ffn_bwd(x, w, dh, one, None, ws)
    gs.gs_ffn_bwd(x, w, dh, None, two, ws)
    assert torch.equal(one, dx) and torch.equal(two, dw)
    start = torch.randn_like(dw)
    acc = start.clone()
    gs.gs_ffn_bwd(x, w, dh, None, acc, ws, accumulate=True)
    assert torch.equal(acc, start + dw)
    low = start.to(x.dtype)
    want = (low.float() + dw).to(x.dtype)
    gs.gs_ffn_bwd(x, w, dh, None, low, ws, accumulate=True)
    assert torch.equal(low, want)


def test_nothing_to_do(gs):
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), _rand(96, 64)
    ws = _ffn_ws(gs, 0, 64, 48)
    h, dw = torch.empty(0, 48, dtype=x.dtype, device="cuda"), torch.ones(96, 64, device="cuda")
    gs.gs_ffn_fwd(x, w, h, ws)
    gs.gs_ffn_bwd(x, w, h, torch.empty_like(x), dw, ws, accumulate=True)
    assert (dw == 1).all()
    gs.gs_ffn_bwd(x, w, h, torch.empty_like(x), dw, ws)
    assert (dw == 0).all()
    q = torch.empty(0, 2, 16, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    s, a = torch.randn(3, 2, 16, 16, device="cuda"), torch.tensor([-0.5, 0.0], device="cuda")
    aws = _attn_ws(gs, 0, 2, 2, 16, 16, 3)
    out, ds = torch.empty_like(s), torch.empty_like(s)
    gs.gs_linear_attn_fwd(q, q, q, a, q, group_offsets=off, state=s, state_out=out, workspace=aws)
    gs.gs_linear_attn_bwd(q, q, q, a, q, q, q, q, group_offsets=off, dstate_out=s, dstate=ds, workspace=aws)
    assert torch.equal(out, s) and torch.equal(ds, s)
    gs.gs_linear_attn_step(q, q, q, a, torch.empty(0, 2, 16, 16, device="cuda"), q)


def test_states_in_place(gs):
    T, H, D = 500, 2, 64
    q, k, v = (_rand(T, H, D, seed=i) for i in range(3))
    a, s = torch.tensor([-0.1, 0.0], device="cuda"), torch.randn(1, H, D, D, device="cuda")
    ws = _attn_ws(gs, T, H, H, D, D)
    o, out = torch.empty_like(q), torch.empty_like(s)
    gs.gs_linear_attn_fwd(q, k, v, a, o, state=s, state_out=out, workspace=ws)
    again = torch.empty_like(q)
    gs.gs_linear_attn_fwd(q, k, v, a, again, state=s, state_out=s, workspace=ws)
    assert torch.equal(o, again) and torch.equal(s, out)
    ds = torch.randn_like(s)
    d, want = [torch.empty_like(q) for _ in range(3)], torch.empty_like(s)
    gs.gs_linear_attn_bwd(q, k, v, a, q, *d, dstate_out=ds, dstate=want, workspace=ws)
    e = [torch.empty_like(q) for _ in range(3)]
    gs.gs_linear_attn_bwd(q, k, v, a, q, *e, dstate_out=ds, dstate=ds, workspace=ws)
    assert torch.equal(ds, want) and all(torch.equal(x, y) for x, y in zip(d, e))


def test_repeated_calls_streams_and_graphs(gs):
    """The same bits each time, on another stream, and from captured graphs that share
    their workspaces and are replayed in turn with other inputs."""
    T, H, K, D, Ch, F = 600, 4, 2, 64, 200, 264
    q, do = _rand(T, H, D), _rand(T, H, D, seed=3)
    k, v = _rand(T, K, D, seed=1), _rand(T, K, D, seed=2)
    x, w, dh = _rand(T, Ch, seed=4), _rand(2 * F, Ch, seed=5, std=0.1), _rand(T, F, seed=6)
    a = -torch.exp2(-torch.arange(1.0, H + 1, device="cuda"))
    aws, fws = _attn_ws(gs, T, H, K, D, D), _ffn_ws(gs, T, Ch, F)

    def buffers():
        e = torch.empty_like
        return [e(q), torch.empty(1, H, D, D, device="cuda"), e(q), e(k), e(v), torch.empty(1, H, D, D, device="cuda"),
                torch.empty(T, F, dtype=x.dtype, device="cuda"), e(x), e(w)]

    def run(b, stream=None):
        gs.gs_linear_attn_fwd(q, k, v, a, b[0], state_out=b[1], workspace=aws, stream=stream)
        gs.gs_linear_attn_bwd(q, k, v, a, do, b[2], b[3], b[4], dstate=b[5], workspace=aws, stream=stream)
        gs.gs_ffn_fwd(x, w, b[6], fws, stream=stream)
        gs.gs_ffn_bwd(x, w, dh, b[7], b[8], fws, stream=stream)

    want, other = buffers(), buffers()
    run(want)
    for _ in range(3):
        run(other)
        assert all(torch.equal(p, r) for p, r in zip(want, other))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for t in other:
        t.zero_()
    torch.cuda.synchronize()
    run(other, stream=side)
    side.synchronize()
    assert all(torch.equal(p, r) for p, r in zip(want, other))
    graphs, outs = [], [buffers(), buffers()]
    for b in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(b)
        graphs.append(g)
    for step in range(3):
        for t in (q, k, v, do, x, w, dh):
            t.copy_(t.flip(0))
        run(want)
        for g, b in zip(graphs, outs):
            for t in b:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, r) for p, r in zip(want, b)), step
    gs.gs_linear_attn_status()
    assert gs.gs_workspace_status(fws) == gs.GS_OK


def test_refusals(gs):
    x, w, h = _rand(8, 32), _rand(64, 32), _rand(8, 32)
    ws = _ffn_ws(gs, 8, 32, 32)
    q, s = _rand(8, 2, 16), torch.zeros(1, 2, 16, 16, device="cuda")
    a, aws = torch.zeros(2, device="cuda"), _attn_ws(gs, 8, 2, 2, 16, 16)
    bad = [
        lambda: gs.gs_ffn_fwd(x.float(), w.float(), h.float(), ws),
        lambda: gs.gs_ffn_fwd(x, w.half(), h, ws),
        lambda: gs.gs_ffn_fwd(x.cpu(), w, h, ws),
        lambda: gs.gs_ffn_fwd(x, w[:63], h, ws),
        lambda: gs.gs_ffn_fwd(x, w[:, :31], h, ws),
        lambda: gs.gs_ffn_fwd(x, w, h[:, :31], ws),
        lambda: gs.gs_ffn_fwd(x, w, h.t()[:8], ws),
        lambda: gs.gs_ffn_fwd(x, w, h, ws, act="relu"),
        lambda: gs.gs_ffn_bwd(x, w, h, torch.empty_like(x), None, ws[:-1]),
        lambda: gs.gs_ffn_fwd(x, w, h, ws[1:]),
        lambda: gs.gs_ffn_fwd(x, w, h, ws.view(torch.int32)),
        lambda: gs.gs_ffn_fwd(x, w, h, None),
        lambda: gs.gs_ffn_fwd(x[0], w, h, ws),
        lambda: gs.gs_ffn_bwd(x, w, h, x[:, :31], None, ws),
        lambda: gs.gs_ffn_bwd(x, w, h, None, w.half(), ws),
        lambda: gs.gs_ffn_fwd(x, w, h[:1].expand(8, 32), ws),
        lambda: gs.gs_linear_attn_fwd(q.float(), q.float(), q.float(), a, q, workspace=aws),
        lambda: gs.gs_linear_attn_fwd(q, q.half(), q, a, q, workspace=aws),
        lambda: gs.gs_linear_attn_fwd(q, q[:7], q, a, q, workspace=aws),
        lambda: gs.gs_linear_attn_fwd(q[:, :1], q, q, a[:1], q[:, :1], workspace=aws),
        lambda: gs.gs_linear_attn_fwd(q, q, q, a[:1], q, workspace=aws),
        lambda: gs.gs_linear_attn_fwd(q, q, q, a.double(), q, workspace=aws),
        lambda: gs.gs_linear_attn_fwd(q, q, q, a, q[..., :15], workspace=aws),
        lambda: gs.gs_linear_attn_fwd(q, q, q, a, q),
        lambda: gs.gs_linear_attn_fwd(q, q, q, a, torch.empty_like(q), workspace=aws[:64]),
        lambda: gs.gs_linear_attn_fwd(q, q, q, a, q, state=s[0], workspace=aws),
        lambda: gs.gs_linear_attn_fwd(q, q, q, a, q, group_offsets=torch.zeros(3, device="cuda"), workspace=aws),
        lambda: gs.gs_linear_attn_fwd(q, q, q, a, q, group_offsets=torch.zeros(1, dtype=torch.int32, device="cuda"),
                                      workspace=aws),
        lambda: gs.gs_linear_attn_fwd(q, q, q, a, q[:1].expand(8, 2, 16), workspace=aws),
        lambda: gs.gs_linear_attn_fwd(*[_rand(8, 2, 129)] * 3, a, _rand(8, 2, 129), workspace=aws),
        lambda: gs.gs_linear_attn_step(q, q, q, a, s, torch.empty_like(q)),
        lambda: gs.gs_linear_attn_step(q, q, q, a, None, torch.empty_like(q)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, gs.GSError)):
            call()
            pytest.fail("call %d was taken" % i)


# --------------------------------------------------------------------------
# gradients against differences


def test_gradients_against_differences(gs):
    """Along a direction the loss, in 64 bits, changes as the gradients say: differences of
    width e are off by e^2, the gradients by their rounding (two at EPS, at random)."""
    torch.manual_seed(0)
    T, H, K, D, E = 150, 4, 2, 24, 40
    dt = torch.bfloat16
    q, k, v = (torch.randn(T, h, d).to(dt) for h, d in ((H, D), (K, D), (K, E)))
    s, do, ds = torch.randn(1, H, D, E), torch.randn(T, H, E).to(dt), torch.randn(1, H, D, E)
    a = torch.tensor([-0.5, -0.1, -0.01, 0.0])
    d = [torch.empty_like(t).cuda() for t in (q, k, v)] + [torch.empty_like(s).cuda()]
    gs.gs_linear_attn_bwd(q.cuda(), k.cuda(), v.cuda(), a.cuda(), do.cuda(), *d[:3], state=s.cuda(),
                          dstate_out=ds.cuda(), dstate=d[3], scale=0.3, workspace=_attn_ws(gs, T, H, K, D, E))
    at = [t.double() for t in (q, k, v, s)]
    for i in range(4):
        step = torch.randn_like(at[i])
        loss = []
        for e in (1e-3, -1e-3):
            x = list(at)
            x[i] = at[i] + e * step
            out, last = plain.attn(*x[:3], a, [0, T], x[3], 0.3)
            loss.append((out * do.double()).sum() + (last * ds.double()).sum())
        want, got = (loss[0] - loss[1]) / 2e-3, (d[i].double().cpu() * step).sum()
        noise = d[i].double().norm().item() * EPS[dt] * 4  # a random direction's share of the rounding
        assert abs(got - want) <= noise + 1e-5 * abs(want), i
    Ch, F = 72, 56
    x, w, dh = torch.randn(T, Ch).to(dt), (torch.randn(2 * F, Ch) * 0.2).to(dt), torch.randn(T, F).to(dt)
    for act in ("silu", "gelu"):
        dx, dw = torch.empty_like(x).cuda(), torch.empty(2 * F, Ch).cuda()
        gs.gs_ffn_bwd(x.cuda(), w.cuda(), dh.cuda(), dx, dw, _ffn_ws(gs, T, Ch, F), act=act)
        for t, grad in ((x, dx), (w, dw)):
            step = torch.randn(t.shape, dtype=torch.float64)
            loss = [(plain.ffn(x.double() + e * step if t is x else x.double(),
                               w.double() + e * step if t is w else w.double(), act)[0] * dh.double()).sum()
                    for e in (1e-4, -1e-4)]
            want, got = (loss[0] - loss[1]) / 2e-4, (grad.double().cpu() * step).sum()
            assert abs(got - want) <= grad.double().norm().item() * EPS[dt] * 4 + 1e-5 * abs(want), act


# --------------------------------------------------------------------------
# sizes


def test_block_past_two_to_the_31_elements(gs):
    """h has 2.2e9 elements: rows from all over against the same rows alone."""
    T, Ch, F = 1050000, 64, 2104
    x, w = _rand(T, Ch), _rand(2 * F, Ch, seed=1, std=0.2)
    h = torch.empty(T, F, dtype=x.dtype, device="cuda")
    ws = _ffn_ws(gs, T, Ch, F)
    gs.gs_ffn_fwd(x, w, h, ws)
    rows = torch.tensor([0, 1, 255, 256, 524288, 1020700, 1020701, T - 257, T - 1], device="cuda")
    rows = torch.cat([rows, torch.arange(T - 300, T - 260, device="cuda")])
    few = torch.empty(len(rows), F, dtype=x.dtype, device="cuda")
    gs.gs_ffn_fwd(x[rows], w, few, ws)
    assert torch.equal(h[rows], few)
    dx, part = torch.empty_like(x), torch.empty(len(rows), Ch, dtype=x.dtype, device="cuda")
    gs.gs_ffn_bwd(x, w, h, dx, None, ws)
    gs.gs_ffn_bwd(x[rows], w, few, part, None, ws)
    # sums in another order where tiles are shared out
    assert (dx[rows].float() - part.float()).norm() <= EPS[x.dtype] * part.float().norm()
    assert gs.gs_workspace_status(ws) == gs.GS_OK


def test_attention_past_two_to_the_31_elements(gs):
    """2.2e9 elements an array: the end of the stream alone, from the state that the tokens
    before it leave, and the gradients there."""
    T, H, D = 2100000, 16, 64
    cut = T - 1000
    q, k, v = (torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda").normal_() for _ in range(3))
    a = -torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
    out, s = torch.empty_like(q), torch.empty(1, H, D, D, device="cuda")
    ws = _attn_ws(gs, T, H, H, D, D)
    gs.gs_linear_attn_fwd(q, k, v, a, out, state_out=s, workspace=ws)
    head, end = torch.empty_like(s), torch.empty_like(s)
    tail = torch.empty(T - cut, H, D, dtype=q.dtype, device="cuda")
    part = torch.empty(cut, H, D, dtype=q.dtype, device="cuda")
    gs.gs_linear_attn_fwd(q[:cut], k[:cut], v[:cut], a, part, state_out=head, workspace=ws)
    gs.gs_linear_attn_fwd(q[cut:], k[cut:], v[cut:], a, tail, state=head, state_out=end, workspace=ws)
    close = lambda x, y, b: (x.float() - y.float()).norm() <= b * y.float().norm()  # noqa: E731
    assert close(out[cut:], tail, 2 * EPS[q.dtype]) and close(s, end, 1e-5)
    del part, tail
    d = [torch.empty_like(q) for _ in range(3)]
    ds = torch.empty_like(s)
    gs.gs_linear_attn_bwd(q, k, v, a, out, *d, dstate=ds, workspace=ws)
    e = [torch.empty(T - cut, H, D, dtype=q.dtype, device="cuda") for _ in range(3)]
    gs.gs_linear_attn_bwd(q[cut:], k[cut:], v[cut:], a, out[cut:], *e, state=head, dstate=end, workspace=ws)
    for x, y in zip(d, e):
        assert close(x[cut:], y, 2 * EPS[q.dtype])
    f = [torch.empty(1000, H, D, dtype=q.dtype, device="cuda") for _ in range(3)]
    # the first tokens' gradients from the state gradient that the others leave
    dmid = torch.empty_like(s)
    g = [torch.empty(T - 1000, H, D, dtype=q.dtype, device="cuda") for _ in range(3)]
    mid = torch.empty_like(s)
    gs.gs_linear_attn_fwd(q[:1000], k[:1000], v[:1000], a, torch.empty_like(f[0]), state_out=mid, workspace=ws)
    gs.gs_linear_attn_bwd(q[1000:], k[1000:], v[1000:], a, out[1000:], *g, state=mid, dstate=dmid, workspace=ws)
    first = torch.empty_like(s)
    gs.gs_linear_attn_bwd(q[:1000], k[:1000], v[:1000], a, out[:1000], *f, dstate_out=dmid, dstate=first, workspace=ws)
    for x, y in zip(d, f):
        assert close(x[:1000], y, 2 * EPS[q.dtype])
    assert close(ds, first, 1e-5)
    gs.gs_linear_attn_status()


def test_shared_heads_past_two_to_the_31_elements(gs):
    """2.2e9 elements of the query heads' gradients: the last and the first tokens' beside those of a call on the last
    ones alone, and of one on the first with the state gradient that the others leave."""
    T, H, K, D = 2200000, 16, 2, 64
    cut = T - 1000
    q, do = (torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda").normal_() for _ in range(2))
    k, v = (torch.empty(T, K, D, dtype=torch.bfloat16, device="cuda").normal_() for _ in range(2))
    a = -torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
    ws = _attn_ws(gs, T, H, K, D, D)
    close = lambda x, y: (x.float() - y.float()).norm() <= 2 * EPS[q.dtype] * y.float().norm()  # noqa: E731
    dq, dk, dv = (torch.empty_like(t) for t in (q, k, v))
    gs.gs_linear_attn_bwd(q, k, v, a, do, dq, dk, dv, workspace=ws)
    tail = [torch.empty_like(t[cut:]) for t in (q, k, v)]
    gs.gs_linear_attn_bwd(q[cut:], k[cut:], v[cut:], a, do[cut:], *tail, workspace=ws)
    assert close(dk[cut:], tail[1]) and close(dv[cut:], tail[2])
    mid = torch.empty(1, H, D, D, device="cuda")
    rest = [torch.empty_like(t[1000:]) for t in (q, k, v)]
    gs.gs_linear_attn_bwd(q[1000:], k[1000:], v[1000:], a, do[1000:], *rest, dstate=mid, workspace=ws)
    first = [torch.empty_like(t[:1000]) for t in (q, k, v)]
    gs.gs_linear_attn_bwd(q[:1000], k[:1000], v[:1000], a, do[:1000], *first, dstate_out=mid, workspace=ws)
    for x, y in zip((dq, dk, dv), first):
        assert close(x[:1000], y)
    gs.gs_linear_attn_status()


def test_many_groups(gs):
    """Thousands of short groups, some empty, against each alone in a few."""
    G, H, D = 5000, 2, 16
    gen = torch.Generator().manual_seed(0)
    n = torch.randint(0, 9, (G,), generator=gen)
    n[::7] = 0
    n[123] = 400
    off = torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)])
    T = int(off[-1])
    q, k, v = (_rand(T, H, D, seed=i) for i in range(3))
    a = torch.tensor([-0.2, 0.0], device="cuda")
    s0, s = torch.randn(G, H, D, D, device="cuda"), torch.empty(G, H, D, D, device="cuda")
    out = torch.empty_like(q)
    gs.gs_linear_attn_fwd(q, k, v, a, out, group_offsets=off.to(torch.int32).cuda(), state=s0, state_out=s,
                          workspace=_attn_ws(gs, T, H, H, D, D, G))
    for g in (0, 1, 7, 122, 123, 124, 2500, G - 1):
        b, e = int(off[g]), int(off[g + 1])
        want, last = plain.attn(q[b:e].double().cpu(), k[b:e].double().cpu(), v[b:e].double().cpu(), a.cpu(), [0, e - b],
                                s0[g:g + 1].double().cpu(), D ** -0.5)
        assert (s[g].double().cpu() - last[0]).norm() <= 1e-5 * last.norm()
        if e > b:
            assert (out[b:e].double().cpu() - want).norm() <= 2 * EPS[q.dtype] * want.norm()


@pytest.mark.parametrize("E", [41, 44])
def test_many_states(gs, E):
    """More elements of the states than the machine has threads, a group of many segments among short ones."""
    G, H, D = 60, 4, 40
    gen = torch.Generator().manual_seed(E)
    n = torch.randint(0, 90, (G,), generator=gen)
    n[3], n[17], n[41] = 0, 3001, 300
    off = torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)])
    T = int(off[-1])
    q, k = (_rand(T, H, D, seed=i) for i in range(2))
    v, do = (_rand(T, H, E, seed=i) for i in (2, 3))
    a = torch.tensor([-0.2, 0.0, -0.01, -0.001], device="cuda")
    s0, ds, s, d0 = (torch.randn(G, H, D, E, device="cuda") for _ in range(4))
    out, dq, dk, dv = (torch.empty_like(t) for t in (v, q, k, v))
    ws = _attn_ws(gs, T, H, H, D, E, G)
    kw = dict(group_offsets=off.to(torch.int32).cuda(), state=s0, workspace=ws)
    gs.gs_linear_attn_fwd(q, k, v, a, out, state_out=s, **kw)
    gs.gs_linear_attn_bwd(q, k, v, a, do, dq, dk, dv, dstate_out=ds, dstate=d0, **kw)
    for g in (0, 2, 3, 16, 17, 18, 41, G - 1):
        b, e = int(off[g]), int(off[g + 1])
        ins = [t[b:e].double().cpu().requires_grad_(True) for t in (q, k, v)]
        first = s0[g:g + 1].double().cpu().requires_grad_(True)
        want, last = plain.attn(*ins, a.cpu(), [0, e - b], first, D ** -0.5)
        total = (want * do[b:e].double().cpu()).sum() + (last * ds[g:g + 1].double().cpu()).sum()
        grads = torch.autograd.grad(total, ins + [first], allow_unused=True)
        # states: keys in two terms or more, 2^-17 each at most, and sums in fp32
        for x, y in ((s[g], last[0].detach()), (d0[g], grads[3][0])):
            assert (x.double().cpu() - y).norm() <= 2.0 ** -16 * y.norm()
        # three roundings to 16 bits that know nothing of one another: sqrt(3) half steps
        for x, y in ((out, want.detach()), (dq, grads[0]), (dk, grads[1]), (dv, grads[2])):
            if e > b:
                assert (x[b:e].double().cpu() - y).norm() <= 2 * EPS[q.dtype] * y.norm()


# --------------------------------------------------------------------------
# waits


@pytest.mark.parametrize("T,Ch,F,stops", [
    (256, 200, 128, (0, 1, 3)),          # one pair, four steps
    (3000, 700, 1500, (0, 5, 6, 7, 15)),  # rings full; the second of a pair's two tiles of 11 steps
])
def test_the_block_gives_up_and_the_context_survives(gs, T, Ch, F, stops):
    """Operands that never come: the waits run out (100 ms), the kernel waits for what is
    under way, flags the error and returns; the next call on the workspace is right."""
    L, vp = gs.lib(), C.c_void_p
    L.gs_selftest_ffn_timeout.restype = C.c_int
    L.gs_selftest_ffn_timeout.argtypes = [C.c_int64, C.c_int32, C.c_int32, vp, vp, vp, vp, C.c_size_t, C.c_int32, vp]
    x, w = _rand(T, Ch), _rand(2 * F, Ch, seed=1, std=0.1)
    ws = _ffn_ws(gs, T, Ch, F)
    want, got = (torch.empty(T, F, dtype=x.dtype, device="cuda") for _ in range(2))
    gs.gs_ffn_fwd(x, w, want, ws)
    stream = torch.cuda.current_stream().cuda_stream
    for steps in stops:
        st = L.gs_selftest_ffn_timeout(T, Ch, F, x.data_ptr(), w.data_ptr(), got.data_ptr(), ws.data_ptr(), ws.numel(),
                                       steps, stream)
        assert st == gs.GS_ERR_TIMEOUT, steps
        assert gs.gs_workspace_status(ws) == gs.GS_OK  # read and cleared
        got.fill_(7.0)
        gs.gs_ffn_fwd(x, w, got, ws)
        assert gs.gs_workspace_status(ws) == gs.GS_OK and torch.equal(got, want), steps
    st = L.gs_selftest_ffn_timeout(T, Ch, F, x.data_ptr(), w.data_ptr(), got.data_ptr(), ws.data_ptr(), ws.numel(),
                                   1 << 20, stream)
    assert st == gs.GS_OK and torch.equal(got, want)
