"""Linear attention with decays on the GPU against its plain 64-bit form.

Tolerances come from the arithmetic.  Let A be the same sum with every factor's magnitude
in its place.  The decayed products and the states are rounded once each before they are
multiplied on (half a step, EPS of their magnitude: EPS A in all), keys inside a segment
are taken to 2^-16, powers of the decay to 2^-20 and sums of up to 512 terms at a time
to 2^-15 of A."""
import pytest
import torch

import block_plain as plain

pytestmark = pytest.mark.gpu

EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -24}


@pytest.fixture(scope="module")
def gs():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_splatting_differentiable_gs_gb300 as gs
    return gs


def _heads(T, H, D, dt, g, std=1.0, layout="packed"):
    """Random heads in a layout of their own on the GPU, and in 64 bits."""
    v = (torch.randn(T, H, D, generator=g) * std).to(dt)
    if layout == "heads first":
        m = torch.empty(H, T, D, dtype=dt, device="cuda").transpose(0, 1)
    elif layout == "odd":
        m = torch.empty(T * (H * D + 5) + 1, dtype=dt, device="cuda")[1:].view(T, H * D + 5)[:, :H * D].view(T, H, D) \
            if T * H * D else torch.empty(T, H, D, dtype=dt, device="cuda")
    else:
        m = torch.empty(T, H + 2, D, dtype=dt, device="cuda")[:, 1:H + 1]
    m.copy_(v)
    return m, v.double()


def _close(got, want, bound, what):
    got = got.double().cpu()
    assert got.shape == want.shape
    over = ~((got - want).abs() <= bound)
    assert not over.any(), (what, int(over.sum()), float((got - want).abs().max()),
                            float(((got - want).abs() / bound).max()))


CASES = [  # tokens, query heads, key heads, dim, vdim, offsets, states, layout
    (1, 1, 1, 64, 64, None, True, "packed"),
    (1, 4, 2, 8, 16, None, False, "packed"),
    (2, 2, 2, 1, 1, None, True, "packed"),
    (63, 3, 3, 64, 64, None, True, "heads first"),
    (64, 2, 1, 64, 64, None, True, "packed"),
    (65, 2, 2, 32, 48, None, True, "odd"),
    (130, 4, 2, 57, 41, None, True, "odd"),
    (200, 6, 2, 72, 64, [0, 64, 64, 65, 193, 200], True, "packed"),
    (200, 2, 2, 128, 128, [0, 1, 129, 200], True, "packed"),
    (300, 4, 1, 128, 91, [0, 0, 150, 280], True, "packed"),     # rows behind the last group
    (333, 2, 2, 64, 64, None, False, "packed"),
    (700, 3, 1, 80, 16, [0, 333, 700], False, "odd"),
]


def _want(q, k, v, a, offsets, state, scale, grads=None, dlast=None):
    """Results and, with every factor's magnitude in its place, what the bounds go by."""
    def run(q, k, v, state, grads, dlast):
        leaves = [t.detach().clone().requires_grad_(True) for t in (q, k, v)]
        s = state.detach().clone().requires_grad_(True) if state is not None else None
        out, last = plain.attn(*leaves, a, offsets, s, scale)
        if grads is None:
            return [out.detach(), last.detach()]
        total = (out * grads).sum() + ((last * dlast).sum() if dlast is not None else 0)
        ins = leaves + ([s] if s is not None else [])
        g = torch.autograd.grad(total, ins, allow_unused=True)
        return [torch.zeros_like(i) if x is None else x for x, i in zip(g, ins)]

    mag = lambda t: t.abs() if t is not None else None  # noqa: E731
    return (run(q, k, v, state, grads, dlast),
            run(mag(q), mag(k), mag(v), mag(state), mag(grads), mag(dlast)))


def _bound(want, mag, dt):
    return want.abs() * EPS[dt] + (EPS[dt] * 1.01 + 2.0 ** -14) * mag + TINY[dt] * (1 + mag)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H,K,D,E,offsets,states,layout", CASES)
def test_linear_attn(gs, dt, T, H, K, D, E, offsets, states, layout):
    g = torch.Generator().manual_seed(T + D)
    q, qd = _heads(T, H, D, dt, g, layout=layout)
    k, kd = _heads(T, K, D, dt, g, layout=layout)
    v, vd = _heads(T, K, E, dt, g, layout=layout)
    do, dod = _heads(T, H, E, dt, g, layout=layout)
    a = -torch.exp2(-torch.linspace(0, 8, H + 1)[:H])
    if H > 2:
        a[1], a[2] = 0.0, -40.0  # no decay; one that leaves next to nothing
    off = [0, T] if offsets is None else offsets
    G, scale = len(off) - 1, D ** -0.5
    s0 = torch.randn(G, H, D, E, generator=g) if states else None
    ds = torch.randn(G, H, D, E, generator=g) if states else None
    args = dict(group_offsets=None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda(),
                state=s0.cuda() if states else None)
    dbl = lambda t: t.double() if t is not None else None  # noqa: E731
    ws = torch.full((gs.gs_linear_attn_workspace_bytes(T, H, K, D, E, G),), 0xff, dtype=torch.uint8, device="cuda")
    end = off[-1]

    (out, last), (out_m, last_m) = _want(qd, kd, vd, a, off, dbl(s0), scale)
    got, got_last = torch.full_like(do, 9.0), torch.empty(G, H, D, E, device="cuda")
    gs.gs_linear_attn_fwd(q, k, v, a.cuda(), got, state_out=got_last, workspace=ws, **args)
    _close(got[:end], out[:end], _bound(out, out_m, dt)[:end], "out")
    assert (got[end:] == 9.0).all()
    _close(got_last, last, 2.0 ** -18 * last_m + 1e-37, "last states")
    only = torch.full_like(do, 9.0)
    gs.gs_linear_attn_fwd(q, k, v, a.cuda(), only, workspace=ws, **args)  # without the last states
    _close(only[:end], out[:end], _bound(out, out_m, dt)[:end], "out alone")

    want, mag = _want(qd, kd, vd, a, off, dbl(s0), scale, dod, dbl(ds))
    dq, dk, dv = (torch.full_like(t, 9.0) for t in (q, k, v))
    d0 = torch.empty(G, H, D, E, device="cuda") if states else None
    gs.gs_linear_attn_bwd(q, k, v, a.cuda(), do, dq, dk, dv, dstate_out=ds.cuda() if states else None, dstate=d0,
                          workspace=ws, **args)
    for name, x, w, m in zip(("dq", "dk", "dv"), (dq, dk, dv), want, mag):
        _close(x[:end], w[:end], _bound(w, m, dt)[:end], name)
        assert (x[end:] == 9.0).all(), name
    if states:
        _close(d0, want[3], 2.0 ** -18 * mag[3] + 1e-37, "dstate")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,D", [(64, 64), (150, 16), (130, 128)])
def test_whole_numbers_are_exact(gs, dt, T, D):
    """Without a decay and with few, small whole numbers every intermediate value is exact:
    outputs are the rounded true ones, bit for bit."""
    g = torch.Generator().manual_seed(T)
    H, E = 2, D
    q, k, v = (torch.where(torch.rand(T, H, D, generator=g) < 0.2, torch.randint(-1, 2, (T, H, D), generator=g), 0)
               .to(dt) for _ in range(3))
    a = torch.zeros(H)
    want, last = plain.attn(q.double(), k.double(), v.double(), a, [0, T], None, 1.0)
    out, s = torch.empty(T, H, E, dtype=dt, device="cuda"), torch.empty(1, H, D, E, device="cuda")
    ws = torch.empty(gs.gs_linear_attn_workspace_bytes(T, H, H, D, E), dtype=torch.uint8, device="cuda")
    gs.gs_linear_attn_fwd(q.cuda(), k.cuda(), v.cuda(), a.cuda(), out, state_out=s, scale=1.0, workspace=ws)
    assert torch.equal(out.cpu(), want.to(dt)) and torch.equal(s.cpu(), last.float())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,H,K,D,E", [(1, 1, 1, 64, 64), (3, 4, 2, 128, 128), (5, 6, 2, 57, 41), (2, 2, 2, 1, 3),
                                       (300, 2, 1, 16, 100)])
def test_steps(gs, dt, B, H, K, D, E):
    """Single tokens, several after one another."""
    g = torch.Generator().manual_seed(B + D)
    a = -torch.exp2(-torch.linspace(0, 8, H + 1)[:H])
    s = torch.randn(B, H, D, E, generator=g)
    state, want = s.cuda(), s.double()
    d = torch.exp(a.double())[:, None, None]
    for i in range(3):
        q, qd = _heads(B, H, D, dt, g, layout="odd" if D % 2 else "packed")
        k, kd = _heads(B, K, D, dt, g)
        v, vd = _heads(B, K, E, dt, g)
        out = torch.empty(B, H, E, dtype=dt, device="cuda")
        gs.gs_linear_attn_step(q, k, v, a.cuda(), state, out)
        kd, vd = kd.repeat_interleave(H // K, 1), vd.repeat_interleave(H // K, 1)
        want = d * want + kd[..., None] * vd[:, :, None]
        o = D ** -0.5 * (qd[:, :, None] @ want)[:, :, 0]
        m = D ** -0.5 * (qd.abs()[:, :, None] @ want.abs())[:, :, 0]
        # the decay and a fused update, 2^-22 a step; a sum of D terms
        _close(state, want, (i + 1) * 2.0 ** -21 * (want.abs() + 8), "state")
        _close(out, o, o.abs() * EPS[dt] + (D + 16) * 2.0 ** -23 * (m + 8) + TINY[dt], "out")
