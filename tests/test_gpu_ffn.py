"""The gated feed-forward block on the GPU against its plain 64-bit form.

Tolerances come from the arithmetic.  A sum of n products on the tensor cores adds 16 of
them at a time to an fp32 sum that is cut, 2^-23 of it at most: n / 16 cuts, and as many
again for what is cut in aligning the 16, off the sum of magnitudes.  A rounding to the
type is half a step, EPS of the value."""
import pytest
import torch

import block_plain as plain

pytestmark = pytest.mark.gpu

EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -24, torch.float32: 1e-38}
CUT = 2.0 ** -23
# silu: an exponential, a sum and a reciprocal of 2^-22 each; gelu: an error function off
# by 2.6e-7 (absolute, of values up to 1)
ACT = 2.6e-7 + 2.0 ** -20


@pytest.fixture(scope="module")
def gs():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_splatting_differentiable_gs_gb300 as gs
    return gs


def _mat(rows, cols, dt, g, std=1.0, pad=0, offset=0):
    """Random values as a slice of a wider GPU matrix, and the same in 64 bits."""
    v = (torch.randn(rows, cols, generator=g) * std).to(dt)
    flat = torch.full((rows * (cols + pad) + offset + 1,), 7.0, dtype=dt, device="cuda")
    m = flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    m.copy_(v)
    return m, v.double()


def _empty(rows, cols, dt, pad=0, offset=0):
    flat = torch.full((rows * (cols + pad) + offset + 1,), 9.0, dtype=dt, device="cuda")
    return flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], flat


def _sum_error(n, magnitudes):
    return (n / 8 + 4) * CUT * magnitudes


def _close(got, want, bound, what):
    got = got.double().cpu()
    assert got.shape == want.shape
    over = ~((got - want).abs() <= bound)
    assert not over.any(), (what, int(over.sum()), float((got - want).abs().max()),
                            float(((got - want).abs() / bound).max()))


def _bounds(x, w, dh, act, dt):
    """64-bit results of both directions, and how far off each may be."""
    F, C = w.shape[0] // 2, x.shape[1]
    h, gate, up = plain.ffn(x, w, act)
    f, df = plain.act_both(gate, act)
    e_gate = _sum_error(C, x.abs() @ w[:F].abs().t())
    e_up = _sum_error(C, x.abs() @ w[F:].abs().t())
    # |act'| <= 1.13, |act''| <= 0.8
    e_f = 1.13 * e_gate + ACT * (1 + gate.abs())
    e_df = 0.8 * e_gate + ACT * (1 + gate.abs())
    b_h = e_f * up.abs() + f.abs() * e_up + e_f * e_up + h.abs() * 2 * EPS[torch.float32]
    out = {"h": (h, b_h + (h.abs() + b_h) * EPS[dt] + TINY[dt])}
    if dh is None:
        return out
    dg, du = dh * up * df, dh * f
    e_dg = dh.abs() * (e_df * up.abs() + df.abs() * e_up + e_df * e_up) + dg.abs() * 3 * EPS[torch.float32]
    e_du = dh.abs() * e_f + du.abs() * EPS[torch.float32]
    e_dg = e_dg + (dg.abs() + e_dg) * EPS[dt] + TINY[dt]
    e_du = e_du + (du.abs() + e_du) * EPS[dt] + TINY[dt]
    d, e = torch.cat([dg, du], 1), torch.cat([e_dg, e_du], 1)
    big = d.abs() + e
    dx, dw = d @ w, d.t() @ x
    out["dx"] = (dx, e @ w.abs() + _sum_error(2 * F + 128, big @ w.abs()))
    out["dw"] = (dw, e.t() @ x.abs() + _sum_error(x.shape[0] + 64, big.t() @ x.abs()))
    return out


def _stored(want, bound, dt):
    return want, bound + (want.abs() + bound) * EPS[dt] + TINY[dt]


SHAPES = [  # tokens, channels, hidden, padding of the rows, offset of the first
    (1, 64, 128, 0, 0),
    (1, 1, 1, 0, 0),
    (3, 8, 8, 0, 0),
    (7, 17, 9, 0, 1),          # odd in everything
    (16, 200, 136, 0, 0),
    (17, 1024, 64, 0, 0),
    (64, 72, 264, 8, 8),
    (65, 65, 129, 3, 0),
    (128, 256, 128, 0, 0),
    (200, 96, 100, 0, 0),      # padded halves
    (256, 384, 1024, 0, 0),
    (257, 130, 257, 0, 3),
    (600, 520, 300, 64, 0),
    (1000, 64, 2000, 0, 0),
    (8, 1000, 100, 0, 0),      # few tokens, on either side of the steps between their forms
    (9, 1031, 24, 0, 0),
    (31, 2056, 16, 0, 2),
    (32, 520, 40, 8, 0),
    (33, 520, 40, 8, 0),
    (300, 300, 3001, 0, 0),    # dx's sums split over several pairs
]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,C,F,pad,offset", SHAPES)
def test_ffn(gs, dt, act, T, C, F, pad, offset):
    g = torch.Generator().manual_seed(T * 7 + C + F)
    x, xd = _mat(T, C, dt, g, pad=pad, offset=offset)
    w, wd = _mat(2 * F, C, dt, g, std=C ** -0.5, pad=pad, offset=offset)
    dh, dhd = _mat(T, F, dt, g, pad=pad, offset=offset)
    ws = torch.zeros(gs.gs_ffn_workspace_bytes(T, C, F), dtype=torch.uint8, device="cuda")
    ws[256:] = 0xff  # NaN in every type: nothing in it is read before it is written
    want = _bounds(xd, wd, dhd, act, dt)
    h, h_all = _empty(T, F, dt, pad, offset)
    gs.gs_ffn_fwd(x, w, h, ws, act=act)
    _close(h, *want["h"], "h")
    h.fill_(9.0)
    assert (h_all == 9.0).all()  # nothing beside it
    for dw_dt in (dt, torch.float32):
        dx, dx_all = _empty(T, C, dt, pad, offset)
        dw, dw_all = _empty(2 * F, C, dw_dt, pad, offset)
        gs.gs_ffn_bwd(x, w, dh, dx, dw, ws, act=act)
        _close(dx, *_stored(*want["dx"], dt), "dx")
        _close(dw, *_stored(*want["dw"], dw_dt), "dw")
        dx.fill_(9.0)
        dw.fill_(9.0)
        assert (dx_all == 9.0).all() and (dw_all == 9.0).all()
    assert gs.gs_workspace_status(ws) == gs.GS_OK
