"""Linear attention where single values are broken or far apart: what they have no part in is
as it is without them, and fp16 reaches as far as its outputs do.

Tolerances as in test_gpu_linear_attn.py: EPS of the magnitudes for the two roundings to the
type on the way, half a step of the result."""
import pytest
import torch

import test_gpu_block_long as long

pytestmark = pytest.mark.gpu
EPS = long.EPS


@pytest.fixture(scope="module")
def gs():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_splatting_differentiable_gs_gb300 as gs
    return gs


def _inputs(T, H, D, E, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k, v, do = (rand(T, H, n).to(dt) for n in (D, D, E, E))
    return q, k, v, do, rand(1, H, D, E), rand(1, H, D, E), -torch.exp2(-8 * torch.rand(H, generator=g, device="cuda"))


def _run(gs, q, k, v, do, s0, ds, a, scale):
    T, H, D = q.shape
    E = v.shape[2]
    ws = torch.empty(gs.gs_linear_attn_workspace_bytes(T, H, H, D, E), dtype=torch.uint8, device="cuda")
    out, last, d0 = torch.empty_like(do), torch.empty_like(s0), torch.empty_like(s0)
    dq, dk, dv = (torch.empty_like(x) for x in (q, k, v))
    kw = dict(state=s0, scale=scale, workspace=ws)
    gs.gs_linear_attn_fwd(q, k, v, a, out, state_out=last, **kw)
    gs.gs_linear_attn_bwd(q, k, v, a, do, dq, dk, dv, dstate_out=ds, dstate=d0, **kw)
    return dict(out=out, last=last, dq=dq, dk=dk, dv=dv, d0=d0)


def _bounds(q, k, v, do, s0, ds, a, scale, dt):
    """64-bit results and how far off each may be."""
    dbl = [x.double() for x in (q, k, v, a)]
    args = lambda f: ([f(x) for x in dbl[:3]] + [dbl[3], [0, q.shape[0]], f(s0.double()), scale,  # noqa: E731
                                                f(do.double()), f(ds.double())])
    want, mag = long._results(*args(lambda x: x)), long._results(*args(torch.abs))
    names = ("out", "last", "dq", "dk", "dv", "d0")
    tol = {n: (2.0 ** -16 * m + 1e-37 if n in ("last", "d0") else
               w.abs() * EPS[dt] + (EPS[dt] * 1.01 + 2.0 ** -14) * m + long.TINY[dt] * (1 + m))
           for n, w, m in zip(names, want, mag)}
    return dict(zip(names, want)), tol


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,D,E", [(400, 64, 64), (300, 128, 128), (300, 72, 41)])
def test_a_broken_channel_leaves_the_others(gs, dt, bad, T, D, E):
    """A broken value has no part in the other channels of values, outputs and states, nor a
    broken key or query in the states' other rows."""
    H, scale, at = 2, D ** -0.5, 170
    ins = _inputs(T, H, D, E, dt, D)
    v, k = ins[2].clone(), ins[1].clone()
    want, tol = _bounds(*ins, scale, dt)
    v[at, 1, 3] = bad
    got = _run(gs, ins[0], ins[1], v, *ins[3:], scale)
    keep = torch.arange(E, device="cuda") != 3
    for n in ("out", "dv"):  # (dv has nothing of v in it)
        cols = slice(None) if n == "dv" else keep
        long._close(got[n][..., cols], want[n][..., cols], tol[n][..., cols], n)
    long._close(got["last"][..., keep], want["last"][..., keep], tol["last"][..., keep], "last")
    long._close(got["d0"], want["d0"], tol["d0"], "d0")
    assert not torch.isfinite(got["last"][0, 1, :, 3]).any() and not torch.isfinite(got["out"][at:, 1, 3]).any()
    k[at, 1, 5] = bad
    got = _run(gs, ins[0], k, *ins[2:], scale)
    rows = torch.arange(D, device="cuda") != 5
    long._close(got["last"][:, :, rows], want["last"][:, :, rows], tol["last"][:, :, rows], "last")
    assert not torch.isfinite(got["last"][0, 1, 5]).any()
    long._close(got["d0"], want["d0"], tol["d0"], "d0")
    early = slice(0, at)  # (a key has no part in the outputs before it)
    long._close(got["out"][early], want["out"][early], tol["out"][early], "out")


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,E", [(64, 64), (128, 128), (72, 41)])
@pytest.mark.parametrize("qs,ks,vs,dos", [
    (300.0, 300.0, 2.0 ** -10, 2.0 ** -10),        # products of queries and keys past 65504
    (2.0 ** -10, 2.0 ** -10, 2.0 ** 8, 2.0 ** -6),  # and below 2^-14
    (2.0 ** -6, 2.0 ** -6, 300.0, 300.0),          # of values and their outputs' gradients
    (2.0 ** 6, 2.0 ** 4, 2.0 ** -12, 2.0 ** -8),
])
def test_products_beyond_the_types_range(gs, dt, D, E, qs, ks, vs, dos):
    """Outputs and gradients are in the type's range; the products on their way are not."""
    T, H, scale = 300, 2, D ** -0.5
    q, k, v, do, s0, ds, a = _inputs(T, H, D, E, dt, E)
    q, k, v, do = ((x.float() * s).to(dt) for x, s in ((q, qs), (k, ks), (v, vs), (do, dos)))
    want, tol = _bounds(q, k, v, do, s0, ds, a, scale, dt)
    got = _run(gs, q, k, v, do, s0, ds, a, scale)
    assert all(float(want[n].abs().max()) < 60000 for n in ("out", "dq", "dk", "dv"))
    for n in want:
        long._close(got[n], want[n], tol[n], n)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,E", [(64, 64), (128, 128)])
def test_decays_that_leave_nothing(gs, dt, D, E):
    """log_decay of minus infinity: a token's output is its own product, and the state its own
    key and value; beside it a head without a decay."""
    T, H, scale = 300, 2, D ** -0.5
    q, k, v, do, s0, ds, _ = _inputs(T, H, D, E, dt, D)
    a = torch.tensor([float("-inf"), 0.0], device="cuda")
    want, tol = _bounds(q, k, v, do, s0, ds, a.clamp(min=-1e9), scale, dt)
    got = _run(gs, q, k, v, do, s0, ds, a, scale)
    for n in want:
        long._close(got[n], want[n], tol[n], n)
    own = scale * (q.double() * k.double()).sum(-1, keepdim=True) * v.double()
    assert (got["out"][:, 0].double() - own[:, 0]).norm() <= 2 * EPS[dt] * own[:, 0].norm()
    s, out = s0.clone(), torch.empty_like(do[:1])
    gs.gs_linear_attn_step(q[:1], k[:1], v[:1], a, s, out, scale=scale)
    assert torch.equal(s[0, 0], k[0, 0, :, None].float() * v[0, 0].float())
    assert (out[0, 0].double() - own[0, 0]).norm() <= 2 * EPS[dt] * own[0, 0].norm()
