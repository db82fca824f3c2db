"""Forms of the network operators' calls at the ends of what they accept, against
the plain 64-bit forms.  Tolerances: u = 2^-24 for each rounding in fp32."""
import pytest
import torch

import net_plain as plain

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def gs():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_splatting_differentiable_gs_gb300 as gs
    return gs


def _gen(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("center", [False, True])
def test_norm_weight_after_the_block_counts_only_with_the_norm(gs, center):
    """Without the norm after the block its weight takes no part: outputs and gradients
    are those of the same call without it, and its own gradient is zero."""
    T, C, G = 12, 72, 2
    g = _gen(1)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, block, dxo, dy, gate = r(T, C), r(T, C), r(T, C), r(T, C), r(G, C)
    scale, w_post = r(C), 1 + r(C)
    off = torch.tensor([0, 5, T], dtype=torch.int32)
    kw = dict(gate=gate.cuda(), group_offsets=off.cuda(), res_scale=scale.cuda(), post=False, center=center)
    ws = torch.empty(gs.gs_gated_norm_workspace_bytes(C, G), dtype=torch.uint8, device="cuda")
    results = []
    for w in (w_post.cuda(), None):
        xo, y, st = (torch.empty(T, n, device="cuda") for n in (C, C, 4))
        gs.gs_gated_norm_fwd(x.cuda(), block.cuda(), xo, y, st, w_post=w, **kw)
        o = {k: torch.full(s, 7.0, device="cuda") for k, s in
             (("dw_pre", (C,)), ("dw_post", (C,)), ("dres_scale", (C,)), ("dgate", (G, C)))}
        dx, db = torch.empty(T, C, device="cuda"), torch.empty(T, C, device="cuda")
        gs.gs_gated_norm_bwd(xo, block.cuda(), st, dxo.cuda(), dy.cuda(), dx, db, w_post=w, workspace=ws, **o,
                             **kw)
        results.append(dict(xo=xo, y=y, st=st, dx=dx, db=db, **o))
    for name in results[0]:
        assert torch.equal(results[0][name], results[1][name]), name
    assert not results[0]["dw_post"].any()
    # and against the formula: u = block, so that d(u gate scale) needs no weight
    d = results[0]["dx"].double().cpu()
    of = plain.group_of(T, off, G)
    terms = d * block.double()
    for name, want, mag in (
            ("dres_scale", (terms * gate.double()[of]).sum(0), (terms * gate.double()[of]).abs().sum(0)),
            ("dgate", torch.stack([(terms * scale.double())[of == i].sum(0) for i in range(G)]),
             torch.stack([(terms * scale.double()).abs()[of == i].sum(0) for i in range(G)]))):
        err = (results[0][name].double().cpu() - want).abs()
        assert (err <= 2 * (T + 4) * U * mag).all(), name  # T terms, then the factors
