"""Calls without tokens, or with a set of no heads, in the layouts that a program has
them: slices of packed projections, outputs of their own."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gs():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_splatting_differentiable_gs_gb300 as gs
    return gs


@pytest.mark.parametrize("T,hq,hk", [(0, 4, 2), (3, 4, 0), (3, 0, 2), (0, 0, 0)])
def test_rope_of_nothing(gs, T, hq, hk):
    packed = torch.randn(T, hq + 2 * hk, 16, device="cuda")
    q, k = packed[:, :hq], packed[:, hq:hq + hk]
    pos = torch.ones(T, 1, dtype=torch.int32, device="cuda")
    rope = gs.Rope([16])
    qo, ko = torch.empty(T, hq, 16, device="cuda"), torch.empty(T, hk, 16, device="cuda")
    gs.gs_rope(rope, pos, q, k, q_out=qo, k_out=ko)
    before = packed.clone()
    gs.gs_rope(rope, pos, q, k)
    assert torch.equal(packed[:, :hq], qo) and torch.equal(packed[:, hq:hq + hk], ko)
    assert torch.equal(packed[:, hq + hk:], before[:, hq + hk:])


def test_matrices_of_nothing(gs):
    packed = torch.empty(0, 96, device="cuda").bfloat16()
    a, b = packed[:, :40], packed[:, 40:80]
    own = lambda: torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    ck = [gs.act8_empty(0, 40) for _ in range(3)]
    gs.gs_act8_encode(a, *ck[0])
    gs.gs_act8_decode(*ck[0], own())
    gs.gs_glu_fwd(a, b, own(), *ck[0], *ck[1])
    gs.gs_glu_bwd(*ck[0], *ck[1], own(), a, b, *ck[2])
    st = torch.empty(0, 4, device="cuda")
    gs.gs_gated_norm_fwd(a, b, own(), own(), st, y_q=ck[0][0], y_e=ck[0][1])
    ws = torch.zeros(gs.gs_act8_wgrad_workspace_bytes(0, 40, 40), dtype=torch.uint8, device="cuda")
    dw = torch.full((40, 50), 3.0, device="cuda")
    gs.gs_act8_wgrad(a, *ck[0], dw[:, :40], ws)
    assert not dw[:, :40].any() and (dw[:, 40:] == 3).all()
    ws = torch.empty(gs.gs_gated_norm_workspace_bytes(40), dtype=torch.uint8, device="cuda")
    dw_pre = torch.full((40,), 3.0, device="cuda")
    gs.gs_gated_norm_bwd(a, b, st, None, own(), own(), own(), dw_pre=dw_pre, workspace=ws)
    assert not dw_pre.any()
    torch.cuda.synchronize()
