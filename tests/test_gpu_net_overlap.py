"""A call reads what the call before it on the stream wrote, whatever it is: the
kernels of the network operators begin while the one before them ends."""
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


@pytest.mark.parametrize("graph", [False, True])
def test_norm_backward_after_the_calls_that_write_its_weights(gs, graph):
    """The gate comes from a gated unit and the weights from checkpoints, in the calls
    right before; each round has other values in the same buffers.  Few rows, so that
    the row kernel leaves room for the sums' kernel beside the one before it."""
    T, C, G = 4, 1024, 3
    g = torch.Generator().manual_seed(11)
    rounds = 12
    x, block, dx_out, dy = (torch.randn(T, C, generator=g).cuda() for _ in range(4))
    offsets = torch.tensor([0, 1, 1, 4], dtype=torch.int32).cuda()
    raw = torch.randn(rounds, G, C, generator=g).cuda()
    held = [[gs.act8_empty(1, C) for _ in range(2)] for _ in range(rounds)]
    values = []
    for ck in held:
        for q, e in ck:
            gs.gs_act8_encode((1 + torch.rand(1, C, generator=g)).cuda(), q, e)
        row = [torch.empty(1, C, device="cuda") for _ in ck]
        for (q, e), v in zip(ck, row):
            gs.gs_act8_decode(q, e, v)
        values.append([v[0].double().cpu() for v in row])
    gate, w_post, scale = (torch.zeros(G, C, device="cuda"), torch.zeros(1, C, device="cuda"),
                           torch.zeros(1, C, device="cuda"))
    one, shift = torch.ones(G, C, device="cuda"), torch.empty(G, C, device="cuda")
    stats = torch.empty(T, 4, device="cuda")
    xo, y = torch.empty(T, C, device="cuda"), torch.empty(T, C, device="cuda")
    gs.gs_gated_norm_fwd(x, block, xo, y, stats, post=True)
    ws = torch.empty(gs.gs_gated_norm_workspace_bytes(C, G), dtype=torch.uint8, device="cuda")
    dx, db = torch.empty(T, C, device="cuda"), torch.empty(T, C, device="cuda")
    out = [dict(dw_post=torch.empty(C, device="cuda"), dres_scale=torch.empty(C, device="cuda"),
                dgate=torch.empty(G, C, device="cuda")) for _ in range(rounds)]

    def run():
        for i in range(rounds):
            gs.gs_act8_decode(*held[i][0], w_post)
            gs.gs_act8_decode(*held[i][1], scale)
            gs.gs_glu_fwd(raw[i], one, gate)
            gs.gs_gated_norm_bwd(x, block, stats, dx_out, dy, dx, db, w_post=w_post[0], gate=gate,
                                 group_offsets=offsets, res_scale=scale[0], workspace=ws, **out[i])

    if graph:
        run()
        for o in out:
            for v in o.values():
                v.fill_(9.0)
        rec = torch.cuda.CUDAGraph()
        with torch.cuda.graph(rec):
            run()
        rec.replay()
    else:
        run()
    torch.cuda.synchronize()
    # d, the gradient of the sum, does not depend on the gate; e_G = sum of d n(block)
    st = stats.double().cpu()
    n = (block.double().cpu() - st[:, :1]) * st[:, 1:2]
    d = dx.double().cpu()
    of = (plain.group_of(T, offsets.cpu(), G)[None] == torch.arange(G)[:, None]).double()
    e, mag = of @ (d * n), of @ (d * n).abs()
    for i, o in enumerate(out):
        w, s = values[i]
        gt = plain.act(raw[i].double().cpu(), "silu")
        bound = 80 * U  # the sums' chain, d and n in fp32 and the factors' roundings
        for got, want, m in ((o["dgate"], s * w * e, s * w * mag),
                             (o["dres_scale"], (gt * w * e).sum(0), (gt.abs() * w * mag).sum(0)),
                             (o["dw_post"], (gt * s * e).sum(0), (gt.abs() * s * mag).sum(0))):
            assert ((got.double().cpu() - want).abs() <= bound * m + 1e-30).all(), i


def test_weight_gradient_after_the_calls_that_write_its_checkpoint(gs):
    """Encoded into the same arrays each round, by the call right before."""
    T, N, K, rounds = 300, 70, 96, 10
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(rounds, T, K, generator=g, device="cuda") * torch.exp2(
        torch.randint(-8, 8, (rounds, T, 1), generator=g, device="cuda").float())
    dy = torch.randn(T, N, generator=g, device="cuda").bfloat16()
    ws = torch.zeros(gs.gs_act8_wgrad_workspace_bytes(T, N, K), dtype=torch.uint8, device="cuda")
    want, got = (torch.empty(rounds, N, K, device="cuda") for _ in range(2))
    for i in range(rounds):  # each with a checkpoint of its own, and a pause
        q, e = gs.act8_empty(T, K)
        gs.gs_act8_encode(x[i], q, e)
        torch.cuda.synchronize()
        gs.gs_act8_wgrad(dy, q, e, want[i], ws)
        torch.cuda.synchronize()
    q, e = gs.act8_empty(T, K)
    for i in range(rounds):
        gs.gs_act8_encode(x[i], q, e)
        gs.gs_act8_wgrad(dy, q, e, got[i], ws)
    assert torch.equal(got, want)
