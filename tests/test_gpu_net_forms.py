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


TOP = {torch.float16: 65504.0, torch.bfloat16: float(torch.finfo(torch.bfloat16).max),
       torch.float32: float(torch.finfo(torch.float32).max)}


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C", [32, 40, 33])
def test_checkpoint_of_the_largest_numbers_reads_back_finite(gs, dt, C):
    """The step nearest to a type's largest numbers can lie above them: such a value
    reads as the type's largest number, everything else as it is held."""
    top = TOP[dt]
    x = torch.full((4, C), 0.0)
    x[0, 0], x[0, 5] = top, -top
    x[1] = top * 0.994          # above 127 / 128 of the power of two
    x[2, ::2], x[2, 1::2] = -top, top * 0.7
    x[3] = top * 0.25
    x = x.to(dt)
    q, e = gs.act8_empty(4, C)
    gs.gs_act8_encode(x.cuda(), q, e)
    wq, we = plain.encode(x)
    assert torch.equal(q.cpu(), wq) and torch.equal(e.cpu(), we)
    held = plain.decode(wq, we, C)
    back = torch.empty(4, C, dtype=dt, device="cuda")
    gs.gs_act8_decode(q, e, back)
    want = held.clamp(-top, top)
    assert torch.equal(back.double().cpu(), want)
    # read in the other types: finite where the type holds the value before rounding
    for other in (torch.bfloat16, torch.float32):
        out = torch.empty(4, C, dtype=other, device="cuda")
        gs.gs_act8_decode(q, e, out)
        assert torch.equal(out.double().cpu(), held.clamp(-TOP[other], TOP[other]))


def test_checkpoint_above_a_type_reads_as_infinity(gs):
    """Values that a type does not hold, whatever their rounding, convert as ever."""
    x = torch.tensor([[1e5, -7e4, 66100.0, 65000.0] + [1.0] * 28, [3e38, 1e30, -1e20, 1.0] + [0.0] * 28])
    q, e = gs.act8_empty(2, 32)
    gs.gs_act8_encode(x.cuda(), q, e)
    out = torch.empty(2, 32, dtype=torch.float16, device="cuda")
    gs.gs_act8_decode(q, e, out)
    step = torch.exp2(e.cpu().double() - 127)
    held = plain.decode(q.cpu(), e.cpu(), 32)
    want = held.float().half()
    within = (held.abs() - 0.5 * step <= 65504) & torch.isinf(want)
    want = torch.where(within, torch.sign(held) * 65504, want.double())
    assert torch.equal(out.double().cpu(), want)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C", [64, 37])
def test_gated_unit_at_the_largest_numbers(gs, act, dt, C):
    """At a type's largest numbers act is v or 0 and its derivative 1 or 0: no NaN."""
    top = TOP[dt]
    gate = torch.where(torch.arange(C) % 2 == 0, torch.tensor(top), torch.tensor(-top)).to(dt)[None].repeat(3, 1)
    up, dh = torch.full((3, C), 0.5).to(dt), torch.full((3, C), 0.25).to(dt)
    h = torch.empty(3, C, dtype=dt, device="cuda")
    g8, u8 = gs.act8_empty(3, C), gs.act8_empty(3, C)
    gs.gs_glu_fwd(gate.cuda(), up.cuda(), h, *g8, *u8, act=act)
    on = (gate > 0).double()
    assert torch.equal(h.double().cpu().abs(), on * float(torch.tensor(top).to(dt).double() * 0.5))
    dg, du = torch.empty_like(h), torch.empty_like(h)
    gs.gs_glu_bwd(*g8, *u8, dh.cuda(), dg, du, act=act)
    assert torch.equal(dg.double().cpu().abs(), on * 0.125)
    held = torch.finfo(torch.float32).max  # the checkpoint's values are taken in fp32
    want = (torch.tensor(held) * 0.25).to(dt).double()
    assert torch.equal(du.double().cpu().abs(), on * want)


def test_fp32_gelu_keeps_its_relative_accuracy(gs):
    """gelu(v) = v Phi(v) in fp32, in the tail too.  Phi is half the complementary error
    function of -v / sqrt 2: 4 units in the last place (8 u) of the function, 2 u for the
    halving's and product's roundings; the argument's rounding (constant and product, 2 u
    relative) moves Phi by at most (v^2 + 1) times that where v < 0."""
    v = torch.cat([-torch.logspace(-4, 0.9, 3000, dtype=torch.float64), torch.zeros(1, dtype=torch.float64),
                   torch.logspace(-4, 1.5, 3000, dtype=torch.float64)]).float()
    v = torch.cat([v, v[:7]])[:6008 // 8 * 8].view(8, -1)
    tail = (v.double() ** 2 + 1) * (v < 0)
    for width in (v.shape[1], v.shape[1] - 1):  # rows on 16-byte boundaries, and not
        x = v[:, :width].cuda().contiguous()
        h = torch.empty_like(x)
        gs.gs_glu_fwd(x, None, h, act="gelu")
        want = x.double() * 0.5 * torch.special.erfc(-x.double() / 2 ** 0.5)
        err = (h.double() - want).abs().cpu()
        bound = want.abs().cpu() * (12 + 2 * tail[:, :width]) * U + 1e-38
        assert (err <= bound).all(), float((err / want.abs().cpu().clamp_min(1e-300) / U).max())


def test_fp32_gelu_derivative(gs):
    """dgate = dh (Phi + v phi) at the held values: the roundings above on Phi, and on
    v phi those of its exponential (argument v^2 / 2 at 3 u, 4 u of its own) and of two products."""
    q0 = torch.arange(-127, 128)
    T, C = 8, 256
    q = torch.zeros(T, C, dtype=torch.int8)
    q[:, :255] = q0.to(torch.int8)
    e = torch.empty(T, C // 32, dtype=torch.uint8)
    for t in range(T):
        e[t] = 127 - 4 - t  # steps 1/16 and finer
    v = plain.decode(q, e, C)
    dg = torch.empty(T, C, device="cuda")
    gs.gs_glu_bwd(q.cuda(), e.cuda(), None, None, torch.ones(T, C, device="cuda"), dg, None, act="gelu")
    phi = torch.exp(-0.5 * v * v) * (0.5 / torch.pi) ** 0.5
    big = 0.5 * torch.special.erfc(-v / 2 ** 0.5)
    bound = (big * (12 + 2 * (v * v + 1) * (v < 0)) + (v * phi).abs() * (8 + 2 * v * v)) * U + 2 * U * (big + v * phi).abs()
    err = (dg.double().cpu() - (big + v * phi)).abs()
    assert (err <= bound + 1e-38).all(), float((err / bound).max())


@pytest.mark.parametrize("C", [96, 70])
def test_gated_unit_of_groups_that_are_not_numbers(gs, C):
    """Such a group gives NaN in both gradients, its neighbours do not."""
    gate, up, dh = (torch.randn(4, C, generator=_gen(i)) for i in range(3))
    gate[1, 40], up[2, 3] = float("nan"), float("inf")
    g8, u8 = gs.act8_empty(4, C), gs.act8_empty(4, C)
    gs.gs_act8_encode(gate.cuda(), *g8)
    gs.gs_act8_encode(up.cuda(), *u8)
    dg, du = torch.empty(4, C, device="cuda"), torch.empty(4, C, device="cuda")
    for act in ("silu", "gelu"):
        gs.gs_glu_bwd(*g8, *u8, dh.cuda(), dg, du, act=act)
        want = torch.zeros(4, C, dtype=torch.bool)
        want[1, 32:64] = True
        assert torch.equal(torch.isnan(du.cpu()), want)
        want[2, :32] = True
        assert torch.equal(torch.isnan(dg.cpu()), want)


def test_rope_in_place_where_a_stride_is_never_taken(gs):
    """One token, or one head: the stride between them does not matter."""
    import ctypes as C
    rope = gs.Rope([8])
    pos = torch.tensor([[3]] * 4, dtype=torch.int32).cuda()
    x = torch.randn(4, 4, 8, generator=_gen(8)).cuda()
    want = torch.empty_like(x)
    gs.gs_rope(rope, pos, x, q_out=want)
    for tokens, heads, strides in ((1, 4, (32, 8, 999, 8)), (4, 1, (32, 8, 32, 999)), (4, 4, (32, 8, 32, 8))):
        y = x.clone()
        sets = gs.net._HEADS.pack(y.data_ptr(), y.data_ptr(), *strides, heads)
        assert gs.lib().gs_rope(tokens, 1, rope._dims, rope.turns, 0, 0, pos.data_ptr(), 8, 2, sets, 1,
                                torch.cuda.current_stream().cuda_stream) == gs.GS_OK
        assert torch.equal(y[:tokens, :heads], want[:tokens, :heads])
        y[:tokens, :heads] = x[:tokens, :heads]
        assert torch.equal(y, x)


@pytest.mark.parametrize("scale", [1.0, -3.0])
def test_rope_far_positions_lose_nothing(gs, scale):
    """The angle of a position up to 2^31 in either direction is good to fp32's rounding:
    the bound is that of small positions, with angles from 60 digits."""
    import math
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    at = [2 ** 31 - 1, -2 ** 31, 123456789, -987654321, 2 ** 30 + 1, 7]
    x = torch.randn(len(at), 2, 64, generator=_gen(1))
    got = torch.empty(len(at), 2, 64, device="cuda")
    gs.gs_rope(gs.Rope([64], scale=scale), torch.tensor(at, dtype=torch.int32)[:, None].cuda(), x.cuda(), q_out=got)
    ang = torch.empty(len(at), 32, dtype=torch.float64)
    for j in range(32):
        f = Decimal(scale) * (Decimal(10000).ln() * Decimal(-2 * j) / 64).exp() / two_pi
        for i, p in enumerate(at):
            t = p * f
            ang[i, j] = float(t - t.to_integral_value()) * 2 * math.pi
    u, v = x[..., :32].double(), x[..., 32:].double()
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    want = torch.cat([u * c - v * s, u * s + v * c], -1)
    pair = torch.cat([u.abs() + v.abs()] * 2, -1)
    err = (got.double().cpu() - want).abs()
    assert (err <= 10 * U * pair + U * want.abs()).all(), float((err / pair).max() / U)


def test_weight_gradient_of_the_smallest_numbers(gs):
    """A wide gradient's terms reach down to bf16's smallest step, 2^-133: one token, so
    that dw = dy x to fp32's rounding (three terms, their sum) but for what lies below it."""
    N, K = 120, 64
    big = 2.0 ** 100
    dy = torch.randn(1, N, generator=_gen(3)) * torch.logspace(-30, -39, N)
    x = torch.full((1, K), big)
    q, e = gs.act8_empty(1, K)
    gs.gs_act8_encode(x.cuda(), q, e)
    ws = torch.zeros(gs.gs_act8_wgrad_workspace_bytes(1, N, K, torch.float32), dtype=torch.uint8, device="cuda")
    dw = torch.empty(N, K, device="cuda")
    gs.gs_act8_wgrad(dy.cuda(), q, e, dw, ws)
    want = dy.double().t() * big
    err = (dw.double().cpu() - want).abs()
    assert (err <= 4 * U * want.abs() + 2.0 ** -133 * big).all(), float((err / big).max() * 2 ** 133)
