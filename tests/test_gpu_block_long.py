"""Linear attention with several chunks a segment, and the feed-forward block's sums that are
shared out, against 64-bit forms: what large calls use.

Tolerances come from the arithmetic.  Linear attention: as in test_gpu_linear_attn.py (EPS of
the magnitudes for the two roundings to the type and half a step of the result); states are
sums in fp32 of chunks of 128 tokens, whose keys are 3 terms at most (24 cuts of 2^-23 on the
tensor cores) with weights of up to nine powers (2^-22 each), decayed once a chunk.
Feed-forward block: test_gpu_ffn.py's bounds."""
import ctypes as C

import pytest
import torch

import test_gpu_ffn as few

pytestmark = pytest.mark.gpu

EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -24}
CHUNK = 128
PARTIALS = 4 * 128 * 256 * 4 * 96  # bytes of the partial sums of dw, the workspace's last part


@pytest.fixture(scope="module")
def gs():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_splatting_differentiable_gs_gb300 as gs
    return gs


def _selftest(gs):
    L, vp = gs.lib(), C.c_void_p
    L.gs_selftest_linear_attn.argtypes = [vp, vp, C.c_int32, vp, vp, vp, C.c_size_t, C.c_int32, C.c_int32, vp]
    L.gs_selftest_linear_attn_chunks.argtypes = [vp, C.c_int32, C.c_int32]
    return L


def _packed(gs, q, k, v, a, offs, state, scale, *others):
    """The C call's structure, and the heads of q, k, v and the others."""
    (T, H, D), K, E = q.shape, k.shape[1], v.shape[2]
    x = gs.net._ATTN.pack(T, H, K, D, E, 1 if offs is None else offs.numel() - 1, gs.net.DTYPES[q.dtype], scale,
                          a.data_ptr(), 0 if offs is None else offs.data_ptr(), 0 if state is None else state.data_ptr())
    heads = [n for t in (q, k, v) + others for n in (t.data_ptr(), t.stride(0), t.stride(1))]
    return x, (gs.net._ATTN_HEADS4 if len(others) == 1 else gs.net._ATTN_HEADS7).pack(*heads)


def _close(got, want, bound, what):
    got = got.double()
    assert got.shape == want.shape
    over = ~((got - want).abs() <= bound)
    assert not over.any(), (what, int(over.sum()), float((got - want).abs().max()),
                            float(((got - want).abs() / bound).max()))


def _attn(q, k, v, a, offsets, state, scale):
    """(out, last states) of [T, h, D] heads, every pair of tokens at once; differentiable."""
    T, h, _ = q.shape
    rep = h // k.shape[1]
    q, k, v = (x.transpose(0, 1) for x in (q, k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)))
    off = torch.tensor(offsets, device=q.device)
    at = torch.arange(T, device=q.device)
    of = torch.searchsorted(off[1:].contiguous(), at, right=True)  # a token's group; past the last: none
    inside = of < len(offsets) - 1
    gap = at[:, None] - at
    a = a.double()[:, None, None]
    decay = torch.where((gap >= 0) & (of[:, None] == of) & inside, torch.exp(a * gap.clamp(min=0)), 0.0)
    of = of.clamp(max=len(offsets) - 2)
    out = ((q @ k.transpose(1, 2)) * decay) @ v
    left = torch.where(inside, torch.exp(a[:, 0] * (off[1:][of] - 1 - at).clamp(min=0)), 0.0)
    part = k * left[..., None]
    last = torch.stack([part[:, b:e].transpose(1, 2) @ v[:, b:e] for b, e in zip(offsets, offsets[1:])])
    if state is not None:
        since = torch.where(inside, torch.exp(a[:, 0] * (at - off[:-1][of] + 1)), 0.0)
        out = out + since[..., None] * (q[:, :, None] @ state.transpose(0, 1)[:, of])[:, :, 0]
        last = last + torch.exp(a[None] * (off[1:] - off[:-1])[:, None, None, None]) * state
    return scale * out.transpose(0, 1), last


def _results(q, k, v, a, offsets, state, scale, do, dlast):
    """out, last states, dq, dk, dv, dstate."""
    leaves = [x.detach().clone().requires_grad_(True) for x in (q, k, v, state)]
    out, last = _attn(*leaves[:3], a, offsets, leaves[3], scale)
    return [out.detach(), last.detach()] + list(
        torch.autograd.grad((out * do).sum() + (last * dlast).sum(), leaves))


def _check_attn(call, dt, T, H, K, D, E, offsets, seed, pick):
    """`call` runs both directions; the key heads `pick` and their query heads are looked at."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, do = rand(T, H, D).to(dt), rand(T, H, E).to(dt)
    k, v = rand(T, K, D).to(dt), rand(T, K, E).to(dt)
    off = [0, T] if offsets is None else offsets
    G, scale, rep, end = len(off) - 1, D ** -0.5, H // K, off[-1]
    a = -torch.exp2(-12.0 * torch.rand(H, generator=g, device="cuda"))
    a[::5] = 0.0
    s0, ds = rand(G, H, D, E), rand(G, H, D, E)
    out, dq, dk, dv = (torch.full_like(x, 9.0) for x in (do, q, k, v))
    last, d0 = (torch.full_like(s0, 9.0) for _ in range(2))
    offs = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    call(q, k, v, a, offs, s0, scale, out, last, do, dq, dk, dv, ds, d0)
    for x in (out, dq, dk, dv):
        assert (x[end:] == 9.0).all()
    eps, chunks = EPS[dt], -(-T // CHUNK)
    for key in pick:
        hs, ks = slice(key * rep, (key + 1) * rep), slice(key, key + 1)
        ins = [x.double() for x in (q[:, hs], k[:, ks], v[:, ks], a[hs])], [x.double() for x in (
            s0[:, hs], do[:, hs], ds[:, hs])]
        want = _results(*ins[0], off, ins[1][0], scale, *ins[1][1:])
        mag = _results(*[x.abs() for x in ins[0][:3]], ins[0][3], off, ins[1][0].abs(), scale,
                       *[x.abs() for x in ins[1][1:]])
        got = [out[:, hs], last[:, hs], dq[:, hs], dk[:, ks], dv[:, ks], d0[:, hs]]
        for i, name in enumerate(("out", "last states", "dq", "dk", "dv", "dstate")):
            if i in (1, 5):
                _close(got[i], want[i], (2.0 ** -17 + chunks * 2.0 ** -20) * mag[i] + 1e-37, (name, key))
            else:
                _close(got[i][:end], want[i][:end], (want[i].abs() * eps + (eps * 1.01 + 2.0 ** -14) * mag[i]
                                                     + TINY[dt] * (1 + mag[i]))[:end], (name, key))


# (dim, vdim), tokens, query heads, key heads, groups: heads so many that segments of several
# chunks are chosen
LONG = [
    (64, 64, 700, 256, 256, None),
    (64, 64, 1000, 160, 40, None),
    (72, 41, 700, 160, 40, None),
    (72, 41, 650, 96, 96, [0, 130, 130, 641]),
    (64, 128, 700, 96, 96, None),
    (128, 64, 1000, 64, 16, None),
    (128, 128, 700, 128, 32, None),
    (128, 128, 1000, 64, 64, [0, 999]),
]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,E,T,H,K,offsets", LONG)
def test_attention_of_many_heads(gs, dt, D, E, T, H, K, offsets):
    G = 1 if offsets is None else len(offsets) - 1
    ws = torch.full((gs.gs_linear_attn_workspace_bytes(T, H, K, D, E, G),), 0xff, dtype=torch.uint8, device="cuda")
    shape = gs.net._ATTN.pack(T, H, K, D, E, G, gs.net.DTYPES[dt], 1.0, 0, 0, 0)
    assert all(_selftest(gs).gs_selftest_linear_attn_chunks(shape, back, 1) >= 2 for back in (0, 1))

    def call(q, k, v, a, offs, s0, scale, out, last, do, dq, dk, dv, ds, d0):
        kw = dict(group_offsets=offs, state=s0, scale=scale, workspace=ws)
        gs.gs_linear_attn_fwd(q, k, v, a, out, state_out=last, **kw)
        gs.gs_linear_attn_bwd(q, k, v, a, do, dq, dk, dv, dstate_out=ds, dstate=d0, **kw)

    _check_attn(call, dt, T, H, K, D, E, offsets, T + D, (0, 1, K // 2, K - 1))
    gs.gs_linear_attn_status()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("chunks", [2, 3, 5])
@pytest.mark.parametrize("D,E,H,K,offsets", [
    (64, 64, 3, 3, None),
    (64, 64, 4, 1, [0, 640, 641, 641, 1297]),
    (72, 41, 2, 2, [0, 511, 1270]),
    (72, 41, 4, 2, None),
    (40, 128, 2, 1, [0, 129, 1300]),
    (64, 128, 2, 2, None),
    (128, 32, 3, 1, None),
    (128, 128, 2, 2, [0, 300, 1200]),
    (128, 128, 2, 1, None),
])
def test_segments_of_several_chunks(gs, dt, chunks, D, E, H, K, offsets):
    """Segments as long as is asked for, the last one of a group ragged."""
    T, L = 1300, _selftest(gs)
    ws = torch.full((1 << 27,), 0xff, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream

    def call(q, k, v, a, offs, s0, scale, out, last, do, dq, dk, dv, ds, d0):
        x, heads = _packed(gs, q, k, v, a, offs, s0, scale, out)
        assert L.gs_selftest_linear_attn(x, heads, 0, None, last.data_ptr(), ws.data_ptr(), ws.numel(), chunks, -1,
                                         stream) == gs.GS_OK
        x, heads = _packed(gs, q, k, v, a, offs, s0, scale, do, dq, dk, dv)
        assert L.gs_selftest_linear_attn(x, heads, 1, ds.data_ptr(), d0.data_ptr(), ws.data_ptr(), ws.numel(), chunks, -1,
                                         stream) == gs.GS_OK

    _check_attn(call, dt, T, H, K, D, E, offsets, chunks + D, range(K))


@pytest.mark.parametrize("D,E,H,K", [(64, 64, 4, 4), (64, 64, 4, 2), (128, 128, 2, 2), (72, 41, 2, 1)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_the_attention_gives_up_and_the_context_survives(gs, dt, D, E, H, K):
    """Products that never come: the waits run out (20 ms), the blocks wait for what is under
    way, flag the error and end; the next call is right."""
    T, L = 700, _selftest(gs)
    g = torch.Generator(device="cuda").manual_seed(D)
    q, k, v, do = (torch.randn(T, h, d, generator=g, device="cuda").to(dt) for h, d in ((H, D), (K, D), (K, E), (H, E)))
    a = torch.full((H,), -0.01, device="cuda")
    ws = torch.full((1 << 27,), 0xff, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    out, grads = torch.empty_like(do), [torch.empty_like(x) for x in (q, k, v)]
    s, ds = (torch.empty(1, H, D, E, device="cuda") for _ in range(2))
    fwd, bwd = _packed(gs, q, k, v, a, None, None, 0.1, out), _packed(gs, q, k, v, a, None, None, 0.1, do, *grads)

    def run(products):
        res = [L.gs_selftest_linear_attn(*fwd, 0, None, s.data_ptr(), ws.data_ptr(), ws.numel(), 3, products, stream)]
        res.append(L.gs_selftest_linear_attn(*bwd, 1, None, ds.data_ptr(), ws.data_ptr(), ws.numel(), 3, products, stream))
        return res

    assert run(-1) == [gs.GS_OK] * 2
    want = [x.clone() for x in (out, s, *grads, ds)]
    for products in (0, 1, 2, 3, 5):  # (a chunk of the sums takes one, of the outputs two, of the gradients two or four)
        assert run(products) == [gs.GS_ERR_TIMEOUT] * 2, products
        gs.gs_linear_attn_status()  # read and cleared
        for x in (out, s, *grads, ds):
            x.fill_(7.0)
        assert run(-1) == [gs.GS_OK] * 2
        assert all(torch.equal(x, y) for x, y in zip(want, (out, s, *grads, ds))), products
    assert run(1 << 20) == [gs.GS_OK] * 2


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,C,F,pad,offset,shared", [
    (1400, 64, 64, 0, 0, True),        # one tile of dw, shared by several pairs
    (2000, 130, 97, 3, 1, True),       # odd channels and hidden, rows that start anywhere
    (3000, 520, 300, 0, 0, True),
    (1300, 1500, 1801, 0, 0, False),   # more tiles of dw than pairs, too short to be shared
    (1700, 1500, 1801, 0, 0, True),    # and with a rest that is
    (2600, 776, 2500, 8, 0, True),
])
def test_shared_sums_of_the_weight_gradient(gs, dt, T, C, F, pad, offset, shared):
    g = torch.Generator().manual_seed(T + C)
    x, xd = few._mat(T, C, dt, g, pad=pad, offset=offset)
    w, wd = few._mat(2 * F, C, dt, g, std=C ** -0.5, pad=pad, offset=offset)
    dh, dhd = few._mat(T, F, dt, g, pad=pad, offset=offset)
    ws = torch.zeros(gs.gs_ffn_workspace_bytes(T, C, F), dtype=torch.uint8, device="cuda")
    ws[256:] = 0xff
    want = few._bounds(xd, wd, dhd, "silu", dt)
    h, _ = few._empty(T, F, dt, pad, offset)
    gs.gs_ffn_fwd(x, w, h, ws)
    few._close(h, *want["h"], "h")
    for dw_dt in (dt, torch.float32):
        dx, dx_all = few._empty(T, C, dt, pad, offset)
        dw, dw_all = few._empty(2 * F, C, dw_dt, pad, offset)
        gs.gs_ffn_bwd(x, w, dh, dx, dw, ws)
        few._close(dx, *few._stored(*want["dx"], dt), "dx")
        few._close(dw, *few._stored(*want["dw"], dw_dt), "dw")
        if dw_dt is torch.float32:
            start = torch.randn(2 * F, C, generator=g)
            added, added_all = few._empty(2 * F, C, dw_dt, pad, offset)
            added.copy_(start)
            gs.gs_ffn_bwd(x, w, dh, None, added, ws, accumulate=True)
            assert torch.equal(added, start.cuda() + dw)
            added.fill_(9.0)
            assert (added_all == 9.0).all()
        dx.fill_(9.0)
        dw.fill_(9.0)
        assert (dx_all == 9.0).all() and (dw_all == 9.0).all()
    assert bool((ws[-PARTIALS:] != 0xff).any()) == shared
    assert gs.gs_workspace_status(ws) == gs.GS_OK


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,C,F", [(32640, 1024, 2432), (200000, 64, 64)])
def test_long_sums_of_the_weight_gradient(gs, dt, T, C, F):
    """dw in fp32 after many tokens, of which the tensor cores sum 2048 at a time.  The gate's
    half, with gate = 0 and up = 2: dgate is dh, exactly, and dw dh^T x.  All terms are positive
    and of alike size, so that a run's partial sums are half of its last one on average: (2048 / 8 + 4)
    cuts of 2^-23 of that; each run, and each pair's share of a tile, is added with a rounding."""
    g = torch.Generator(device="cuda").manual_seed(T)
    x = (torch.rand(T, C, generator=g, device="cuda") / 2 + 0.5).to(dt)
    x[:, 0] = 2.0
    dh = (torch.rand(T, F, generator=g, device="cuda") / 2 + 0.5).to(dt)
    w = torch.zeros(2 * F, C, dtype=dt, device="cuda")
    w[F:, 0] = 1.0
    dw = torch.empty(2 * F, C, device="cuda")
    ws = torch.zeros(gs.gs_ffn_workspace_bytes(T, C, F), dtype=torch.uint8, device="cuda")
    gs.gs_ffn_bwd(x, w, dh, None, dw, ws)
    want = dh.double().t() @ x.double()
    err = ((dw[:F].double() - want) / want).abs()
    assert float(err.max()) <= 130 * 2.0 ** -23 + (T / 2048 + 77) * 2.0 ** -24, (float(err.max()), float(err.mean()))
    assert (dw[F:] == 0).all()


def test_many_tiles_a_pair(gs):
    """Forward and dx of over twice as many tiles as there are pairs."""
    dt, T, C, F = torch.bfloat16, 5300, 2060, 1100
    g = torch.Generator().manual_seed(1)
    x, xd = few._mat(T, C, dt, g)
    w, wd = few._mat(2 * F, C, dt, g, std=C ** -0.5)
    dh, dhd = few._mat(T, F, dt, g)
    ws = torch.zeros(gs.gs_ffn_workspace_bytes(T, C, F), dtype=torch.uint8, device="cuda")
    want = few._bounds(xd, wd, dhd, "gelu", dt)
    h, dx = torch.empty(T, F, dtype=dt, device="cuda"), torch.empty(T, C, dtype=dt, device="cuda")
    gs.gs_ffn_fwd(x, w, h, ws, act="gelu")
    few._close(h, *want["h"], "h")
    gs.gs_ffn_bwd(x, w, dh, dx, None, ws, act="gelu")
    few._close(dx, *few._stored(*want["dx"], dt), "dx")
    assert gs.gs_workspace_status(ws) == gs.GS_OK


@pytest.mark.parametrize("dt,D,E,offsets", [
    (torch.bfloat16, 64, 64, None),
    (torch.float16, 64, 64, [0, 333, 333, 901, 1400]),
    (torch.float16, 72, 41, [0, 7, 650, 1500]),
    (torch.bfloat16, 40, 128, [3, 129, 131, 1111, 1499]),
    (torch.bfloat16, 128, 128, None),
])
def test_shared_heads_with_little_room(gs, dt, D, E, offsets):
    """Gradients of shared heads with room for all tokens and for ever fewer: the same bits,
    nothing beside the room, until the call is refused."""
    T, H, K = 1500, 8, 2
    g = torch.Generator(device="cuda").manual_seed(D)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k, v, do = (rand(T, h, d).to(dt) for h, d in ((H, D), (K, D), (K, E), (H, E)))
    G = 1 if offsets is None else len(offsets) - 1
    a, s0, ds = -torch.exp2(-rand(H).abs() * 8), rand(G, H, D, E), rand(G, H, D, E)
    offs = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    token = 4 * H * sum(64 if d <= 64 else 128 for d in (D, E))
    asked = gs.gs_linear_attn_workspace_bytes(T, H, K, D, E, G)
    room = torch.empty(asked + T * token, dtype=torch.uint8, device="cuda")

    def run(size):
        room.fill_(0xff)
        out = [torch.full_like(x, 9.0) for x in (q, k, v, s0)]
        gs.gs_linear_attn_bwd(q, k, v, a, do, *out[:3], group_offsets=offs, state=s0, dstate_out=ds, dstate=out[3],
                              workspace=room[:size])
        assert (room[size:] == 0xff).all()
        return out

    want = run(room.numel())
    assert all(torch.equal(x, y) for x, y in zip(want, run(asked)))
    sizes, size = 0, asked
    try:
        while size > 0:
            assert all(torch.equal(x, y) for x, y in zip(want, run(size))), size
            sizes, size = sizes + 1, size - 100 * token
    except gs.GSError:
        pass
    assert sizes >= 3 and size > 0


@pytest.mark.parametrize("back", [False, True])
def test_tokens_outside_the_groups_are_not_read(gs, back):
    """Rows that are copied first: a value that only tokens outside the groups hold is nowhere
    in the workspace."""
    T, H, D, dt, mark = 120, 2, 41, torch.float16, 1234.0
    q, k, v, do = (few._empty(T, H * D, dt, 3, 1)[0].unflatten(1, (H, D)) for _ in range(4))
    offs = torch.tensor([5, 60, 101], dtype=torch.int32, device="cuda")
    a = torch.full((H,), -0.1, device="cuda")
    for x in (q, k, v, do):
        x.copy_(torch.rand(T, H, D, device="cuda"))
        x[:5], x[101:] = mark, mark
    ws = torch.zeros(gs.gs_linear_attn_workspace_bytes(T, H, H, D, D, 2), dtype=torch.uint8, device="cuda")
    out = [torch.full_like(q, 9.0) for _ in range(4)]
    if back:
        gs.gs_linear_attn_bwd(q, k, v, a, do, *out[:3], group_offsets=offs, workspace=ws)
    else:
        gs.gs_linear_attn_fwd(q, k, v, a, out[0], group_offsets=offs, workspace=ws)
    used = ws[:ws.numel() // 2 * 2].view(dt)
    assert (used != 0).any() and not (used == mark).any()
    assert all((x[:5] == 9.0).all() and (x[101:] == 9.0).all() for x in out)


def test_ranges_captured_and_on_another_stream(gs):
    """Shared heads with little room: replayed with other inputs, and on a stream beside one that
    is busy with the same inputs and a workspace of its own."""
    T, H, K, D, dt = 1500, 8, 2, 64, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v, do = (torch.randn(T, h, D, generator=g, device="cuda").to(dt) for h in (H, K, K, H))
    a = torch.linspace(-1.0, 0.0, H, device="cuda")
    offs = torch.tensor([0, 300, 1450], dtype=torch.int32, device="cuda")
    size = gs.gs_linear_attn_workspace_bytes(T, H, K, D, D, 2)
    small = size - 500 * 4 * H * 128
    rooms = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]

    def run(out, room, n, stream=None):
        gs.gs_linear_attn_bwd(q, k, v, a, do, *out, group_offsets=offs, workspace=room[:n], stream=stream)

    new = lambda: [torch.zeros_like(x) for x in (q, k, v)]  # noqa: E731
    want, got, other = new(), new(), new()
    run(got, rooms[0], small)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(got, rooms[0], small)
    for _ in range(3):
        for x in (q, k, v, do):
            x.copy_(x.flip(0))
        run(want, rooms[0], size)
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for x in got:
        x.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        run(got, rooms[0], small)
        run(other, rooms[1], small, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(want, got, other))
