"""CPU checks of the network operators' host side: the frequency table, sizes
and the refusals of the C ABI.  No call here reaches the GPU."""
import ctypes as C
import math

import pytest
import torch

import net_plain


class Heads(C.Structure):  # gs_heads
    _fields_ = [("src", C.c_void_p), ("dst", C.c_void_p), ("in_token", C.c_int64),
                ("in_head", C.c_int64), ("out_token", C.c_int64), ("out_head", C.c_int64),
                ("heads", C.c_int32)]


class Norm(C.Structure):  # gs_norm
    _fields_ = [("tokens", C.c_int64), ("channels", C.c_int32), ("groups", C.c_int32),
                ("flags", C.c_int32), ("dtype", C.c_int32), ("res_dtype", C.c_int32),
                ("eps", C.c_float), ("w_pre", C.c_void_p), ("w_post", C.c_void_p),
                ("res_scale", C.c_void_p), ("gate", C.c_void_p), ("group_offsets", C.c_void_p)]


class Ckpt(C.Structure):  # gs_ckpt
    _fields_ = [("q", C.c_void_p), ("e", C.c_void_p), ("q_stride", C.c_int64),
                ("e_stride", C.c_int64)]


@pytest.fixture(scope="module")
def gs():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_splatting_differentiable_gs_gb300 as gs
    return gs


def test_rope_turns_are_fractions_of_a_turn(gs):
    r = gs.Rope([4, 6], base=[10000.0, 100.0], scale=[1.0, 2.5])
    want = [1.0, 1e-2] + [2.5 * 100.0 ** (-2 * j / 6) for j in range(3)]
    for got, f in zip(r.turns, want):
        # a double holds 53 of the 64 bits
        assert abs(got / 2.0 ** 64 - f / (2 * math.pi)) < 2 ** -52
    # a negative frequency and one above a turn per step wrap
    r = gs.Rope([2, 2], base=1.0, scale=[-1.0, 7.0])
    assert abs(r.turns[0] / 2.0 ** 64 - (1 - 1 / (2 * math.pi))) < 2 ** -52
    assert abs(r.turns[1] / 2.0 ** 64 - (7 / (2 * math.pi) - 1)) < 2 ** -50


@pytest.mark.parametrize("dims,base,scale", [([3], 1e4, 1.0), ([0], 1e4, 1.0), ([-2, 4], 1e4, 1.0),
                                             ([258], 1e4, 1.0), ([128, 130], 1e4, 1.0),
                                             ([8], 0.0, 1.0), ([8], -1.0, 1.0),
                                             ([8], math.nan, 1.0), ([8], 1e4, math.inf)])
def test_rope_refuses_bad_sections(gs, dims, base, scale):
    with pytest.raises(gs.GSError, match="invalid argument"):
        gs.Rope(dims, base=base, scale=scale)


def test_rope_refuses_axis_counts(gs):
    for dims in ([], [2] * 5):
        with pytest.raises(ValueError):
            gs.Rope(dims)
    with pytest.raises(ValueError):
        gs.Rope([2, 2], base=[1.0])


def _a16(buf):
    return C.c_void_p((C.addressof(buf) + 15) & ~15)


def test_rope_refusals(gs):
    L, bad = gs.lib(), gs.GS_ERR_INVALID_ARG
    r = gs.Rope([8, 8])
    buf = C.create_string_buffer(4096)
    p = _a16(buf)

    def call(tokens=4, axes=2, dims=r._dims, turns=r.turns, pos=p, dim=16, dtype=0, src=p, dst=p,
             heads=1, n_sets=1, sets=None):
        s = (Heads * 2)()
        for h in s:
            h.src, h.dst, h.heads = src, dst, heads
            h.in_token = h.out_token = 16 * max(heads, 1)
            h.in_head = h.out_head = 16
        return L.gs_rope(tokens, axes, dims, turns, 0, 0, pos, dim, dtype,
                         s if sets is None else sets[0], n_sets, None)

    assert call(tokens=-1) == bad and call(tokens=1 << 31) == bad
    assert call(axes=0) == bad and call(axes=5) == bad
    assert call(dims=None) == bad and call(turns=None) == bad
    assert call(dim=14) == bad and call(dim=257) == bad          # sections wider than the head
    assert call(dtype=3) == bad and call(dtype=-1) == bad
    assert call(pos=None) == bad and call(pos=C.c_void_p(p.value + 2)) == bad
    assert call(src=None) == bad and call(dst=None) == bad
    assert call(src=p.value + 1) == bad                         # half an element
    assert call(heads=-1) == bad and call(n_sets=0) == bad and call(n_sets=3) == bad
    assert call(sets=[None]) == bad
    assert call(tokens=0) == gs.GS_OK and call(heads=0) == gs.GS_OK


def _norm(gs, **kw):
    p = Norm()
    p.tokens, p.channels, p.groups, p.eps = 4, 8, 1, 1e-6
    p.flags = gs.net.NORM_POST
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def test_norm_refusals(gs):
    L, bad = gs.lib(), gs.GS_ERR_INVALID_ARG
    buf = C.create_string_buffer(1 << 16)
    p = _a16(buf).value

    def fwd(n, x=p, block=p, x_out=p, y=p, stats=p, q=None, e=None, qs=32):
        return L.gs_gated_norm_fwd(None if n is None else C.byref(n), x, 8, block, 8, x_out, 8, y,
                                   8, stats, q, qs, e, 1, None)

    assert fwd(None) == bad
    for kw in (dict(tokens=-1), dict(tokens=1 << 31), dict(channels=0), dict(channels=8193),
               dict(groups=0), dict(dtype=3), dict(dtype=0, res_dtype=1), dict(dtype=2, res_dtype=0),
               dict(flags=4), dict(eps=-1.0), dict(eps=math.nan), dict(groups=2),
               dict(groups=2, gate=p), dict(w_pre=p + 2), dict(gate=p + 1), dict(res_scale=p + 1)):
        assert fwd(_norm(gs, **kw)) == bad, kw
    n = _norm(gs)
    assert fwd(n, x=None) == bad and fwd(n, stats=None) == bad and fwd(n, stats=p + 4) == bad
    assert fwd(n, block=None) == bad and fwd(n, x_out=None) == bad      # one without the other
    assert fwd(n, block=None, x_out=None, y=None) == bad                # nothing to do
    assert fwd(n, q=p) == bad and fwd(n, e=p) == bad
    assert fwd(n, q=p, e=p, y=None) == bad
    assert fwd(n, q=p + 4, e=p) == bad and fwd(n, q=p, e=p, qs=40) == bad
    assert fwd(n, x=p + 1) == bad and fwd(n, y=p + 1) == bad
    assert fwd(_norm(gs, tokens=0), x=None, block=None, x_out=None, y=None, stats=None) == gs.GS_OK

    ws = gs.gs_gated_norm_workspace_bytes(8, 1)
    assert ws > 0 and gs.gs_gated_norm_workspace_bytes(0, 1) == 0
    assert gs.gs_gated_norm_workspace_bytes(8, 0) == 0

    def bwd(n, x=p, block=p, stats=p, dxo=p, dy=p, dx=p, db=p, w=p, dgate=None, work=p, size=ws):
        return L.gs_gated_norm_bwd(C.byref(n), x, 8, block, 8, stats, dxo, 8, dy, 8, dx, 8, db, 8,
                                   w, None, dgate, None, work, size, None)

    assert bwd(n, x=None) == bad and bwd(n, stats=None) == bad and bwd(n, dx=None) == bad
    assert bwd(n, dxo=None, dy=None) == bad
    assert bwd(n, db=None) == bad and bwd(n, block=None) == bad
    assert bwd(n, dgate=p) == bad                                       # no gate
    assert bwd(n, work=None) == bad and bwd(n, size=ws - 1) == bad and bwd(n, work=p + 8) == bad


def test_act8_refusals(gs):
    L, bad = gs.lib(), gs.GS_ERR_INVALID_ARG
    buf = C.create_string_buffer(1 << 16)
    p = _a16(buf).value

    def enc(T=2, ch=8, dt=0, x=p, q=p, qs=32, e=p, fn=L.gs_act8_encode):
        if fn is L.gs_act8_encode:
            return fn(T, ch, dt, x, 8, q, qs, e, 1, None)
        return fn(T, ch, dt, q, qs, e, 1, x, 8, None)

    for fn in (L.gs_act8_encode, L.gs_act8_decode):
        for kw in (dict(T=-1), dict(T=1 << 31), dict(ch=0), dict(dt=3), dict(x=None), dict(q=None),
                   dict(e=None), dict(q=p + 8), dict(qs=24), dict(x=p + 1)):
            assert enc(fn=fn, **kw) == bad, kw
        assert enc(fn=fn, T=0, x=None, q=None, e=None) == gs.GS_OK

    ck = Ckpt(p, p, 32, 1)
    none = Ckpt()
    odd = Ckpt(p + 4, p, 32, 1)

    def fwd(act=0, gate=p, up=p, h=p, g8=ck, u8=ck, T=2):
        return L.gs_glu_fwd(T, 8, 0, act, gate, 8, up, 8, h, 8, C.byref(g8), C.byref(u8), None)

    assert fwd(act=2) == bad and fwd(act=-1) == bad
    assert fwd(gate=None) == bad and fwd(h=None) == bad
    assert fwd(up=None) == bad                       # a checkpoint of what is not there
    assert fwd(g8=odd) == bad and fwd(u8=odd) == bad
    assert fwd(T=0, gate=None) == gs.GS_OK

    def bwd(act=0, dh=p, dg=p, du=p, g8=ck, u8=ck, h8=none, T=2):
        return L.gs_glu_bwd(T, 8, 0, act, C.byref(g8), C.byref(u8), dh, 8, dg, 8, du, 8,
                            C.byref(h8), None)

    assert bwd(act=5) == bad and bwd(dh=None) == bad and bwd(dg=None) == bad
    assert bwd(du=None) == bad and bwd(u8=none) == bad and bwd(g8=none) == bad
    assert bwd(h8=odd) == bad
    assert bwd(T=0) == gs.GS_OK

    need = gs.gs_act8_wgrad_workspace_bytes(2, 8, 8)
    assert need >= 256 and gs.gs_act8_wgrad_workspace_bytes(-1, 8, 8) == 0

    def wg(T=2, rows=8, ch=8, dt=0, dy=p, q=p, qs=32, e=p, dw=p, out=2, ws=p, size=None):
        size = gs.gs_act8_wgrad_workspace_bytes(2, 8, 8) if size is None else size
        return L.gs_act8_wgrad(T, rows, ch, dt, dy, 8, q, qs, e, 1, dw, 8, out, 0, ws, size, None)

    for kw in (dict(T=-1), dict(rows=0), dict(ch=0), dict(dt=3), dict(dy=None), dict(q=None),
               dict(e=None), dict(dw=None), dict(out=1), dict(out=3), dict(ws=None),
               dict(size=need - 1), dict(ws=p + 8), dict(q=p + 8), dict(qs=40), dict(dw=p + 2),
               dict(dy=p + 1)):
        assert wg(**kw) == bad, kw


def test_checkpoint_shapes(gs):
    assert gs.act8_shapes(5, 1) == ((5, 32), (5, 1))
    assert gs.act8_shapes(5, 64) == ((5, 64), (5, 2))
    assert gs.act8_shapes(0, 65) == ((0, 96), (0, 3))


def test_wrappers_refuse_host_tensors(gs):
    x = torch.zeros(2, 8)
    q, e = gs.act8_empty(2, 8, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        gs.gs_act8_encode(x, q, e)
    with pytest.raises(ValueError, match="CUDA"):
        gs.gs_gated_norm_fwd(x, x, x, x, torch.zeros(2, 4))
    with pytest.raises(ValueError, match="CUDA"):
        gs.gs_rope(gs.Rope([8]), torch.zeros(2, 1, dtype=torch.int32), x[:, None])


def test_plain_checkpoint_is_the_nearest_step():
    """The plain form used by the GPU tests: |error| <= step / 2, the largest
    magnitude within 127 steps and above 63.5 of them."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(6, 70, generator=g) * torch.exp2(torch.randint(-30, 30, (6, 1), generator=g))
    q, e = net_plain.encode(x)
    v = net_plain.decode(q, e, 70)
    step = torch.exp2(e.double() - 127).repeat_interleave(32, 1)[:, :70]
    assert ((v - x.double()).abs() <= step / 2).all()
    big = torch.nn.functional.pad(x, (0, 26)).view(6, 3, 32).abs().amax(2).double()
    unit = torch.exp2(e.double() - 127)
    assert (big <= 127 * unit).all() and (big > 63.5 * unit).all()


def test_packed_structures_have_the_c_layout(gs):
    for packed, struct in ((gs.net._HEADS, Heads), (gs.net._NORM, Norm), (gs.net._CKPT, Ckpt)):
        assert packed.size == C.sizeof(struct)
    p = Norm.from_buffer_copy(gs.net._NORM.pack(1 << 40, 2, 3, 4, 5, 6, 0.5, 7, 8, 9, 10, 11))
    assert (p.tokens, p.channels, p.groups, p.flags, p.dtype, p.res_dtype, p.eps) == (1 << 40, 2, 3, 4, 5, 6, 0.5)
    assert (p.w_pre, p.w_post, p.res_scale, p.gate, p.group_offsets) == (7, 8, 9, 10, 11)
    h = Heads.from_buffer_copy(gs.net._HEADS.pack(1, 2, 3, 4, 5, 6, 7))
    assert (h.src, h.dst, h.in_token, h.in_head, h.out_token, h.out_head, h.heads) == (1, 2, 3, 4, 5, 6, 7)
    k = Ckpt.from_buffer_copy(gs.net._CKPT.pack(1, 2, 3, 4))
    assert (k.q, k.e, k.q_stride, k.e_stride) == (1, 2, 3, 4)
