"""CPU checks of the block operators' arguments at the C ABI: what is refused is refused
before anything is enqueued (here nothing can be: there is no GPU), and the binding's
structures are the header's."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def gs():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_splatting_differentiable_gs_gb300 as gs
    return gs


def _aligned(size=1 << 16):
    buf = C.create_string_buffer(size)
    return buf, (C.addressof(buf) + 255) & ~255


class Attn(C.Structure):  # gs_linear_attn
    _fields_ = [("tokens", C.c_int64), ("q_heads", C.c_int32), ("k_heads", C.c_int32), ("dim", C.c_int32),
                ("vdim", C.c_int32), ("groups", C.c_int32), ("dtype", C.c_int32), ("scale", C.c_float),
                ("log_decay", C.c_void_p), ("group_offsets", C.c_void_p), ("state", C.c_void_p)]


class Heads(C.Structure):  # gs_attn_heads
    _fields_ = [("p", C.c_void_p), ("token", C.c_int64), ("head", C.c_int64)]


def test_structures(gs):
    a = Attn.from_buffer_copy(gs.net._ATTN.pack(1 << 40, 2, 3, 4, 5, 6, 7, 0.5, 8, 9, 10))
    assert [getattr(a, f) for f, _ in Attn._fields_] == [1 << 40, 2, 3, 4, 5, 6, 7, 0.5, 8, 9, 10]
    h = (Heads * 4).from_buffer_copy(gs.net._ATTN_HEADS4.pack(*range(1, 13)))
    assert [(x.p, x.token, x.head) for x in h] == [(1, 2, 3), (4, 5, 6), (7, 8, 9), (10, 11, 12)]
    assert C.sizeof(Heads) * 7 == gs.net._ATTN_HEADS7.size and C.sizeof(Attn) == gs.net._ATTN.size


def _ffn(gs, p, size, tokens=300, channels=64, hidden=48, dtype=0, act=0, x=None, xs=64, w=None, ws=64, h=None, hs=48,
         workspace=None):
    at = lambda v: p if v is None else v  # noqa: E731
    return gs.lib().gs_ffn_fwd(tokens, channels, hidden, dtype, act, at(x), xs, at(w), ws, at(h), hs, at(workspace), size,
                               None)


@pytest.mark.parametrize("change", [
    dict(tokens=-1), dict(tokens=1 << 31), dict(channels=0), dict(hidden=0), dict(channels=(1 << 20) + 1),
    dict(hidden=(1 << 20) + 1), dict(dtype=2), dict(dtype=-1), dict(act=2), dict(x=0), dict(w=0), dict(h=0),
    dict(workspace=0), dict(hs=47), dict(hs=0), dict(ws=1 << 38),
])
def test_ffn_refusals(gs, change):
    keep, p = _aligned()
    assert _ffn(gs, p, 1 << 40, **change) == gs.GS_ERR_INVALID_ARG
    for odd in ("x", "w", "h"):
        assert _ffn(gs, p, 1 << 40, **{odd: p + 1}) == gs.GS_ERR_INVALID_ARG
    assert _ffn(gs, p, gs.gs_ffn_workspace_bytes(300, 64, 48, False) - 1) == gs.GS_ERR_INVALID_ARG
    assert _ffn(gs, p, 1 << 40, workspace=p + 8) == gs.GS_ERR_INVALID_ARG


def test_ffn_backward_refusals(gs):
    keep, p = _aligned()
    L, size = gs.lib(), gs.gs_ffn_workspace_bytes(300, 64, 48)
    call = lambda dx=p, dxs=64, dw=p, dws=64, dt=2, dh=p, n=size: L.gs_ffn_bwd(  # noqa: E731
        300, 64, 48, 0, 0, p, 64, p, 64, dh, 48, dx, dxs, dw, dws, dt, 0, p, n, None)
    bad = gs.GS_ERR_INVALID_ARG
    assert call(dt=1) == bad and call(dws=63) == bad and call(dxs=63) == bad and call(dh=None) == bad
    assert call(dw=p + 2) == bad and call(n=size - 1) == bad
    assert call(dx=None, dw=None) == gs.GS_OK  # nothing wanted


def test_workspace_sizes(gs):
    assert gs.gs_ffn_workspace_bytes(1 << 31, 64, 64) == 0
    assert gs.gs_ffn_workspace_bytes(100, 0, 64) == 0
    assert 0 < gs.gs_ffn_workspace_bytes(0, 64, 64, False) < gs.gs_ffn_workspace_bytes(100, 64, 64, False)
    assert gs.gs_linear_attn_workspace_bytes(100, 4, 3, 64, 64) == 0
    assert gs.gs_linear_attn_workspace_bytes(100, 4, 2, 129, 64) == 0
    assert gs.gs_linear_attn_workspace_bytes(100, 4, 2, 64, 64, groups=0) == 0
    one = gs.gs_linear_attn_workspace_bytes(100, 4, 2, 64, 64)
    assert 0 < one < gs.gs_linear_attn_workspace_bytes(100, 4, 2, 64, 64, groups=9)
    # the sums over shared heads and the copies of odd rows are in the backward's
    assert gs.gs_linear_attn_workspace_bytes(100, 4, 2, 64, 64, backward=False) < one


def test_attention_refusals(gs):
    keep, p = _aligned()
    L, bad = gs.lib(), gs.GS_ERR_INVALID_ARG

    def call(heads=None, size=1 << 40, ws=p, step=False, into=p, **change):
        a = Attn(300, 4, 2, 16, 24, 1, 0, 1.0, p, None, None)
        for k, v in change.items():
            setattr(a, k, v)
        h = (Heads * 4)(Heads(p, 64, 16), Heads(p, 32, 16), Heads(p, 48, 24), Heads(p, 96, 24))
        for i, v in (heads or {}).items():
            h[i] = Heads(*v)
        r = C.byref
        return (L.gs_linear_attn_step(r(a), h, into, None) if step
                else L.gs_linear_attn_fwd(r(a), h, None, ws, size, None))

    for step in (False, True):
        for change in (dict(tokens=-1), dict(tokens=1 << 31), dict(q_heads=0), dict(k_heads=0), dict(k_heads=3),
                       dict(q_heads=65536), dict(dim=0), dict(dim=129), dict(vdim=0), dict(vdim=129), dict(dtype=2),
                       dict(groups=0), dict(log_decay=None), dict(log_decay=p + 2), dict(state=p + 2)):
            assert call(step=step, **change) == bad, (step, change)
        for i in range(4):
            assert call({i: (None, 96, 24)}, step=step) == bad
            assert call({i: (p + 1, 96, 24)}, step=step) == bad
        for strides in ((95, 24), (96, 23), (0, 24), (96, 0), (24, 24)):  # outputs that overlap
            assert call({3: (p, *strides)}, step=step) == bad, strides
    assert call(groups=2) == bad              # groups without offsets
    assert call(size=64) == bad and call(ws=None) == bad and call(ws=p + 8) == bad
    assert call(step=True, into=None) == bad and call(step=True, into=p + 2) == bad
    assert L.gs_linear_attn_fwd(None, None, None, p, 1 << 40, None) == bad
