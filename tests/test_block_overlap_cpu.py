"""CPU checks of the block operators' arguments at the C ABI with arrays of their own: outputs
at an input's address are refused, and so is everything else that is refused for itself."""
import pytest
import torch

FREE = pytest.mark.skipif(torch.cuda.is_available(),
                          reason="the addresses are nobody's: only where nothing can be launched")


@pytest.fixture(scope="module")
def gs():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_splatting_differentiable_gs_gb300 as gs
    return gs


def at(i):
    return (1 << 40) + (i << 36)


def _ffn(gs, back=False, tokens=300, channels=64, hidden=48, dtype=0, act=0, x=at(0), xs=64, w=at(1), ws=64, h=at(2), hs=48,
         dx=at(3), dxs=64, dw=at(4), dws=64, dt=2, room=at(5), size=1 << 40):
    L = gs.lib()
    if back:
        return L.gs_ffn_bwd(tokens, channels, hidden, dtype, act, x, xs, w, ws, h, hs, dx, dxs, dw, dws, dt, 0, room, size,
                            None)
    return L.gs_ffn_fwd(tokens, channels, hidden, dtype, act, x, xs, w, ws, h, hs, room, size, None)


@pytest.mark.parametrize("change", [
    dict(tokens=-1), dict(tokens=1 << 31), dict(channels=0), dict(hidden=0), dict(channels=(1 << 20) + 1),
    dict(hidden=(1 << 20) + 1), dict(dtype=2), dict(dtype=-1), dict(act=2), dict(x=0), dict(w=0), dict(h=0),
    dict(room=0), dict(room=at(5) + 8), dict(ws=1 << 38), dict(x=at(0) + 1), dict(w=at(1) + 1), dict(h=at(2) + 1),
])
def test_ffn_refusals(gs, change):
    for back in (False, True):
        assert _ffn(gs, back, **change) == gs.GS_ERR_INVALID_ARG
        assert _ffn(gs, back, size=gs.gs_ffn_workspace_bytes(300, 64, 48, back) - 1) == gs.GS_ERR_INVALID_ARG


@pytest.mark.parametrize("back,change", [
    (False, dict(h=at(0))), (False, dict(h=at(1))), (False, dict(hs=47)), (False, dict(hs=0)),
    (True, dict(dx=at(0))), (True, dict(dx=at(1))), (True, dict(dw=at(0))), (True, dict(dw=at(3))),
    (True, dict(dxs=63)), (True, dict(dws=63)), (True, dict(dt=1)), (True, dict(dw=at(4) + 2)), (True, dict(dx=at(3) + 1)),
])
def test_ffn_outputs_in_place(gs, back, change):
    assert _ffn(gs, back, **change) == gs.GS_ERR_INVALID_ARG


@FREE
def test_ffn_accepts(gs):
    assert _ffn(gs) == gs.GS_ERR_CUDA and _ffn(gs, True) == gs.GS_ERR_CUDA
    assert _ffn(gs, tokens=3) == gs.GS_ERR_CUDA


def _attn(gs, kind, heads=None, size=1 << 40, room=at(9), into=at(8), tokens=300, q_heads=4, k_heads=2, dim=16, vdim=16,
          groups=1, dtype=0, log_decay=at(7), offsets=0, state=0):
    a = gs.net._ATTN.pack(tokens, q_heads, k_heads, dim, vdim, groups, dtype, 1.0, log_decay, offsets, state)
    q, k, v = (at(0), q_heads * dim, dim), (at(1), k_heads * dim, dim), (at(2), k_heads * vdim, vdim)
    out = (at(3), q_heads * vdim, vdim)
    h = [q, k, v, out] + ([(p + at(4) - at(0), t, e) for p, t, e in (q, k, v)] if kind == "bwd" else [])
    for i, x in (heads or {}).items():
        h[i] = x
    L, flat = gs.lib(), [x for t in h for x in t]
    if kind == "bwd":
        return L.gs_linear_attn_bwd(a, gs.net._ATTN_HEADS7.pack(*flat), None, None, room, size, None)
    if kind == "step":
        return L.gs_linear_attn_step(a, gs.net._ATTN_HEADS4.pack(*flat), into, None)
    return L.gs_linear_attn_fwd(a, gs.net._ATTN_HEADS4.pack(*flat), None, room, size, None)


@pytest.mark.parametrize("kind", ["fwd", "bwd", "step"])
def test_attention_refusals(gs, kind):
    bad = gs.GS_ERR_INVALID_ARG
    for change in (dict(tokens=-1), dict(tokens=1 << 31), dict(q_heads=0), dict(k_heads=0), dict(k_heads=3),
                   dict(q_heads=65536), dict(dim=0), dict(dim=129), dict(vdim=0), dict(vdim=129), dict(dtype=2),
                   dict(groups=0), dict(log_decay=0), dict(log_decay=at(7) + 2), dict(state=at(8) + 2)):
        assert _attn(gs, kind, **change) == bad, change
    inputs = 4 if kind == "bwd" else 3
    for i in range(7 if kind == "bwd" else 4):
        assert _attn(gs, kind, {i: (0, 96, 24)}) == bad and _attn(gs, kind, {i: (at(i) + 1, 96, 24)}) == bad
        if i < inputs:
            continue
        for strides in ((15, 16), (64, 15), (0, 16), (64, 0), (16, 16)):  # outputs that overlap
            assert _attn(gs, kind, {i: (at(i), *strides)}) == bad, strides
        for j in range(i if kind != "step" else 0):  # an input's address, or another output's
            for strides in ((64, 16), (32, 16), (128, 32)):
                assert _attn(gs, kind, {i: (at(j), *strides)}) == bad, (i, j)
    if kind == "step":
        assert _attn(gs, kind, into=None) == bad and _attn(gs, kind, into=at(8) + 2) == bad
    else:
        assert _attn(gs, kind, size=64) == bad and _attn(gs, kind, room=None) == bad and _attn(gs, kind, groups=2) == bad
        assert _attn(gs, kind, room=at(9) + 8) == bad


def test_steps_in_place(gs):
    """Refused: other strides, shared key heads, rows that reach into the next one's."""
    bad = gs.GS_ERR_INVALID_ARG
    assert _attn(gs, "step", {3: (at(0), 128, 16)}) == bad and _attn(gs, "step", {3: (at(0), 64, 20)}) == bad
    assert _attn(gs, "step", {2: (at(2), 64, 16), 3: (at(2), 64, 16)}) == bad
    assert _attn(gs, "step", {1: (at(1), 64, 16), 3: (at(1), 64, 16)}) == bad
    assert _attn(gs, "step", {0: (at(0), 32, 8), 3: (at(0), 32, 8)}, vdim=8) == bad


@FREE
def test_attention_accepts(gs):
    for kind in ("fwd", "bwd", "step"):
        assert _attn(gs, kind) == gs.GS_ERR_CUDA
    assert _attn(gs, "step", {3: (at(0), 64, 16)}) == gs.GS_ERR_CUDA
    for i in (1, 2):
        assert _attn(gs, "step", {3: (at(i), 64, 16)}, k_heads=4) == gs.GS_ERR_CUDA
