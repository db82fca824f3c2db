"""Outputs of the block operators where inputs lie: refused, or right."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gs():
    import __graft_entry__
    __graft_entry__.build()
    import gaussian_splatting_differentiable_gs_gb300 as gs
    return gs


def _rand(*shape, seed=0, dt=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dt)


def test_gradients_over_their_inputs_are_refused(gs):
    T, H, D = 300, 2, 32
    qkv = _rand(T, 3, H, D)
    q, k, v = before = qkv.unbind(1)
    before = [t.clone() for t in before]
    do, a = _rand(T, H, D, seed=1), torch.full((H,), -0.1, device="cuda")
    ws = torch.empty(gs.gs_linear_attn_workspace_bytes(T, H, H, D, D), dtype=torch.uint8, device="cuda")
    new = lambda: torch.empty_like(do)  # noqa: E731
    for grads in ((q, new(), new()), (new(), k, new()), (new(), new(), v), (new(), v, new()), (do, new(), new())):
        with pytest.raises(gs.GSError):
            gs.gs_linear_attn_bwd(q, k, v, a, do, *grads, workspace=ws)
    one = new()
    with pytest.raises(gs.GSError):
        gs.gs_linear_attn_bwd(q, k, v, a, do, one, one, new(), workspace=ws)
    with pytest.raises(gs.GSError):
        gs.gs_linear_attn_fwd(q, k, v, a, v, workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(before, (q, k, v)))
    # another part of the same packed buffer is none of theirs
    packed = torch.empty(T, 6, H, D, dtype=qkv.dtype, device="cuda")
    packed[:, :3] = qkv
    q, k, v, *grads = packed.unbind(1)
    want = [new() for _ in range(3)]
    gs.gs_linear_attn_bwd(*before, a, do, *want, workspace=ws)
    gs.gs_linear_attn_bwd(q, k, v, a, do, *grads, workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(want, grads))

    x, w = _rand(300, 64), _rand(128, 64, seed=2)
    fws = torch.zeros(gs.gs_ffn_workspace_bytes(300, 64, 64), dtype=torch.uint8, device="cuda")
    dw = torch.empty_like(w)
    for call in (lambda: gs.gs_ffn_fwd(x, w, x, fws), lambda: gs.gs_ffn_bwd(x, w, _rand(300, 64), x, None, fws),
                 lambda: gs.gs_ffn_bwd(x, w, _rand(300, 64), dw[:1].expand(300, 64), dw, fws)):
        with pytest.raises((gs.GSError, ValueError)):
            call()


@pytest.mark.parametrize("B,H,D", [(1, 3, 64), (5, 4, 40), (3, 2, 7)])
def test_single_tokens_in_place(gs, B, H, D):
    """out where q, k or v was, as a slice of a packed projection too."""
    a = torch.linspace(-0.5, 0.0, H, device="cuda")
    for place in range(3):
        for packed in (False, True):
            t = list(_rand(B, 3, H, D, seed=place).unbind(1))
            if not packed:
                t = [x.contiguous() for x in t]
            s, want_s = (_rand(B, H, D, D, seed=9, dt=torch.float32) for _ in range(2))
            want = torch.empty(B, H, D, dtype=t[0].dtype, device="cuda")
            gs.gs_linear_attn_step(*t, a, want_s, want)
            gs.gs_linear_attn_step(*t, a, s, t[place])
            assert torch.equal(t[place], want) and torch.equal(s, want_s)


def test_single_tokens_over_shared_heads_are_refused(gs):
    """Two query heads of one key head would write where the other still reads."""
    B, D = 3, 32
    room = _rand(B, 4, D)
    q, kv, a = _rand(B, 4, D, seed=1), room[:, :2], torch.zeros(4, device="cuda")
    s = torch.zeros(B, 4, D, D, device="cuda")
    with pytest.raises(gs.GSError):
        gs.gs_linear_attn_step(q, kv, kv.clone(), a, s, room)
    with pytest.raises(gs.GSError):
        gs.gs_linear_attn_step(q, kv.clone(), kv, a, s, room)
    gs.gs_linear_attn_step(q, kv, kv, a, s, q)


def test_heads_without_channels_are_refused(gs):
    q, v, a = _rand(4, 2, 0), _rand(4, 2, 8), torch.zeros(2, device="cuda")
    ws, s = torch.empty(1 << 20, dtype=torch.uint8, device="cuda"), torch.empty(4, 2, 0, 8, device="cuda")
    out = torch.empty_like(v)
    for scale in (None, 1.0):
        with pytest.raises(ValueError):
            gs.gs_linear_attn_fwd(q, q, v, a, out, scale=scale, workspace=ws)
        with pytest.raises(ValueError):
            gs.gs_linear_attn_bwd(q, q, v, a, out, q, q, v.clone(), scale=scale, workspace=ws)
        with pytest.raises(ValueError):
            gs.gs_linear_attn_step(q, q, v, a, s, out, scale=scale)
        with pytest.raises((ValueError, gs.GSError)):
            gs.gs_linear_attn_fwd(v, v, q, a, q, scale=scale, workspace=ws)
