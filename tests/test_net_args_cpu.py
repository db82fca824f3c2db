"""CPU checks of the network operators' arguments at the C ABI: what is refused is refused
before anything is enqueued (here nothing can be: there is no GPU)."""
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
    return buf, (C.addressof(buf) + 15) & ~15


@pytest.mark.parametrize("dtype,tokens", [(2, 1 << 30), (1, 1 << 30), (0, (1 << 31) - 32), (2, 715827904)])
def test_wgrad_refuses_lengths_beyond_the_tensor_map_first(gs, dtype, tokens):
    """Two bf16 terms of an fp16 gradient, three of an fp32 one: 2^31 - 64 rows in all."""
    keep, p = _aligned()
    L = gs.lib()
    call = lambda size: L.gs_act8_wgrad(tokens, 8, 8, dtype, p, 8, p, 32, p, 1, p, 8, 2, 0, p, size, None)  # noqa: E731
    assert call(1 << 62) == gs.GS_ERR_INVALID_ARG
    assert L.gs_act8_wgrad_workspace_bytes(tokens, 8, 8, dtype) == 0
    assert L.gs_act8_wgrad_workspace_bytes(tokens // 4, 8, 8, dtype) > 0


class Heads(C.Structure):  # gs_heads
    _fields_ = [("src", C.c_void_p), ("dst", C.c_void_p), ("in_token", C.c_int64),
                ("in_head", C.c_int64), ("out_token", C.c_int64), ("out_head", C.c_int64),
                ("heads", C.c_int32)]


def test_rope_refuses_in_place_with_other_strides(gs):
    keep, p = _aligned()
    r = gs.Rope([8])

    def call(strides):
        s = (Heads * 1)(Heads(p, p, *strides, 2))
        return gs.lib().gs_rope(3, 1, r._dims, r.turns, 0, 0, p, 8, 0, s, 1, None)

    assert call((32, 8, 16, 8)) == gs.GS_ERR_INVALID_ARG     # another stride between tokens
    assert call((32, 8, 32, 16)) == gs.GS_ERR_INVALID_ARG    # between heads


class Norm(C.Structure):  # gs_norm
    _fields_ = [("tokens", C.c_int64), ("channels", C.c_int32), ("groups", C.c_int32),
                ("flags", C.c_int32), ("dtype", C.c_int32), ("res_dtype", C.c_int32),
                ("eps", C.c_float), ("w_pre", C.c_void_p), ("w_post", C.c_void_p),
                ("res_scale", C.c_void_p), ("gate", C.c_void_p), ("group_offsets", C.c_void_p)]


class Ckpt(C.Structure):  # gs_ckpt
    _fields_ = [("q", C.c_void_p), ("e", C.c_void_p), ("q_stride", C.c_int64),
                ("e_stride", C.c_int64)]


@pytest.mark.parametrize("es", [0, 1, -2])
def test_exponent_rows_must_not_overlap(gs, es):
    """40 channels: two exponents a row."""
    keep, p = _aligned()
    L, bad = gs.lib(), gs.GS_ERR_INVALID_ARG
    ws = gs.gs_act8_wgrad_workspace_bytes(2, 8, 40)
    good, short = Ckpt(p, p, 64, 2), Ckpt(p, p, 64, es)
    r = C.byref
    assert L.gs_act8_encode(2, 40, 0, p, 40, p, 64, p, es, None) == bad
    assert L.gs_act8_decode(2, 40, 0, p, 64, p, es, p, 40, None) == bad
    assert L.gs_glu_fwd(2, 40, 0, 0, p, 40, p, 40, p, 40, r(short), r(good), None) == bad
    assert L.gs_glu_fwd(2, 40, 0, 0, p, 40, p, 40, p, 40, r(good), r(short), None) == bad
    for cks in ((short, good, good), (good, short, good), (good, good, short)):
        assert L.gs_glu_bwd(2, 40, 0, 0, r(cks[0]), r(cks[1]), p, 40, p, 40, p, 40, r(cks[2]), None) == bad
    n = Norm(2, 40, 1, 1, 0, 0, 1e-6)
    assert L.gs_gated_norm_fwd(r(n), p, 40, p, 40, p, 40, p, 40, p, p, 64, p, es, None) == bad
    assert L.gs_act8_wgrad(2, 8, 40, 0, p, 8, p, 64, p, es, p, 40, 2, 0, p, ws, None) == bad


def test_tensors_of_another_device_than_the_current_one_are_refused(gs, monkeypatch):
    """The library launches on the current device, so that is whose stream is taken."""
    class Tensor:
        def __init__(self, device):
            self.device = device

        def get_device(self):
            return self.device

    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(gs.net, "_current_device", lambda: 1)
    monkeypatch.setattr(gs.net, "_raw_stream", lambda device: 1000 + device)
    assert gs.net._stream(None, Tensor(1)) == 1001 and gs.net._stream(Stream, Tensor(1)) == 77
    for stream in (None, Stream):
        with pytest.raises(ValueError, match="current device"):
            gs.net._stream(stream, Tensor(0))


def _turns(dims, base, scale):
    """Each pair's frequency in turns times 2^64, modulo 2^64, to 60 digits."""
    from decimal import Decimal, getcontext
    getcontext().prec = 90
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")
    out = []
    for d, b, s in zip(dims, base, scale):
        for j in range(d // 2):
            f = Decimal(s) * (Decimal(b).ln() * Decimal(-2 * j) / Decimal(d)).exp() / two_pi * 2 ** 64
            out.append(f % 2 ** 64)
    return out


@pytest.mark.parametrize("dims,base,scale", [
    ([64], [10000.0], [1.0]), ([128], [500000.0], [0.25]), ([16, 24, 24], [10000.0, 100.0, 7.5], [1.0, 0.5, 2.0]),
    ([6, 10], [1.0, 1e6], [-1.0, 3.0]), ([256], [1e4], [-0.125]), ([2, 30], [0.5, 0.001], [7.0, 1e-3]),
    ([34], [1e300], [1e-9]), ([22], [3.0], [12345.678]), ([8], [1e4], [0.0])])
def test_rope_turns_to_the_last_of_their_bits(gs, dims, base, scale):
    """64 bits of each frequency: a position times it, modulo 2^64, is off by 2^-64 of a turn
    times the position."""
    r = gs.Rope(dims, base=base, scale=scale)
    want = _turns(dims, base, scale)
    assert len(want) == sum(dims) // 2
    for got, f in zip(r.turns, want):
        off = abs(int(got) - f)
        assert min(off, 2 ** 64 - off) <= 1, (int(got), f)


def test_rope_turns_at_the_ends_of_the_bases(gs):
    """Frequencies that are next to nothing, and one that is no finite number."""
    for base in (1.7e308, 1e308):
        r = gs.Rope([256], base=base)
        want = _turns([256], [base], [1.0])
        assert all(abs(int(got) - f) <= 1 for got, f in zip(r.turns, want))
    assert gs.Rope([4], base=5e-324, scale=0.0).turns[1] == 0
    with pytest.raises(gs.GSError, match="invalid argument"):
        gs.Rope([64], base=1e-310, scale=1e30)


def test_matrices_in_place_with_other_strides_are_refused(gs):
    """Rows would be written before others are read there."""
    keep, p = _aligned()
    L, bad, r = gs.lib(), gs.GS_ERR_INVALID_ARG, C.byref
    ck, other = Ckpt(p, p, 32, 1), p + 4096
    assert L.gs_glu_bwd(2, 8, 0, 0, r(ck), r(ck), p, 8, p, 16, other, 8, None, None) == bad
    n = Norm(2, 8, 1, 1, 0, 0, 1e-6)
    assert L.gs_gated_norm_fwd(r(n), p, 8, other, 8, p, 16, other, 8, other, None, 0, None, 0, None) == bad
    bwd = lambda dx, dxs, db, dbs: L.gs_gated_norm_bwd(  # noqa: E731
        r(n), other, 8, other, 8, other, p, 8, p + 2048, 8, dx, dxs, db, dbs, None, None, None, None, None, 0, None)
    assert bwd(p, 16, other, 8) == bad and bwd(other, 8, p + 2048, 16) == bad
