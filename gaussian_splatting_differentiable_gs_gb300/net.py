"""Network operators (include/gs_net.h): multi-axis rotary positions, gated
norms and 8-bit activation checkpoints, for a network that predicts Gaussians
from views.  As in the package itself, each gs_* function only checks and
marshals its arguments and calls the C ABI function of the same name.

Matrices are CUDA tensors [tokens, channels] whose last axis is contiguous;
rows may have any stride (a slice of a packed projection, say)."""
import ctypes as C

import torch

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
GROUP = 32
NORM_POST, NORM_CENTER = 1, 2
ACTS = {"silu": 0, "gelu": 1}
ROPE_MAX_AXES = 4


class _Heads(C.Structure):
    _fields_ = [("src", C.c_void_p), ("dst", C.c_void_p), ("in_token", C.c_int64),
                ("in_head", C.c_int64), ("out_token", C.c_int64), ("out_head", C.c_int64),
                ("heads", C.c_int32)]


class _Norm(C.Structure):
    _fields_ = [("tokens", C.c_int64), ("channels", C.c_int32), ("groups", C.c_int32),
                ("flags", C.c_int32), ("dtype", C.c_int32), ("res_dtype", C.c_int32),
                ("eps", C.c_float), ("w_pre", C.c_void_p), ("w_post", C.c_void_p),
                ("res_scale", C.c_void_p), ("gate", C.c_void_p), ("group_offsets", C.c_void_p)]


class _Ckpt(C.Structure):
    _fields_ = [("q", C.c_void_p), ("e", C.c_void_p), ("q_stride", C.c_int64),
                ("e_stride", C.c_int64)]


def declare(L):
    """Argument types of the network calls, set once by lib()."""
    vp, i64, i32, sz = C.c_void_p, C.c_int64, C.c_int32, C.c_size_t
    L.gs_rope_turns.argtypes = [i32, vp, vp, vp, vp]
    L.gs_rope.argtypes = [i64, i32, vp, vp, i32, i32, vp, i32, i32, vp, i32, vp]
    L.gs_gated_norm_fwd.argtypes = [vp, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, i64, vp, i64,
                                    vp]
    L.gs_gated_norm_workspace_bytes.argtypes = [i32, i32]
    L.gs_gated_norm_workspace_bytes.restype = sz
    L.gs_gated_norm_bwd.argtypes = [vp, vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, i64, vp, i64,
                                    vp, vp, vp, vp, vp, sz, vp]
    L.gs_act8_encode.argtypes = [i64, i32, i32, vp, i64, vp, i64, vp, i64, vp]
    L.gs_act8_decode.argtypes = [i64, i32, i32, vp, i64, vp, i64, vp, i64, vp]
    L.gs_glu_fwd.argtypes = [i64, i32, i32, i32, vp, i64, vp, i64, vp, i64, vp, vp, vp]
    L.gs_glu_bwd.argtypes = [i64, i32, i32, i32, vp, vp, vp, i64, vp, i64, vp, i64, vp, vp]
    L.gs_act8_wgrad_workspace_bytes.argtypes = [i64, i32, i32, i32]
    L.gs_act8_wgrad_workspace_bytes.restype = sz
    L.gs_act8_wgrad.argtypes = [i64, i32, i32, i32, vp, i64, vp, i64, vp, i64, vp, i64, i32, i32,
                                vp, sz, vp]


from . import _check, _stream, lib  # noqa: E402  (the package defines these first)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _mat(t, name, shape=None, dtype=None):
    """A CUDA matrix with a contiguous last axis, of the given shape and type."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 2:
        raise ValueError("%s must be a CUDA matrix" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s is %s, expected %s" % (name, t.dtype, dtype))
    if t.dtype not in DTYPES and t.dtype not in (torch.int8, torch.uint8):
        raise ValueError("%s: unsupported type %s" % (name, t.dtype))
    if t.numel() and t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s: the last axis must be contiguous" % name)
    return t


def _vec(t, name, n, dtype=torch.float32):
    if t is None:
        return None
    if (not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype or t.numel() != n
            or not t.is_contiguous()):
        raise ValueError("%s must be a contiguous CUDA %s tensor of %d entries" % (name, dtype, n))
    return t.data_ptr()


def act8_shapes(tokens, channels):
    """Shapes of a checkpoint's q (int8) and e (uint8) arrays."""
    ld = -(-channels // GROUP) * GROUP
    return (tokens, ld), (tokens, ld // GROUP)


def act8_empty(tokens, channels, device="cuda"):
    """A new checkpoint's arrays (q, e) for [tokens, channels] values."""
    qs, es = act8_shapes(tokens, channels)
    return (torch.empty(qs, dtype=torch.int8, device=device),
            torch.empty(es, dtype=torch.uint8, device=device))


def _act8(q, e, tokens, channels, name):
    qs, es = act8_shapes(tokens, channels)
    _mat(q, name + "_q", qs, torch.int8)
    _mat(e, name + "_e", es, torch.uint8)
    return _Ckpt(q.data_ptr(), e.data_ptr(), q.stride(0), e.stride(0))


# --------------------------------------------------------------------------
# rotary positions


class Rope:
    """The frequencies of a rotary embedding with several axes: dims[a]
    channels of a head turn with position a (base and scale: one value or one
    per axis).  Computed once on the host."""

    def __init__(self, dims, base=10000.0, scale=1.0, interleaved=False):
        self.dims = [int(d) for d in dims]
        n = len(self.dims)
        if not 1 <= n <= ROPE_MAX_AXES:
            raise ValueError("1..%d axes" % ROPE_MAX_AXES)
        base = [float(b) for b in (base if isinstance(base, (list, tuple)) else [base] * n)]
        scale = [float(s) for s in (scale if isinstance(scale, (list, tuple)) else [scale] * n)]
        if len(base) != n or len(scale) != n:
            raise ValueError("one base and one scale per axis")
        self.interleaved = bool(interleaved)
        self._dims = (C.c_int32 * n)(*self.dims)
        self.turns = (C.c_uint64 * max(1, sum(self.dims) // 2))()
        _check("gs_rope_turns", lib().gs_rope_turns(
            n, self._dims, (C.c_double * n)(*base), (C.c_double * n)(*scale), self.turns))


def gs_rope(rope, positions, q, k=None, q_out=None, k_out=None, inverse=False, stream=None):
    """Rotates q (and k) [tokens, heads, head_dim] by the positions [tokens,
    axes] (int32); in place where no output is given.  inverse: the opposite
    rotation, which is the backward pass.  Returns (q_out, k_out)."""
    q_out = q if q_out is None else q_out
    k_out = k if k_out is None else k_out
    pairs = [(q, q_out, "q")] + ([(k, k_out, "k")] if k is not None else [])
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    tokens, dim = q.shape[0], q.shape[-1]
    sets = (_Heads * len(pairs))()
    for s, (src, dst, name) in zip(sets, pairs):
        for t in (src, dst):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 3:
                raise ValueError("%s must be a CUDA [tokens, heads, head_dim] tensor" % name)
            if t.dtype != q.dtype or t.dtype not in DTYPES:
                raise ValueError("%s: type %s" % (name, t.dtype))
            if t.shape[0] != tokens or t.shape[2] != dim or t.shape != src.shape:
                raise ValueError("%s: shape %s" % (name, tuple(t.shape)))
            if t.numel() and dim > 1 and t.stride(2) != 1:
                raise ValueError("%s: the last axis must be contiguous" % name)
        if src.data_ptr() == dst.data_ptr() and src.stride() != dst.stride():
            raise ValueError("%s: in place with other strides" % name)
        s.src, s.dst, s.heads = src.data_ptr(), dst.data_ptr(), src.shape[1]
        s.in_token, s.in_head = src.stride(0), src.stride(1)
        s.out_token, s.out_head = dst.stride(0), dst.stride(1)
    n = len(rope.dims)
    if (not isinstance(positions, torch.Tensor) or not positions.is_cuda
            or positions.dtype != torch.int32 or tuple(positions.shape) != (tokens, n)
            or not positions.is_contiguous()):
        raise ValueError("positions must be a contiguous CUDA int32 [%d, %d] tensor" % (tokens, n))
    _check("gs_rope", lib().gs_rope(tokens, n, rope._dims, rope.turns, int(rope.interleaved),
                                    int(bool(inverse)), positions.data_ptr(), dim,
                                    DTYPES[q.dtype], sets, len(pairs), _stream(stream)))
    return q_out, k_out


# --------------------------------------------------------------------------
# gated norms


def _norm_args(x, other, w_pre, w_post, gate, group_offsets, res_scale, post, center, eps):
    tokens, c = x.shape
    p = _Norm()
    p.tokens, p.channels, p.eps = tokens, c, float(eps)
    p.flags = (NORM_POST if post else 0) | (NORM_CENTER if center else 0)
    p.dtype, p.res_dtype = DTYPES[other.dtype], DTYPES[x.dtype]
    p.w_pre = _vec(w_pre, "w_pre", c)
    p.w_post = _vec(w_post, "w_post", c)
    p.res_scale = _vec(res_scale, "res_scale", c)
    p.groups = 1
    if gate is not None:
        if gate.dim() != 2 or gate.shape[1] != c or gate.shape[0] < 1:
            raise ValueError("gate must be [groups, channels]")
        p.groups = gate.shape[0]
        p.gate = _vec(gate, "gate", gate.numel(), other.dtype)
        if group_offsets is None and p.groups > 1:
            raise ValueError("gate: more than one group needs group_offsets")
        p.group_offsets = _vec(group_offsets, "group_offsets", p.groups + 1, torch.int32)
    elif group_offsets is not None:
        raise ValueError("group_offsets without a gate")
    return p


def gs_gated_norm_fwd(x, block, x_out, y, stats, w_pre=None, w_post=None, gate=None,
                      group_offsets=None, res_scale=None, y_q=None, y_e=None, post=True,
                      center=False, eps=1e-6, stream=None):
    """x_out = x + res_scale * gate[group] * (w_post * norm(block)), y = w_pre
    * norm(x_out).  block, x_out None: y = w_pre * norm(x) only; y None: the
    sum only; post False: no norm of the block.  gate [groups, channels] with
    group_offsets int32 [groups + 1] (one group: None).  stats: float32
    [tokens, 4] for the backward.  y_q, y_e: y's 8-bit checkpoint."""
    _mat(x, "x")
    shape = tuple(x.shape)
    other = y if y is not None else block
    if other is None:
        raise ValueError("neither block nor y")
    _mat(other, "y or block", shape)
    for t, name, dt in ((block, "block", other.dtype), (x_out, "x_out", x.dtype),
                        (y, "y", other.dtype)):
        if t is not None:
            _mat(t, name, shape, dt)
    if (y_q is None) != (y_e is None):
        raise ValueError("y_q and y_e come together")
    ck = _act8(y_q, y_e, *shape, name="y") if y_q is not None else _Ckpt()
    p = _norm_args(x, other, w_pre, w_post, gate, group_offsets, res_scale, post, center, eps)
    st = lambda t: 0 if t is None else t.stride(0)  # noqa: E731
    _check("gs_gated_norm_fwd", lib().gs_gated_norm_fwd(
        C.byref(p), x.data_ptr(), x.stride(0), _ptr(block), st(block), _ptr(x_out), st(x_out),
        _ptr(y), st(y), _vec(stats, "stats", 4 * shape[0]), ck.q, ck.q_stride, ck.e, ck.e_stride,
        _stream(stream)))


def gs_gated_norm_workspace_bytes(channels, groups=1):
    return int(lib().gs_gated_norm_workspace_bytes(channels, groups))


def gs_gated_norm_bwd(x_out, block, stats, dx_out, dy, dx, dblock, w_pre=None, w_post=None,
                      gate=None, group_offsets=None, res_scale=None, dw_pre=None, dw_post=None,
                      dgate=None, dres_scale=None, workspace=None, post=True, center=False,
                      stream=None):
    """Backward of gs_gated_norm_fwd from its x_out, block and stats: writes
    dx, dblock and, where given, the fp32 sums dw_pre, dw_post, dres_scale
    [channels] and dgate [groups, channels].  dx_out or dy None: zero.  The
    sums need a uint8 workspace of gs_gated_norm_workspace_bytes()."""
    _mat(x_out, "x_out")
    shape = tuple(x_out.shape)
    other = dy if dy is not None else block
    if other is None:
        raise ValueError("neither block nor dy")
    _mat(other, "dy or block", shape)
    for t, name, dt in ((block, "block", other.dtype), (dx_out, "dx_out", x_out.dtype),
                        (dy, "dy", other.dtype), (dx, "dx", x_out.dtype),
                        (dblock, "dblock", other.dtype)):
        if t is not None:
            _mat(t, name, shape, dt)
    p = _norm_args(x_out, other, w_pre, w_post, gate, group_offsets, res_scale, post, center, 0.0)
    c, st = shape[1], lambda t: 0 if t is None else t.stride(0)  # noqa: E731
    _check("gs_gated_norm_bwd", lib().gs_gated_norm_bwd(
        C.byref(p), x_out.data_ptr(), x_out.stride(0), _ptr(block), st(block),
        _vec(stats, "stats", 4 * shape[0]), _ptr(dx_out), st(dx_out), _ptr(dy), st(dy), _ptr(dx),
        st(dx), _ptr(dblock), st(dblock), _vec(dw_pre, "dw_pre", c), _vec(dw_post, "dw_post", c),
        _vec(dgate, "dgate", p.groups * c), _vec(dres_scale, "dres_scale", c),
        None if workspace is None else _vec(workspace, "workspace", workspace.numel(), torch.uint8),
        0 if workspace is None else workspace.numel(), _stream(stream)))


# --------------------------------------------------------------------------
# 8-bit activation checkpoints


def gs_act8_encode(x, q, e, stream=None):
    """Writes the 8-bit checkpoint (q, e) of x [tokens, channels]."""
    _mat(x, "x")
    ck = _act8(q, e, *x.shape, name="x")
    _check("gs_act8_encode", lib().gs_act8_encode(
        x.shape[0], x.shape[1], DTYPES[x.dtype], x.data_ptr(), x.stride(0), ck.q, ck.q_stride,
        ck.e, ck.e_stride, _stream(stream)))


def gs_act8_decode(q, e, x, stream=None):
    """Reads a checkpoint's values into x [tokens, channels]."""
    _mat(x, "x")
    ck = _act8(q, e, *x.shape, name="x")
    _check("gs_act8_decode", lib().gs_act8_decode(
        x.shape[0], x.shape[1], DTYPES[x.dtype], ck.q, ck.q_stride, ck.e, ck.e_stride,
        x.data_ptr(), x.stride(0), _stream(stream)))


def gs_glu_fwd(gate, up, h, gate_q=None, gate_e=None, up_q=None, up_e=None, act="silu",
               stream=None):
    """h = act(gate) * up (up None: act(gate)), and the 8-bit checkpoints of
    gate and up where their arrays are given."""
    _mat(gate, "gate")
    shape = tuple(gate.shape)
    if up is not None:
        _mat(up, "up", shape, gate.dtype)
    _mat(h, "h", shape, gate.dtype)
    g8 = _act8(gate_q, gate_e, *shape, name="gate") if gate_q is not None else _Ckpt()
    u8 = _act8(up_q, up_e, *shape, name="up") if up_q is not None else _Ckpt()
    _check("gs_glu_fwd", lib().gs_glu_fwd(
        shape[0], shape[1], DTYPES[gate.dtype], ACTS[act], gate.data_ptr(), gate.stride(0),
        _ptr(up), 0 if up is None else up.stride(0), h.data_ptr(), h.stride(0), C.byref(g8),
        C.byref(u8), _stream(stream)))


def gs_glu_bwd(gate_q, gate_e, up_q, up_e, dh, dgate, dup, h_q=None, h_e=None, act="silu",
               stream=None):
    """Gradients of gate and up at the checkpoints' values; h_q, h_e: the
    checkpoint of h at those values, for the next product's weight gradient.
    up_q, up_e, dup None: a unit without up."""
    _mat(dh, "dh")
    shape = tuple(dh.shape)
    _mat(dgate, "dgate", shape, dh.dtype)
    if dup is not None:
        _mat(dup, "dup", shape, dh.dtype)
    g8 = _act8(gate_q, gate_e, *shape, name="gate")
    u8 = _act8(up_q, up_e, *shape, name="up") if up_q is not None else _Ckpt()
    h8 = _act8(h_q, h_e, *shape, name="h") if h_q is not None else _Ckpt()
    _check("gs_glu_bwd", lib().gs_glu_bwd(
        shape[0], shape[1], DTYPES[dh.dtype], ACTS[act], C.byref(g8), C.byref(u8), dh.data_ptr(),
        dh.stride(0), dgate.data_ptr(), dgate.stride(0), _ptr(dup),
        0 if dup is None else dup.stride(0), C.byref(h8), _stream(stream)))


def gs_act8_wgrad_workspace_bytes(tokens, rows, channels, dtype=torch.bfloat16):
    return int(lib().gs_act8_wgrad_workspace_bytes(tokens, rows, channels, DTYPES[dtype]))


def gs_act8_wgrad(dy, q, e, dw, workspace, accumulate=False, stream=None):
    """dw [rows, channels] (float32 or bfloat16) = dy^T [rows, tokens] times
    the values of the checkpoint (q, e) of [tokens, channels]; accumulate adds
    to dw.  workspace: uint8, gs_act8_wgrad_workspace_bytes() bytes, its first
    256 zero before the first call."""
    _mat(dy, "dy")
    tokens, rows = dy.shape
    _mat(dw, "dw")
    if dw.shape[0] != rows:
        raise ValueError("dw has %d rows, dy %d columns" % (dw.shape[0], rows))
    if dw.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("dw: type %s" % dw.dtype)
    ck = _act8(q, e, tokens, dw.shape[1], name="x")
    _check("gs_act8_wgrad", lib().gs_act8_wgrad(
        tokens, rows, dw.shape[1], DTYPES[dy.dtype], dy.data_ptr(), dy.stride(0), ck.q,
        ck.q_stride, ck.e, ck.e_stride, dw.data_ptr(), dw.stride(0), DTYPES[dw.dtype],
        int(bool(accumulate)), _vec(workspace, "workspace", workspace.numel(), torch.uint8),
        workspace.numel(), _stream(stream)))
