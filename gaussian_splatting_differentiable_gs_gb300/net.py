"""Network operators (include/gs_net.h): multi-axis rotary positions, gated
norms and 8-bit activation checkpoints, for a network that predicts Gaussians
from views.  As in the package itself, each gs_* function only checks and
marshals its arguments and calls the C ABI function of the same name.

Matrices are CUDA tensors [tokens, channels] whose last axis is contiguous;
rows may have any stride (a slice of a packed projection, say).

Results go into the tensors that the caller gives.  The calls are not autograd
functions: a tensor that requires a gradient is taken as it is and gets none; each
operator's backward pass is a call of its own (examples/predict_gaussians.py chains
them)."""
import ctypes as C
import struct

import torch

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
GROUP = 32
NORM_POST, NORM_CENTER = 1, 2
ACTS = {"silu": 0, "gelu": 1}
ROPE_MAX_AXES = 4


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


from . import _check, lib  # noqa: E402  (the package defines these first)

# A call's cost on the host is most of a small call's time, so what every call
# does is kept short: one comparison per property, structures packed in one go.
_NORM = struct.Struct("qiiiiifPPPPP")
_HEADS = struct.Struct("PPqqqqi4x")
_CKPT = struct.Struct("PPqq")
_NO_CKPT = _CKPT.pack(0, 0, 0, 0)
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _stream(stream, t):
    """The given stream, or the current one; kernels run on the current device."""
    device = t.get_device()
    if device != _current_device():
        raise ValueError("tensors on cuda:%d, but the current device is cuda:%d"
                         % (device, _current_device()))
    return _raw_stream(device) if stream is None else stream.cuda_stream


def _refuse_mat(t, name, shape, dtype):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 2:
        raise ValueError("%s must be a CUDA matrix" % name)
    if shape is not None and t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype != dtype:
        raise ValueError("%s is %s, expected %s" % (name, t.dtype, dtype))
    raise ValueError("%s: the last axis must be contiguous" % name)


def _mat(t, name, shape, dtype):
    """Checks a CUDA matrix with a contiguous last axis, of the given shape and type."""
    try:
        if (t.shape == shape and t.dtype is dtype and t.is_cuda
                and (t.stride(1) == 1 or shape[1] == 1 or shape[0] == 0)):
            return t
    except (AttributeError, IndexError, TypeError):
        pass
    return _refuse_mat(t, name, shape, dtype)


def _first(t, name):
    """Checks a call's first matrix, which sets the shape: (shape, type's number)."""
    code = DTYPES.get(getattr(t, "dtype", None))
    if code is None or not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError("%s must be a CUDA matrix of bfloat16, float16 or float32" % name)
    _mat(t, name, t.shape, t.dtype)
    return t.shape, code


def _vec(t, name, n, dtype=torch.float32):
    if t is None:
        return 0
    try:
        if t.dtype is dtype and t.is_cuda and t.numel() == n and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    raise ValueError("%s must be a contiguous CUDA %s tensor of %d entries" % (name, dtype, n))


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
    """Checks a checkpoint's arrays: (q, q's stride, e, e's stride)."""
    groups = -(-channels // GROUP)
    _mat(q, name, (tokens, groups * GROUP), torch.int8)
    _mat(e, name, (tokens, groups), torch.uint8)
    return q.data_ptr(), q.stride(0), e.data_ptr(), e.stride(0)


def _ckpt(q, e, tokens, channels, name):
    if q is None and e is None:
        return _NO_CKPT
    qp, qs, ep, es = _act8(q, e, tokens, channels, name)
    return _CKPT.pack(qp, ep, qs, es)


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
        self.interleaved = 1 if interleaved else 0
        self._dims = (C.c_int32 * n)(*self.dims)
        self.turns = (C.c_uint64 * max(1, sum(self.dims) // 2))()
        _check("gs_rope_turns", lib().gs_rope_turns(
            n, self._dims, (C.c_double * n)(*base), (C.c_double * n)(*scale), self.turns))


def _heads(src, dst, name, like):
    """Checks one set of heads and packs its gs_heads."""
    try:
        shape = src.shape
        if not (src.dtype is like.dtype and dst.dtype is like.dtype and src.is_cuda and dst.is_cuda
                and dst.shape == shape and len(shape) == 3 and shape[0] == like.shape[0]
                and shape[2] == like.shape[2]):
            raise ValueError("%s must be CUDA %s tensors [%d, heads, %d]"
                             % (name, like.dtype, like.shape[0], like.shape[-1]))
    except AttributeError:
        raise ValueError("%s must be a CUDA [tokens, heads, head_dim] tensor" % name) from None
    (it, ih, i1), (ot, oh, o1) = src.stride(), dst.stride()
    if (i1 != 1 or o1 != 1) and shape[2] > 1 and src.numel():
        raise ValueError("%s: the last axis must be contiguous" % name)
    a, b = src.data_ptr(), dst.data_ptr()
    # (tensors without entries have no address)
    if a == b and a and ((it != ot and shape[0] > 1) or (ih != oh and shape[1] > 1)):
        raise ValueError("%s: in place with other strides" % name)
    return _HEADS.pack(a, b, it, ih, ot, oh, shape[1])


def gs_rope(rope, positions, q, k=None, q_out=None, k_out=None, inverse=False, stream=None):
    """Rotates q (and k) [tokens, heads, head_dim] by the positions [tokens,
    axes] (int32); in place where no output is given.  inverse: the opposite
    rotation, which is the backward pass.  Returns (q_out, k_out)."""
    code = DTYPES.get(getattr(q, "dtype", None))
    if code is None or q.dim() != 3:
        raise ValueError("q must be a CUDA [tokens, heads, head_dim] tensor")
    if q_out is None:
        q_out = q
    sets, n_sets = _heads(q, q_out, "q", q), 1
    if k is not None:
        if k_out is None:
            k_out = k
        sets, n_sets = sets + _heads(k, k_out, "k", q), 2
    elif k_out is not None:
        raise ValueError("k_out without k")
    tokens, n = q.shape[0], len(rope.dims)
    pos = _vec(positions, "positions", tokens * n, torch.int32)
    if positions.shape != (tokens, n):
        raise ValueError("positions must be [%d, %d]" % (tokens, n))
    _check("gs_rope", lib().gs_rope(tokens, n, rope._dims, rope.turns, rope.interleaved,
                                    1 if inverse else 0, pos, q.shape[2], code, sets, n_sets,
                                    _stream(stream, q)))
    return q_out, k_out


# --------------------------------------------------------------------------
# gated norms


def _norm_args(shape, code, res_code, dtype, w_pre, w_post, gate, group_offsets, res_scale, post,
               center, eps):
    """The packed gs_norm, and its number of groups."""
    c, groups, gp, op = shape[1], 1, 0, 0
    if gate is not None:
        if gate.dim() != 2 or gate.shape[1] != c or gate.shape[0] < 1:
            raise ValueError("gate must be [groups, channels]")
        groups = gate.shape[0]
        gp = _vec(gate, "gate", groups * c, dtype)
        if group_offsets is None and groups > 1:
            raise ValueError("gate: more than one group needs group_offsets")
        op = _vec(group_offsets, "group_offsets", groups + 1, torch.int32)
    elif group_offsets is not None:
        raise ValueError("group_offsets without a gate")
    return _NORM.pack(shape[0], c, groups, (NORM_POST if post else 0) | (NORM_CENTER if center else 0),
                      code, res_code, eps, _vec(w_pre, "w_pre", c), _vec(w_post, "w_post", c),
                      _vec(res_scale, "res_scale", c), gp, op), groups


def _opt(t, name, shape, dtype):
    """(pointer, row stride) of a matrix that may be None."""
    if t is None:
        return None, 0
    _mat(t, name, shape, dtype)
    return t.data_ptr(), t.stride(0)


def gs_gated_norm_fwd(x, block, x_out, y, stats, w_pre=None, w_post=None, gate=None,
                      group_offsets=None, res_scale=None, y_q=None, y_e=None, post=True,
                      center=False, eps=1e-6, stream=None):
    """x_out = x + res_scale * gate[group] * (w_post * norm(block)), y = w_pre
    * norm(x_out).  block, x_out None: y = w_pre * norm(x) only; y None: the
    sum only; post False: no norm of the block, and no w_post.  gate [groups, channels] with
    group_offsets int32 [groups + 1] (one group: None).  stats: float32
    [tokens, 4] for the backward.  y_q, y_e: y's 8-bit checkpoint."""
    shape, res_code = _first(x, "x")
    other = y if y is not None else block
    if other is None:
        raise ValueError("neither block nor y")
    dt = other.dtype
    if (y_q is None) != (y_e is None):
        raise ValueError("y_q and y_e come together")
    b, bs = _opt(block, "block", shape, dt)
    xo, xos = _opt(x_out, "x_out", shape, x.dtype)
    yp, ys = _opt(y, "y", shape, dt)
    q, qs, e, es = _act8(y_q, y_e, *shape, name="y's checkpoint") if y_q is not None else (None, 0, None, 0)
    p, _ = _norm_args(shape, DTYPES.get(dt, -1), res_code, dt, w_pre, w_post, gate, group_offsets,
                      res_scale, post, center, eps)
    _check("gs_gated_norm_fwd", lib().gs_gated_norm_fwd(
        p, x.data_ptr(), x.stride(0), b, bs, xo, xos, yp, ys, _vec(stats, "stats", 4 * shape[0]), q,
        qs, e, es, _stream(stream, x)))


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
    shape, res_code = _first(x_out, "x_out")
    other = dy if dy is not None else block
    if other is None:
        raise ValueError("neither block nor dy")
    dt, rt, c = other.dtype, x_out.dtype, shape[1]
    b, bs = _opt(block, "block", shape, dt)
    dxo, dxos = _opt(dx_out, "dx_out", shape, rt)
    dyp, dys = _opt(dy, "dy", shape, dt)
    dxp, dxs = _opt(dx, "dx", shape, rt)
    db, dbs = _opt(dblock, "dblock", shape, dt)
    p, groups = _norm_args(shape, DTYPES.get(dt, -1), res_code, dt, w_pre, w_post, gate,
                           group_offsets, res_scale, post, center, 0.0)
    size = 0 if workspace is None else workspace.numel()
    _check("gs_gated_norm_bwd", lib().gs_gated_norm_bwd(
        p, x_out.data_ptr(), x_out.stride(0), b, bs, _vec(stats, "stats", 4 * shape[0]), dxo, dxos,
        dyp, dys, dxp, dxs, db, dbs, _vec(dw_pre, "dw_pre", c), _vec(dw_post, "dw_post", c),
        _vec(dgate, "dgate", groups * c), _vec(dres_scale, "dres_scale", c),
        _vec(workspace, "workspace", size, torch.uint8), size, _stream(stream, x_out)))


# --------------------------------------------------------------------------
# 8-bit activation checkpoints


def gs_act8_encode(x, q, e, stream=None):
    """Writes the 8-bit checkpoint (q, e) of x [tokens, channels]."""
    (tokens, c), code = _first(x, "x")
    q, qs, e, es = _act8(q, e, tokens, c, "x's checkpoint")
    _check("gs_act8_encode", lib().gs_act8_encode(tokens, c, code, x.data_ptr(), x.stride(0), q, qs,
                                                  e, es, _stream(stream, x)))


def gs_act8_decode(q, e, x, stream=None):
    """Reads a checkpoint's values into x [tokens, channels]."""
    (tokens, c), code = _first(x, "x")
    q, qs, e, es = _act8(q, e, tokens, c, "x's checkpoint")
    _check("gs_act8_decode", lib().gs_act8_decode(tokens, c, code, q, qs, e, es, x.data_ptr(),
                                                  x.stride(0), _stream(stream, x)))


def gs_glu_fwd(gate, up, h, gate_q=None, gate_e=None, up_q=None, up_e=None, act="silu",
               stream=None):
    """h = act(gate) * up (up None: act(gate)), and the 8-bit checkpoints of
    gate and up where their arrays are given."""
    shape, code = _first(gate, "gate")
    u, us = _opt(up, "up", shape, gate.dtype)
    _mat(h, "h", shape, gate.dtype)
    g8 = _ckpt(gate_q, gate_e, *shape, name="gate's checkpoint")
    u8 = _ckpt(up_q, up_e, *shape, name="up's checkpoint")
    _check("gs_glu_fwd", lib().gs_glu_fwd(
        shape[0], shape[1], code, ACTS[act], gate.data_ptr(), gate.stride(0), u, us, h.data_ptr(),
        h.stride(0), g8, u8, _stream(stream, gate)))


def gs_glu_bwd(gate_q, gate_e, up_q, up_e, dh, dgate, dup, h_q=None, h_e=None, act="silu",
               stream=None):
    """Gradients of gate and up at the checkpoints' values; h_q, h_e: the
    checkpoint of h at those values, for the next product's weight gradient.
    up_q, up_e, dup None: a unit without up."""
    shape, code = _first(dh, "dh")
    _mat(dgate, "dgate", shape, dh.dtype)
    u, us = _opt(dup, "dup", shape, dh.dtype)
    g8 = _ckpt(gate_q, gate_e, *shape, name="gate's checkpoint")
    u8 = _ckpt(up_q, up_e, *shape, name="up's checkpoint")
    h8 = _ckpt(h_q, h_e, *shape, name="h's checkpoint")
    _check("gs_glu_bwd", lib().gs_glu_bwd(
        shape[0], shape[1], code, ACTS[act], g8, u8, dh.data_ptr(), dh.stride(0), dgate.data_ptr(),
        dgate.stride(0), u, us, h8, _stream(stream, dh)))


def gs_act8_wgrad_workspace_bytes(tokens, rows, channels, dtype=torch.bfloat16):
    return int(lib().gs_act8_wgrad_workspace_bytes(tokens, rows, channels, DTYPES[dtype]))


def gs_act8_wgrad(dy, q, e, dw, workspace, accumulate=False, stream=None):
    """dw [rows, channels] (float32 or bfloat16) = dy^T [rows, tokens] times
    the values of the checkpoint (q, e) of [tokens, channels]; accumulate adds
    to dw.  workspace: uint8, gs_act8_wgrad_workspace_bytes() bytes, its first
    256 zero before the first call."""
    (tokens, rows), code = _first(dy, "dy")
    (n, c), out_code = _first(dw, "dw")
    if n != rows:
        raise ValueError("dw has %d rows, dy %d columns" % (n, rows))
    if dw.dtype is torch.float16:
        raise ValueError("dw: type %s" % dw.dtype)
    q, qs, e, es = _act8(q, e, tokens, c, "x's checkpoint")
    size = workspace.numel()
    _check("gs_act8_wgrad", lib().gs_act8_wgrad(
        tokens, rows, c, code, dy.data_ptr(), dy.stride(0), q, qs, e, es, dw.data_ptr(),
        dw.stride(0), out_code, 1 if accumulate else 0,
        _vec(workspace, "workspace", size, torch.uint8), size, _stream(stream, dy)))
