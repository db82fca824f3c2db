"""Network operators (include/gs_net.h): multi-axis rotary positions, gated
norms, 8-bit activation checkpoints, the gated feed-forward block and linear
attention with decays, for a network that predicts Gaussians from views.  As in
the package itself, each gs_* function only checks and marshals its arguments and
calls the C ABI function of the same name.

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
    L.gs_ffn_workspace_bytes.argtypes = [i64, i32, i32, i32]
    L.gs_ffn_workspace_bytes.restype = sz
    L.gs_ffn_fwd.argtypes = [i64, i32, i32, i32, i32, vp, i64, vp, i64, vp, i64, vp, sz, vp]
    L.gs_ffn_bwd.argtypes = [i64, i32, i32, i32, i32, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64,
                             i32, i32, vp, sz, vp]
    L.gs_linear_attn_workspace_bytes.argtypes = [vp, i32]
    L.gs_linear_attn_workspace_bytes.restype = sz
    L.gs_linear_attn_fwd.argtypes = [vp, vp, vp, vp, sz, vp]
    L.gs_linear_attn_bwd.argtypes = [vp, vp, vp, vp, vp, sz, vp]
    L.gs_linear_attn_step.argtypes = [vp, vp, vp, vp]
    L.gs_linear_attn_status.argtypes = [vp]


from . import _check, lib  # noqa: E402  (the package defines these first)

# A call's cost on the host is most of a small call's time, so what every call
# does is kept short: one comparison per property, structures packed in one go.
_NORM = struct.Struct("qiiiiifPPPPP")
_HEADS = struct.Struct("PPqqqqi4x")
_CKPT = struct.Struct("PPqq")
_NO_CKPT = _CKPT.pack(0, 0, 0, 0)
_ATTN = struct.Struct("qiiiiiifPPP")
_ATTN_HEADS4, _ATTN_HEADS7 = struct.Struct("Pqq" * 4), struct.Struct("Pqq" * 7)
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


# --------------------------------------------------------------------------
# the gated feed-forward block

# (a tensor's device is -1 on the CPU, so that one comparison says both that it is on a
# GPU and on which)


def _refuse_device(t, name, device):
    raise ValueError("%s is on %s, not on cuda:%d" % (name, getattr(t, "device", "no device"), device))


def _workspace(t, device):
    """(pointer, size) of a workspace."""
    try:
        if t.dtype is torch.uint8 and t.get_device() == device and t.is_contiguous():
            return t.data_ptr(), t.numel()
    except AttributeError:
        pass
    if t is None:
        return 0, 0
    raise ValueError("workspace must be a contiguous uint8 tensor on cuda:%d" % device)


def gs_ffn_workspace_bytes(tokens, channels, hidden, backward=True):
    return int(lib().gs_ffn_workspace_bytes(tokens, channels, hidden, 1 if backward else 0))


def _ffn_args(x, w, h, name, workspace, act):
    """Checks what both directions have: the C call's arguments up to h's, and the workspace's."""
    try:
        dt, device = x.dtype, x.get_device()
        tokens, c = x.shape
        rows, wc = w.shape
        (xs, x1), (ws, w1), (hs, h1) = x.stride(), w.stride(), h.stride()
        hidden = rows // 2
        if ((dt is torch.bfloat16 or dt is torch.float16) and w.dtype is dt and h.dtype is dt and wc == c
                and rows > 0 and not rows & 1 and h.shape == (tokens, hidden)
                and device == w.get_device() == h.get_device() >= 0
                and (x1 == 1 or c == 1 or not tokens) and (w1 == 1 or c == 1)
                and (h1 == 1 or hidden == 1 or not tokens)):
            return ((tokens, c, hidden, DTYPES[dt], ACTS[act], x.data_ptr(), xs, w.data_ptr(), ws, h.data_ptr(), hs),
                    _workspace(workspace, device))
    except (AttributeError, TypeError, KeyError):
        if act not in ACTS:
            raise ValueError("act: one of %s" % ", ".join(ACTS)) from None
    except ValueError as e:
        if "unpack" not in str(e):
            raise
    # something is wrong: say what
    (tokens, c), code = _first(x, "x")
    if code == 2:
        raise ValueError("x: bfloat16 or float16")
    if getattr(w, "dim", int)() != 2 or w.shape[0] % 2 or not w.shape[0]:
        raise ValueError("w must be [2 * hidden, channels]")
    _mat(w, "w", (w.shape[0], c), x.dtype)
    _mat(h, name, (tokens, w.shape[0] // 2), x.dtype)
    for t, n in ((w, "w"), (h, name)):
        if t.get_device() != x.get_device():
            _refuse_device(t, n, x.get_device())
    raise ValueError("x, w, %s: not as documented" % name)


def gs_ffn_fwd(x, w, h, workspace, act="silu", stream=None):
    """h [tokens, hidden] = act(x w_gate^T) * (x w_up^T) in one kernel, with w [2 * hidden,
    channels] the gate's rows and then up's; bfloat16 or float16.  workspace: uint8,
    gs_ffn_workspace_bytes() bytes, its first 256 zero before the first call."""
    args, ws = _ffn_args(x, w, h, "h", workspace, act)
    status = lib().gs_ffn_fwd(*args, *ws, _stream(stream, x))
    if status:
        _check("gs_ffn_fwd", status)


def gs_ffn_bwd(x, w, dh, dx, dw, workspace, act="silu", accumulate=False, stream=None):
    """From dh, the gradient of h: dx [tokens, channels] and dw [2 * hidden, channels] (of
    x's type or float32; accumulate adds to it); either may be None.  Gate and up are
    formed again from x, so that nothing else is kept from the forward pass."""
    args, ws = _ffn_args(x, w, dh, "dh", workspace, act)
    d, ds = _opt(dx, "dx", x.shape, x.dtype)
    g, gs_, code = None, 0, args[3]
    if dw is not None:
        if dw.dtype is not x.dtype and dw.dtype is not torch.float32:
            raise ValueError("dw: type %s" % dw.dtype)
        _mat(dw, "dw", w.shape, dw.dtype)
        g, gs_, code = dw.data_ptr(), dw.stride(0), DTYPES[dw.dtype]
    device = x.get_device()
    for t, n in ((dx, "dx"), (dw, "dw")):
        if t is not None and t.get_device() != device:
            _refuse_device(t, n, device)
    _check("gs_ffn_bwd", lib().gs_ffn_bwd(*args, d, ds, g, gs_, code, 1 if accumulate else 0, *ws,
                                          _stream(stream, x)))


# --------------------------------------------------------------------------
# linear attention


def _attn(q, k, v, out, name, log_decay, group_offsets, state, scale):
    """Checks what every call has: (the packed gs_linear_attn, pointers and strides of q, k,
    v and out, shape of the states, device)."""
    try:
        dt, device = q.dtype, q.get_device()
        tokens, hq, dim = q.shape
        tk, hk, dk = k.shape
        tv, hv, vdim = v.shape
        (qa, qb, q1), (ka, kb, k1), (va, vb, v1), (oa, ob, o1) = q.stride(), k.stride(), v.stride(), out.stride()
        if ((dt is torch.bfloat16 or dt is torch.float16) and k.dtype is dt and v.dtype is dt and out.dtype is dt
                and tk == tokens == tv and dk == dim and dim and hk == hv and hk and hq and not hq % hk
                and out.shape == (tokens, hq, vdim)
                and device == k.get_device() == v.get_device() == out.get_device() >= 0
                and ((q1 == k1 == v1 == o1 == 1) or not tokens
                     or ((q1 == k1 == 1 or dim == 1) and (v1 == o1 == 1 or vdim == 1)))):
            groups = 1 if group_offsets is None else group_offsets.numel() - 1
            if groups < 1:
                raise ValueError("group_offsets must have groups + 1 entries")
            states = (groups, hq, dim, vdim)
            return (_ATTN.pack(tokens, hq, hk, dim, vdim, groups, DTYPES[dt], dim ** -0.5 if scale is None else scale,
                               _entries(log_decay, "log_decay", (hq,), torch.float32, device),
                               0 if group_offsets is None else
                               _entries(group_offsets, "group_offsets", (groups + 1,), torch.int32, device),
                               0 if state is None else _entries(state, "state", states, torch.float32, device)),
                    (q.data_ptr(), qa, qb, k.data_ptr(), ka, kb, v.data_ptr(), va, vb, out.data_ptr(), oa, ob),
                    states, device)
    except (AttributeError, TypeError):
        pass
    except ValueError as e:
        if "unpack" not in str(e):
            raise
    # something is wrong: say what
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.dim() != 3 or not t.is_cuda or DTYPES.get(t.dtype, 2) == 2:
            raise ValueError("%s must be a CUDA [tokens, heads, dim] tensor of bfloat16 or float16" % n)
    tokens, hq, dim = q.shape
    hk, vdim = k.shape[1], v.shape[2]
    if not hk or not hq or hq % hk:
        raise ValueError("%d query heads do not share %d key heads evenly" % (hq, hk))
    if not dim:
        raise ValueError("q: heads without channels")
    for t, n, shape in ((q, "q", (tokens, hq, dim)), (k, "k", (tokens, hk, dim)), (v, "v", (tokens, hk, vdim)),
                        (out, name, (tokens, hq, vdim))):
        _attn_heads(t, n, shape, q.dtype, q.get_device())
    raise ValueError("q, k, v, %s: not as documented" % name)


def _attn_heads(t, name, shape, dtype, device):
    """(pointer, stride between tokens, between heads)."""
    try:
        a, b, c = t.stride()
        if (t.shape == shape and t.dtype is dtype and t.get_device() == device >= 0
                and (c == 1 or shape[2] == 1 or not shape[0])):
            return t.data_ptr(), a, b
    except (AttributeError, ValueError, TypeError):
        pass
    if getattr(t, "shape", None) == shape and t.dtype is dtype and t.is_cuda:
        if t.get_device() != device:
            _refuse_device(t, name, device)
        raise ValueError("%s: the last axis must be contiguous" % name)
    raise ValueError("%s must be a CUDA %s tensor %s" % (name, dtype, list(shape)))


def _entries(t, name, shape, dtype, device):
    """The pointer of a contiguous tensor of that shape; 0 for None."""
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        if t is None:
            return 0
    raise ValueError("%s must be a contiguous %s tensor %s on q's device" % (name, dtype, list(shape)))


def gs_linear_attn_workspace_bytes(tokens, q_heads, k_heads, dim, vdim, groups=1, backward=True):
    """What a call needs at most (0: refused); less where every row starts on a 16-byte boundary."""
    return int(lib().gs_linear_attn_workspace_bytes(
        _ATTN.pack(tokens, q_heads, k_heads, dim, vdim, groups, 0, 1.0, 0, 0, 0), 1 if backward else 0))


def gs_linear_attn_fwd(q, k, v, log_decay, out, group_offsets=None, state=None, state_out=None, scale=None,
                       workspace=None, stream=None):
    """out [tokens, q_heads, vdim]: S <- e^log_decay S + k v^T, out = scale q S token after
    token (scale: dim ** -0.5 where none is given), for q [tokens, q_heads, dim], k [tokens,
    k_heads, dim], v [tokens, k_heads, vdim] of bfloat16 or float16 and log_decay float32
    [q_heads], 0 or less.  Groups of tokens (group_offsets int32 [groups + 1]; None: one)
    each go from their state to state_out, float32 [groups, q_heads, dim, vdim] (None: zeros;
    not wanted).  workspace: uint8, gs_linear_attn_workspace_bytes() bytes."""
    a, heads, states, device = _attn(q, k, v, out, "out", log_decay, group_offsets, state, scale)
    status = lib().gs_linear_attn_fwd(
        a, _ATTN_HEADS4.pack(*heads),
        0 if state_out is None else _entries(state_out, "state_out", states, torch.float32, device),
        *_workspace(workspace, device), _stream(stream, q))
    if status:
        _check("gs_linear_attn_fwd", status)


def gs_linear_attn_bwd(q, k, v, log_decay, dout, dq, dk, dv, group_offsets=None, state=None, dstate_out=None,
                       dstate=None, scale=None, workspace=None, stream=None):
    """Backward of gs_linear_attn_fwd from its inputs, dout and (None: zeros) the gradient of
    its last states: dq, dk, dv and, where given, dstate, the gradient of the first states."""
    a, heads, states, device = _attn(q, k, v, dout, "dout", log_decay, group_offsets, state, scale)
    dt, f32 = q.dtype, torch.float32
    _check("gs_linear_attn_bwd", lib().gs_linear_attn_bwd(
        a, _ATTN_HEADS7.pack(*heads, *_attn_heads(dq, "dq", q.shape, dt, device),
                             *_attn_heads(dk, "dk", k.shape, dt, device), *_attn_heads(dv, "dv", v.shape, dt, device)),
        _entries(dstate_out, "dstate_out", states, f32, device), _entries(dstate, "dstate", states, f32, device),
        *_workspace(workspace, device), _stream(stream, q)))


def gs_linear_attn_step(q, k, v, log_decay, state, out, scale=None, stream=None):
    """One token of each of q.shape[0] streams: updates state, float32 [streams, q_heads, dim,
    vdim], in place and writes out [streams, q_heads, vdim]."""
    a, heads, states, device = _attn(q, k, v, out, "out", log_decay, None, None, scale)
    status = lib().gs_linear_attn_step(
        a, _ATTN_HEADS4.pack(*heads),
        _entries(state, "state", (q.shape[0],) + states[1:], torch.float32, device), _stream(stream, q))
    if status:
        _check("gs_linear_attn_step", status)


def gs_linear_attn_status(stream=None):
    """Synchronises, and raises if a wait for the tensor cores ran out on the current device."""
    s = torch.cuda.current_stream() if stream is None else stream
    _check("gs_linear_attn_status", lib().gs_linear_attn_status(s.cuda_stream))
