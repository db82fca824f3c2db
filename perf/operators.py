"""The network operators that are measured, case by case.

The cases come from a network that predicts Gaussians from views: a token per 16x16 pixel tile (256x256 images: 256
tokens; one 1080p view: 120 x 68 = 8160; the four views of the ring scene: 32640), widths and head counts generic.

  rope   rotary positions with several axes on queries and keys, forward and backward (the inverse rotation)
  norm   norm after a block, gate, residual scale, residual sum and norm before the next block; forward, backward
  act8   activation checkpoints in 8 bits: written and read back ("encode"); a gated unit's forward that keeps only the
         checkpoint and its backward from it ("glu"); the weight gradient from a checkpoint ("wgrad")

A checkpoint holds, per token, groups of 32 channels: signed bytes q and one biased exponent e, value = q * 2^(e - 127),
e the smallest (>= 1) with the group's largest magnitude <= 127 * 2^(e - 127); q is rounded to nearest, ties to even.
Rows are padded with zeros to whole groups.
"""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GROUP = 32
EPS = 1e-6


def listed():
    return [
        # a 256x256 image's tokens, every head small: a call's latency
        dict(name="rope_tiny_f16", op="rope", tokens=256, q_heads=6, k_heads=6, head_dim=64, axes="32,32",
             interleaved=False, inverse=False, dtype="f16"),
        # one 1080p view, queries and keys inside the packed projection, shared key heads
        dict(name="rope_view_bf16", op="rope", tokens=8160, q_heads=16, k_heads=4, head_dim=64, axes="16,24,24",
             interleaved=False, inverse=False, dtype="bf16"),
        # gradients of four views' queries and keys, neighbouring pairs, part of the head left unrotated
        dict(name="rope_ring_bwd_f32", op="rope", tokens=32640, q_heads=12, k_heads=12, head_dim=80, axes="20,26,26",
             interleaved=True, inverse=True, dtype="f32"),
        # the tiny image again, centred norms, the checkpoint of y written and read back
        dict(name="norm_tiny_fwd_f16", op="norm", dir="fwd", tokens=256, width=384, groups=1, center=True, post=True,
             gate=True, scale=True, ckpt=True, dtype="f16", res="f16"),
        # four views, a gate per view
        dict(name="norm_ring_fwd_bf16", op="norm", dir="fwd", tokens=32640, width=1024, groups=4, center=False,
             post=True, gate=True, scale=True, ckpt=False, dtype="bf16", res="bf16"),
        dict(name="norm_ring_bwd_bf16", op="norm", dir="bwd", tokens=32640, width=1024, groups=4, center=False,
             post=True, gate=True, scale=True, ckpt=False, dtype="bf16", res="bf16"),
        # views of different sizes (one of them empty), an odd width, in 32 bits
        dict(name="norm_ragged_bwd_f32", op="norm", dir="bwd", tokens=5003, width=997, groups=7, center=True,
             post=True, gate=True, scale=True, ckpt=False, dtype="f32", res="f32"),
        # the smallest checkpoint
        dict(name="act8_tiny_encode_bf16", op="act8", kind="encode", tokens=256, width=384, dtype="bf16"),
        # a gated unit's training pass over four views: only the 8-bit checkpoint lives between the two directions
        dict(name="act8_ring_glu_bf16", op="act8", kind="glu", tokens=32640, width=2816, act="silu", dtype="bf16"),
        # the same at an odd width
        dict(name="act8_odd_glu_f16", op="act8", kind="glu", tokens=8160, width=1361, act="gelu", dtype="f16"),
        # weight gradient of the gated unit's input projection
        dict(name="act8_ring_wgrad_bf16", op="act8", kind="wgrad", tokens=32640, rows=5632, width=1024, dtype="bf16",
             out="f32"),
        # weight gradient of the head that writes the 59 parameters of a Gaussian, its gradient in 32 bits
        dict(name="act8_head_wgrad_f32", op="act8", kind="wgrad", tokens=8160, rows=59, width=1024, dtype="f32",
             out="f32"),
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of its range; whole multiples of 8 half of the time."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        v = max(lo, v // 8 * 8)
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["rope", "norm", "norm", "act8", "act8", "act8"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "rope":
        head_dim, axes = rng.choice([(32, "8,12,12"), (64, "32,32"), (64, "16,24,24"), (80, "20,26,26"),
                                     (96, "32,32,32"), (128, "32,48,48"), (72, "12,12,12,12"), (64, "64")])
        k_heads = rng.choice([1, 2, 4, 6, 8])
        q_heads = k_heads * rng.choice([1, 2, 4])
        cap = 32640 * 24 * 80 // ((q_heads + k_heads) * head_dim)
        return dict(op="rope", tokens=_size(rng, 1, min(32640, cap)), q_heads=q_heads, k_heads=k_heads,
                    head_dim=head_dim, axes=axes, interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5,
                    dtype=dtype)
    if op == "norm":
        width = _size(rng, 32, 4096)
        tokens = _size(rng, 1, min(32640, 32640 * 1024 // width))
        return dict(op="norm", dir=rng.choice(["fwd", "bwd"]), tokens=tokens, width=width,
                    groups=rng.choice([1, 2, 4, 7, 16]), center=rng.random() < 0.5, post=rng.random() < 0.8,
                    gate=rng.random() < 0.8, scale=rng.random() < 0.8, ckpt=rng.random() < 0.3, dtype=dtype,
                    res="f32" if rng.random() < 0.3 else dtype)
    kind = rng.choice(["encode", "glu", "wgrad"])
    if kind == "encode":
        width = _size(rng, 1, 4096)
        return dict(op="act8", kind="encode", tokens=_size(rng, 1, min(32640, 32640 * 2816 // width)), width=width,
                    dtype=dtype)
    if kind == "glu":
        width = _size(rng, 16, 5632)
        return dict(op="act8", kind="glu", tokens=_size(rng, 1, min(32640, 32640 * 2816 // width)), width=width,
                    act=rng.choice(["silu", "gelu"]), dtype=dtype)
    rows, width = _size(rng, 1, 5632), _size(rng, 16, 4096)
    return dict(op="act8", kind="wgrad", tokens=_size(rng, 1, min(32640, 32640 * 5632 * 1024 // (rows * width))),
                rows=rows, width=width, dtype=dtype, out=rng.choice(["f32", "bf16"]))


# ------------------------------------------------------------------------------------------------------------------
# inputs


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _activations(g, tokens, width, dtype):
    """Activations: unit normal with a few channels ten times as large, as residual streams and units have them."""
    x = _normal(g, tokens, width)
    x *= torch.where(torch.rand(width, generator=g, device="cuda") < 0.01, 10.0, 1.0)
    return x.to(dtype)


def _offsets(case, g):
    """Where each group's (view's) tokens begin: equal parts for up to four groups, else ragged with an empty one."""
    T, G = case["tokens"], case["groups"]
    if G <= 4:
        cuts = [T * i // G for i in range(G + 1)]
        return torch.tensor(cuts, dtype=torch.int32, device="cuda")
    cuts = torch.randint(0, T + 1, (G - 1,), generator=g, device="cuda").sort().values
    cuts[1] = cuts[0]
    ends = torch.tensor([0, T], device="cuda")
    return torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)


def _positions(tokens, axes):
    """(view, row, column) of each token on grids 120 wide and 68 high (16 x 16 for a 256 x 256 image)."""
    w, h = (16, 16) if tokens <= 256 else (120, 68)
    t = torch.arange(tokens, device="cuda")
    cols = [t // (w * h), t % (w * h) // w, t % w, t % 5]
    pick = {1: [2], 2: [1, 2], 3: [0, 1, 2], 4: [0, 1, 2, 3]}[axes]
    return torch.stack([cols[i] for i in pick], 1).to(torch.int32).contiguous()


def _padded(width):
    return -(-width // GROUP) * GROUP


def _encode(x):
    """(q, e) of the checkpoint of x [tokens, width]."""
    tokens, width = x.shape
    x = torch.nn.functional.pad(x.float(), (0, _padded(width) - width)).view(tokens, -1, GROUP)
    big = x.abs().amax(2).contiguous()
    bits = big.view(torch.int32)
    e = (bits >> 23) - 6 + ((bits & 0x7FFFFF) > 0x7E0000).to(torch.int32)
    e = e.clamp(min=1)
    inv = ((254 - e) << 23).view(torch.float32)
    q = torch.round(x * inv[:, :, None]).to(torch.int8)
    return q.view(tokens, -1), e.to(torch.uint8)


def _decode(q, e, width, dtype):
    """The values that a checkpoint stands for."""
    step = (e.to(torch.int32) << 23).view(torch.float32)
    x = q.view(q.shape[0], -1, GROUP).float() * step[:, :, None]
    return x.view(q.shape[0], -1)[:, :width].to(dtype)


def _ckpt(tokens, width):
    ld = _padded(width)
    return (torch.empty(tokens, ld, dtype=torch.int8, device="cuda"),
            torch.empty(tokens, ld // GROUP, dtype=torch.uint8, device="cuda"))


def _stats(x, center):
    x = x.float()
    mean = x.mean(1) if center else torch.zeros_like(x[:, 0])
    return mean, torch.rsqrt((x - mean[:, None]).square().mean(1) + EPS)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, T, S = DTYPE[case["dtype"]], case["tokens"], {"case": case}
    if case["op"] == "rope":
        D, hq, hk = case["head_dim"], case["q_heads"], case["k_heads"]
        axes = [int(a) for a in case["axes"].split(",")]
        packed = _normal(g, T, hq + 2 * hk, D, dtype=dt)  # queries, keys, values of the projection
        S.update(q=packed[:, :hq], k=packed[:, hq:hq + hk], positions=_positions(T, len(axes)), dims=axes,
                 q_out=torch.empty(T, hq, D, dtype=dt, device="cuda"),
                 k_out=torch.empty(T, hk, D, dtype=dt, device="cuda"))
        return S
    if case["op"] == "norm":
        C, G, rt = case["width"], case["groups"], DTYPE[case["res"]]
        S["w_pre"] = 1 + _normal(g, C, std=0.1)
        S["w_post"] = 1 + _normal(g, C, std=0.1) if case["post"] else None
        S["scale"] = 0.3 + _normal(g, C, std=0.05) if case["scale"] else None
        S["gate"] = _normal(g, G, C, std=0.5, dtype=dt) if case["gate"] else None
        S["offsets"] = _offsets(case, g) if case["gate"] else None
        S["x"] = _activations(g, T, C, rt)  # backward: the sum that the forward wrote
        S["block"] = _activations(g, T, C, dt)
        if case["dir"] == "fwd":
            S.update(x_out=torch.empty(T, C, dtype=rt, device="cuda"), y=torch.empty(T, C, dtype=dt, device="cuda"),
                     stats=torch.empty(T, 4, device="cuda"))
            if case["ckpt"]:
                S["y_q"], S["y_e"] = _ckpt(T, C)
                S["y_back"] = torch.empty(T, C, dtype=dt, device="cuda")
        else:
            post = _stats(S["block"], case["center"]) if case["post"] else (torch.zeros(T, device="cuda"),) * 2
            S["stats"] = torch.stack([*post, *_stats(S["x"], case["center"])], 1).contiguous()
            S["dx_out"] = _normal(g, T, C, std=1e-2, dtype=rt)
            S["dy"] = _normal(g, T, C, std=1e-2, dtype=dt)
            S.update(dx=torch.empty(T, C, dtype=rt, device="cuda"), dblock=torch.empty(T, C, dtype=dt, device="cuda"),
                     dw_pre=torch.empty(C, device="cuda"),
                     dw_post=torch.empty(C, device="cuda") if case["post"] else None,
                     dscale=torch.empty(C, device="cuda") if case["scale"] else None,
                     dgate=torch.empty(G, C, device="cuda") if case["gate"] else None)
            # room for the column sums, kept from call to call
            S["workspace"] = torch.empty(8 * (2048 + G) * C + 256, dtype=torch.uint8, device="cuda")
        return S
    W = case["width"]
    if case["kind"] == "encode":
        S["x"] = _activations(g, T, W, dt)
        S["q"], S["e"] = _ckpt(T, W)
        S["out"] = torch.empty(T, W, dtype=dt, device="cuda")
    elif case["kind"] == "glu":
        packed = _activations(g, T, 2 * W, dt)  # gate and up of one projection
        S.update(gate=packed[:, :W], up=packed[:, W:], dh=_normal(g, T, W, std=1e-2, dtype=dt))
        S["gate_q"], S["gate_e"] = _ckpt(T, W)
        S["up_q"], S["up_e"] = _ckpt(T, W)
        S["h"] = torch.empty(T, W, dtype=dt, device="cuda")
        dpacked = torch.empty(T, 2 * W, dtype=dt, device="cuda")
        S["dgate"], S["dup"] = dpacked[:, :W], dpacked[:, W:]
    else:
        S["dy"] = _normal(g, T, case["rows"], std=1e-2, dtype=dt)
        S["q"], S["e"] = _encode(_activations(g, T, W, torch.bfloat16))
        S["dw"] = torch.empty(case["rows"], W, dtype=DTYPE[case["out"]], device="cuda")
        # room for partial sums and for the parts of a gradient that is not in 16 bits, kept from call to call
        S["workspace"] = torch.zeros(wgrad_room(case), dtype=torch.uint8, device="cuda")
    return S


def wgrad_room(case):
    """Three 16-bit parts of a padded gradient, and 128 MiB of partial sums."""
    rows, tokens = -(-case["rows"] // 256) * 256, -(-case["tokens"] // 64) * 64
    return 6 * tokens * rows + (128 << 20)


# ------------------------------------------------------------------------------------------------------------------
# one pass


def run(S):
    return (_own if own else _plain)[_kind(S["case"])](S)


def _kind(case):
    return {"rope": "rope", "norm": "norm_" + case.get("dir", ""), "act8": case.get("kind")}[case["op"]]


def _plain_rope(S):
    c = S["case"]
    out = []
    parts = []
    for a, d in enumerate(S["dims"]):
        f = 10000.0 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float32) / d)
        parts.append(S["positions"][:, a, None].float() * f)
    angle = torch.cat(parts, 1)[:, None, :]
    cos, sin = angle.cos(), angle.sin() * (-1.0 if c["inverse"] else 1.0)
    for x in (S["q"], S["k"]):
        y = x.float().clone()
        at, pair = 0, 0
        for d in S["dims"]:
            n = d // 2
            first = slice(at, at + d, 2) if c["interleaved"] else slice(at, at + n)
            second = slice(at + 1, at + d, 2) if c["interleaved"] else slice(at + n, at + d)
            u, v = x[..., first].float(), x[..., second].float()
            co, si = cos[..., pair:pair + n], sin[..., pair:pair + n]
            y[..., first] = u * co - v * si
            y[..., second] = u * si + v * co
            at, pair = at + d, pair + n
        out.append(y.to(x.dtype))
    return out


def _rows_of_gate(S):
    T = S["case"]["tokens"]
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    return torch.searchsorted(S["offsets"], t, right=True) - 1


def _plain_norm_fwd(S):
    c = S["case"]
    x, b = S["x"].float(), S["block"].float()
    T = c["tokens"]
    mean_b = rstd_b = torch.zeros(T, device="cuda")
    u = b
    if c["post"]:
        mean_b, rstd_b = _stats(b, c["center"])
        u = (b - mean_b[:, None]) * rstd_b[:, None] * S["w_post"]
    if c["scale"]:
        u = u * S["scale"]
    if c["gate"]:
        u = u * S["gate"].float()[_rows_of_gate(S)]
    x = x + u
    mean, rstd = _stats(x, c["center"])
    y = ((x - mean[:, None]) * rstd[:, None] * S["w_pre"]).to(S["y"].dtype)
    out = [x.to(S["x"].dtype), y, torch.stack([mean_b, rstd_b, mean, rstd], 1)]
    if c["ckpt"]:
        q, e = _encode(y)
        out.append(_decode(q, e, c["width"], y.dtype))
    return out


def _norm_back(h, n, rstd, center):
    back = h - n * (h * n).mean(1, keepdim=True)
    if center:
        back = back - h.mean(1, keepdim=True)
    return back * rstd[:, None]


def _plain_norm_bwd(S):
    c = S["case"]
    mean_b, rstd_b, mean, rstd = S["stats"].unbind(1)
    dy = S["dy"].float()
    n = (S["x"].float() - mean[:, None]) * rstd[:, None]
    d = S["dx_out"].float() + _norm_back(dy * S["w_pre"], n, rstd, c["center"])
    m = S["block"].float()
    if c["post"]:
        m = (m - mean_b[:, None]) * rstd_b[:, None]
    u = m * S["w_post"] if c["post"] else m
    k = torch.ones_like(S["w_pre"])[None]
    if c["gate"]:
        group = _rows_of_gate(S)
        k = S["gate"].float()[group]
    s = S["scale"] if c["scale"] else 1.0
    du = d * k * s
    db = _norm_back(du * S["w_post"], m, rstd_b, c["center"]) if c["post"] else du
    out = [d.to(S["dx"].dtype), db.to(S["dblock"].dtype), (dy * n).sum(0)]
    if c["post"]:
        out.append((du * m).sum(0))
    if c["scale"]:
        out.append((d * k * u).sum(0))
    if c["gate"]:
        of_group = (group[None] == torch.arange(c["groups"], device="cuda")[:, None]).float()
        out.append(of_group @ (d * s * u))
    return out


def _plain_encode(S):
    q, e = _encode(S["x"])
    return _decode(q, e, S["case"]["width"], S["x"].dtype)


def _act(x, name):
    """The unit's function and its derivative."""
    if name == "silu":
        s = torch.sigmoid(x)
        return x * s, s * (1 + x * (1 - s))
    phi = 0.5 * (1 + torch.erf(x * 0.5 ** 0.5))
    return x * phi, phi + x * torch.exp(-0.5 * x * x) * (0.5 / math.pi) ** 0.5


def _plain_glu(S):
    c = S["case"]
    dt = S["gate"].dtype
    f, _ = _act(S["gate"].float(), c["act"])
    h = (f * S["up"].float()).to(dt)
    gate = _decode(*_encode(S["gate"]), c["width"], torch.float32)
    up = _decode(*_encode(S["up"]), c["width"], torch.float32)
    f, df = _act(gate, c["act"])
    dh = S["dh"].float()
    return [h, (dh * up * df).to(dt), (dh * f).to(dt)]


def _plain_wgrad(S):
    x = _decode(S["q"], S["e"], S["case"]["width"], torch.float32)
    return (S["dy"].float().t() @ x).to(S["dw"].dtype)


_plain = {"rope": _plain_rope, "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "encode": _plain_encode,
          "glu": _plain_glu, "wgrad": _plain_wgrad}


def _gs():
    import gaussian_splatting_differentiable_gs_gb300 as gs
    return gs


def _own_rope(S):
    gs, c = _gs(), S["case"]
    if "rope" not in S:
        S["rope"] = gs.Rope(S["dims"], base=10000.0, interleaved=c["interleaved"])  # frequencies, kept with the network
    gs.gs_rope(S["rope"], S["positions"], S["q"], S["k"], q_out=S["q_out"], k_out=S["k_out"], inverse=c["inverse"])
    return [S["q_out"], S["k_out"]]


def _own_norm_fwd(S):
    gs, c = _gs(), S["case"]
    gs.gs_gated_norm_fwd(S["x"], S["block"], S["x_out"], S["y"], S["stats"], w_pre=S["w_pre"], w_post=S["w_post"],
                         gate=S["gate"], group_offsets=S["offsets"], res_scale=S["scale"], y_q=S.get("y_q"),
                         y_e=S.get("y_e"), post=c["post"], center=c["center"], eps=EPS)
    out = [S["x_out"], S["y"], S["stats"]]
    if c["ckpt"]:
        gs.gs_act8_decode(S["y_q"], S["y_e"], S["y_back"])
        out.append(S["y_back"])
    return out


def _own_norm_bwd(S):
    gs, c = _gs(), S["case"]
    gs.gs_gated_norm_bwd(S["x"], S["block"], S["stats"], S["dx_out"], S["dy"], S["dx"], S["dblock"],
                         w_pre=S["w_pre"], w_post=S["w_post"], gate=S["gate"], group_offsets=S["offsets"],
                         res_scale=S["scale"], dw_pre=S["dw_pre"], dw_post=S["dw_post"], dgate=S["dgate"],
                         dres_scale=S["dscale"], workspace=S["workspace"], post=c["post"], center=c["center"])
    return [t for t in (S["dx"], S["dblock"], S["dw_pre"], S["dw_post"], S["dscale"], S["dgate"]) if t is not None]


def _own_encode(S):
    gs = _gs()
    gs.gs_act8_encode(S["x"], S["q"], S["e"])
    gs.gs_act8_decode(S["q"], S["e"], S["out"])
    return S["out"]


def _own_glu(S):
    gs, act = _gs(), S["case"]["act"]
    kept = (S["gate_q"], S["gate_e"], S["up_q"], S["up_e"])
    gs.gs_glu_fwd(S["gate"], S["up"], S["h"], *kept, act=act)
    gs.gs_glu_bwd(*kept, S["dh"], S["dgate"], S["dup"], act=act)
    return [S["h"], S["dgate"], S["dup"]]


def _own_wgrad(S):
    _gs().gs_act8_wgrad(S["dy"], S["q"], S["e"], S["dw"], S["workspace"])
    return S["dw"]


_own = {"rope": _own_rope, "norm_fwd": _own_norm_fwd, "norm_bwd": _own_norm_bwd, "encode": _own_encode,
        "glu": _own_glu, "wgrad": _own_wgrad}


# ------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without, and its results in 64 bits


def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}
    b, T = size[case["dtype"]], case["tokens"]
    if case["op"] == "rope":
        n = T * (case["q_heads"] + case["k_heads"])
        axes = [int(a) for a in case["axes"].split(",")]
        return {"bytes": 2 * b * n * case["head_dim"] + 4 * T * len(axes), "flops": 3 * n * sum(axes)}
    if case["op"] == "norm":
        C, r = case["width"], size[case["res"]]
        gate = case["groups"] * C if case["gate"] else 0
        if case["dir"] == "fwd":  # x, block -> x', y; with a checkpoint its bytes out and in, and the values
            kept = T * (2 * (_padded(C) + _padded(C) // GROUP) + C * b) if case["ckpt"] else 0
            return {"bytes": T * C * (2 * r + 2 * b) + 16 * T + 12 * C + gate * b + kept, "flops": 14 * T * C}
        return {"bytes": T * C * (3 * r + 3 * b) + 16 * T + 24 * C + gate * (b + 4), "flops": 28 * T * C}
    W = case["width"]
    held = T * (_padded(W) + _padded(W) // GROUP)
    if case["kind"] == "encode":
        return {"bytes": 2 * T * W * b + 2 * held, "flops": 4 * T * W}
    if case["kind"] == "glu":  # gate, up -> h, checkpoint; checkpoint, dh -> dgate, dup
        return {"bytes": 6 * T * W * b + 4 * held, "flops": 40 * T * W}
    out = case["rows"] * W * size[case["out"]]
    return {"bytes": T * case["rows"] * b + held + out, "flops": 2 * T * case["rows"] * W}


def exact(case, seed):
    S = prepare(case, seed)
    return _exact[_kind(case)](S)


def _exact_rope(S):
    c = S["case"]
    sign = -1j if c["inverse"] else 1j
    out = []
    for x in (S["q"], S["k"]):
        whole = []
        at = 0
        for a, d in enumerate(S["dims"]):
            z = x[..., at:at + d].double()
            z = z.unflatten(-1, (d // 2, 2)) if c["interleaved"] else z.unflatten(-1, (2, d // 2)).transpose(-1, -2)
            f = torch.exp(-math.log(10000.0) * 2 / d * torch.arange(d // 2, device="cuda", dtype=torch.float64))
            turn = torch.exp(sign * (S["positions"][:, a].double()[:, None] * f))[:, None]
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
            z = z if c["interleaved"] else z.transpose(-1, -2)
            whole.append(z.flatten(-2))
            at += d
        out.append(torch.cat(whole + [x[..., at:].double()], -1))
    return out


def _exact_norm(S, leaf):
    """The forward in 64 bits: (x', y, statistics), from the tensors of `leaf`."""
    c = S["case"]

    def moments(v):
        m = v.mean(1, keepdim=True) if c["center"] else torch.zeros_like(v[:, :1])
        return m, ((v - m) ** 2).mean(1, keepdim=True).add(EPS).pow(-0.5)

    t = leaf["block"]
    none = torch.zeros_like(t[:, :1])
    first = (none, none)
    if c["post"]:
        first = moments(t)
        t = (t - first[0]) * first[1] * leaf["w_post"]
    if c["gate"]:
        counts = (S["offsets"][1:] - S["offsets"][:-1]).long()
        t = t * torch.repeat_interleave(leaf["gate"], counts, 0)
    if c["scale"]:
        t = t * leaf["scale"]
    return t, first, moments


def _leaves(S, grad):
    names = [k for k in ("block", "w_pre", "w_post", "scale", "gate") if S[k] is not None]
    return {k: S[k].double().requires_grad_(grad) for k in names}


def _exact_norm_fwd(S):
    c = S["case"]
    leaf = _leaves(S, False)
    t, first, moments = _exact_norm(S, leaf)
    x = S["x"].double() + t
    m, r = moments(x)
    y = (x - m) * r * leaf["w_pre"]
    out = [x, y, torch.cat([*first, m, r], 1)]
    if c["ckpt"]:
        out.append(_held(y.to(S["y"].dtype)))
    return out


def _exact_norm_bwd(S):
    c = S["case"]
    leaf = _leaves(S, True)
    t, _, moments = _exact_norm(S, leaf)
    x = S["x"].double().requires_grad_(True)
    m, r = moments(x)
    y = (x - m) * r * leaf["w_pre"]
    dx, dw = torch.autograd.grad(y, (x, leaf["w_pre"]), S["dy"].double())
    d = S["dx_out"].double() + dx
    names = [k for k in ("block", "w_post", "scale", "gate") if k in leaf]
    return [d, *_in_order(torch.autograd.grad(t, [leaf[k] for k in names], d), dw)]


def _in_order(grads, dw):
    return [grads[0], dw, *grads[1:]]


def _held(x):
    """The checkpoint's values of x, from the definition: the least power of two that reaches, then the nearest step."""
    T, W = x.shape
    x = torch.nn.functional.pad(x.double(), (0, _padded(W) - W)).unflatten(1, (-1, GROUP))
    m, k = torch.frexp(x.abs().amax(2, keepdim=True) / 127)
    k = (k - (m == 0.5).int()).clamp(min=-126).long()
    step = ((k + 1023) << 52).view(torch.float64)  # 2^k to the last bit
    return ((x / step).round() * step).flatten(1)[:, :W]


def _exact_glu(S):
    act = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[S["case"]["act"]]
    h = act(S["gate"].double()) * S["up"].double()
    gate, up = _held(S["gate"]).requires_grad_(True), _held(S["up"]).requires_grad_(True)
    return [h, *torch.autograd.grad(act(gate) * up, (gate, up), S["dh"].double())]


def _exact_wgrad(S):
    T, W = S["dy"].shape[0], S["case"]["width"]
    step = ((S["e"].long() + (1023 - 127)) << 52).view(torch.float64)
    x = (S["q"].double().view(T, -1, GROUP) * step[..., None]).flatten(1)[:, :W]
    return torch.einsum("tn,tk->nk", S["dy"].double(), x)


_exact = {"rope": _exact_rope, "norm_fwd": _exact_norm_fwd, "norm_bwd": _exact_norm_bwd,
          "encode": lambda S: _held(S["x"]), "glu": _exact_glu, "wgrad": _exact_wgrad}
