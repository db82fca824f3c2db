"""More network operators that are measured, case by case.

The cases come from a network that predicts Gaussians from views: a token per 16x16 pixel tile (256x256 images: 256
tokens; one 1080p view: 120 x 68 = 8160; the four views of the ring scene: 32640), widths and head counts generic.

  ffn   gated feed-forward block, h = act(x Wg^T) * (x Wu^T) with W = [Wg; Wu], and its backward pass from x alone
  attn  linear attention with a decay for each head: S_t = d S_{t-1} + k_t v_t^T, o_t = scale q_t S_t, over groups of
        tokens (views), each from a state to a state; its backward pass; and the step that takes single tokens

Queries and keys of a head have `dim` channels, values `vdim`; query head h reads key head h // (q_heads / k_heads) and
has a decay and a state of its own.
"""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16}
CHUNK = 64


def listed():
    return [
        # one token of a stream of views: the weights are read for it alone
        dict(name="ffn_token_fwd_bf16", op="ffn", dir="fwd", tokens=1, width=1024, hidden=2816, act="silu",
             dtype="bf16"),
        # a 256x256 image's tokens in a small network: a call's latency
        dict(name="ffn_tiny_fwd_f16", op="ffn", dir="fwd", tokens=256, width=384, hidden=1024, act="gelu", dtype="f16"),
        # four views through a block, both directions
        dict(name="ffn_ring_fwd_bf16", op="ffn", dir="fwd", tokens=32640, width=1024, hidden=2816, act="silu",
             dtype="bf16"),
        dict(name="ffn_ring_bwd_bf16", op="ffn", dir="bwd", tokens=32640, width=1024, hidden=2816, act="silu",
             dtype="bf16"),
        # odd sizes: rows that start anywhere
        dict(name="ffn_odd_bwd_f16", op="ffn", dir="bwd", tokens=5003, width=997, hidden=1361, act="gelu", dtype="f16"),
        # the tiny image's heads
        dict(name="attn_tiny_fwd_f16", op="attn", dir="fwd", tokens=256, q_heads=6, k_heads=6, dim=64, vdim=64,
             groups=1, state=False, dtype="f16"),
        # four views as one stream that goes on from a state and leaves one, both directions
        dict(name="attn_ring_fwd_bf16", op="attn", dir="fwd", tokens=32640, q_heads=16, k_heads=16, dim=64, vdim=64,
             groups=1, state=True, dtype="bf16"),
        dict(name="attn_ring_bwd_bf16", op="attn", dir="bwd", tokens=32640, q_heads=16, k_heads=16, dim=64, vdim=64,
             groups=1, state=True, dtype="bf16"),
        # wide heads, shared key heads, a view each for itself
        dict(name="attn_wide_fwd_bf16", op="attn", dir="fwd", tokens=8160, q_heads=8, k_heads=2, dim=128, vdim=128,
             groups=4, state=False, dtype="bf16"),
        # views of different sizes (one of them empty), odd heads, shared key heads
        dict(name="attn_ragged_bwd_f16", op="attn", dir="bwd", tokens=5003, q_heads=8, k_heads=4, dim=72, vdim=41,
             groups=7, state=True, dtype="f16"),
        # single tokens: one stream, and 256 of them side by side
        dict(name="attn_step_one_bf16", op="attn", dir="step", tokens=1, q_heads=16, k_heads=16, dim=64, vdim=64,
             dtype="bf16"),
        dict(name="attn_step_many_bf16", op="attn", dir="step", tokens=256, q_heads=16, k_heads=4, dim=64, vdim=64,
             dtype="bf16"),
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of its range; whole multiples of 8 half of the time."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        v = max(lo, v // 8 * 8)
    return v


def draw(rng):
    dtype = rng.choice(["bf16", "f16"])
    if rng.random() < 0.5:
        width, hidden = _size(rng, 32, 2048), _size(rng, 32, 5632)
        few = rng.random() < 0.25  # a stream's tokens
        most = 32 if few else min(32640, 32640 * 1024 * 2816 // (width * hidden))
        return dict(op="ffn", dir="fwd" if few else rng.choice(["fwd", "bwd"]), tokens=_size(rng, 1, most), width=width,
                    hidden=hidden, act=rng.choice(["silu", "gelu"]), dtype=dtype)
    dim, vdim = rng.choice([(64, 64), (64, 64), (128, 128), (32, 32), (48, 48), (80, 80), (96, 96), (64, 128), (72, 64),
                            (57, 91), (16, 64)])
    k_heads = rng.choice([1, 2, 4, 6, 8])
    q_heads = k_heads * rng.choice([1, 1, 2, 4])
    case = dict(op="attn", dir=rng.choice(["fwd", "fwd", "bwd", "bwd", "step"]), q_heads=q_heads, k_heads=k_heads,
                dim=dim, vdim=vdim, dtype=dtype)
    wide = q_heads * max(dim, vdim)
    if case["dir"] == "step":
        return dict(case, tokens=_size(rng, 1, min(512, 256 * 16 * 64 * 64 // (q_heads * dim * vdim))))
    return dict(case, tokens=_size(rng, 1, min(32640, 32640 * 16 * 64 // wide)), groups=rng.choice([1, 2, 4, 7, 16]),
                state=rng.random() < 0.5)


# ------------------------------------------------------------------------------------------------------------------
# inputs


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


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


def ffn_room(case):
    """Room that a block's calls keep: rows laid out anew, the projections' gradient, 128 MiB of partial sums."""
    T, C, F = case["tokens"], -(-case["width"] // 8) * 8, -(-case["hidden"] // 8) * 8
    return (1 << 16) + (128 << 20) + 2 * (T * C + 2 * case["hidden"] * C + 2 * T * F)


def attn_room(case):
    """Room for the states between the tokens: two for each 64 tokens of a group, padded to 64 or 128 channels."""
    d = 64 if max(case["dim"], case["vdim"]) <= 64 else 128
    return (1 << 16) + 8 * (case["tokens"] // 64 + case["groups"] + 1) * case["q_heads"] * d * d


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, T, S = DTYPE[case["dtype"]], case["tokens"], {"case": case}
    if case["op"] == "ffn":
        C, F = case["width"], case["hidden"]
        S["x"] = _normal(g, T, C, dtype=dt)
        S["w"] = _normal(g, 2 * F, C, std=C ** -0.5, dtype=dt)
        S["workspace"] = torch.zeros(ffn_room(case), dtype=torch.uint8, device="cuda")
        if case["dir"] == "fwd":
            S["h"] = torch.empty(T, F, dtype=dt, device="cuda")
        else:
            S["dh"] = _normal(g, T, F, dtype=dt)
            S["dx"] = torch.empty(T, C, dtype=dt, device="cuda")
            S["dw"] = torch.empty(2 * F, C, dtype=dt, device="cuda")
        return S
    hq, hk, D, E = case["q_heads"], case["k_heads"], case["dim"], case["vdim"]
    S["log_decay"] = -torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda") / hq)
    S["scale"] = D ** -0.5

    def heads(make):  # queries, keys and values of one projection
        flat = make(T, hq * D + hk * D + hk * E)
        parts = flat.split([hq * D, hk * D, hk * E], 1)
        return [p.unflatten(1, (h, d)) for p, h, d in zip(parts, (hq, hk, hk), (D, D, E))]

    S["q"], S["k"], S["v"] = heads(lambda *s: _normal(g, *s, dtype=dt))
    if case["dir"] == "step":
        S["state"] = _normal(g, T, hq, D, E)
        S["out"] = torch.empty(T, hq, E, dtype=dt, device="cuda")
        return S
    G = case["groups"]
    S["offsets"] = _offsets(case, g) if G > 1 else None
    S["state"] = _normal(g, G, hq, D, E) if case["state"] else None
    S["workspace"] = torch.empty(attn_room(case), dtype=torch.uint8, device="cuda")
    if case["dir"] == "fwd":
        S["out"] = torch.empty(T, hq, E, dtype=dt, device="cuda")
        S["state_out"] = torch.empty(G, hq, D, E, device="cuda") if case["state"] else None
    else:
        S["dout"] = _normal(g, T, hq, E, dtype=dt)
        S["dq"], S["dk"], S["dv"] = heads(lambda *s: torch.empty(*s, dtype=dt, device="cuda"))
        S["dstate_out"] = _normal(g, G, hq, D, E, std=0.1) if case["state"] else None
        S["dstate"] = torch.empty(G, hq, D, E, device="cuda") if case["state"] else None
    return S


# ------------------------------------------------------------------------------------------------------------------
# one pass


def run(S):
    return (_own if own else _plain)[_kind(S["case"])](S)


def _kind(case):
    return case["op"] + "_" + case["dir"]


def _act(x, name):
    """The block's function and its derivative."""
    if name == "silu":
        s = torch.sigmoid(x)
        return x * s, s * (1 + x * (1 - s))
    phi = 0.5 * (1 + torch.erf(x * 0.5 ** 0.5))
    return x * phi, phi + x * torch.exp(-0.5 * x * x) * (0.5 / math.pi) ** 0.5


def _plain_ffn_fwd(S):
    x, w = S["x"], S["w"]
    gate, up = (x.float() @ w.float().t()).chunk(2, 1)
    return (_act(gate, S["case"]["act"])[0] * up).to(x.dtype)


def _plain_ffn_bwd(S):
    dt, x, w = S["x"].dtype, S["x"].float(), S["w"].float()
    gate, up = (x @ w.t()).chunk(2, 1)
    f, df = _act(gate, S["case"]["act"])
    dh = S["dh"].float()
    d = torch.cat([dh * up * df, dh * f], 1)
    return [(d @ w).to(dt), (d.t() @ x).to(dt)]


class _Chunks:
    """The groups' tokens in chunks: chunk s of the groups one after the other holds the tokens [start, end)."""

    def __init__(self, S):
        c = S["case"]
        T, G = c["tokens"], c["groups"]
        off = S["offsets"].long() if S["offsets"] is not None else torch.tensor([0, T], device="cuda")
        first = off // CHUNK + torch.arange(G + 1, device="cuda")  # a group's first chunk: no two groups share one
        s = torch.arange(T // CHUNK + G, device="cuda")
        self.group = (torch.searchsorted(first, s, right=True) - 1).clamp(0, G - 1)
        self.begin, self.stop = off[self.group], off[self.group + 1]
        self.start = torch.minimum(self.begin + (s - first[self.group]) * CHUNK, self.stop)
        self.end = torch.minimum(self.start + CHUNK, self.stop)
        i = torch.arange(CHUNK, device="cuda")
        at = self.start[:, None] + i
        self.valid = at < self.end[:, None]
        self.at = torch.where(self.valid, at, T)  # T: a row of zeros, and where what is not wanted goes
        self.T, self.G = T, G
        self.a = S["log_decay"]
        self.off = off
        # within a chunk, decays from one token to a later one
        gap = i[:, None] - i
        self.inner = torch.where(gap >= 0, torch.exp(self.a[:, None, None] * gap.clamp(min=0)), 0.0)

    def rows(self, x, heads):
        """[chunks, heads, CHUNK, dim] in 32 bits; shared heads for each that reads them."""
        x = torch.cat([x.float(), x.new_zeros(1, *x.shape[1:], dtype=torch.float32)])
        return x[self.at].transpose(1, 2).repeat_interleave(heads // x.shape[1], 1)

    def back(self, y, heads, dtype):
        """The tokens' rows, summed over the heads that share one."""
        n, h, L, d = y.shape
        y = y.view(n, heads, h // heads, L, d).sum(2).transpose(1, 2)
        out = torch.zeros(self.T + 1, heads, d, device="cuda")
        out[self.at.flatten()] = y.reshape(n * L, heads, d)
        return out[:self.T].to(dtype)

    def decay(self, gap, where=True):
        """d^gap for each head in front: [heads, *gap.shape], 0 where there is none."""
        e = torch.exp(self.a.view(-1, *[1] * gap.dim()) * gap.clamp(min=0))
        return torch.where((gap >= 0) & where, e, 0.0)

    def between(self, per_chunk, edge, forward):
        """States at the chunks' starts (ends, backward) and the groups' ends (starts), from each chunk's part."""
        n, h, d, e = per_chunk.shape
        same = self.group[:, None] == self.group
        s = torch.arange(n, device="cuda")
        flat = per_chunk.transpose(0, 1).flatten(2)
        if forward:
            gap, earlier = self.start[:, None] - self.end, s[:, None] > s
            to_edge, last = self.start - self.begin, self.off[1:, None] - self.end
        else:
            gap, earlier = self.start - self.end[:, None], s[:, None] < s
            to_edge, last = self.stop - self.end, self.start - self.off[:-1, None]
        of = self.group == torch.arange(self.G, device="cuda")[:, None]
        inside = (self.decay(gap, same & earlier) @ flat).view(h, n, d, e).transpose(0, 1)
        final = (self.decay(last, of) @ flat).view(h, self.G, d, e).transpose(0, 1)
        if edge is not None:
            inside = inside + self.decay(to_edge).t()[:, :, None, None] * edge[self.group]
            final = final + self.decay(self.off[1:] - self.off[:-1]).t()[:, :, None, None] * edge
        return inside, final


def _states(S, c, k, v):
    """Keys' part of each chunk, and the states at the chunks' starts and the groups' ends."""
    left = c.decay((c.end - 1)[:, None] - c.start[:, None] - torch.arange(CHUNK, device="cuda")).transpose(0, 1)
    return left, c.between((k * left[..., None]).transpose(2, 3) @ v, S["state"], True)


def _plain_attn_fwd(S):
    c, hq = _Chunks(S), S["case"]["q_heads"]
    q, k, v = (c.rows(S[n], hq) for n in "qkv")
    _, (state, final) = _states(S, c, k, v)
    since = c.decay(torch.arange(1, CHUNK + 1, device="cuda"))[..., None]
    o = ((q @ k.transpose(2, 3)) * c.inner) @ v + since * (q @ state)
    out = [c.back(S["scale"] * o, hq, S["q"].dtype)]
    return out + [final] if S["state_out"] is not None else out


def _plain_attn_bwd(S):
    c, hq, dt = _Chunks(S), S["case"]["q_heads"], S["q"].dtype
    q, k, v, do = (c.rows(S[n], hq) for n in ("q", "k", "v", "dout"))
    q = q * S["scale"]
    left, (state, _) = _states(S, c, k, v)
    since = c.decay(torch.arange(1, CHUNK + 1, device="cuda"))[..., None]
    back, dstate = c.between((q * since).transpose(2, 3) @ do, S["dstate_out"], False)
    p = (q @ k.transpose(2, 3)) * c.inner
    dp = (do @ v.transpose(2, 3)) * c.inner
    dq = S["scale"] * (dp @ k + since * (do @ state.transpose(2, 3)))
    dk = dp.transpose(2, 3) @ q + left[..., None] * (v @ back.transpose(2, 3))
    dv = p.transpose(2, 3) @ do + left[..., None] * (k @ back)
    hk = S["case"]["k_heads"]
    out = [c.back(dq, hq, dt), c.back(dk, hk, dt), c.back(dv, hk, dt)]
    return out + [dstate] if S["dstate"] is not None else out


def _plain_attn_step(S):
    rep = S["case"]["q_heads"] // S["case"]["k_heads"]
    k, v = (S[n].float().repeat_interleave(rep, 1) for n in "kv")
    S["state"].mul_(torch.exp(S["log_decay"])[:, None, None]).add_(k[..., None] * v[:, :, None])
    o = (S["q"].float()[:, :, None] @ S["state"])[:, :, 0]
    return [(S["scale"] * o).to(S["q"].dtype), S["state"]]


_plain = {"ffn_fwd": _plain_ffn_fwd, "ffn_bwd": _plain_ffn_bwd, "attn_fwd": _plain_attn_fwd,
          "attn_bwd": _plain_attn_bwd, "attn_step": _plain_attn_step}


def _gs():
    import gaussian_splatting_differentiable_gs_gb300 as gs
    return gs


def _own_ffn_fwd(S):
    _gs().gs_ffn_fwd(S["x"], S["w"], S["h"], S["workspace"], act=S["case"]["act"])
    return S["h"]


def _own_ffn_bwd(S):
    _gs().gs_ffn_bwd(S["x"], S["w"], S["dh"], S["dx"], S["dw"], S["workspace"], act=S["case"]["act"])
    return [S["dx"], S["dw"]]


def _own_attn_fwd(S):
    _gs().gs_linear_attn_fwd(S["q"], S["k"], S["v"], S["log_decay"], S["out"], group_offsets=S["offsets"],
                             state=S["state"], state_out=S["state_out"], scale=S["scale"], workspace=S["workspace"])
    return [S["out"]] + ([S["state_out"]] if S["state_out"] is not None else [])


def _own_attn_bwd(S):
    _gs().gs_linear_attn_bwd(S["q"], S["k"], S["v"], S["log_decay"], S["dout"], S["dq"], S["dk"], S["dv"],
                             group_offsets=S["offsets"], state=S["state"], dstate_out=S["dstate_out"],
                             dstate=S["dstate"], scale=S["scale"], workspace=S["workspace"])
    return [S["dq"], S["dk"], S["dv"]] + ([S["dstate"]] if S["dstate"] is not None else [])


def _own_attn_step(S):
    _gs().gs_linear_attn_step(S["q"], S["k"], S["v"], S["log_decay"], S["state"], S["out"], scale=S["scale"])
    return [S["out"], S["state"]]


_own = {"ffn_fwd": _own_ffn_fwd, "ffn_bwd": _own_ffn_bwd, "attn_fwd": _own_attn_fwd, "attn_bwd": _own_attn_bwd,
        "attn_step": _own_attn_step}


# ------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without, and its results in 64 bits


def work(case):
    T = case["tokens"]
    if case["op"] == "ffn":
        C, F = case["width"], case["hidden"]
        if case["dir"] == "fwd":
            return {"bytes": 2 * (T * C + 2 * F * C + T * F), "flops": 4 * T * C * F}
        return {"bytes": 2 * (2 * T * C + 4 * F * C + T * F), "flops": 12 * T * C * F}
    hq, hk, D, E = case["q_heads"], case["k_heads"], case["dim"], case["vdim"]
    state = 4 * hq * D * E
    once = 2 * T * (hq * D + hk * D + hk * E)  # queries, keys and values
    if case["dir"] == "step":
        return {"bytes": once + 2 * T * hq * E + 2 * T * state, "flops": 5 * T * hq * D * E}
    held = 2 * case["groups"] * state if case["state"] else 0
    # a state's update and its reading take 4 D E flops a token and head
    if case["dir"] == "fwd":
        return {"bytes": once + 2 * T * hq * E + held, "flops": 4 * T * hq * D * E}
    return {"bytes": 2 * once + 2 * T * hq * E + 3 * held // 2, "flops": 10 * T * hq * D * E}


def exact(case, seed):
    return _exact[_kind(case)](prepare(case, seed))


def _exact_ffn(S):
    act = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[S["case"]["act"]]
    x, w = S["x"].double().requires_grad_(), S["w"].double().requires_grad_()
    F = S["case"]["hidden"]
    h = act(torch.einsum("tc,fc->tf", x, w[:F])) * torch.einsum("tc,fc->tf", x, w[F:])
    return x, w, h


def _exact_ffn_fwd(S):
    with torch.no_grad():
        return _exact_ffn(S)[2]


def _exact_ffn_bwd(S):
    x, w, h = _exact_ffn(S)
    return list(torch.autograd.grad(h, (x, w), S["dh"].double()))


def _of_head(S, name):
    """A tensor in 64 bits, a row for each query head."""
    x = S[name].double()
    return x.repeat_interleave(S["case"]["q_heads"] // x.shape[1], 1)


def _spans(S):
    return S["offsets"].tolist() if S["offsets"] is not None else [0, S["case"]["tokens"]]


def _recurrence(S, first, second, edge, read, spans):
    """M <- d M + first_t second_t^T token after token, and what `read` says of each; the last M of each span."""
    d = S["log_decay"].double().exp()[:, None, None]
    ends = []
    for g, tokens in enumerate(spans):
        M = edge[g].double() if edge is not None else torch.zeros(
            first.shape[1], first.shape[2], second.shape[2], dtype=torch.float64, device="cuda")
        for t in tokens:
            M = torch.baddbmm(d * M, first[t][:, :, None], second[t][:, None])
            read(t, M)
        ends.append(M)
    return torch.stack(ends)


def _exact_attn_fwd(S):
    q, k, v = (_of_head(S, n) for n in "qkv")
    cuts = _spans(S)
    out = torch.zeros(*q.shape[:2], v.shape[2], dtype=torch.float64, device="cuda")

    def read(t, M):
        torch.bmm(q[t][:, None], M, out=out[t][:, None])

    final = _recurrence(S, k, v, S["state"], read, [range(a, b) for a, b in zip(cuts, cuts[1:])])
    return [out * S["scale"]] + ([final] if S["state_out"] is not None else [])


def _exact_attn_bwd(S):
    q, k, v, do = (_of_head(S, n) for n in ("q", "k", "v", "dout"))
    q = q * S["scale"]
    cuts = _spans(S)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)

    def of_query(t, M):
        torch.bmm(M, do[t][:, :, None], out=dq[t][:, :, None])

    def of_key(t, M):
        torch.bmm(M, v[t][:, :, None], out=dk[t][:, :, None])
        torch.bmm(k[t][:, None], M, out=dv[t][:, None])

    _recurrence(S, k, v, S["state"], of_query, [range(a, b) for a, b in zip(cuts, cuts[1:])])
    # backward the decay comes after the token: the gradient of the state that a token's sum goes into
    edge = S["dstate_out"].double() if S["dstate_out"] is not None else None
    d = S["log_decay"].double().exp()[:, None, None]
    last = _recurrence(S, q, do, edge / d if edge is not None else None, of_key,
                       [range(b - 1, a - 1, -1) for a, b in zip(cuts, cuts[1:])])
    share = S["case"]["q_heads"] // S["case"]["k_heads"]
    dk, dv = (x.unflatten(1, (-1, share)).sum(2) for x in (dk, dv))
    return [dq * S["scale"], dk, dv] + ([d * last] if S["dstate"] is not None else [])


def _exact_attn_step(S):
    q, k, v = (_of_head(S, n) for n in "qkv")
    M = S["log_decay"].double().exp()[:, None, None] * S["state"].double() + torch.einsum("bhd,bhe->bhde", k, v)
    return [torch.einsum("bhd,bhde->bhe", q, M) * S["scale"], M]


_exact = {"ffn_fwd": _exact_ffn_fwd, "ffn_bwd": _exact_ffn_bwd, "attn_fwd": _exact_attn_fwd,
          "attn_bwd": _exact_attn_bwd, "attn_step": _exact_attn_step}
