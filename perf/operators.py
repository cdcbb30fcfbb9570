"""Measured cases of the operators around the memory: the short causal convolution, the selective
scan and the norm with rotation of queries and keys.

Each case names an operator and a direction with its sizes. ``prepare`` makes the inputs on the GPU,
``run`` makes one pass (the plain torch form, or the library's entry points where ``own`` is true),
``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # The convolution over the keys' third of a fused q, k, v projection (token-major rows), written
        # head-major for the chunk kernel: the prompt shape of the chunk-parallel workload.
        {"name": "conv_prompt", "op": "conv_fwd", "io": "bf16", "B": 8, "H": 16, "T": 4096, "d": 128, "K": 4,
         "silu": True, "bias": False, "ragged": False, "state": False},
        # A small padded batch in fp32: odd width, three taps, a cached tail in and out, ragged lengths.
        {"name": "conv_ragged", "op": "conv_fwd", "io": "f32", "B": 3, "H": 5, "T": 777, "d": 83, "K": 3,
         "silu": False, "bias": True, "ragged": True, "state": True},
        # A training step's backward pass of the same convolution.
        {"name": "conv_train", "op": "conv_bwd", "io": "bf16", "B": 4, "H": 16, "T": 4096, "d": 128, "K": 4,
         "silu": True, "bias": True, "ragged": False, "state": False},
        # One token for each sequence of the decode workload: the smallest call, where latency counts.
        {"name": "conv_token", "op": "conv_step", "io": "bf16", "N": 256, "H": 32, "d": 128, "K": 4,
         "silu": True, "bias": True},
        # One long prompt of a state-space layer: few rows, so the sequence has to be split.
        {"name": "scan_prompt", "op": "scan_fwd", "io": "bf16", "B": 1, "H": 1, "T": 16384, "dk": 16, "dv": 2048,
         "softplus": True, "z": True, "skip": True, "ragged": False, "state": True},
        # A training batch, queries and keys of each head on their own.
        {"name": "scan_batch", "op": "scan_fwd", "io": "bf16", "B": 4, "H": 16, "T": 2048, "dk": 16, "dv": 128,
         "softplus": True, "z": True, "skip": True, "ragged": False, "state": False},
        # A short padded batch in fp32 with odd sizes and steps given as they are.
        {"name": "scan_ragged", "op": "scan_fwd", "io": "f32", "B": 3, "H": 2, "T": 301, "dk": 11, "dv": 75,
         "softplus": False, "z": False, "skip": True, "ragged": True, "state": True},
        # The backward pass of a training step.
        {"name": "scan_train", "op": "scan_bwd", "io": "bf16", "B": 2, "H": 16, "T": 2048, "dk": 16, "dv": 128,
         "softplus": True, "z": True, "skip": True, "ragged": False, "state": True},
        # One token for each sequence of the decode workload.
        {"name": "scan_token", "op": "scan_step", "io": "bf16", "N": 256, "H": 32, "dk": 16, "dv": 128,
         "softplus": True, "z": True, "skip": True},
        # Queries and keys of the chunk-parallel workload, token-major in, head-major out, rotated whole.
        {"name": "norm_prompt", "op": "norm_fwd", "io": "bf16", "B": 8, "Hq": 16, "Hk": 16, "T": 4096, "d": 128,
         "norm": "rms", "weight": True, "rot": 128, "layout": "half", "ragged": False},
        # One token for each of 256 sequences at positions of its own, shared keys, half of the width rotated.
        {"name": "norm_token", "op": "norm_fwd", "io": "bf16", "B": 256, "Hq": 32, "Hk": 8, "T": 1, "d": 128,
         "norm": "l2", "weight": False, "rot": 64, "layout": "pairs", "ragged": False},
        # The backward pass of a training step, shared keys.
        {"name": "norm_train", "op": "norm_bwd", "io": "bf16", "B": 4, "Hq": 16, "Hk": 4, "T": 2048, "d": 128,
         "norm": "rms", "weight": True, "rot": 128, "layout": "half", "ragged": False},
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_fwd", "scan_bwd", "scan_step",
                     "norm_fwd", "norm_fwd", "norm_bwd"])
    io = rng.choice(["bf16", "bf16", "f32"])
    kind, way = op.split("_")
    ragged, state = rng.random() < 0.4, rng.random() < 0.5
    case = {"op": op, "io": io}
    if kind == "conv":
        H, d, K = rng.randint(1, 24), rng.choice([16, 32, 64, 128, 256, rng.randint(1, 200)]), rng.randint(1, 8)
        act = {"silu": rng.random() < 0.7, "bias": rng.random() < 0.5}
        if way == "step":
            return case | {"N": _log(rng, 1, 512), "H": H, "d": d, "K": K} | act
        room = (1 << 26) // (H * d)
        T = _log(rng, 1, min(32768, room))
        B = _log(rng, 1, max(1, min(64, room // T)))
        return case | {"B": B, "H": H, "T": T, "d": d, "K": K, "ragged": ragged, "state": state} | act
    if kind == "scan":
        H, dk = rng.choice([1, 1, 2, 4, 16]), rng.choice([16, 16, 16, 4, 8, 32, 64, rng.randint(1, 64)])
        dv = rng.choice([64, 128, 1024, 2048, rng.randint(1, 600)])
        more = {"softplus": rng.random() < 0.8, "z": rng.random() < 0.6, "skip": rng.random() < 0.7}
        if way == "step":
            return case | {"N": _log(rng, 1, max(1, min(512, (1 << 24) // (H * dk * dv)))), "H": H, "dk": dk, "dv": dv} | more
        room = max(1, (1 << (27 if way == "fwd" else 26)) // (H * dk * dv))
        T = _log(rng, 1, min(16384, room))
        B = _log(rng, 1, max(1, min(16, room // T)))
        return case | {"B": B, "H": H, "T": T, "dk": dk, "dv": dv, "ragged": ragged, "state": state} | more
    Hk = rng.randint(1, 8)
    Hq = Hk * rng.choice([1, 2, 4])
    d = rng.choice([32, 64, 128, 256, 2 * rng.randint(1, 100)])
    rot = rng.choice([d, d, 0, 2 * rng.randint(1, d // 2)])
    room = (1 << 26) // ((Hq + Hk) * d)
    T = _log(rng, 1, min(32768, room))
    B = _log(rng, 1, max(1, min(256, room // T)))
    return case | {"B": B, "Hq": Hq, "Hk": Hk, "T": T, "d": d, "norm": rng.choice(["rms", "l2", "none"]),
                   "weight": rng.random() < 0.6, "rot": rot, "layout": rng.choice(["half", "pairs"]), "ragged": ragged}


# ---- inputs ----------------------------------------------------------------------------------

def _lengths(gen, c):
    """Lengths of a padded batch: from an empty sequence to a full one."""
    if not c["ragged"]:
        return None
    n = torch.randint(0, c["T"] + 1, (c["B"],), generator=gen, device="cuda", dtype=torch.int32)
    n[0] = c["T"]
    return n


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    io = DTYPES[c["io"]]

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    def heads(B, H, T, d, parts=1, dtype=io):
        """(B, H, T, d), a view of the middle of `parts` token-major projections that were made together."""
        x = normal(B, T, parts, H, d, dtype=dtype)
        return x[:, :, parts // 2].transpose(1, 2)

    kind, way = c["op"].split("_")
    s = {"case": c}
    if kind == "conv":
        H, d, K = c["H"], c["d"], c["K"]
        s["w"] = normal(H, d, K, scale=1.0 / math.sqrt(K))
        s["bias"] = normal(H, d, scale=0.1) if c["bias"] else None
        if way == "step":
            s["x"] = normal(c["N"], 3, H, d, dtype=io)[:, 1]
            s["state"] = normal(c["N"], H, K - 1, d, dtype=io)
            s["state_out"] = torch.empty_like(s["state"])
            s["y"] = torch.empty(c["N"], H, d, dtype=io, device="cuda")
            return s
        B, T = c["B"], c["T"]
        s["x"] = heads(B, H, T, d, parts=3)
        s["lengths"] = _lengths(gen, c)
        s["state"] = normal(B, H, K - 1, d, dtype=io) if c["state"] else None
        if way == "fwd":
            s["y"] = torch.zeros(B, H, T, d, dtype=io, device="cuda")
        else:
            s["dy"] = normal(B, H, T, d)
            s["dstate_out"] = normal(B, H, K - 1, d) if c["state"] else None
        return s
    if kind == "scan":
        H, dk, dv = c["H"], c["dk"], c["dv"]
        # decay rates 1 .. dk of each channel, and steps between 0.001 and 0.1, as such layers start out with
        s["A"] = -(torch.arange(1, dk + 1, device="cuda").float() * torch.exp(normal(H, dv, dk, scale=0.1))).contiguous()
        step = torch.exp(torch.rand(H, dv, generator=gen, device="cuda") * math.log(100.0) + math.log(0.001))
        s["D"] = normal(H, dv, scale=0.2) + 1.0 if c["skip"] else None
        s["delta_bias"] = step + torch.log(-torch.expm1(-step)) if c["softplus"] else None
        B, T = (c["N"], 1) if way == "step" else (c["B"], c["T"])
        v, delta, z = heads(B, H, T, dv, parts=2), heads(B, H, T, dv), heads(B, H, T, dv, parts=2)
        if c["softplus"]:
            delta.mul_(0.5)
        else:
            delta.copy_(torch.exp(0.5 * delta.float()) * step[:, None])
        q, k = heads(B, H, T, dk, parts=2), heads(B, H, T, dk, parts=2)
        s["z"] = z if c["z"] else None
        if way == "step":
            s |= {"q": q[:, :, 0], "k": k[:, :, 0], "v": v[:, :, 0], "delta": delta[:, :, 0],
                  "z": s["z"][:, :, 0] if c["z"] else None, "S": normal(B, H, dv, dk, scale=0.3)}
            s["S_out"] = torch.empty_like(s["S"])
            s["o"] = torch.empty(B, H, dv, dtype=io, device="cuda")
            return s
        s |= {"q": q, "k": k, "v": v, "delta": delta, "lengths": _lengths(gen, c)}
        s["S0"] = normal(B, H, dv, dk, scale=0.3) if c["state"] else None
        if way == "fwd":
            s["o"] = torch.zeros(B, T, H, dv, dtype=io, device="cuda").transpose(1, 2)
        else:
            s["dO"] = heads(B, H, T, dv, dtype=torch.float32)
            s["dS_T"] = normal(B, H, dv, dk) if c["state"] else None
        return s
    B, T, d, rot = c["B"], c["T"], c["d"], c["rot"]
    s["q"], s["k"] = heads(B, c["Hq"], T, d), heads(B, c["Hk"], T, d)
    s["wq"] = normal(d, scale=0.2) + 1.0 if c["weight"] else None
    s["wk"] = normal(d, scale=0.2) + 1.0 if c["weight"] else None
    s["freq"] = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda").float() / max(rot, 1)) if rot else None
    # every sequence goes on from a position of its own
    start = torch.randint(0, 32768, (B, 1), generator=gen, device="cuda")
    s["positions"] = (start + torch.arange(T, device="cuda")).to(torch.int32) if rot else None
    s["lengths"] = _lengths(gen, c)
    if way == "fwd":
        s["q_out"] = torch.zeros(B, c["Hq"], T, d, dtype=io, device="cuda")
        s["k_out"] = torch.zeros(B, c["Hk"], T, d, dtype=io, device="cuda")
    else:
        s["dq_out"], s["dk_out"] = normal(B, c["Hq"], T, d), normal(B, c["Hk"], T, d)
    return s


# ---- the plain forms, in 32 bits ---------------------------------------------------------------

def _inside(lengths, B, T, device):
    """(B, 1, T, 1): which tokens are in their sequence."""
    t = torch.arange(T, device=device)
    n = torch.full((B,), T, device=device) if lengths is None else lengths.long()
    return (t[None, :] < n[:, None])[:, None, :, None]


def _silu_grad(p):
    g = torch.sigmoid(p)
    return g * (1 + p * (1 - g))


def _conv_windows(x, state, K):
    """x in 32 bits behind its cached tail (B, H, K-1+T, d)."""
    B, H, T, d = x.shape
    tail = x.new_zeros(B, H, K - 1, d) if state is None else state
    return torch.cat([tail.float(), x.float()], 2)


def _conv_tail_index(lengths, B, T, K, device):
    """Rows of the extended input that are the tail behind the last token: (B, K-1)."""
    n = torch.full((B,), T, device=device) if lengths is None else lengths.long()
    return n[:, None] + torch.arange(K - 1, device=device)


def _conv_pre(ext, w, bias):
    p = (ext.unfold(2, w.shape[-1], 1) * w[:, None]).sum(-1)
    return p if bias is None else p + bias[:, None]


def _conv_fwd(s):
    c, x = s["case"], s["x"]
    B, H, T, d = x.shape
    K = c["K"]
    ext = _conv_windows(x, s["state"], K)
    p = _conv_pre(ext, s["w"], s["bias"])
    y = p * torch.sigmoid(p) if c["silu"] else p
    y = torch.where(_inside(s["lengths"], B, T, x.device), y.to(x.dtype), s["y"])
    at = _conv_tail_index(s["lengths"], B, T, K, x.device)[:, None, :, None].expand(B, H, K - 1, d)
    return {"y": y, "state": ext.gather(2, at).to(x.dtype)}


def _conv_bwd(s):
    c, x, w = s["case"], s["x"], s["w"]
    B, H, T, d = x.shape
    K = c["K"]
    ext = _conv_windows(x, s["state"], K)
    inside = _inside(s["lengths"], B, T, x.device)
    dp = torch.where(inside, s["dy"], 0.0)
    if c["silu"]:
        dp = dp * _silu_grad(_conv_pre(ext, w, s["bias"]))
    pad = torch.cat([dp.new_zeros(B, H, K - 1, d), dp, dp.new_zeros(B, H, K - 1, d)], 2)
    # row e of the extended input is under tap j of the token e - j
    dext = (pad.unfold(2, K, 1) * w.flip(-1)[:, None]).sum(-1)
    dw = (dp[..., None] * ext.unfold(2, K, 1)).sum((0, 2))
    if s["dstate_out"] is not None:
        at = _conv_tail_index(s["lengths"], B, T, K, x.device)[:, None, :, None].expand(B, H, K - 1, d)
        dext.scatter_add_(2, at, s["dstate_out"])
    out = {"dx": dext[:, :, K - 1:].contiguous(), "dw": dw}
    if s["bias"] is not None:
        out["dbias"] = dp.sum((0, 2))
    if s["state"] is not None:
        out["dstate"] = dext[:, :, :K - 1].contiguous()
    return out


def _conv_step(s):
    c, x = s["case"], s["x"]
    ext = torch.cat([s["state"].float(), x.float()[:, :, None]], 2)
    p = (ext * s["w"].transpose(1, 2)).sum(2)
    if s["bias"] is not None:
        p = p + s["bias"]
    y = p * torch.sigmoid(p) if c["silu"] else p
    return {"y": y.to(x.dtype), "state": ext[:, :, 1:].to(x.dtype)}


def _linear_scan(a, b):
    """S_t = a_t S_{t-1} + b_t along the third axis, by doubling."""
    step = 1
    while step < a.shape[2]:
        b = torch.cat([b[:, :, :step], b[:, :, step:] + a[:, :, step:] * b[:, :, :-step]], 2)
        a = torch.cat([a[:, :, :step], a[:, :, step:] * a[:, :, :-step]], 2)
        step *= 2
    return b


def _scan_step_size(s, delta):
    x = delta.float()
    if s["delta_bias"] is not None:
        x = x + s["delta_bias"][:, None]
    if not s["case"]["softplus"]:
        return x
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _scan_states(s, inside):
    """Step sizes, decays and states of the scan: (B,H,T,dv), (B,H,T,dv,dk) twice."""
    dt = torch.where(inside, _scan_step_size(s, s["delta"]), 0.0)
    a = torch.exp(dt[..., None] * s["A"][:, None])
    b = (dt * s["v"].float())[..., None] * s["k"].float()[:, :, :, None]
    b = torch.where(inside[..., None], b, 0.0)
    if s["S0"] is not None:
        b[:, :, 0] += a[:, :, 0] * s["S0"]
    return dt, a, _linear_scan(a, b)


def _scan_fwd(s):
    c, v, q = s["case"], s["v"], s["q"]
    inside = _inside(s["lengths"], c["B"], c["T"], v.device)
    _, _, S = _scan_states(s, inside)
    o = (S * q.float()[:, :, :, None]).sum(-1)
    if s["D"] is not None:
        o = o + s["D"][:, None] * v.float()
    if s["z"] is not None:
        z = s["z"].float()
        o = o * (z * torch.sigmoid(z))
    return {"o": torch.where(inside, o.to(v.dtype), s["o"]), "S": S[:, :, -1].clone()}


def _scan_bwd(s):
    c, q, k, v = s["case"], s["q"].float(), s["k"].float(), s["v"].float()
    inside = _inside(s["lengths"], c["B"], c["T"], v.device)
    dt, a, S = _scan_states(s, inside)
    before = torch.zeros_like(S[:, :, :1]) if s["S0"] is None else s["S0"][:, :, None]
    before = torch.cat([before, S[:, :, :-1]], 2)
    dy = torch.where(inside, s["dO"], 0.0)
    out = {}
    if s["z"] is not None:
        z = s["z"].float()
        y = (S * q[:, :, :, None]).sum(-1)
        if s["D"] is not None:
            y = y + s["D"][:, None] * v
        out["dz"] = dy * y * _silu_grad(z)
        dy = dy * (z * torch.sigmoid(z))
    out["dq"] = (dy[..., None] * S).sum(3)
    del S
    g = dy[..., None] * q[:, :, :, None]
    if s["dS_T"] is not None:
        g[:, :, -1] += s["dS_T"]
    # G_t = g_t + a_{t+1} G_{t+1}: the same scan from the other end
    later = torch.cat([a[:, :, 1:], torch.ones_like(a[:, :, :1])], 2)
    g = _linear_scan(later.flip(2), g.flip(2)).flip(2)
    if s["S0"] is not None:
        out["dS0"] = a[:, :, 0] * g[:, :, 0]
    out["dk"] = (g * (dt * v)[..., None]).sum(3)
    gk = (g * k[:, :, :, None]).sum(-1)
    out["dv"] = dt * gk
    if s["D"] is not None:
        out["dv"] = out["dv"] + s["D"][:, None] * dy
        out["dD"] = (dy * v).sum((0, 2))
    g = g * a * before
    out["dA"] = (g * dt[..., None]).sum((0, 2))
    ddt = (g * s["A"][:, None]).sum(-1) + v * gk
    if c["softplus"]:
        x = s["delta"].float() + s["delta_bias"][:, None]
        ddt = ddt * torch.sigmoid(x)
    out["ddelta"] = torch.where(inside, ddt, 0.0)
    if s["delta_bias"] is not None:
        out["ddelta_bias"] = out["ddelta"].sum((0, 2))
    return out


def _scan_step(s):
    v, q, k = s["v"].float(), s["q"].float(), s["k"].float()
    dt = _scan_step_size(s, s["delta"][:, :, None])[:, :, 0]
    S = torch.exp(dt[..., None] * s["A"]) * s["S"] + (dt * v)[..., None] * k[:, :, None]
    o = (S * q[:, :, None]).sum(-1)
    if s["D"] is not None:
        o = o + s["D"] * v
    if s["z"] is not None:
        z = s["z"].float()
        o = o * (z * torch.sigmoid(z))
    return {"o": o.to(s["v"].dtype), "S": S}


def _angles(s):
    """Angles (B, T, rot/2) in 64 bits: a far position times a frequency needs them."""
    return s["positions"].double()[..., None] * s["freq"].double()


def _rotate(x, c, cos, sin):
    """The first `rot` channels of (B, H, T, d) rotated by the angles of (B, 1, T, rot/2)."""
    r = c["rot"]
    if r == 0:
        return x
    y = x.clone()
    if c["layout"] == "half":
        x1, x2 = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    else:
        x1, x2 = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    return y


def _rstd(x, c):
    """One over the norm of each row; 0 where there is nothing to divide by."""
    if c["norm"] == "none":
        return torch.ones_like(x[..., :1])
    n = (x * x).sum(-1, keepdim=True)
    n = (n / x.shape[-1] if c["norm"] == "rms" else n) + 1e-6
    return torch.where(n == 0, 0.0, 1.0 / torch.sqrt(n))


def _norm_fwd(s):
    c = s["case"]
    cos = sin = None
    if c["rot"]:
        angle = _angles(s)[:, None]
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    inside = _inside(s["lengths"], c["B"], c["T"], s["q"].device)
    out = {}
    for name, w in (("q", s["wq"]), ("k", s["wk"])):
        x = s[name].float()
        n = x * _rstd(x, c)
        n = n if w is None else n * w
        out[name] = torch.where(inside, _rotate(n, c, cos, sin).to(s[name].dtype), s[name + "_out"])
    return out


def _norm_bwd(s):
    c = s["case"]
    cos = sin = None
    if c["rot"]:
        angle = _angles(s)[:, None]
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    inside = _inside(s["lengths"], c["B"], c["T"], s["q"].device)
    out = {}
    for name, w in (("q", s["wq"]), ("k", s["wk"])):
        x = s[name].float()
        g = torch.where(inside, s["d" + name + "_out"], 0.0)
        g = _rotate(g, c, cos, -sin if c["rot"] else None)
        r = _rstd(x, c)
        n = x * r
        if w is not None:
            out["dw" + name] = (g * n).sum((0, 1, 2))
            g = g * w
        if c["norm"] == "none":
            out["d" + name] = g
        else:
            m = (g * n).sum(-1, keepdim=True)
            out["d" + name] = r * (g - n * (m / c["d"] if c["norm"] == "rms" else m))
    return out


PLAIN = {"conv_fwd": _conv_fwd, "conv_bwd": _conv_bwd, "conv_step": _conv_step, "scan_fwd": _scan_fwd,
         "scan_bwd": _scan_bwd, "scan_step": _scan_step, "norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd}


# ---- the library's calls -------------------------------------------------------------------------

def _own(s):
    from delta_rule_linear_falcon_b200 import falcon as F
    c = s["case"]
    op = c["op"]
    if op.startswith("conv"):
        act = "silu" if c["silu"] else "none"
        if op == "conv_step":
            y = F.falcon_conv_step(s["x"], s["w"], s["state"], bias=s["bias"], act=act, state_out=s["state_out"], y=s["y"])
            return {"y": y, "state": s["state_out"]}
        if op == "conv_fwd":
            y, state = F.falcon_conv_fwd(s["x"], s["w"], bias=s["bias"], act=act, state=s["state"],
                                         lengths=s["lengths"], y=s["y"], want_state=True)
            return {"y": y, "state": state}
        g = F.falcon_conv_bwd(s["x"], s["w"], s["dy"], bias=s["bias"], act=act, state=s["state"],
                              lengths=s["lengths"], dstate_out=s["dstate_out"])
        return {n: t for n, t in g.items() if t is not None}
    if op.startswith("scan"):
        more = {"D": s["D"], "z": s["z"], "delta_bias": s["delta_bias"], "softplus": c["softplus"]}
        if op == "scan_step":
            o = F.falcon_scan_step(s["q"], s["k"], s["v"], s["delta"], s["A"], s["S"], S_out=s["S_out"], o=s["o"], **more)
            return {"o": o, "S": s["S_out"]}
        if op == "scan_fwd":
            o, S = F.falcon_scan_fwd(s["q"], s["k"], s["v"], s["delta"], s["A"], S0=s["S0"], lengths=s["lengths"],
                                     o=s["o"], want_state=True, **more)
            return {"o": o, "S": S}
        g = F.falcon_scan_bwd(s["q"], s["k"], s["v"], s["delta"], s["A"], s["dO"], S0=s["S0"], lengths=s["lengths"],
                              dS_T=s["dS_T"], **more)
        return {n: t for n, t in g.items() if t is not None}
    more = {"wq": s["wq"], "wk": s["wk"], "norm": c["norm"], "eps": 1e-6, "rot": c["rot"], "layout": c["layout"],
            "freq": s["freq"], "positions": s["positions"], "lengths": s["lengths"]}
    if op == "norm_fwd":
        q, k = F.falcon_qknorm_fwd(s["q"], s["k"], q_out=s["q_out"], k_out=s["k_out"], **more)
        return {"q": q, "k": k}
    g = F.falcon_qknorm_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], **more)
    return {n: t for n, t in g.items() if t is not None}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---- the work that a pass cannot do without --------------------------------------------------------

def work(case):
    c = case
    e = 2 if c["io"] == "bf16" else 4
    kind, way = c["op"].split("_")
    if kind == "conv":
        H, d, K = c["H"], c["d"], c["K"]
        rows = c["N"] if way == "step" else c["B"] * c["T"]
        n = rows * H * d
        weights = 4 * H * d * (K + (1 if c["bias"] else 0))
        act = 4 if c["silu"] else 0
        if way == "step":
            return {"bytes": n * e * (2 + 2 * (K - 1)) + weights, "flops": n * (2 * K + act)}
        tail = c["B"] * H * (K - 1) * d
        if way == "fwd":
            return {"bytes": 2 * e * n + e * tail * (2 if c["state"] else 1) + weights, "flops": n * (2 * K + act)}
        return {"bytes": n * (e + 8) + (tail * (e + 8) if c["state"] else 0) + 2 * weights,
                "flops": n * (4 * K + (2 * K + 8 if c["silu"] else 0))}
    if kind == "scan":
        H, dk, dv = c["H"], c["dk"], c["dv"]
        B, T = (c["N"], 1) if way == "step" else (c["B"], c["T"])
        rows = B * H * T
        params = 4 * H * dv * (dk + (1 if c["skip"] else 0) + (1 if c["softplus"] else 0))
        state = 4 * B * H * dv * dk
        wide = 3 if c["z"] else 2
        if way != "bwd":
            states = 2 if way == "step" or c["state"] else 1
            return {"bytes": rows * e * ((wide + 1) * dv + 2 * dk) + params + states * state, "flops": rows * dv * (7 * dk + 12)}
        return {"bytes": rows * (e * (wide * dv + 2 * dk) + 4 * ((wide + 1) * dv + 2 * dk)) + 2 * params
                + (3 * state if c["state"] else 0), "flops": rows * dv * (24 * dk + 30)}
    n = c["B"] * c["T"] * (c["Hq"] + c["Hk"]) * c["d"]
    if way == "fwd":
        return {"bytes": 2 * e * n, "flops": n * 8}
    return {"bytes": n * (e + 8), "flops": n * 14}


# ---- the definitions in 64 bits -----------------------------------------------------------------

def _f64(s, *names, grad=False):
    got = []
    for n in names:
        x = s.get(n)
        got.append(None if x is None else x.detach().double().clone().requires_grad_(grad))
    return got


def _exact_conv(s, x, w, bias, state):
    """The convolution as one sum for each tap over shifted rows."""
    c = s["case"]
    B, H, T, d = x.shape
    K = c["K"]
    rows = torch.nn.functional.pad(x, (0, 0, K - 1, 0))
    if state is not None:
        rows = rows + torch.nn.functional.pad(state, (0, 0, 0, T))
    p = sum(rows[:, :, j:j + T] * w[:, None, :, j] for j in range(K))
    if bias is not None:
        p = p + bias[:, None]
    y = torch.nn.functional.silu(p) if c["silu"] else p
    ends = [T] * B if s.get("lengths") is None else s["lengths"].tolist()
    return y, torch.stack([rows[b, :, ends[b]:ends[b] + K - 1] for b in range(B)])


def _exact_scan(s, q, k, v, delta, A, D, z, bias, S):
    """The recurrence, token by token; a sequence that has ended keeps its state."""
    c = s["case"]
    B, H, T, dv = v.shape
    x = delta if bias is None else delta + bias[:, None]
    dt = torch.nn.functional.softplus(x, threshold=1000.0) if c["softplus"] else x
    ends = torch.full((B,), T, device=v.device) if s.get("lengths") is None else s["lengths"]
    S = v.new_zeros(B, H, dv, c["dk"]) if S is None else S
    rows = []
    for t in range(T):
        new = S * torch.exp(dt[:, :, t, :, None] * A) + (dt[:, :, t] * v[:, :, t]).unsqueeze(-1) * k[:, :, t].unsqueeze(2)
        S = new if s.get("lengths") is None else torch.where((ends > t)[:, None, None, None], new, S)
        rows.append(torch.einsum("bhvk,bhk->bhv", S, q[:, :, t]))
    y = torch.stack(rows, 2)
    if D is not None:
        y = y + D[:, None] * v
    if z is not None:
        y = y * torch.nn.functional.silu(z)
    return y, S


def _exact_norm(s, x, w):
    c = s["case"]
    n = x
    if c["norm"] != "none":
        ss = x.pow(2).mean(-1, keepdim=True) if c["norm"] == "rms" else x.pow(2).sum(-1, keepdim=True)
        n = x * torch.rsqrt(ss + 1e-6)
    n = n if w is None else n * w
    r = c["rot"]
    if not r:
        return n
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), _angles(s))[:, None]
    if c["layout"] == "half":
        t = torch.complex(n[..., :r // 2], n[..., r // 2:r]) * turn
        return torch.cat([t.real, t.imag, n[..., r:]], -1)
    t = torch.view_as_real(torch.view_as_complex(n[..., :r].unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
    return torch.cat([t, n[..., r:]], -1)


def exact(case, seed):
    c = case
    kind, way = c["op"].split("_")
    if kind == "scan" and way == "bwd" and c["B"] * c["H"] * c["T"] * c["dk"] * c["dv"] > 1 << 27:
        return None  # the states of every token in 64 bits, with their gradients, would not fit
    s = prepare(case, seed)
    if way == "step":
        # a step is a sequence of one token
        s["case"] = c = c | {"B": c["N"], "T": 1}
        for n in ("x", "q", "k", "v", "delta", "z"):
            if s.get(n) is not None:
                s[n] = s[n].unsqueeze(2)
    grad = way == "bwd"
    with torch.set_grad_enabled(grad):
        if kind == "conv":
            x, w, bias, state = _f64(s, "x", "w", "bias", "state", grad=grad)
            y, tail = _exact_conv(s, x, w, bias, state)
            if way == "step":
                return {"y": y[:, :, 0], "state": tail}
            inside = _inside(s["lengths"], c["B"], c["T"], x.device)
            if way == "fwd":
                return {"y": torch.where(inside, y, 0.0), "state": tail}
            loss = (torch.where(inside, y, 0.0) * s["dy"]).sum()
            if s["dstate_out"] is not None:
                loss = loss + (tail * s["dstate_out"]).sum()
            want = {"dx": x, "dw": w, "dbias": bias, "dstate": state}
        elif kind == "scan":
            leaves = _f64(s, "q", "k", "v", "delta", "A", "D", "z", "delta_bias", "S" if way == "step" else "S0", grad=grad)
            y, S = _exact_scan(s, *leaves)
            if way == "step":
                return {"o": y[:, :, 0], "S": S}
            inside = _inside(s["lengths"], c["B"], c["T"], y.device)
            if way == "fwd":
                return {"o": torch.where(inside, y, 0.0), "S": S}
            loss = (torch.where(inside, y, 0.0) * s["dO"]).sum()
            if s["dS_T"] is not None:
                loss = loss + (S * s["dS_T"]).sum()
            want = dict(zip(("dq", "dk", "dv", "ddelta", "dA", "dD", "dz", "ddelta_bias", "dS0"), leaves))
        else:
            q, k, wq, wk = _f64(s, "q", "k", "wq", "wk", grad=grad)
            yq, yk = _exact_norm(s, q, wq), _exact_norm(s, k, wk)
            inside = _inside(s["lengths"], c["B"], c["T"], q.device)
            if way == "fwd":
                return {"q": torch.where(inside, yq, 0.0), "k": torch.where(inside, yk, 0.0)}
            loss = (torch.where(inside, yq, 0.0) * s["dq_out"]).sum() + (torch.where(inside, yk, 0.0) * s["dk_out"]).sum()
            want = {"dq": q, "dk": k, "dwq": wq, "dwk": wk}
        want = {n: x for n, x in want.items() if x is not None}
        return dict(zip(want, torch.autograd.grad(loss, list(want.values()))))
