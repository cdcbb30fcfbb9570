"""GPU parity of the operators around the memory (short convolution, selective scan, q/k norm with
rotation), forward, backward and single token, against the 64-bit forms of oracle/operators.py.

Bounds, with u = 2^-24 (half a step of fp32) and M the same sum over absolute values, formed in 64 bits:
  conv      |p - p*| <= (K + 1) u M; silu has slope <= 1.1 and its exponential and quotient are good to
            2^-21 (1 + |p|): 2^-21 (K + 2 + M) M covers both;
  scan      a step's exponential is good to 2^-22 and its two roundings to 2 u, at most T of them multiply;
            a step size to 2^-21, which enters a term once and its decay as x e^-x <= 1: (T + 8) 2^-21 M;
  gradients the same chain twice, against the largest entry of the array: (T + 64) 2^-20;
  norm      16 additions in sequence, one reciprocal root (2^-22), an angle to 2^-21: 2^-18 of the row's largest;
bf16 outputs add the rounding of one value, 2^-8 of it.
"""
import ctypes

import pytest
import torch

from oracle import operators as O
from test_gpu_parity import F  # noqa: F401

pytestmark = pytest.mark.gpu
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Draw:
    """Seeded inputs as (64-bit values on the CPU, tensor on the GPU), equal after rounding to the type."""

    def __init__(self, seed):
        self.g = gen(seed)

    def __call__(self, *shape, dtype=torch.float32, scale=1.0, make=None, order=None):
        x = torch.randn(*shape, generator=self.g) * scale
        x = (make(x) if make else x).to(dtype)
        return x.double(), place(x, order)


def place(x, order):
    """The tensor on the GPU: dense, token-major rows, every other row of a wider array, or off alignment."""
    x = x.cuda()
    if order is None:
        return x
    if order == "token":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if order == "slice":    # the second of three projections that were made together
        w = torch.full(x.shape[:1] + x.shape[2:3] + (3,) + x.shape[1:2] + x.shape[3:], float("nan"), dtype=x.dtype, device="cuda")
        v = w[:, :, 1].transpose(1, 2)
        v.copy_(x)
        return v
    if order == "odd":      # rows one element off alignment, with a gap behind each
        w = torch.full(x.shape[:3] + (x.shape[3] + 3,), float("nan"), dtype=x.dtype, device="cuda")
        v = w[..., 1:1 + x.shape[3]]
        v.copy_(x)
        return v
    raise ValueError(order)


def host(t):
    return t.detach().cpu().double()


def close(got, want, bound, what=""):
    got = host(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), what
    off = (got - want).abs() - bound
    assert want.numel() == 0 or float(off.max()) <= 0, (what, float((got - want).abs().max()), float(off.max()))


def half_step(io, want):
    return 2.0 ** -8 * want.abs() if io == "bf16" else 0.0


def gradients_close(got, want, T, skip=()):
    tol = (T + 64) * 2.0 ** -20
    for n, w in want.items():
        if n in skip:
            continue
        close(got[n], w, tol * float(w.abs().max()) if w.numel() else 0.0, n)


# ------------------------------------------------------------------ convolution

def conv_inputs(seed, io, B, H, T, d, K, bias, state, order):
    r = Draw(seed)
    dt = IO[io]
    a = {"x": r(B, H, T, d, dtype=dt, order=order), "w": r(H, d, K, scale=K ** -0.5), "bias": r(H, d) if bias else (None, None),
         "state": r(B, H, K - 1, d, dtype=dt) if state else (None, None)}
    return {n: v[0] for n, v in a.items()}, {n: v[1] for n, v in a.items()}, r


CONV = [  # io, B, H, T, d, K, act, bias, state, order, lengths
    ("bf16", 2, 3, 65, 64, 4, "silu", True, True, None, None),
    ("bf16", 2, 3, 65, 64, 4, "silu", False, False, "slice", None),
    ("bf16", 2, 2, 200, 128, 4, "silu", True, True, "token", [200, 77]),
    ("bf16", 3, 2, 33, 16, 2, "none", True, True, "odd", [33, 0, 1]),
    ("f32", 2, 5, 37, 83, 3, "none", True, True, "slice", [37, 2]),
    ("f32", 2, 2, 37, 20, 4, "silu", False, True, None, [5, 37]),
    ("f32", 1, 1, 1, 1, 1, "silu", True, False, None, None),
    ("f32", 1, 2, 2, 4, 8, "silu", True, True, None, None),
    ("bf16", 1, 2, 3, 8, 8, "none", False, False, None, None),
    ("bf16", 4, 1, 7, 24, 5, "silu", True, True, "token", [7, 3, 0, 4]),
    ("f32", 1, 3, 70, 36, 6, "silu", True, True, None, None),
    ("bf16", 1, 3, 70, 40, 7, "silu", True, True, "slice", None),
    ("f32", 2, 3, 0, 12, 4, "silu", True, True, None, None),
    ("bf16", 1, 40, 300, 32, 4, "silu", True, False, None, None),
]


@pytest.mark.parametrize("io,B,H,T,d,K,act,bias,state,order,lengths", CONV)
def test_conv_fwd(F, io, B, H, T, d, K, act, bias, state, order, lengths):
    h, g, _ = conv_inputs(1, io, B, H, T, d, K, bias, state, order)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    if lengths:   # what lies behind a sequence's end is not read
        for b, e in enumerate(lengths):
            g["x"][b, :, e:] = float("nan")
    y = torch.full((B, H, T, d), 7.0, dtype=IO[io], device="cuda")
    y, tail = F.falcon_conv_fwd(g["x"], g["w"], bias=g["bias"], act=act, state=g["state"], lengths=n, y=y, want_state=True)
    want, tail_w = O.conv(h["x"], h["w"], bias=h["bias"], act=act, state=h["state"], lengths=lengths)
    ab = lambda x: None if x is None else x.abs()
    M, _ = O.conv(ab(h["x"]), ab(h["w"]), bias=ab(h["bias"]), act="none", state=ab(h["state"]), lengths=lengths)
    for b in range(B):
        e = T if lengths is None else lengths[b]
        assert (y[b, :, e:] == 7.0).all()
        y[b, :, e:] = 0
    close(y, want, 2.0 ** -21 * (K + 2 + M) * M + half_step(io, want))
    assert torch.equal(host(tail), tail_w)


@pytest.mark.parametrize("io,B,H,T,d,K,act,bias,state,order,lengths", CONV)
def test_conv_bwd(F, io, B, H, T, d, K, act, bias, state, order, lengths):
    h, g, r = conv_inputs(2, io, B, H, T, d, K, bias, state, order)
    dy, dy_g = r(B, H, T, d, order=order)
    ds, ds_g = r(B, H, K - 1, d)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    if lengths:
        for b, e in enumerate(lengths):
            g["x"][b, :, e:] = float("nan")
            dy_g[b, :, e:] = float("nan")
    got = F.falcon_conv_bwd(g["x"], g["w"], dy_g, bias=g["bias"], act=act, state=g["state"], lengths=n, dstate_out=ds_g)
    leaves = {k: v.clone().requires_grad_() for k, v in h.items() if v is not None}
    y, tail = O.conv(leaves["x"], leaves["w"], bias=leaves.get("bias"), act=act, state=leaves.get("state"), lengths=lengths)
    want = O.gradients((y, tail), (dy, ds), leaves)
    names = {"x": "dx", "w": "dw", "bias": "dbias", "state": "dstate"}
    gradients_close(got, {names[k]: v for k, v in want.items()}, max(T, 1))
    for k, v in names.items():
        assert (got[v] is None) == (k not in want)


@pytest.mark.parametrize("io,N,H,d,K,act", [("bf16", 5, 3, 64, 4, "silu"), ("f32", 3, 2, 7, 4, "silu"), ("f32", 1, 1, 1, 1, "none"),
                                            ("bf16", 2, 2, 24, 2, "none"), ("bf16", 300, 4, 128, 4, "silu"), ("f32", 4, 2, 16, 8, "silu")])
def test_conv_step_continues_the_prompt(F, io, N, H, d, K, act):
    """A prompt, then its next token from the tail in place, is the prompt with one more token."""
    h, g, r = conv_inputs(3, io, N, H, 6, d, K, True, True, None)
    y, tail = F.falcon_conv_fwd(g["x"], g["w"], bias=g["bias"], act=act, state=g["state"], want_state=True)
    y5, t5 = F.falcon_conv_fwd(g["x"][:, :, :5], g["w"], bias=g["bias"], act=act, state=g["state"], want_state=True)
    assert torch.equal(y5, y[:, :, :5])
    out = F.falcon_conv_step(g["x"][:, :, 5], g["w"], t5, bias=g["bias"], act=act)
    assert torch.equal(out, y[:, :, 5]) and torch.equal(t5, tail)


def test_conv_state_in_place(F):
    h, g, _ = conv_inputs(4, "bf16", 2, 3, 50, 64, 4, True, True, None)
    y, tail = F.falcon_conv_fwd(g["x"], g["w"], state=g["state"], want_state=True)
    s = g["state"].clone()
    for n in ([50, 50], [1, 0], [2, 3]):
        lens = torch.tensor(n, dtype=torch.int32, device="cuda")
        _, want = F.falcon_conv_fwd(g["x"], g["w"], state=g["state"], want_state=True, lengths=lens)
        s.copy_(g["state"])
        F.falcon_conv_fwd(g["x"], g["w"], state=s, state_out=s, lengths=lens)
        assert torch.equal(s, want)


def test_conv_lengths_are_clamped(F):
    h, g, _ = conv_inputs(5, "f32", 3, 2, 9, 16, 4, False, False, None)
    lens = torch.tensor([-5, 100, 4], dtype=torch.int32, device="cuda")
    y, tail = F.falcon_conv_fwd(g["x"], g["w"], lengths=lens, y=torch.zeros(3, 2, 9, 16, device="cuda"), want_state=True)
    want, tail_w = O.conv(h["x"], h["w"], lengths=[0, 9, 4])
    close(y, want, 1e-5)
    assert torch.equal(host(tail), tail_w)


# ------------------------------------------------------------------ selective scan

def scan_inputs(seed, io, B, H, T, dk, dv, softplus, z, skip, state, order):
    r = Draw(seed)
    dt = IO[io]
    # steps around 0.1 (softplus of -2), decay rates up to about 3
    a = {"q": r(B, H, T, dk, dtype=dt, order=order), "k": r(B, H, T, dk, dtype=dt, order=order),
         "v": r(B, H, T, dv, dtype=dt, order=order),
         "delta": r(B, H, T, dv, dtype=dt, order=order, make=None if softplus else lambda x: 0.1 * x.abs()),
         "A": r(H, dv, dk, make=lambda x: -x.abs()), "D": r(H, dv) if skip else (None, None),
         "z": r(B, H, T, dv, dtype=dt, order=order) if z else (None, None),
         "delta_bias": r(H, dv, make=lambda x: x - 2) if softplus else (None, None),
         "S0": r(B, H, dv, dk) if state else (None, None)}
    return {n: v[0] for n, v in a.items()}, {n: v[1] for n, v in a.items()}, r


def scan_bound(h, softplus, lengths, T):
    """(bound of o, bound of S) from the same sums over absolute values."""
    p = {n: (x.abs() if x is not None and n in ("q", "k", "v", "D", "S0") else x) for n, x in h.items() if n != "z"}
    Mo, MS = O.scan(**p, softplus=softplus, lengths=lengths)
    if h["z"] is not None:
        Mo = Mo * (h["z"] * torch.sigmoid(h["z"])).abs()
    return (T + 8) * 2.0 ** -21 * Mo, (T + 8) * 2.0 ** -21 * MS


SCAN = [  # io, B, H, T, dk, dv, softplus, z, skip, state, order, lengths
    ("bf16", 2, 3, 40, 16, 64, True, True, True, True, None, None),
    ("bf16", 2, 3, 40, 16, 64, True, True, True, False, "slice", [40, 17]),
    ("f32", 3, 2, 61, 11, 75, False, False, True, True, "token", [61, 0, 1]),
    ("f32", 1, 1, 1, 1, 1, True, False, False, True, None, None),
    ("f32", 1, 2, 2, 3, 5, True, True, False, False, None, None),
    ("f32", 2, 1, 9, 4, 130, True, True, True, True, "odd", [8, 9]),
    ("bf16", 1, 1, 17, 8, 33, True, True, True, True, None, None),
    ("f32", 1, 2, 50, 20, 40, True, True, True, True, None, None),
    ("bf16", 1, 2, 23, 32, 100, False, True, True, True, "token", None),
    ("f32", 2, 1, 30, 64, 48, True, True, True, True, None, [30, 16]),
    ("f32", 1, 1, 20, 128, 20, True, False, True, True, None, None),
    ("bf16", 1, 1, 33, 65, 37, True, True, True, True, "slice", None),
    ("f32", 2, 2, 0, 16, 24, True, True, True, True, None, None),
    ("bf16", 1, 1, 24, 16, 600, True, True, True, True, None, None),
    ("bf16", 2, 1, 900, 16, 40, True, True, True, True, None, [900, 333]),     # split into segments
    ("f32", 1, 1, 700, 5, 9, True, True, True, True, "token", None),           # split into segments
]


@pytest.mark.parametrize("io,B,H,T,dk,dv,softplus,z,skip,state,order,lengths", SCAN)
def test_scan_fwd(F, io, B, H, T, dk, dv, softplus, z, skip, state, order, lengths):
    h, g, _ = scan_inputs(10, io, B, H, T, dk, dv, softplus, z, skip, state, order)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    if lengths:
        for b, e in enumerate(lengths):
            for x in ("q", "k", "v", "delta", "z"):
                if g[x] is not None:
                    g[x][b, :, e:] = float("nan")
    want, S_w = O.scan(**h, softplus=softplus, lengths=lengths)
    bo, bS = scan_bound(h, softplus, lengths, T)
    for ws in (None, torch.empty(16, dtype=torch.uint8, device="cuda")):   # split where it pays; never split
        o = torch.full((B, T, H, dv), 7.0, dtype=IO[io], device="cuda").transpose(1, 2)
        o, S = F.falcon_scan_fwd(**g, softplus=softplus, lengths=n, o=o, workspace=ws)
        for b in range(B):
            e = T if lengths is None else lengths[b]
            assert (o[b, :, e:] == 7.0).all()
            o[b, :, e:] = 0
        close(o, want, bo + half_step(io, want), "o")
        close(S, S_w, bS, "S")


@pytest.mark.parametrize("io,B,H,T,dk,dv,softplus,z,skip,state,order,lengths", SCAN)
def test_scan_bwd(F, io, B, H, T, dk, dv, softplus, z, skip, state, order, lengths):
    h, g, r = scan_inputs(11, io, B, H, T, dk, dv, softplus, z, skip, state, order)
    dO, dO_g = r(B, H, T, dv, order=order)
    dS, dS_g = r(B, H, dv, dk) if state else (None, None)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    if lengths:
        for b, e in enumerate(lengths):
            for x in ("q", "k", "v", "delta", "z"):
                if g[x] is not None:
                    g[x][b, :, e:] = float("nan")
            dO_g[b, :, e:] = float("nan")
    got = F.falcon_scan_bwd(**{("S0" if k == "S0" else k): v for k, v in g.items()}, dO=dO_g, softplus=softplus, lengths=n, dS_T=dS_g)
    leaves = {k: v.clone().requires_grad_() for k, v in h.items() if v is not None}
    outs = O.scan(**{k: leaves.get(k) for k in h}, softplus=softplus, lengths=lengths)
    want = O.gradients(outs, (dO, dS), leaves)
    gradients_close(got, {"d" + k if k != "delta_bias" else "ddelta_bias": v for k, v in want.items()}, T)
    for k in h:
        assert (got["d" + k] is None) == (h[k] is None)


@pytest.mark.parametrize("io,N,H,dk,dv,z", [("bf16", 3, 2, 16, 64, True), ("f32", 2, 1, 11, 75, False), ("f32", 1, 1, 1, 1, True),
                                            ("bf16", 2, 2, 4, 200, True), ("f32", 1, 2, 64, 33, True), ("bf16", 1, 1, 128, 40, True),
                                            ("f32", 2, 3, 6, 130, True), ("bf16", 1, 1, 32, 64, False)])
def test_scan_step(F, io, N, H, dk, dv, z):
    h, g, _ = scan_inputs(12, io, N, H, 1, dk, dv, True, z, True, True, None)
    want, S_w = O.scan(**h)
    bo, bS = scan_bound(h, True, None, 1)
    one = {k: (v if v is None or k in ("A", "D", "delta_bias", "S0") else v[:, :, 0]) for k, v in g.items()}
    S = one.pop("S0")
    S_out = torch.empty_like(S)
    o = F.falcon_scan_step(S=S, S_out=S_out, **one)
    close(o, want[:, :, 0], bo[:, :, 0] + half_step(io, want[:, :, 0]), "o")
    close(S_out, S_w, bS, "S")
    o2 = F.falcon_scan_step(S=S, **one)     # in place
    assert torch.equal(o2, o) and torch.equal(S, S_out)


def test_scan_state_in_place_when_split(F):
    h, g, _ = scan_inputs(13, "f32", 1, 1, 2000, 16, 32, True, True, True, True, None)
    o, S = F.falcon_scan_fwd(**g)
    S0 = g.pop("S0").clone()
    o2, S2 = F.falcon_scan_fwd(**g, S0=S0, S_out=S0)
    assert torch.equal(o, o2) and torch.equal(S, S2)


def test_scan_shared_keys(F):
    """q and k broadcast over heads (stride 0): the same as copies of them."""
    h, g, r = scan_inputs(14, "bf16", 2, 4, 37, 16, 32, True, True, True, False, None)
    for n in ("q", "k"):
        g[n] = g[n][:, :1].expand(-1, 4, -1, -1)
    a = F.falcon_scan_fwd(**g)
    b = F.falcon_scan_fwd(**{**g, "q": g["q"].contiguous(), "k": g["k"].contiguous()})
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dO = torch.randn(2, 4, 37, 32, device="cuda")
    ga, gb = F.falcon_scan_bwd(**g, dO=dO), F.falcon_scan_bwd(**{**g, "q": g["q"].contiguous(), "k": g["k"].contiguous()}, dO=dO)
    assert torch.equal(ga["dk"], gb["dk"]) and ga["dk"].shape == (2, 4, 37, 16)


def test_scan_strong_and_weak_decays(F):
    """Decays from exp(-0) to exp(-300) (which underflows to 0) beside each other, over a split sequence."""
    h, g, r = scan_inputs(15, "f32", 1, 1, 600, 16, 8, True, False, False, True, None)
    rates = torch.cat([torch.zeros(4), torch.logspace(-3, 3.5, 12)]).expand(1, 8, 16)
    h["A"], g["A"] = -rates.double(), (-rates).contiguous().cuda()
    want, S_w = O.scan(**h)
    bo, bS = scan_bound(h, True, None, 600)
    o, S = F.falcon_scan_fwd(**g)
    close(o, want, bo)
    close(S, S_w, bS + 1e-37)
    dO, dO_g = r(1, 1, 600, 8)
    got = F.falcon_scan_bwd(**g, dO=dO_g)
    leaves = {k: v.clone().requires_grad_() for k, v in h.items() if v is not None}
    want = O.gradients(O.scan(**{k: leaves.get(k) for k in h}), (dO, None), leaves)
    gradients_close(got, {"d" + k: v for k, v in want.items()}, 600)


def test_softplus_over_its_range(F):
    """Steps from e^-30 to 90: one token, A = 0, k = v = 1, so that the state is the step itself."""
    x = torch.linspace(-30, 90, 481).reshape(1, 1, 1, 481)
    one = torch.ones(1, 1, 1, 1)
    o, S = F.falcon_scan_fwd(one.cuda(), one.cuda(), torch.ones_like(x).cuda(), x.cuda(), torch.zeros(1, 481, 1).cuda())
    want = torch.nn.functional.softplus(x.double(), threshold=1e9)
    close(o, want, 2.0 ** -21 * 4 * want)


# ------------------------------------------------------------------ norm and rotation

NORM = [  # io, B, Hq, Hk, T, d, norm, weight, rot, layout, order, lengths, far
    ("bf16", 2, 4, 2, 33, 128, "rms", True, 128, "half", "slice", None, False),
    ("bf16", 2, 4, 1, 33, 64, "l2", False, 32, "pairs", "token", [33, 5], True),
    ("f32", 2, 3, 3, 17, 128, "rms", True, 64, "half", None, [0, 17], True),
    ("f32", 1, 2, 1, 5, 256, "l2", True, 256, "half", None, None, False),
    ("bf16", 1, 2, 2, 9, 256, "none", False, 256, "pairs", None, None, True),
    ("f32", 1, 5, 2, 7, 46, "rms", True, 46, "half", "slice", None, True),
    ("bf16", 1, 5, 2, 7, 40, "rms", True, 22, "pairs", "odd", None, True),
    ("bf16", 1, 3, 1, 7, 96, "rms", True, 24, "half", "token", None, True),
    ("f32", 3, 1, 1, 1, 2, "l2", False, 2, "half", None, None, True),
    ("f32", 1, 1, 1, 3, 1, "rms", True, 0, "half", None, None, False),
    ("bf16", 1, 1, 2, 3, 200, "l2", True, 0, "half", None, None, False),
    ("bf16", 70, 32, 8, 1, 128, "rms", True, 128, "half", None, None, True),
    ("f32", 1, 2, 0, 6, 32, "rms", True, 32, "half", None, None, False),
    ("f32", 1, 0, 2, 6, 16, "rms", False, 16, "pairs", None, None, False),
    ("bf16", 1, 2, 2, 6, 80, "rms", False, 80, "half", None, None, False),
    ("bf16", 1, 2, 2, 6, 16, "none", False, 0, "half", None, None, False),
]


def norm_inputs(seed, io, B, Hq, Hk, T, d, weight, rot, order, far):
    r = Draw(seed)
    q, k = r(B, Hq, T, d, dtype=IO[io], order=order, scale=3.0), r(B, Hk, T, d, dtype=IO[io], order=order, scale=0.1)
    wq, wk = (r(d), r(d)) if weight else ((None, None), (None, None))
    freq = (10000.0 ** (-torch.arange(0, rot, 2).float() / rot)) if rot else None
    pos = torch.randint(-1000, 2 ** 31 - 1, (B, T), generator=r.g, dtype=torch.int32) if far else None
    return q, k, wq, wk, freq, pos, r


@pytest.mark.parametrize("io,B,Hq,Hk,T,d,norm,weight,rot,layout,order,lengths,far", NORM)
def test_qknorm_fwd(F, io, B, Hq, Hk, T, d, norm, weight, rot, layout, order, lengths, far):
    q, k, wq, wk, freq, pos, _ = norm_inputs(20, io, B, Hq, Hk, T, d, weight, rot, order, far)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    kw = dict(norm=norm, rot=rot, layout=layout)
    dev = lambda t: None if t is None else t.cuda()
    qo = torch.full((B, Hq, T, d), 7.0, dtype=IO[io], device="cuda") if Hq else None
    ko = torch.full((B, Hk, T, d), 7.0, dtype=IO[io], device="cuda") if Hk else None
    qo, ko = F.falcon_qknorm_fwd(q[1] if Hq else None, k[1] if Hk else None, wq=wq[1], wk=wk[1], freq=dev(freq), positions=dev(pos),
                                 lengths=n, q_out=qo, k_out=ko, **kw)
    for x, w, o in ((q, wq, qo), (k, wk, ko)):
        if o is None:
            continue
        want = O.qknorm(x[0], w=w[0], freq=freq, positions=pos, lengths=lengths, **kw)
        for b in range(B):
            e = T if lengths is None else lengths[b]
            assert (o[b, :, e:] == 7.0).all()
            o[b, :, e:] = 0
        big = O.qknorm(x[0], w=w[0], norm=norm, lengths=lengths).abs().amax(-1, keepdim=True)
        # a far angle is exact to 2^31 * 2^-53 * pi turns before its reduction, below the other terms
        close(o, want, 2.0 ** -18 * big + half_step(io, want))


@pytest.mark.parametrize("io,B,Hq,Hk,T,d,norm,weight,rot,layout,order,lengths,far", NORM)
def test_qknorm_bwd(F, io, B, Hq, Hk, T, d, norm, weight, rot, layout, order, lengths, far):
    q, k, wq, wk, freq, pos, r = norm_inputs(21, io, B, Hq, Hk, T, d, weight, rot, order, far)
    gq, gk = r(B, Hq, T, d, order=order), r(B, Hk, T, d)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    if lengths:
        for b, e in enumerate(lengths):
            for t in (q[1], k[1], gq[1], gk[1]):
                t[b, :, e:] = float("nan")
    kw = dict(norm=norm, rot=rot, layout=layout)
    dev = lambda t: None if t is None else t.cuda()
    got = F.falcon_qknorm_bwd(q[1] if Hq else None, k[1] if Hk else None, gq[1] if Hq else None, gk[1] if Hk else None, wq=wq[1],
                              wk=wk[1], freq=dev(freq), positions=dev(pos), lengths=n, **kw)
    rows = B * T * max(Hq, Hk)
    for name, x, w, g in (("q", q, wq, gq), ("k", k, wk, gk)):
        if x[0].numel() == 0:
            assert got["d" + name] is None
            continue
        leaves = {"x": x[0].clone().requires_grad_(), "w": w[0].clone().requires_grad_() if weight else None}
        out = O.qknorm(leaves["x"], w=leaves["w"], freq=freq, positions=pos, lengths=lengths, **kw)
        want = O.gradients([out], [g[0]], leaves)
        # dx = r (u - xr m) is a difference: with e = 2^-18 (relative) on each of its two terms its error is at most
        # e r (|u| + |xr| sum |u xr|), whatever is left of it (for d = 1 and eps = 0 nothing is)
        r0 = O.qknorm(torch.ones_like(x[0]), norm="none", lengths=lengths)
        u = O.gradients([O.qknorm(leaves["x"], w=w[0] if weight else None, freq=freq, positions=pos, lengths=lengths, rot=rot,
                                  layout=layout, norm="none")], [g[0]], {"x": leaves["x"]})["x"].abs()
        xr = O.qknorm(x[0], norm=norm, lengths=lengths).abs()
        root = torch.where(x[0] == 0, r0, xr / x[0].abs()) if norm != "none" else r0
        both = root * (u + xr * ((u * xr).sum(-1, keepdim=True) / (d if norm == "rms" else 1) if norm != "none" else 0))
        close(got["d" + name], want["x"], 2.0 ** -16 * float(want["x"].abs().max()) + 2.0 ** -18 * both, name)
        if weight:
            close(got["dw" + name], want["w"], (2.0 ** -18 + rows * 2.0 ** -24) * float(want["w"].abs().max()), "dw" + name)


def test_qknorm_in_place_and_empty_rows(F):
    q, k, wq, wk, freq, pos, _ = norm_inputs(22, "bf16", 2, 4, 2, 9, 64, True, 64, "token", True)
    q[1][1, :, 3] = 0          # rows with nothing to normalise
    kw = dict(wq=wq[1], wk=wk[1], norm="l2", eps=0.0, rot=64, freq=freq.cuda(), positions=pos.cuda())
    a, b = F.falcon_qknorm_fwd(q[1], k[1], **kw)
    assert (a[1, :, 3] == 0).all() and torch.isfinite(a).all()
    g = F.falcon_qknorm_bwd(q[1], k[1], a.float(), b.float(), **kw)
    assert torch.isfinite(g["dq"]).all() and (g["dq"][1, :, 3] == 0).all()
    F.falcon_qknorm_fwd(q[1], k[1], q_out=q[1], k_out=k[1], **kw)
    assert torch.equal(q[1], a) and torch.equal(k[1], b)


def test_norm_of_a_row_with_nan_stays_in_the_row(F):
    q, k, *_ = norm_inputs(23, "f32", 1, 2, 1, 5, 64, False, 0, None, False)
    a, _ = F.falcon_qknorm_fwd(q[1], k[1])
    q[1][0, 1, 2, 7] = float("nan")
    b, _ = F.falcon_qknorm_fwd(q[1], k[1])
    assert b[0, 1, 2].isnan().all()
    b[0, 1, 2] = a[0, 1, 2]
    assert torch.equal(a, b)


# ------------------------------------------------------------------ calls as such

def test_repeated_calls_give_the_same_bits(F):
    h, g, r = scan_inputs(30, "bf16", 2, 2, 300, 16, 160, True, True, True, True, None)
    dO = r(2, 2, 300, 160)[1]
    a, b = F.falcon_scan_bwd(**g, dO=dO), F.falcon_scan_bwd(**g, dO=dO)
    assert all(torch.equal(a[n], b[n]) for n in a)
    h, c, r = conv_inputs(31, "bf16", 2, 3, 700, 64, 4, True, True, None)
    dy = r(2, 3, 700, 64)[1]
    a, b = (F.falcon_conv_bwd(c["x"], c["w"], dy, bias=c["bias"], state=c["state"]) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_the_binding_refuses(F):
    x = torch.zeros(1, 2, 3, 8, device="cuda")
    w = torch.zeros(2, 8, 4, device="cuda")
    for bad in (dict(w=torch.zeros(2, 7, 4, device="cuda")), dict(bias=torch.zeros(8, device="cuda")),
                dict(state=torch.zeros(1, 2, 4, 8, device="cuda")), dict(act="relu"),
                dict(lengths=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(x=x[..., ::2], w=torch.zeros(2, 4, 4, device="cuda")),
                dict(y=torch.zeros(1, 2, 3, 7, device="cuda"))):
        with pytest.raises(ValueError):
            F.falcon_conv_fwd(**{"x": x, "w": w, **bad})
    for bad in (dict(w=w.double()), dict(lengths=torch.zeros(1, device="cuda")), dict(x=x.half()), dict(state=torch.zeros(1, 2, 3, 8))):
        with pytest.raises(TypeError):
            F.falcon_conv_fwd(**{"x": x, "w": w, **bad})
    with pytest.raises(F.FalconError) as e:
        F.falcon_conv_fwd(x, torch.zeros(2, 8, 9, device="cuda"))
    assert e.value.status == F.FALCON_ERR_UNSUPPORTED
    with pytest.raises(F.FalconError) as e:
        F.falcon_conv_fwd(x, w, y=x)
    assert e.value.status == F.FALCON_ERR_INVALID_ARG
    with pytest.raises(F.FalconError) as e:     # one row for all tokens as an output
        F.falcon_qknorm_fwd(x, x, q_out=x[:, :, :1].clone().expand(-1, -1, 3, -1))
    assert e.value.status == F.FALCON_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="freq"):
        F.falcon_qknorm_fwd(x, x, rot=8, freq=torch.ones(8, device="cuda"))
    with pytest.raises(F.FalconError):
        F.falcon_qknorm_fwd(x, x, rot=8)
    A = -torch.ones(2, 8, 8, device="cuda")
    with pytest.raises(ValueError, match="A must"):
        F.falcon_scan_fwd(x, x, x, x, A[:1])
    with pytest.raises(F.FalconError) as e:     # a workspace that is given has to do
        F.falcon_scan_bwd(x, x, x, x, A, x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == F.FALCON_ERR_WORKSPACE
    assert F.falcon_check_device_errors() == F.FALCON_OK


def test_workspace_sizes(F):
    """A split needs its states and sums of steps between the segments; unsplit problems need nothing."""
    L = F.lib()
    few = F.FalconScanArgs(io_dtype=1, B=1, H=1, T=8192, dk=16, dv=64, flags=1, A=0x1000)
    for n in ("q", "k", "v", "delta"):
        setattr(few, n, F.FalconView(0x1000, 0, 0, 64))
    need = L.falcon_scan_workspace_size(ctypes.byref(few))
    assert need > 0 and need % (64 * 17 * 4) == 0
    few.T = 16
    assert L.falcon_scan_workspace_size(ctypes.byref(few)) == 0
