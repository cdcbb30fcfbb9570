"""The plans of large calls, on small tensors: runs of the convolution that reuse every stage of their ring and end inside
a batch, and walks of several segments of the scan's backward pass. Each case says which plan it is for (tests/plans.py).

The 64-bit forms are whole-tensor ones on the GPU, held to oracle/operators.py's on the CPU. Bounds, besides those of
test_gpu_operators.py that hold value by value, in the Euclidean norm of an array, where roundings add up as independent
ones and a product held in 11 bits shows (2^-11 / sqrt(12) = 2^-12.8 of the result):
  convolution  a value passes K products, one exponential and one quotient (2^-22 each at most), a gradient the slope from
               the same: 2^-19; sums over tokens add 2^-24 sqrt(160) of a run and less behind it;
  scan         the error of a decay's exponential (2^-23 in the mean at most) is the same for all of T steps at worst, and
               about eight roundings come on top: (T + 8) 2^-23.
"""
import pytest
import torch

import plans
from oracle import operators as O
from test_gpu_operators import F, IO, half_step, place, scan_inputs  # noqa: F401

pytestmark = pytest.mark.gpu


def norm_close(got, want, tol, what):
    want = want.detach()
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    off, size = float((got.double() - want).norm()), float(want.norm())
    assert off <= tol * size, (what, off / size if size else off, tol)


def inside(lengths, B, T):
    n = torch.full((B,), T, device="cuda") if lengths is None else lengths.long().clamp(0, T)
    return (torch.arange(T, device="cuda") < n[:, None])[:, None, :, None], n


def conv64(x, w, bias, act, state, lengths):
    """(y, state_out) of include/falcon.h's formula, all tokens at once; y is 0 behind a sequence's end."""
    B, H, T, d = x.shape
    K = w.shape[2]
    there, n = inside(lengths, B, T)
    ext = torch.cat([state if state is not None else x.new_zeros(B, H, K - 1, d), torch.where(there, x, 0)], 2)
    p = sum(w[:, :, j][:, None] * ext[:, :, j:j + T] for j in range(K)) + (bias[:, None] if bias is not None else 0)
    y = p / (1 + torch.exp(-p)) if act == "silu" else p
    rows = (n[:, None] + torch.arange(K - 1, device=x.device))[:, None, :, None].expand(B, H, K - 1, d)
    return torch.where(there, y, 0), ext.gather(2, rows)


def scan64(q, k, v, delta, A, D, z, delta_bias, S0, lengths, softplus=True):
    B, H, T, dk = k.shape
    there, _ = inside(lengths, B, T)
    dt = delta if delta_bias is None else delta + delta_bias[:, None]
    if softplus:
        dt = torch.nn.functional.softplus(dt, threshold=1e9)
    S = S0 if S0 is not None else v.new_zeros(B, H, v.shape[3], dk)
    rows = []
    for t in range(T):
        d = dt[:, :, t, :, None]
        S = torch.where(there[:, :, t, :, None], torch.exp(d * A) * S + d * v[:, :, t, :, None] * k[:, :, t, None, :], S)
        rows.append((S * q[:, :, t, None, :]).sum(-1))
    o = torch.stack(rows, 2)
    if D is not None:
        o = o + D[:, None] * v
    if z is not None:
        o = o * z / (1 + torch.exp(-z))
    return torch.where(there, o, 0), S


def ragged(B, T, on):
    """Ends inside runs, segments and walks: 0, 1 and T among them."""
    if not on:
        return None
    some = [T, 0, 1, T // 2 + 1, T - 1, T // 3, 2, 2 * T // 3 + 1]
    return torch.tensor([some[b % 8] for b in range(B)], dtype=torch.int32, device="cuda")


def fill_behind(t, lengths):
    """NaN behind the ends, where nothing may be read."""
    if lengths is not None and t is not None:
        there, _ = inside(lengths, t.shape[0], t.shape[2])
        t.masked_fill_(~there, float("nan"))


CONV = [  # io, B, H, T, d, K, act, state, order, ragged, runs (forward, backward)
    ("bf16", 8, 16, 500, 128, 4, "silu", True, "slice", True, (14, 39)),
    ("bf16", 8, 16, 1365, 128, 4, "silu", False, "token", False, (37, 105)),
    ("f32", 8, 16, 500, 128, 4, "silu", True, None, True, (28, 39)),
    ("bf16", 600, 1, 104, 4, 4, "silu", True, None, True, (13, 13)),
    ("f32", 600, 1, 296, 4, 3, "none", True, None, True, (37, 37)),
    ("bf16", 600, 1, 1277, 4, 4, "silu", True, None, True, (160, 160)),
    ("bf16", 600, 1, 1401, 4, 4, "silu", True, "odd", True, (88, 88)),      # several turns of the SMs
    ("f32", 600, 1, 299, 5, 4, "silu", True, "odd", True, (38, 38)),
    ("f32", 5000, 1, 1403, 1, 1, "silu", False, None, True, (160, 160)),    # the longest run
    ("bf16", 300, 2, 310, 8, 8, "silu", True, None, True, (39, 39)),
    ("f32", 300, 2, 1270, 8, 8, "silu", True, None, True, (159, 159)),
    ("bf16", 300, 2, 1270, 8, 8, "none", True, "odd", True, (159, 159)),
    ("bf16", 5000, 1, 1403, 2, 8, "silu", True, None, True, (160, 160)),
    ("bf16", 600, 1, 296, 4, 6, "silu", True, None, False, (37, 37)),
]


@pytest.mark.parametrize("io,B,H,T,d,K,act,state,order,rag,runs", CONV)
def test_conv_runs(F, io, B, H, T, d, K, act, state, order, rag, runs):
    wide = order != "odd"
    V = (8 // (2 if io == "bf16" else 4)) if wide else 1
    V = V if d % V == 0 else 1
    V2 = 2 if wide and d % 2 == 0 else 1
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if sms == 148:
        assert (plans.conv_fwd_run(B, H, T, d, K, V, sms), plans.conv_bwd_run(B, H, T, d, K, V2)) == runs
    r = torch.Generator(device="cuda").manual_seed(90)
    rand = lambda *s: torch.randn(*s, generator=r, device="cuda")
    dt = IO[io]
    x, w, bias = place(rand(B, H, T, d).to(dt), order), rand(H, d, K) * K ** -0.5, rand(H, d)
    tail = rand(B, H, K - 1, d).to(dt) if state else None
    dy, dtail = place(rand(B, H, T, d), order), rand(B, H, K - 1, d)
    n = ragged(B, T, rag)
    leaves = {"x": x.double(), "w": w.double(), "bias": bias.double(), "state": None if tail is None else tail.double()}
    for t in leaves.values():
        if t is not None:
            t.requires_grad_()
    want, tail_w = conv64(leaves["x"], leaves["w"], leaves["bias"], act, leaves["state"], n)
    grads = O.gradients((want, tail_w), (torch.where(inside(n, B, T)[0], dy, 0).double(), dtail.double()), leaves)
    with torch.no_grad():
        ab = lambda t: None if t is None else t.abs()
        M, _ = conv64(leaves["x"].abs(), leaves["w"].abs(), leaves["bias"].abs(), "none", ab(leaves["state"]), n)
    for t in (x, dy):
        fill_behind(t, n)
    y0 = torch.full((B, H, T, d), 7.0, dtype=dt, device="cuda")
    y0 = place(y0, order) if order else y0
    y, tail_o = F.falcon_conv_fwd(x, w, bias=bias, act=act, state=tail, lengths=n, y=y0, want_state=True)
    there, _ = inside(n, B, T)
    assert (y.masked_fill(there, 7.0) == 7.0).all()
    y = y.masked_fill(~there, 0.0).double()
    want = want.detach()
    assert float(((y - want).abs() - 2.0 ** -21 * (K + 2 + M) * M - half_step(io, want)).max()) <= 0
    if io == "f32":
        norm_close(y, want, 2.0 ** -19, "y")
    assert torch.equal(tail_o.double(), tail_w.detach())
    args = F.make_conv_args(x, w, bias=bias, act=act, state=tail, lengths=n)
    assert F.falcon_conv_bwd_workspace_size(args) == plans.conv_workspace(B, H, T, d, K)
    got = F.falcon_conv_bwd(x, w, dy, bias=bias, act=act, state=tail, lengths=n, dstate_out=dtail,
                            dx=None if wide else place(torch.empty(B, H, T, d, device="cuda"), order))
    for name, key in (("x", "dx"), ("w", "dw"), ("bias", "dbias"), ("state", "dstate")):
        if name in grads and grads[name].numel():
            norm_close(got[key], grads[name], 2.0 ** -19, key)
    assert not got["dx"].masked_select(~there).any()
    # dx is a sum of K products w dp, |dp| <= 1.1 |dy|, each good to 2^-17 at the worst (slope 2^-20 (1 + |p|)), and of the
    # tail's gradient
    with torch.no_grad():
        up = torch.where(there, dy, 0).double().abs()
        up = torch.cat([up, up.new_zeros(B, H, K - 1, d)], 2)
        rows = (inside(n, B, T)[1][:, None] + torch.arange(K - 1, device="cuda"))[:, None, :, None].expand(B, H, K - 1, d)
        M = up.new_zeros(B, H, T + K - 1, d).scatter_add_(2, rows, dtail.double().abs())[:, :, K - 1:]
        for j in range(K):
            M = M + 1.1 * leaves["w"].abs()[:, :, j][:, None] * up[:, :, K - 1 - j:K - 1 - j + T]
    assert float(((got["dx"].double() - grads["x"]).abs() - 2.0 ** -17 * M).max()) <= 0


SCAN = [  # io, B, H, T, dk, dv, z, state, order, ragged, (segments, of a walk, walks, walks of a block of step 1, blocks a head)
    ("f32", 40, 8, 333, 8, 9, True, True, None, True, (21, 2, 11, 3, 1)),
    ("bf16", 64, 8, 100, 16, 24, True, True, "token", True, (7, 2, 4, 2, 1)),
    ("bf16", 20, 8, 333, 16, 130, True, True, None, True, (21, 2, 11, 3, 2)),
    ("f32", 2, 16, 1000, 16, 128, True, True, None, True, (63, 5, 13, 1, 1)),
    ("f32", 64, 2, 300, 40, 12, False, True, None, True, (19, 2, 10, 4, 1)),
    ("bf16", 32, 8, 300, 100, 10, True, True, "slice", True, (19, 4, 5, 1, 1)),
    ("f32", 512, 2, 300, 3, 5, True, False, "odd", True, (19, 7, 3, 1, 1)),
    ("f32", 100, 4, 300, 16, 8, True, True, None, True, (19, 19, 1, 1, 1)),          # one walk of several segments
    ("bf16", 600, 2, 45, 16, 8, True, True, "odd", True, (3, 3, 1, 1, 1)),
    ("bf16", 1024, 2, 100, 6, 5, False, True, None, False, (7, 7, 1, 1, 1)),
    ("f32", 300, 2, 50, 64, 20, True, True, None, True, (4, 2, 2, 1, 1)),
    ("bf16", 200, 8, 100, 4, 130, True, True, None, True, (7, 7, 1, 1, 2)),
]


@pytest.mark.parametrize("io,B,H,T,dk,dv,z,state,order,rag,plan", SCAN)
def test_scan_backward_walks(F, io, B, H, T, dk, dv, z, state, order, rag, plan):
    p = plans.ScanBwd(B, H, T, dk, dv)
    assert (p.nseg, p.walk, p.nwalk, p.block, p.ngrp) == plan
    h, g, r = scan_inputs(91, io, B, H, T, dk, dv, True, z, True, state, order)
    assert F.falcon_scan_bwd_workspace_size(F.make_scan_args(**g)) == p.bytes
    n = ragged(B, T, rag)
    dO, dO_g = r(B, H, T, dv, order=order)
    dS, dS_g = r(B, H, dv, dk) if state else (None, None)
    leaves = {k: v.cuda().requires_grad_() for k, v in h.items() if v is not None}
    outs = scan64(**{k: leaves.get(k) for k in h}, lengths=n)
    want = O.gradients(outs, (dO.cuda(), None if dS is None else dS.cuda()), leaves)
    for t in [g[x] for x in ("q", "k", "v", "delta", "z")] + [dO_g]:
        fill_behind(t, n)
    o, S = F.falcon_scan_fwd(**g, lengths=n, o=torch.zeros(B, H, T, dv, dtype=IO[io], device="cuda"))
    norm_close(S, outs[1], (T + 8) * 2.0 ** -23, "S")
    if io == "f32":
        norm_close(o, outs[0], (T + 8) * 2.0 ** -23, "o")
    got = F.falcon_scan_bwd(**g, dO=dO_g, lengths=n, dS_T=dS_g)
    for k, w in want.items():
        norm_close(got["d" + k], w, (T + 8) * 2.0 ** -23, "d" + k)
    there, _ = inside(n, B, T)
    for k in ("dq", "dk", "dv", "ddelta") + (("dz",) if z else ()):
        assert not got[k].masked_select(~there).any(), k


SPLIT = [  # io, B, H, T, dk, dv, z, order, ragged
    ("bf16", 1, 2, 900, 20, 48, True, None, False),
    ("f32", 2, 1, 1000, 40, 30, False, "odd", True),
    ("bf16", 3, 1, 1100, 100, 24, True, "token", True),
    ("f32", 2, 2, 1300, 4, 200, True, None, True),
]


@pytest.mark.parametrize("io,B,H,T,dk,dv,z,order,rag", SPLIT)
def test_scan_split(F, io, B, H, T, dk, dv, z, order, rag):
    """Segments joined over every width of the state's rows."""
    h, g, _ = scan_inputs(92, io, B, H, T, dk, dv, True, z, True, True, order)
    n = ragged(B, T, rag)
    assert F.falcon_scan_workspace_size(F.make_scan_args(**g)) > 0
    with torch.no_grad():
        o_w, S_w = scan64(**{k: None if v is None else v.cuda() for k, v in h.items()}, lengths=n)
    for x in ("q", "k", "v", "delta", "z"):
        fill_behind(g[x], n)
    o, S = F.falcon_scan_fwd(**g, lengths=n, o=torch.zeros(B, H, T, dv, dtype=IO[io], device="cuda"))
    norm_close(S, S_w, (T + 8) * 2.0 ** -23, "S")
    # an output of bf16 is off by half a step, 2^-8 of it at most
    norm_close(o, o_w, (T + 8) * 2.0 ** -23 + (2.0 ** -8 if io == "bf16" else 0), "o")


NORM = [  # io, B, Hq, Hk, T, d, norm, rot, layout, order, ragged, units a block of the backward pass takes at least
    ("bf16", 4, 16, 4, 301, 128, "rms", 128, "half", None, True, 5),
    ("bf16", 3, 7, 3, 401, 64, "l2", 32, "pairs", "token", True, 1),
    ("f32", 3, 7, 3, 401, 100, "rms", 60, "half", "slice", True, 4),
    ("bf16", 2, 5, 2, 799, 75, "rms", 30, "half", "odd", True, 4),
    ("f32", 2, 3, 1, 900, 250, "l2", 250, "pairs", None, False, 3),
    ("bf16", 2, 64, 0, 50, 256, "none", 100, "pairs", None, True, 2),
]


@pytest.mark.parametrize("io,B,Hq,Hk,T,d,norm,rot,layout,order,rag,least", NORM)
def test_qknorm_stretches(F, io, B, Hq, Hk, T, d, norm, rot, layout, order, rag, least):
    """Backward, a block takes a stretch of (group of tokens, head) that starts and ends at any head."""
    V = {"bf16": 8, "f32": 4}[io]
    while V > 1 and (order == "odd" or d % V or (layout == "half" and rot % V)):
        V = V // 2 if V > 4 else 1
    packs = d // V
    lanes = 32 if V == 1 or packs > 16 else 16 if packs > 8 else 8 if packs > 4 else 4
    assert plans.ceil(B * T, 256 // lanes) * (Hq + Hk) // (148 * 2) >= least
    r = torch.Generator(device="cuda").manual_seed(93)
    rand = lambda *s: torch.randn(*s, generator=r, device="cuda")
    n = ragged(B, T, rag)
    freq, pos = torch.rand(rot // 2, generator=r, device="cuda"), torch.randint(0, 100000, (B, T), generator=r, device="cuda", dtype=torch.int32)
    x = [place(rand(B, h, T, d).to(IO[io]), order) if h else None for h in (Hq, Hk)]
    up = [place(rand(B, h, T, d), order) if h else None for h in (Hq, Hk)]
    w = [rand(d), rand(d)]
    want = []
    for i, t in enumerate(x):
        if t is None:
            want.append({})
            continue
        leaves = {"x": t.double().cpu().requires_grad_(), "w": w[i].double().cpu().requires_grad_()}
        out = O.qknorm(leaves["x"], w=leaves["w"], norm=norm, rot=rot, layout=layout, freq=freq.cpu(), positions=pos.cpu(),
                       lengths=None if n is None else n.tolist())
        grads = O.gradients([out], [up[i].double().cpu()], leaves)
        want.append({"y": out.detach().cuda(), "x": grads["x"].cuda(), "w": grads["w"].cuda()})
    for t in x + up:
        fill_behind(t, n)
    kw = dict(wq=w[0], wk=w[1], norm=norm, rot=rot, layout=layout, freq=freq, positions=pos, lengths=n)
    y = F.falcon_qknorm_fwd(x[0], x[1], q_out=None if x[0] is None else torch.zeros_like(want[0]["y"], dtype=IO[io]),
                            k_out=None if x[1] is None else torch.zeros_like(want[1]["y"], dtype=IO[io]), **kw)
    got = F.falcon_qknorm_bwd(x[0], x[1], up[0], up[1], **kw)
    # a value: the root (2^-22) and its sums, an angle to 2^-21, three roundings; a gradient the same with two sums of d
    for i, name in enumerate("qk"):
        if not want[i]:
            continue
        norm_close(y[i], want[i]["y"], 2.0 ** -19 + (2.0 ** -8 if io == "bf16" else 0), "y" + name)
        norm_close(got["d" + name], want[i]["x"], 2.0 ** -18, "d" + name)
        norm_close(got["dw" + name], want[i]["w"], 2.0 ** -18, "dw" + name)
        assert not got["d" + name].masked_select(~inside(n, B, T)[0]).any()
