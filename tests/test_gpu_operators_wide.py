"""The operators around the memory over drawn sizes and layouts, and at offsets beyond 32 bits, against the
64-bit forms of oracle/operators.py with the bounds of test_gpu_operators.py."""
import ctypes
import random

import pytest
import torch

from oracle import operators as O
from test_gpu_operators import (F, IO, Draw, close, conv_inputs, gradients_close, half_step, host, norm_inputs,  # noqa: F401
                                scan_bound, scan_inputs)

pytestmark = pytest.mark.gpu
SEEDS = range(16)


def ends(rng, B, T):
    return [rng.choice([0, T, rng.randint(0, T)]) for _ in range(B)] if rng.random() < 0.5 else None


def dev_ends(lengths):
    return None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("seed", SEEDS)
def test_conv_drawn(F, seed):
    rng = random.Random(seed)
    io, K = rng.choice(["bf16", "f32"]), rng.randint(1, 8)
    B, H, T, d = rng.randint(1, 3), rng.randint(1, 5), rng.choice([1, 2, 7, 8, 9, 33, 100, 400]), rng.choice([1, 2, 4, 6, 8, 30, 64, 100])
    order, act, bias, state = rng.choice([None, "token", "slice", "odd"]), rng.choice(["silu", "none"]), rng.random() < 0.5, rng.random() < 0.5
    n = ends(rng, B, T)
    h, g, r = conv_inputs(100 + seed, io, B, H, T, d, K, bias, state, order)
    y = torch.zeros(B, T, H, d, dtype=IO[io], device="cuda").transpose(1, 2) if seed % 2 else torch.zeros(B, H, T, d, dtype=IO[io], device="cuda")
    y, tail = F.falcon_conv_fwd(g["x"], g["w"], bias=g["bias"], act=act, state=g["state"], lengths=dev_ends(n), y=y, want_state=True)
    ab = lambda x: None if x is None else x.abs()
    want, tail_w = O.conv(h["x"], h["w"], bias=h["bias"], act=act, state=h["state"], lengths=n)
    M, _ = O.conv(ab(h["x"]), ab(h["w"]), bias=ab(h["bias"]), act="none", state=ab(h["state"]), lengths=n)
    close(y, want, 2.0 ** -21 * (K + 2 + M) * M + half_step(io, want))
    assert torch.equal(host(tail), tail_w)
    dy, dy_g = r(B, H, T, d, order=rng.choice([None, "token", "odd"]))
    ds, ds_g = r(B, H, K - 1, d)
    got = F.falcon_conv_bwd(g["x"], g["w"], dy_g, bias=g["bias"], act=act, state=g["state"], lengths=dev_ends(n), dstate_out=ds_g)
    leaves = {k: v.clone().requires_grad_() for k, v in h.items() if v is not None}
    out = O.conv(leaves["x"], leaves["w"], bias=leaves.get("bias"), act=act, state=leaves.get("state"), lengths=n)
    want = O.gradients(out, (dy, ds), leaves)
    names = {"x": "dx", "w": "dw", "bias": "dbias", "state": "dstate"}
    gradients_close(got, {names[k]: v for k, v in want.items()}, T)


@pytest.mark.parametrize("seed", SEEDS)
def test_scan_drawn(F, seed):
    rng = random.Random(1000 + seed)
    io = rng.choice(["bf16", "f32"])
    dk, dv = rng.choice([1, 3, 4, 8, 12, 16, 16, 24, 64, 100]), rng.choice([1, 2, 16, 40, 64, 129, 200])
    B, H, T = rng.randint(1, 2), rng.randint(1, 3), rng.choice([1, 2, 8, 15, 16, 17, 50, 130, 300])
    softplus, z, skip, state = (rng.random() < 0.6 for _ in range(4))
    n = ends(rng, B, T)
    h, g, r = scan_inputs(200 + seed, io, B, H, T, dk, dv, softplus, z, skip, state, rng.choice([None, "token", "slice", "odd"]))
    want, S_w = O.scan(**h, softplus=softplus, lengths=n)
    bo, bS = scan_bound(h, softplus, n, T)
    o = torch.zeros(B, H, T, dv, dtype=IO[io], device="cuda")
    o, S = F.falcon_scan_fwd(**g, softplus=softplus, lengths=dev_ends(n), o=o)
    close(o, want, bo + half_step(io, want), "o")
    close(S, S_w, bS, "S")
    dO, dO_g = r(B, H, T, dv, order=rng.choice([None, "token", "odd"]))
    dS, dS_g = r(B, H, dv, dk) if rng.random() < 0.5 else (None, None)
    got = F.falcon_scan_bwd(**g, dO=dO_g, softplus=softplus, lengths=dev_ends(n), dS_T=dS_g)
    leaves = {k: v.clone().requires_grad_() for k, v in h.items() if v is not None}
    outs = O.scan(**{k: leaves.get(k) for k in h}, softplus=softplus, lengths=n)
    gradients_close(got, {"d" + k: v for k, v in O.gradients(outs, (dO, dS), leaves).items()}, T)


@pytest.mark.parametrize("seed", SEEDS)
def test_qknorm_drawn(F, seed):
    rng = random.Random(2000 + seed)
    io, d = rng.choice(["bf16", "f32"]), rng.choice([2, 4, 8, 16, 24, 30, 64, 72, 128, 250, 256])
    B, T, Hq, Hk = rng.randint(1, 3), rng.choice([1, 2, 5, 16, 17, 40]), rng.randint(1, 9), rng.randint(0, 4)
    rot, layout, norm, weight = 2 * rng.randint(0, d // 2), rng.choice(["half", "pairs"]), rng.choice(["rms", "l2", "none"]), rng.random() < 0.6
    n = ends(rng, B, T)
    q, k, wq, wk, freq, pos, r = norm_inputs(300 + seed, io, B, Hq, Hk, T, d, weight, rot, rng.choice([None, "token", "slice", "odd"]), rng.random() < 0.5)
    kw = dict(norm=norm, rot=rot, layout=layout)
    dev = lambda t: None if t is None else t.cuda()
    more = dict(wq=wq[1], wk=wk[1], freq=dev(freq), positions=dev(pos), lengths=dev_ends(n), **kw)
    out = [torch.zeros(B, x, T, d, dtype=IO[io], device="cuda") if x else None for x in (Hq, Hk)]
    out = F.falcon_qknorm_fwd(q[1], k[1] if Hk else None, q_out=out[0], k_out=out[1], **more)
    gq, gk = r(B, Hq, T, d), r(B, Hk, T, d)
    got = F.falcon_qknorm_bwd(q[1], k[1] if Hk else None, gq[1], gk[1] if Hk else None, **more)
    for name, x, w, o, g in (("q", q, wq, out[0], gq), ("k", k, wk, out[1], gk)):
        if o is None:
            continue
        leaves = {"x": x[0].clone().requires_grad_(), "w": w[0].clone().requires_grad_() if weight else None}
        want = O.qknorm(leaves["x"], w=leaves["w"], freq=freq, positions=pos, lengths=n, **kw)
        grads = O.gradients([want], [g[0]], leaves)
        want = want.detach()
        big = O.qknorm(x[0], w=w[0], norm=norm, lengths=n).abs().amax(-1, keepdim=True)
        close(o, want, 2.0 ** -18 * big + half_step(io, want), name)
        # the difference of two terms (see test_gpu_operators.py), each at most 2 |g w| / root with sqrt(d) entries
        u = (g[0].abs() * (w[0].abs().max() if weight else 1)).amax(-1, keepdim=True)
        xn = O.qknorm(x[0], norm=norm)
        root = (xn.abs() / x[0].abs()).amax(-1, keepdim=True)
        close(got["d" + name], grads["x"], 2.0 ** -16 * float(grads["x"].abs().max()) + 2.0 ** -18 * root * u * 2 * (1 + d ** 0.5), "d" + name)
        if weight:
            M = (g[0].abs() * xn.abs()).sum((0, 1, 2)).max() * 2
            close(got["dw" + name], grads["w"], (B * Hq * T + 64) * 2.0 ** -24 * float(M), "dw" + name)


def test_offsets_beyond_32_bits(F):
    """Rows whose offset in their tensor is above 2^31 elements: a batch stride of 2^31 + 2^10 (4.3 GB of bf16)."""
    far = 2 ** 31 + 2 ** 10
    big = torch.empty(far + 2 ** 16, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(1)

    def pair(H, T, d):
        x = torch.randn(2, H, T, d, generator=g).to(torch.bfloat16)
        v = big.as_strided((2, H, T, d), (far, T * d, d, 1))
        v.copy_(x)
        return x.double(), v

    h, x = pair(2, 20, 64)
    w = torch.randn(2, 64, 4, generator=g)
    near, _ = F.falcon_conv_fwd(x.contiguous(), w.cuda())
    y, _ = F.falcon_conv_fwd(x, w.cuda())
    assert torch.equal(y, near)
    out = big.as_strided((2, 2, 20, 64), (far, 1280, 64, 1), 8192)
    F.falcon_conv_fwd(x.contiguous(), w.cuda(), y=out)
    assert torch.equal(out, near)
    f = torch.ones(32, device="cuda")
    near, _ = F.falcon_qknorm_fwd(x.contiguous(), None, rot=64, freq=f)
    F.falcon_qknorm_fwd(x, None, rot=64, freq=f, q_out=out)
    assert torch.equal(out, near)
    A = -torch.rand(2, 64, 64, generator=g).cuda()
    c = x.contiguous()
    near, S = F.falcon_scan_fwd(c, c, c, c, A, z=c)
    o, S2 = F.falcon_scan_fwd(x, x, x, x, A, z=x, o=out)
    assert torch.equal(o, near) and torch.equal(S, S2)
    dO = torch.randn(2, 2, 20, 64, generator=g).cuda()
    a, b = F.falcon_scan_bwd(c, c, c, c, A, dO, z=c), F.falcon_scan_bwd(x, x, x, x, A, dO, z=x)
    assert all(torch.equal(a[n], b[n]) for n in a if a[n] is not None)
    S0 = torch.zeros(2, 2, 64, 64, device="cuda")
    t = lambda v: v[:, :, 7]
    assert torch.equal(F.falcon_scan_step(t(x), t(x), t(x), t(x), A, S0.clone()), F.falcon_scan_step(t(c), t(c), t(c), t(c), A, S0.clone()))


def test_qknorm_backward_in_place(F):
    """dq in dq_out's memory with the same strides, through the C ABI."""
    g = torch.Generator().manual_seed(2)
    q, gq = torch.randn(2, 3, 40, 64, generator=g).cuda(), torch.randn(2, 3, 40, 64, generator=g).cuda()
    freq = torch.rand(32, generator=g).cuda()
    want = F.falcon_qknorm_bwd(q, None, gq, None, norm="l2", rot=64, freq=freq)["dq"]
    view = lambda t: F.FalconView(t.data_ptr(), *t.stride()[:3])
    a = F.FalconQknormArgs(io_dtype=F.FALCON_F32, B=2, Hq=3, Hk=0, T=40, d=64, norm=F.FALCON_NORM_L2, rot=64, rot_layout=F.FALCON_ROT_HALF,
                           eps=1e-6, freq=freq.data_ptr())
    a.q = view(q)
    grads = F.FalconQknormGrads(dq_out=view(gq), dq=view(gq))
    assert F.lib().falcon_qknorm_bwd(ctypes.byref(a), ctypes.byref(grads), None, 0, torch.cuda.current_stream().cuda_stream) == F.FALCON_OK
    assert torch.equal(gq, want)


# Many sequences: a block or thread works through several of them, the last one through fewer. Each sequence is what a
# call on a few of them gives, to the last bit.

FEW = [slice(0, 5), slice(300, 307), slice(-4, None)]


@pytest.mark.parametrize("io,N,H,d,K", [("bf16", 601, 16, 128, 4), ("bf16", 405, 12, 200, 8), ("bf16", 601, 8, 33, 3), ("f32", 601, 16, 128, 4),
                                        ("f32", 405, 16, 101, 6)])
def test_conv_step_of_many_sequences(F, io, N, H, d, K):
    r = torch.Generator(device="cuda").manual_seed(40)
    rand = lambda *s: torch.randn(*s, generator=r, device="cuda")
    x, state = rand(N, H, d).to(IO[io]), rand(N, H, K - 1, d).to(IO[io])
    w, bias = rand(H, d, K), rand(H, d)
    out = torch.empty_like(state)
    y = F.falcon_conv_step(x, w, state, bias=bias, state_out=out)
    for few in FEW:
        part = state[few].clone()
        want = F.falcon_conv_step(x[few], w, part, bias=bias)
        assert torch.equal(y[few], want) and torch.equal(out[few], part)
    assert torch.equal(out[:, :, -1], x) and torch.equal(out[:, :, :-1], state[:, :, 1:])
    assert torch.equal(F.falcon_conv_step(x, w, state, bias=bias), y) and torch.equal(state, out)


@pytest.mark.parametrize("io,N,H,dk,dv", [("bf16", 901, 8, 16, 128), ("f32", 901, 8, 16, 128), ("bf16", 907, 4, 64, 64), ("f32", 701, 8, 15, 100),
                                          ("bf16", 601, 8, 128, 32), ("f32", 2003, 8, 3, 130)])
def test_scan_step_of_many_sequences(F, io, N, H, dk, dv):
    r = torch.Generator(device="cuda").manual_seed(41)
    rand = lambda *s: torch.randn(*s, generator=r, device="cuda")
    seq = {n: rand(N, H, dk if n in "qk" else dv).to(IO[io]) for n in ("q", "k", "v", "delta", "z")}
    par = {"A": -rand(H, dv, dk).exp(), "D": rand(H, dv), "delta_bias": rand(H, dv)}
    S = rand(N, H, dv, dk)
    S_out = torch.empty_like(S)
    o = F.falcon_scan_step(S=S, S_out=S_out, **seq, **par)
    for few in FEW:
        part = S[few].clone()
        want = F.falcon_scan_step(S=part, **{n: x[few] for n, x in seq.items()}, **par)
        assert torch.equal(o[few], want) and torch.equal(S_out[few], part)
    assert torch.equal(F.falcon_scan_step(S=S, **seq, **par), o) and torch.equal(S, S_out)


def test_conv_step_of_the_most_sequences(F):
    """2^31 - 1 rows of one channel: sequence numbers behind the last one pass 31 bits in the last block."""
    N = 2 ** 31 - 1
    x = torch.arange(N, dtype=torch.int32, device="cuda").remainder_(251).to(torch.bfloat16).view(N, 1, 1)
    y = F.falcon_conv_step(x, torch.ones(1, 1, 1, device="cuda"), torch.empty(N, 1, 0, 1, dtype=torch.bfloat16, device="cuda"), act="none")
    assert torch.equal(y, x)
