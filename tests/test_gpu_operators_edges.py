"""Values and sizes at the edge of what the operators around the memory allow, against the 64-bit forms of
oracle/operators.py with the bounds of test_gpu_operators.py."""
import pytest
import torch

from oracle import operators as O
from test_gpu_operators import Draw, F, IO, close, gradients_close, half_step, scan_bound, scan_inputs  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ scan: entries that forget everything

FORGET = [  # io, B, H, T, dk, dv, order, lengths
    ("bf16", 2, 2, 21, 16, 64, None, [21, 13]),        # tokens behind the end inside a chunk of eight
    ("f32", 3, 1, 19, 11, 30, "odd", [19, 0, 1]),
    ("bf16", 1, 2, 37, 40, 24, "token", None),
    ("bf16", 2, 1, 900, 16, 40, None, [900, 101]),     # segments without a token behind a ragged end
    ("f32", 1, 1, 700, 5, 9, None, None),
]


def forgetting(seed, io, B, H, T, dk, dv, order):
    """Inputs whose A has columns of -inf and of a finite value that overflows times log2 e. The 64-bit form gets -1e30
    in their place: the same decays, all 0, and a gradient that is no 0 x inf."""
    h, g, r = scan_inputs(seed, io, B, H, T, dk, dv, True, True, True, True, order)
    for c, x in ((0, float("-inf")), (2, -3e38)):
        h["A"][:, :, c], g["A"][:, :, c] = -1e30, x
    return h, g, r


@pytest.mark.parametrize("io,B,H,T,dk,dv,order,lengths", FORGET)
def test_scan_forgets(F, io, B, H, T, dk, dv, order, lengths):
    h, g, r = forgetting(50, io, B, H, T, dk, dv, order)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    want, S_w = O.scan(**h, lengths=lengths)
    bo, bS = scan_bound(h, True, lengths, T)
    for ws in (None, torch.empty(16, dtype=torch.uint8, device="cuda")):   # split where it pays; never split
        o, S = F.falcon_scan_fwd(**g, lengths=n, o=torch.zeros(B, H, T, dv, dtype=IO[io], device="cuda"), workspace=ws)
        close(o, want, bo + half_step(io, want), "o")
        close(S, S_w, bS, "S")
    dO, dO_g = r(B, H, T, dv)
    dS, dS_g = r(B, H, dv, dk)
    got = F.falcon_scan_bwd(**g, dO=dO_g, lengths=n, dS_T=dS_g)
    leaves = {k: v.clone().requires_grad_() for k, v in h.items()}
    outs = O.scan(**{k: leaves.get(k) for k in h}, lengths=lengths)
    gradients_close(got, {"d" + k: v for k, v in O.gradients(outs, (dO, dS), leaves).items() if k != "delta_bias"}, T)


def test_scan_step_forgets(F):
    h, g, _ = forgetting(51, "f32", 3, 2, 1, 16, 40, None)
    want, S_w = O.scan(**h)
    bo, bS = scan_bound(h, True, None, 1)
    one = {k: (v if k in ("A", "D", "delta_bias", "S0") else v[:, :, 0]) for k, v in g.items()}
    S = one.pop("S0")
    close(F.falcon_scan_step(S=S, **one), want[:, :, 0], bo[:, :, 0], "o")
    close(S, S_w, bS, "S")
    # a step of 0 keeps the state, whatever A is
    one.update(delta=torch.zeros_like(one["delta"]), delta_bias=None, softplus=False)
    kept = S.clone()
    F.falcon_scan_step(S=S, **one)
    assert torch.equal(S, kept)


@pytest.mark.parametrize("B,H,T,dk,dv,lengths", [(2, 2, 21, 16, 64, [21, 13]), (2, 1, 900, 5, 9, [900, 101])])
def test_scan_forgets_with_steps_below_0(F, B, H, T, dk, dv, lengths):
    """dt A <= 0 with both signs turned: A up to +inf, steps as they are given, all below 0."""
    h, g, r = scan_inputs(53, "f32", B, H, T, dk, dv, False, True, True, True, None)
    for x in (h, g):
        x["delta"], x["A"] = -x["delta"], -x["A"]
    for c, x in ((0, float("inf")), (2, 3e38)):
        h["A"][:, :, c], g["A"][:, :, c] = 1e30, x
    h["delta"], g["delta"] = h["delta"] - 2.0 ** -7, g["delta"] - 2.0 ** -7      # no step of 0
    h["delta"] = g["delta"].double().cpu()
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    want, S_w = O.scan(**h, softplus=False, lengths=lengths)
    bo, bS = scan_bound({**h, "delta": -h["delta"], "A": -h["A"]}, False, lengths, T)
    o, S = F.falcon_scan_fwd(**g, softplus=False, lengths=n, o=torch.zeros(B, H, T, dv, device="cuda"))
    close(o, want, bo, "o")
    close(S, S_w, bS, "S")
    dO, dO_g = r(B, H, T, dv)
    got = F.falcon_scan_bwd(**g, dO=dO_g, softplus=False, lengths=n)
    leaves = {k: v.clone().requires_grad_() for k, v in h.items() if v is not None}
    outs = O.scan(**{k: leaves.get(k) for k in h}, softplus=False, lengths=lengths)
    gradients_close(got, {"d" + k: v for k, v in O.gradients(outs, (dO, None), leaves).items()}, T)


def test_scan_nan_in_A_is_seen(F):
    _, g, _ = scan_inputs(52, "f32", 1, 1, 12, 16, 8, True, False, False, True, None)
    g["A"][0, 3, 5] = float("nan")
    _, S = F.falcon_scan_fwd(**g)
    assert S[0, 0, 3, 5].isnan() and int(S.isnan().sum()) == 1


# ------------------------------------------------------------------ gradients of very many sequences

def test_conv_backward_of_2_27_sequences(F):
    """A partial row for each sequence. Whole numbers that fp32 sums hold exactly."""
    N = 2 ** 27 + 3
    at = torch.arange(N, dtype=torch.int32, device="cuda")
    x = ((at % 7 == 0).to(torch.bfloat16) - (at % 11 == 0).to(torch.bfloat16)).view(N, 1, 1, 1)
    dy = (at % 13 - 6).float().view(N, 1, 1, 1)
    one = torch.ones(1, 1, 1, device="cuda")
    g = F.falcon_conv_bwd(x, one, dy, bias=torch.zeros(1, 1, device="cuda"), act="none", dx=torch.empty(N, 1, 1, 1, device="cuda"))
    assert torch.equal(g["dx"], dy)
    assert int(g["dbias"]) == int(dy.sum(dtype=torch.float64)) and int(g["dw"]) == int((dy * x.float()).sum(dtype=torch.float64))


def test_long_column_sums(F):
    """dbias over 2^21 sequences of one token, all terms near 1: a chain of 2^18 fp32 additions in sequence would be off by
    up to 2^18 half steps of 2^-24, 1.6e-2. Handed over after each 2^13, it is 2^13 + 2^5 + a block's few: 5e-4 at worst."""
    N = 2 ** 21
    dy = 1 + torch.rand(N, 1, 1, 1, generator=torch.Generator().manual_seed(5)).cuda() * 2 ** -3
    g = F.falcon_conv_bwd(torch.ones_like(dy), torch.ones(1, 1, 1, device="cuda"), dy, bias=torch.zeros(1, 1, device="cuda"), act="none")
    want = float(dy.sum(dtype=torch.float64))
    assert abs(float(g["dbias"]) - want) <= (2 ** 13 + 2 ** 5 + 16) * 2.0 ** -24 * want


# ------------------------------------------------------------------ norm of very many heads

@pytest.mark.parametrize("io,Hq,Hk,d,T", [("f32", 65000, 5000, 16, 1), ("bf16", 65536, 65536, 4, 1), ("bf16", 65536, 1, 3, 2)])
def test_qknorm_of_many_heads(F, io, Hq, Hk, d, T):
    """A token's heads in as many blocks as a grid takes: the same bits as calls on a thousand heads each."""
    r = torch.Generator(device="cuda").manual_seed(54)
    rand = lambda *s: torch.randn(*s, generator=r, device="cuda")
    q, k, wq, wk = rand(1, Hq, T, d).to(IO[io]), rand(1, Hk, T, d).to(IO[io]), rand(d), rand(d)
    rot = d // 2 * 2
    kw = dict(wq=wq, wk=wk, rot=rot, freq=torch.rand(rot // 2, generator=r, device="cuda"))
    qo, ko = F.falcon_qknorm_fwd(q, k, **kw)
    for x, o in ((q, qo), (k, ko)):
        name = "wq" if x is q else "wk"
        for at in range(0, x.shape[1], 1000):
            few = x[:, at:at + 1000].contiguous()
            assert torch.equal(F.falcon_qknorm_fwd(few, None, **{**kw, "wq": kw[name]})[0], o[:, at:at + 1000])
    want = O.qknorm(q[:, -50:].double().cpu(), w=wq.double().cpu(), rot=rot, freq=kw["freq"].cpu())
    close(qo[:, -50:], want, 2.0 ** -18 * O.qknorm(q[:, -50:].double().cpu(), w=wq.double().cpu()).abs().amax(-1, keepdim=True)
          + half_step(io, want))


# ------------------------------------------------------------------ norm: values that are not finite stay where they are

@pytest.mark.parametrize("order", [None, "odd"])
@pytest.mark.parametrize("io,d,rot,layout", [("bf16", 64, 0, "half"), ("bf16", 64, 0, "pairs"), ("bf16", 64, 32, "half"), ("bf16", 64, 32, "pairs"),
                                             ("bf16", 64, 6, "pairs"), ("bf16", 64, 6, "half"), ("f32", 128, 64, "half"), ("f32", 128, 64, "pairs"),
                                             ("f32", 128, 2, "pairs"), ("bf16", 200, 100, "half"), ("f32", 256, 8, "half"), ("f32", 60, 28, "half")])
def test_channels_that_do_not_turn_are_on_their_own(F, io, d, rot, layout, order):
    """Without a norm, a channel that does not turn is x w forwards and g w backwards: an infinity or a NaN in one reaches
    no other, and the gradient does not depend on x. The others keep the bits of a call without it."""
    r = Draw(55)
    (_, q), (_, g), (_, w) = r(2, 3, 20, d, dtype=IO[io], order=order), r(2, 3, 20, d, order=order), r(d)
    freq = torch.rand(rot // 2, generator=r.g).cuda() if rot else None
    kw = dict(wq=w, norm="none", rot=rot, layout=layout, freq=freq)
    fwd = lambda: F.falcon_qknorm_fwd(q, None, **kw)[0].clone()
    bwd = lambda: F.falcon_qknorm_bwd(q, None, g, None, **kw)
    y, b = fwd(), bwd()
    at = [(0, 0, 3, rot), (1, 2, 19, d - 1), (0, 1, 7, rot + (d - rot) // 2), (1, 0, 0, rot + 1)]
    odd = [float("inf"), float("-inf"), float("nan"), float("inf")]
    keep = [(q[i].clone(), g[i].clone()) for i in at]
    for i, x in zip(at, odd):
        q[i] = x
    got = fwd()
    for i, x in zip(at, odd):
        assert got[i].isnan() if x != x else float(got[i]) == x * (1 if w[i[3]] > 0 else -1)
        got[i] = y[i]
    assert torch.equal(got, y)
    back = bwd()
    assert torch.equal(back["dq"], b["dq"])
    channels = sorted({i[3] for i in at})
    assert not back["dwq"][channels].isfinite().any()
    rest = torch.ones(d, dtype=torch.bool)
    rest[channels] = False
    assert torch.equal(back["dwq"][rest], b["dwq"][rest])
    for i, x, (qx, _) in zip(at, odd, keep):
        q[i], g[i] = qx, x
    back = bwd()
    for i, x in zip(at, odd):
        assert back["dq"][i].isnan() if x != x else float(back["dq"][i]) == x * (1 if w[i[3]] > 0 else -1)
        back["dq"][i] = b["dq"][i]
    assert torch.equal(back["dq"], b["dq"])


@pytest.mark.parametrize("order", [None, "odd"])
def test_norm_of_an_infinity(F, order):
    """A row with an infinity has an infinite root: that channel is inf / inf, the others that do not turn with it are 0."""
    r = Draw(56)
    _, q = r(1, 2, 5, 64, order=order)
    q[0, 1, 2, 40] = float("inf")
    for rot, layout in ((0, "half"), (32, "half"), (32, "pairs"), (6, "pairs")):
        y, _ = F.falcon_qknorm_fwd(q, None, rot=rot, layout=layout, freq=torch.ones(rot // 2, device="cuda") if rot else None)
        row = y[0, 1, 2].clone()
        assert row[40].isnan()
        row[40] = 0
        assert (row == 0).all()
        y[0, 1, 2] = 0
        assert y.isfinite().all()


@pytest.mark.parametrize("d,order", [(64, None), (64, "odd"), (3, None)])
@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_range_of_the_sum_of_squares(F, d, order, norm):
    """eps = 0: entries whose squares fp32 holds are normalised, below that a row counts as 0, above as infinite."""
    r = Draw(57)
    x, q = r(1, 4, 1, d, order=order, make=lambda t: t.sign() + t / 8)
    scale = torch.tensor([2.0 ** -62, 2.0 ** 59, 2.0 ** -70, 2.0 ** 66]).view(1, 4, 1, 1)
    q *= scale.cuda()
    y, _ = F.falcon_qknorm_fwd(q, None, norm=norm, eps=0.0)
    want = O.qknorm(x * scale.double(), norm=norm, eps=0.0)
    close(y[:, :2], want[:, :2], 2.0 ** -18 * want[:, :2].abs().amax(-1, keepdim=True))
    assert (y[:, 2:] == 0).all()
    g = F.falcon_qknorm_bwd(q, None, torch.ones(1, 4, 1, d, device="cuda"), None, norm=norm, eps=0.0)["dq"]
    assert g.isfinite().all() and (g[:, 2:] == 0).all()


# ------------------------------------------------------------------ inputs that repeat, and problems of nothing

@pytest.mark.parametrize("axis", [0, 1, 2])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_inputs_repeated_along_an_axis(F, io, axis):
    """A stride of 0 along batch, heads or tokens: the bits of a call on copies, forwards and backwards."""
    r = Draw(58)
    size = [3, 4, 37]
    one = [1 if i == axis else n for i, n in enumerate(size)]

    def pair(d, dt=IO[io]):
        x = r(*one, d, dtype=dt)[1].expand(*size, d)
        return x, x.contiguous()

    def same(call, *args):
        a, b = (call(*(t[i] for t in args)) for i in (0, 1))
        for x, y in zip(*((t.values() if isinstance(t, dict) else t for t in (a, b)))):
            assert (x is None) == (y is None) and (x is None or torch.equal(x, y))

    x, dy = pair(32), pair(32, torch.float32)
    w = r(4, 32, 4)[1]
    same(lambda x: F.falcon_conv_fwd(x, w, want_state=True), x)
    same(lambda x, dy: F.falcon_conv_bwd(x, w, dy), x, dy)
    freq = torch.rand(16, generator=r.g).cuda()
    same(lambda x: F.falcon_qknorm_fwd(x, None, rot=32, freq=freq), x)
    same(lambda x, dy: F.falcon_qknorm_bwd(x, None, dy, None, wq=w[0, :, 0].contiguous(), rot=32, freq=freq), x, dy)
    A, D = -torch.rand(4, 32, 16, generator=r.g).cuda(), r(4, 32)[1]
    q, k, delta, z = pair(16), pair(16), pair(32), pair(32)
    same(lambda q, k, v, e, z: F.falcon_scan_fwd(q, k, v, e, A, D=D, z=z), q, k, x, delta, z)
    same(lambda q, k, v, e, z, g: F.falcon_scan_bwd(q, k, v, e, A, g, D=D, z=z), q, k, x, delta, z, dy)


@pytest.mark.parametrize("B,H,T", [(0, 2, 5), (2, 3, 0), (0, 1, 0), (2, 0, 5), (0, 0, 5), (1, 0, 0)])
def test_nothing_to_do(F, B, H, T):
    """No sequences, heads or tokens: outputs of that shape, and parameters' gradients of 0."""
    z = lambda *s: torch.zeros(*s, device="cuda")
    x, w = z(B, H, T, 8), z(H, 8, 4)
    y, tail = F.falcon_conv_fwd(x, w, want_state=True)
    assert y.shape == x.shape and tail.shape == (B, H, 3, 8)
    assert F.falcon_conv_step(z(B, H, 8), w, tail).shape == (B, H, 8)
    g = F.falcon_conv_bwd(x, w, x, bias=z(H, 8), state=tail)
    assert g["dw"].shape == w.shape and not g["dw"].any() and not g["dbias"].any()
    A = z(H, 8, 4)
    q = z(B, H, T, 4)
    o, S = F.falcon_scan_fwd(q, q, x, x, A)
    assert o.shape == x.shape and S.shape == (B, H, 8, 4)
    assert F.falcon_scan_step(z(B, H, 4), z(B, H, 4), z(B, H, 8), z(B, H, 8), A, S).shape == (B, H, 8)
    g = F.falcon_scan_bwd(q, q, x, x, A, x, D=z(H, 8), delta_bias=z(H, 8), S0=S)
    assert not g["dA"].any() and not g["dD"].any() and not g["ddelta_bias"].any()
    a, b = F.falcon_qknorm_fwd(x, x, rot=8, freq=z(4))
    assert a.shape == b.shape == x.shape
    g = F.falcon_qknorm_bwd(x, x, x, x, wq=z(8), wk=z(8), rot=8, freq=z(4))
    assert not g["dwq"].any() and not g["dwk"].any()


@pytest.mark.parametrize("dv", [2 ** 31 - 512, 2 ** 31 - 513])
def test_the_widest_scan(F, dv):
    """One token of one head with as many channels as there may be, one column each: channel numbers and offsets at the end
    of 31 bits, in rows of whole 16-byte words and of single elements."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    one = torch.ones(1, 1, 1, 1, dtype=torch.bfloat16, device="cuda")
    v = torch.ones(1, 1, 1, dv, dtype=torch.bfloat16, device="cuda")
    delta = torch.zeros_like(v)
    v[..., -1], delta[..., -1] = 3, 2
    A = torch.zeros(1, dv, 1, device="cuda")
    few = F.falcon_scan_fwd(one, one, v[..., -8:].contiguous(), delta[..., -8:].contiguous(), A[:, -8:].contiguous())
    o, S = F.falcon_scan_fwd(one, one, v, delta, A)
    assert torch.equal(o[..., -8:], few[0]) and torch.equal(S[:, :, -8:], few[1])
    assert (o[..., :-1] == o[0, 0, 0, 0]).all() and (S[:, :, :-1] == S[0, 0, 0, 0]).all()
    y = F.falcon_scan_step(one[:, :, 0], one[:, :, 0], v[:, :, 0], delta[:, :, 0], A, S)    # S twice the step now
    want = F.falcon_scan_step(one[:, :, 0], one[:, :, 0], v[:, :, 0, -8:].contiguous(), delta[:, :, 0, -8:].contiguous(), A[:, -8:].contiguous(), few[1])
    assert torch.equal(y[..., -8:], want) and torch.equal(S[:, :, -8:], few[1])
    assert (y[..., :-1] == y[0, 0, 0]).all() and (S[:, :, :-1] == S[0, 0, 0, 0]).all()
