"""The operators around the memory in a run, as a layer uses them: convolution, q/k norm with rotation and
the fast-weight memory; convolution and scan; prompts that single tokens continue; the backward chain;
side streams and captured graphs."""
import pytest
import torch

import oracle
from oracle import operators as O
from test_gpu_parity import F  # noqa: F401

pytestmark = pytest.mark.gpu
B, H, T, D, K = 2, 3, 50, 32, 4


def layer(seed, T=T, dtype=torch.float32):
    """A fused projection (token-major q, k, v rows), the convolution's and the norm's weights, gates."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    p = {"qkv": r(B, T, 3, H, D).to(dtype), "w": r(3, H, D, K) * 0.5, "wq": 1 + 0.2 * r(D), "wk": 1 + 0.2 * r(D),
         "alpha": torch.sigmoid(r(B, H, T) + 3), "eta": torch.sigmoid(r(B, H, T)),
         "freq": 100.0 ** -(torch.arange(0, D, 2).float() / D)}
    return {n: x.cuda() for n, x in p.items()}


def forward(F, p, pos=None, states=(None,) * 3):
    """(q, k, v) as the memory takes them, and the convolutions' tails."""
    out, tails = [], []
    for i in range(3):
        y, t = F.falcon_conv_fwd(p["qkv"][:, :, i].transpose(1, 2), p["w"][i], state=states[i], want_state=True)
        out.append(y)
        tails.append(t)
    q, k = F.falcon_qknorm_fwd(out[0], out[1], wq=p["wq"], wk=p["wk"], norm="l2", rot=D, freq=p["freq"], positions=pos)
    return (q, k, out[2]), tails, out


def test_memory_layer_and_its_gradients(F):
    """Fused projection -> conv -> norm, rotation -> Falcon-1, and back, against the 64-bit forms of each."""
    p = layer(1)
    (q, k, v), _, (cq, ck, _) = forward(F, p)
    o, S, _ = F.falcon_fwd_recurrent(q, k, v, p["alpha"], p["eta"], rule="falcon1")
    h = {n: x.cpu().double().requires_grad_() for n, x in p.items()}
    c = [O.conv(h["qkv"][:, :, i].transpose(1, 2), h["w"][i])[0] for i in range(3)]
    qh, kh = (O.qknorm(x, w=h[w], norm="l2", rot=D, freq=p["freq"].cpu()) for x, w in ((c[0], "wq"), (c[1], "wk")))
    n = lambda t: t.detach().numpy()
    o_r, S_r, _ = oracle.recurrent(1, n(qh), n(kh), n(c[2]), n(h["alpha"]), n(h["eta"]), 1e-6)
    for got, want in ((o, o_r), (S, S_r)):
        assert float((got.cpu().double() - torch.from_numpy(want)).abs().max()) <= 1e-4 * abs(want).max()
    # backwards: the memory's gradients go into the norm's and the convolution's backward
    dO = torch.randn(B, H, T, D, generator=torch.Generator().manual_seed(2)).cuda()
    m = F.falcon_bwd_recurrent(q, k, v, p["alpha"], p["eta"], dO, rule="falcon1", want_dS0=False)
    m_r = oracle.backward(1, n(qh), n(kh), n(c[2]), n(h["alpha"]), n(h["eta"]), 1e-6, dO.cpu().numpy().astype("float64"))
    g = F.falcon_qknorm_bwd(cq, ck, m["dq"], m["dk"], wq=p["wq"], wk=p["wk"], norm="l2", rot=D, freq=p["freq"])
    dqkv = torch.empty(B, T, 3, H, D, device="cuda")
    dw = []
    for i, dy in enumerate((g["dq"], g["dk"], m["dv"])):
        gi = F.falcon_conv_bwd(p["qkv"][:, :, i].transpose(1, 2), p["w"][i], dy, dx=dqkv[:, :, i].transpose(1, 2))
        dw.append(gi["dw"])
    up = [torch.from_numpy(m_r[x]) for x in ("dq", "dk", "dv")]
    want = O.gradients((qh, kh, c[2]), up, {x: h[x] for x in ("qkv", "w", "wq", "wk")})
    for got, name in ((dqkv, "qkv"), (torch.stack(dw), "w"), (g["dwq"], "wq"), (g["dwk"], "wk")):
        # the memory's gradients are held to 1e-4 of their largest; what follows is a linear map of them
        assert float((got.cpu().double() - want[name]).abs().max()) <= 3e-4 * float(want[name].abs().max()), name


def test_scan_layer_prompt_then_tokens(F):
    """conv -> scan over a prompt, then token by token, is the prompt's continuation."""
    T2, n = 40, 33
    p = layer(3, T2, torch.bfloat16)
    g = torch.Generator().manual_seed(4)
    z, delta = (torch.randn(B, H, T2, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    A = -torch.rand(H, D, D, generator=g).cuda()
    c = [F.falcon_conv_fwd(p["qkv"][:, :, i].transpose(1, 2), p["w"][i])[0] for i in range(3)]
    o, S = F.falcon_scan_fwd(*c, delta, A, z=z)
    tails, heads = [], []
    for i in range(3):
        y, t = F.falcon_conv_fwd(p["qkv"][:, :n, i].transpose(1, 2), p["w"][i], want_state=True)
        heads.append(y)
        tails.append(t)
    o1, S1 = F.falcon_scan_fwd(*heads, delta[:, :, :n], A, z=z[:, :, :n])
    assert torch.equal(o1, o[:, :, :n])
    for t in range(n, T2):
        x = [F.falcon_conv_step(p["qkv"][:, t, i], p["w"][i], tails[i]) for i in range(3)]
        ot = F.falcon_scan_step(*x, delta[:, :, t], A, S1, z=z[:, :, t])
        # the token's kernel adds a row's products in another order: fp32 rounding, then bf16's
        assert float((ot.float() - o[:, :, t].float()).abs().max()) <= 2.0 ** -7 * float(o[:, :, t].float().abs().max())
    assert float((S1 - S).abs().max()) <= 40 * 2.0 ** -21 * float(S.abs().max())


def test_memory_layer_token_by_token(F):
    """conv step -> norm at the token's position -> decode step, against the whole prompt."""
    p = layer(5, 12)
    (q, k, v), _, _ = forward(F, p)
    o, S, _ = F.falcon_fwd_recurrent(q, k, v, p["alpha"], p["eta"], rule="falcon1")
    tails = [torch.zeros(B, H, K - 1, D, device="cuda") for _ in range(3)]
    Sd, kp = torch.zeros(B, H, D, D, device="cuda"), torch.zeros(B, H, D, device="cuda")
    for t in range(12):
        x = [F.falcon_conv_step(p["qkv"][:, t, i], p["w"][i], tails[i]) for i in range(3)]
        pos = torch.full((B, 1), t, dtype=torch.int32, device="cuda")
        qt, kt = F.falcon_qknorm_fwd(x[0][:, :, None], x[1][:, :, None], wq=p["wq"], wk=p["wk"], norm="l2", rot=D,
                                     freq=p["freq"], positions=pos)
        ot = F.falcon_decode_step(Sd, kp, qt[:, :, 0].contiguous(), kt[:, :, 0].contiguous(), x[2],
                                  p["alpha"][:, :, t].contiguous(), p["eta"][:, :, t].contiguous())
        assert float((ot - o[:, :, t]).abs().max()) <= 1e-4 * float(o.abs().max())
    assert float((Sd - S).abs().max()) <= 1e-4 * float(S.abs().max())


def test_side_stream(F):
    p = layer(6)
    (q, k, v), _, _ = forward(F, p)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        y, tail = F.falcon_conv_fwd(p["qkv"][:, :, 0].transpose(1, 2), p["w"][0], want_state=True, stream=handle)
        y2, _ = F.falcon_conv_fwd(p["qkv"][:, :, 1].transpose(1, 2), p["w"][1], stream=handle)
        a, b = F.falcon_qknorm_fwd(y, y2, wq=p["wq"], wk=p["wk"], norm="l2", rot=D, freq=p["freq"], stream=handle)
        s.synchronize()
        assert torch.equal(a, q) and torch.equal(b, k)
    with torch.cuda.stream(s):
        (a, b, c), _, _ = forward(F, p)
    s.synchronize()
    assert torch.equal(a, q) and torch.equal(b, k) and torch.equal(c, v)


def test_captured_layers(F):
    """Forward and backward of a scan layer in one graph, replayed on new inputs; two graphs side by side, each
    with workspaces of its own."""
    T2 = 1500
    g = torch.Generator().manual_seed(7)
    new = lambda: {n: torch.randn(1, 2, T2, d, generator=g).cuda() for n, d in (("q", 16), ("k", 16), ("v", 24), ("delta", 24), ("z", 24))}
    A, dO = -torch.rand(2, 24, 16, generator=g).cuda(), torch.randn(1, 2, T2, 24, generator=g).cuda()
    w = torch.randn(2, 24, 4, generator=g).cuda()

    def run(x):
        v, _ = F.falcon_conv_fwd(x["v"], w)
        o, S = F.falcon_scan_fwd(x["q"], x["k"], v, x["delta"], A, z=x["z"])
        r = F.falcon_scan_bwd(x["q"], x["k"], v, x["delta"], A, dO, z=x["z"])
        c = F.falcon_conv_bwd(x["v"], w, r["dv"])
        return [o, S, r["dq"], r["dk"], r["dA"], r["dz"], r["ddelta"], c["dx"], c["dw"]]

    graphs = []
    for _ in range(2):
        x = new()
        run(x)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(x)
        graphs.append((graph, x, out))
    for _ in range(2):
        want = []
        for graph, x, out in graphs:
            y = new()
            for n in x:
                x[n].copy_(y[n])
            want.append([t.clone() for t in run(x)])
        for graph, _, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for (graph, x, out), w_ in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w_))
