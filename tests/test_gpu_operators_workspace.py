"""Workspaces that the caller keeps: their sizes through the binding, calls with exactly as much, refusals of less, and
captured graphs with workspaces of their own."""
import ctypes

import pytest
import torch

from test_gpu_operators import F, conv_inputs, norm_inputs, scan_inputs  # noqa: F401

pytestmark = pytest.mark.gpu


def calls(F, seed):
    """(size, call with a workspace, name) of every operator that takes one."""
    _, c, r = conv_inputs(seed, "bf16", 3, 4, 700, 64, 4, True, True, "slice")
    dy = r(3, 4, 700, 64)[1]
    _, s, r = scan_inputs(seed + 1, "bf16", 2, 2, 900, 16, 160, True, True, True, True, "token")
    dO = r(2, 2, 900, 160)[1]
    q, k, wq, wk, freq, _, r = norm_inputs(seed + 2, "f32", 2, 4, 2, 90, 64, True, 64, None, False)
    gq, gk = r(2, 4, 90, 64)[1], r(2, 2, 90, 64)[1]
    kw = dict(wq=wq[1], wk=wk[1], rot=64, freq=freq.cuda())
    conv = dict(bias=c["bias"], state=c["state"])
    return [
        (F.falcon_conv_bwd_workspace_size(F.make_conv_args(c["x"], c["w"], **conv)),
         lambda ws: F.falcon_conv_bwd(c["x"], c["w"], dy, workspace=ws, **conv), "falcon_conv_bwd"),
        (F.falcon_scan_bwd_workspace_size(F.make_scan_args(**s)), lambda ws: F.falcon_scan_bwd(**s, dO=dO, workspace=ws), "falcon_scan_bwd"),
        (F.falcon_qknorm_bwd_workspace_size(F.make_qknorm_args(q[1], k[1], **kw)),
         lambda ws: F.falcon_qknorm_bwd(q[1], k[1], gq, gk, workspace=ws, **kw), "falcon_qknorm_bwd"),
        (F.falcon_scan_workspace_size(F.make_scan_args(**s)), lambda ws: F.falcon_scan_fwd(**s, workspace=ws), "falcon_scan_fwd"),
    ]


def flat(out):
    return [t for t in (out.values() if isinstance(out, dict) else out) if t is not None]


def test_exactly_as_much_is_enough(F):
    for size, call, name in calls(F, 60):
        assert size > 0, name
        guard = 4096
        ws = torch.full((size + guard,), 0xA5, dtype=torch.uint8, device="cuda")
        for a, b in zip(flat(call(None)), flat(call(ws[:size]))):
            assert torch.equal(a, b), name
        assert (ws[size:] == 0xA5).all(), name      # nothing behind it is written
        if name != "falcon_scan_fwd":               # which runs the sequence whole
            with pytest.raises(F.FalconError) as e:
                call(ws[:size - 16])
            assert e.value.status == F.FALCON_ERR_WORKSPACE, name


def test_sizes_do_not_need_the_optional_tensors(F):
    """What the documentation names: the sequence tensors and the weights are enough."""
    _, c, _ = conv_inputs(63, "f32", 2, 3, 300, 20, 4, True, True, None)
    _, s, _ = scan_inputs(64, "f32", 1, 1, 2000, 16, 32, True, True, True, True, None)
    few = {n: s[n] for n in ("q", "k", "v", "delta", "A")}
    same = lambda f, a, b: f(a) == f(b) > 0
    assert same(F.falcon_conv_bwd_workspace_size, F.make_conv_args(c["x"], c["w"]), F.make_conv_args(**c))
    assert same(F.falcon_scan_workspace_size, F.make_scan_args(**few), F.make_scan_args(**s))
    assert same(F.falcon_scan_bwd_workspace_size, F.make_scan_args(**few), F.make_scan_args(**s))
    x = c["x"]
    assert same(F.falcon_qknorm_bwd_workspace_size, F.make_qknorm_args(x, None), F.make_qknorm_args(x, x, norm="l2"))
    a = F.make_scan_args(**s, o=torch.empty_like(s["v"]), S_out=s["S0"])
    assert (a.B, a.H, a.T, a.dk, a.dv, a.flags) == (1, 1, 2000, 16, 32, F.FALCON_SCAN_SOFTPLUS) and ctypes.sizeof(a) > 0


def test_graphs_with_workspaces_of_their_own(F):
    """Two graphs captured with kept workspaces, replayed on two streams at once."""
    s0 = torch.cuda.Stream()
    jobs = []
    for seed in (70, 80):
        cs = calls(F, seed)
        ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for size, _, _ in cs]
        want = [[t.clone() for t in flat(call(w))] for (_, call, _), w in zip(cs, ws)]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = [flat(call(w)) for (_, call, _), w in zip(cs, ws)]
        jobs.append((graph, ws, cs, want, out))
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s0):
            jobs[0][0].replay()
        jobs[1][0].replay()
    torch.cuda.synchronize()
    for _, _, _, want, out in jobs:
        for a, b in zip(want, out):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
