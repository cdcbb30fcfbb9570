"""Host checks of the operators around the memory: an output that starts where an input or another output does is
refused (no kernel runs), except where the header allows it."""
import ctypes
import subprocess
import sys

import pytest
import torch

from delta_rule_linear_falcon_b200 import falcon as F
from test_abi_operators import (CUDA, INVALID, L, OK, UNSUPPORTED, conv, conv_grads, qknorm, qknorm_grads, scan, scan_grads,  # noqa: F401
                                view)

R = ctypes.byref
HERE = pytest.mark.skipif(torch.cuda.is_available(), reason="a well-formed call would run")


def same(a, b, src, dst):
    """Field dst of b becomes field src of a."""
    setattr(b, dst, getattr(a, src))


@pytest.mark.parametrize("name", ["q", "k", "v", "delta", "z"])
def test_scan_output_on_an_input(L, name):
    a = scan(dk=64)     # rows of one width
    a.z = view(0x30000, 2, 3, 10, 64)
    same(a, a, name, "o")
    assert L.falcon_scan_fwd(R(a), None, 0, None) == INVALID
    a = scan(dk=64, T=1, S0=0x70000, S_out=0x70000)
    a.z = view(0x30000, 2, 3, 1, 64)
    same(a, a, name, "o")
    assert L.falcon_scan_step(R(a), None) == INVALID


def test_scan_states_on_sequences(L):
    a = scan(io_dtype=0, S0=0x70000, S_out=0x3000)      # v
    assert L.falcon_scan_fwd(R(a), None, 0, None) == INVALID
    a = scan(io_dtype=0, S_out=0x6000)                  # o
    assert L.falcon_scan_fwd(R(a), None, 0, None) == INVALID
    a = scan(io_dtype=0, S0=0x6000)
    assert L.falcon_scan_fwd(R(a), None, 0, None) == INVALID


@pytest.mark.parametrize("grad", ["dq", "dk", "dv", "ddelta", "dz"])
@pytest.mark.parametrize("other", ["dO", "q", "k", "v", "delta", "z"])
def test_scan_gradients_on_inputs(L, grad, other):
    a, g = scan(dk=64, io_dtype=0), scan_grads(dq=view(0x22000, 2, 3, 10, 64), dk=view(0x23000, 2, 3, 10, 64), dz=view(0x26000, 2, 3, 10, 64))
    a.z = view(0x30000, 2, 3, 10, 64)
    same(g if other == "dO" else a, g, other, grad)
    assert L.falcon_scan_bwd(R(a), R(g), 0x10000, 1 << 40, None) == INVALID


@pytest.mark.parametrize("kw", [dict(dq=view(0x23000, 2, 3, 10, 16)), dict(dv=view(0x25000, 2, 3, 10, 64)), dict(dA=0x24000),
                                dict(dS0=0x20000), dict(dD=0x20000)])
def test_scan_gradients_on_each_other(L, kw):
    assert L.falcon_scan_bwd(R(scan()), R(scan_grads(**kw)), 0x10000, 1 << 40, None) == INVALID


def test_scan_gradient_of_the_state_on_the_state(L):
    assert L.falcon_scan_bwd(R(scan(S0=0x40000)), R(scan_grads(dS0=0x40000)), 0x10000, 1 << 40, None) == INVALID


@pytest.mark.parametrize("kw", [dict(state=0x2000), dict(state_out=0x2000), dict(state_out=0x1000)])
def test_conv_outputs(L, kw):
    assert L.falcon_conv_fwd(R(conv(**kw)), None) == INVALID


@pytest.mark.parametrize("a,g", [
    (dict(), dict(dstate_out=0xa000, dstate=0xa000)),      # a row of dstate is written before dstate_out's is read
    (dict(state=0xa000), dict(dstate=0xa000)), (dict(), dict(dbias=0x9000)), (dict(), dict(dstate=0x8000)),
    (dict(io_dtype=0), dict(dx=view(0x1000, 2, 3, 10, 64))), (dict(), dict(dw=0x7000)), (dict(), dict(dstate_out=0x8000))])
def test_conv_gradients(L, a, g):
    assert L.falcon_conv_bwd(R(conv(**a)), R(conv_grads(**g)), 0x10000, 1 << 40, None) == INVALID


@pytest.mark.parametrize("kw", [dict(q_out=view(0x2000, 2, 3, 10, 64)), dict(k_out=view(0x1000, 2, 1, 10, 64)),
                                dict(k_out=view(0x3000, 2, 1, 10, 64))])
def test_qknorm_outputs(L, kw):
    assert L.falcon_qknorm_fwd(R(qknorm(**kw)), None) == INVALID


@pytest.mark.parametrize("kw", [dict(dq=view(0x12000, 2, 3, 10, 64)), dict(dk=view(0x11000, 2, 1, 10, 64)), dict(dk=view(0x13000, 2, 1, 10, 64)),
                                dict(dq=view(0x1000, 2, 3, 10, 64)), dict(dwq=0x13000)])
def test_qknorm_gradients(L, kw):
    assert L.falcon_qknorm_bwd(R(qknorm(io_dtype=0)), R(qknorm_grads(**kw)), 0x10000, 1 << 40, None) == INVALID


@HERE
def test_what_the_header_allows_is_not_refused(L):
    """In place where an entry point says so, inputs on each other, and equal addresses of what is empty: these calls
    get as far as looking for a device."""
    assert L.falcon_conv_fwd(R(conv(state=0x4000, state_out=0x4000)), None) == CUDA
    assert L.falcon_conv_fwd(R(conv(K=1, state=0x2000, state_out=0x1000)), None) == CUDA
    assert L.falcon_conv_fwd(R(conv(T=0, state_out=0x1000)), None) == CUDA
    a = scan(dk=64, S0=0x70000, S_out=0x70000)
    a.k, a.v, a.delta, a.z = a.q, a.q, a.q, a.q
    assert L.falcon_scan_fwd(R(a), None, 0, None) == CUDA
    assert L.falcon_scan_bwd(R(a), R(scan_grads(dS_T=0x40000, dS0=0x40000, dq=view(0x32000, 2, 3, 10, 64), dk=view(0x33000, 2, 3, 10, 64))),
                             0x10000, 1 << 40, None) == CUDA
    a = qknorm()
    a.q_out, a.k_out = a.q, a.k
    assert L.falcon_qknorm_fwd(R(a), None) == CUDA
    a.k = a.q
    a.k_out = view(0x4000, 2, 1, 10, 64)
    a.q_out = view(0x3000, 2, 3, 10, 64)
    assert L.falcon_qknorm_fwd(R(a), None) == CUDA
    g = qknorm_grads()
    g.dq, g.dk = g.dq_out, g.dk_out
    assert L.falcon_qknorm_bwd(R(qknorm()), R(g), None, 0, None) == CUDA
    a = qknorm(Hk=0, k_out=view(0x3000, 2, 0, 10, 64))
    assert L.falcon_qknorm_fwd(R(a), None) == CUDA
    none = scan(B=0)
    none.o = none.q
    assert L.falcon_scan_fwd(R(none), None, 0, None) == OK


@pytest.mark.parametrize("kw", [
    dict(B=8, H=8, T=1000, dk=128, dv=1 << 27),          # the joins' grid: states of 2^33 channels
    dict(B=1 << 20, H=1, T=1 << 15, dk=128, dv=17),      # the sums of dq and dk over a head's two blocks
    dict(B=1 << 24, H=1, T=1 << 16, dk=1, dv=1)])        # the main grid: 2^24 sequences of 128 walks
def test_scan_backward_refuses_before_its_first_launch(L, kw):
    a, g = scan(**kw), scan_grads()
    for s, names in ((a, ("q", "k", "v", "delta")), (g, ("dO", "dq", "dk", "dv", "ddelta"))):
        for i, n in enumerate(names):
            d = kw["dk"] if n in ("q", "k", "dq", "dk") else kw["dv"]
            setattr(s, n, view((0x100000 if s is g else 0x200000) + 0x1000 * i, kw["B"], kw["H"], kw["T"], d))
    assert L.falcon_scan_bwd_workspace_size(R(a)) > 1 << 40
    assert L.falcon_scan_bwd(R(a), R(g), 0x10000, (1 << 64) - 16, None) == UNSUPPORTED


@HERE
def test_in_place_whatever_the_stride_of_an_axis_of_one(L):
    """A single token's rows seen as (B, T, H, d) transposed and as (B, H, T, d): the same memory in the same order."""
    a = qknorm(T=1)
    a.q, a.q_out = F.FalconView(0x1000, 192, 64, 192), F.FalconView(0x1000, 192, 64, 64)
    a.k, a.k_out = F.FalconView(0x2000, 64, 64, 64), F.FalconView(0x2000, 64, 7, 0)
    assert L.falcon_qknorm_fwd(R(a), None) == CUDA
    g = F.FalconQknormGrads()
    g.dq_out, g.dq, g.dk_out, g.dk = a.q, a.q_out, a.k, a.k_out
    b = qknorm(T=1, q=F.FalconView(0x11000, 192, 64, 64), k=F.FalconView(0x12000, 64, 64, 64))
    assert L.falcon_qknorm_bwd(R(b), R(g), None, 0, None) == CUDA
    a.q_out = F.FalconView(0x1000, 192, 65, 64)      # another order
    assert L.falcon_qknorm_fwd(R(a), None) == INVALID


@HERE
@pytest.mark.parametrize("kw", [dict(B=0), dict(T=0)])
def test_nothing_is_in_place(L, kw):
    """Empty tensors of torch all have the address 0, whatever their strides."""
    none = F.FalconView(0, 640, 64, 192)
    a = qknorm(**kw, q=none, k=none, q_out=F.FalconView(0, 640, 10, 64), k_out=F.FalconView(0, 640, 640, 64))
    assert L.falcon_qknorm_fwd(R(a), None) == OK
    g = qknorm_grads(dq_out=none, dk_out=none, dq=F.FalconView(0, 640, 10, 64), dk=F.FalconView(0, 640, 640, 64), dwq=0x9000)
    assert L.falcon_qknorm_bwd(R(a), R(g), None, 0, None) == CUDA


def test_sizes_of_nothing(L):
    """Workspace sizes of no sequences, heads or tokens (in a process of its own: without heads the convolution's once
    divided by zero)."""
    code = """
import sys; sys.path[:0] = {path!r}
import ctypes
from test_abi_operators import B, F, conv, qknorm, scan
L = F.lib()
R = ctypes.byref
for b in (0, 2):
    for h in (0, 3):
        for t in (0, 1, 10):
            n = F.FalconView()
            if b * h == 0:
                assert L.falcon_conv_bwd_workspace_size(R(conv(B=b, H=h, T=t, x=n, w=None))) == 0, (b, h, t)
                assert L.falcon_scan_bwd_workspace_size(R(scan(B=b, H=h, T=t, q=n, k=n, v=n, delta=n, A=None))) == 0, (b, h, t)
                assert L.falcon_qknorm_bwd_workspace_size(R(qknorm(B=b, Hq=h, Hk=0, T=t, q=n, k=n, freq=None))) == 0, (b, h, t)
                assert L.falcon_scan_workspace_size(R(scan(B=b, H=h, T=t, q=n, k=n, v=n, delta=n, A=None))) == 0, (b, h, t)
            else:
                L.falcon_conv_bwd_workspace_size(R(conv(B=b, H=h, T=t)))
                L.falcon_scan_bwd_workspace_size(R(scan(B=b, H=h, T=t)))
                L.falcon_qknorm_bwd_workspace_size(R(qknorm(B=b, Hq=h, T=t)))
print("all")
"""
    r = subprocess.run([sys.executable, "-c", code.format(path=sys.path)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout == "all\n", (r.returncode, r.stderr[-500:])
