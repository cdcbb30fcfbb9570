"""Host checks of the operators around the memory, through the C ABI (no kernel runs): struct layouts,
refusals, workspace sizes, and empty problems."""
import ctypes
import os
import subprocess

import pytest
import torch

from delta_rule_linear_falcon_b200 import build as B
from delta_rule_linear_falcon_b200 import falcon as F

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    B.build()
    return F.lib()


@pytest.mark.parametrize("mirror,ctype", [
    (F.FalconView, "falcon_view_t"), (F.FalconConvArgs, "falcon_conv_args_t"), (F.FalconConvGrads, "falcon_conv_grads_t"),
    (F.FalconScanArgs, "falcon_scan_args_t"), (F.FalconScanGrads, "falcon_scan_grads_t"),
    (F.FalconQknormArgs, "falcon_qknorm_args_t"), (F.FalconQknormGrads, "falcon_qknorm_grads_t")])
def test_struct_layout_matches_header(tmp_path, mirror, ctype):
    fields = [f[0] for f in mirror._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "falcon.h"\nint main(void) {\n'
                   + "".join(f'  printf("{f} %zu\\n", offsetof({ctype}, {f}));\n' for f in fields)
                   + f'  printf("sizeof %zu\\n", sizeof({ctype}));\n  return 0;\n}}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for f in fields:
        assert getattr(mirror, f).offset == int(got[f]), f
    assert ctypes.sizeof(mirror) == int(got["sizeof"])


@pytest.mark.parametrize("packer,mirror", [
    (F._CONV_ARGS, F.FalconConvArgs), (F._CONV_GRADS, F.FalconConvGrads), (F._SCAN_ARGS, F.FalconScanArgs),
    (F._SCAN_GRADS, F.FalconScanGrads), (F._QKNORM_ARGS, F.FalconQknormArgs), (F._QKNORM_GRADS, F.FalconQknormGrads)])
def test_packed_structs_are_the_mirrors(packer, mirror):
    """The calls pack their structs as bytes: the same layout, field by field."""
    flat, count = [], iter(range(1, 1000))

    def fill(s):
        for name, kind in s._fields_:
            if kind is F.FalconView:
                fill(getattr(s, name))
            else:
                x = next(count)
                setattr(s, name, x)
                flat.append(float(x) if kind is ctypes.c_float else x)

    s = mirror()
    fill(s)
    packed = packer.pack(*flat)
    assert len(packed) == ctypes.sizeof(mirror)
    assert bytes(mirror.from_buffer_copy(packed)) == packed
    again = mirror.from_buffer_copy(packed)
    same = lambda a, b: all(same(getattr(a, n), getattr(b, n)) if k is F.FalconView else getattr(a, n) == getattr(b, n)
                            for n, k in a._fields_)
    assert same(s, again)


def view(p, B, H, T, d):
    return F.FalconView(p, H * T * d, T * d, d)


def conv(**kw):
    a = dict(io_dtype=1, B=2, H=3, T=10, d=64, K=4, act=1, w=0x3000, bias=None, lengths=None, state=None, state_out=None)
    a.update({k: v for k, v in kw.items() if k not in ("x", "y")})
    s = F.FalconConvArgs(**a)
    s.x = kw.get("x", view(0x1000, 2, 3, a["T"], 64))
    s.y = kw.get("y", view(0x2000, 2, 3, a["T"], 64))
    return s


CONV_BAD = [
    (dict(io_dtype=3), INVALID), (dict(B=-1), INVALID), (dict(d=0), INVALID), (dict(K=0), INVALID), (dict(act=2), INVALID),
    (dict(K=9), UNSUPPORTED), (dict(T=(1 << 30) + 1), UNSUPPORTED), (dict(H=1 << 30, B=4), UNSUPPORTED),
    (dict(w=None), INVALID), (dict(w=0x3002), INVALID), (dict(bias=0x3001), INVALID), (dict(lengths=0x3002), INVALID),
    (dict(state=0x3001), INVALID), (dict(x=view(None, 2, 3, 10, 64)), INVALID), (dict(x=view(0x1001, 2, 3, 10, 64)), INVALID),
    (dict(x=F.FalconView(0x1000, -1, 640, 64)), INVALID), (dict(x=F.FalconView(0x1000, 1 << 61, 640, 64)), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,expect", CONV_BAD + [
    (dict(y=view(None, 2, 3, 10, 64)), INVALID), (dict(y=view(0x1000, 2, 3, 10, 64)), INVALID),   # y = x
    (dict(y=F.FalconView(0x2000, 640 * 3, 640, 0)), INVALID),       # tokens on top of each other
    (dict(y=F.FalconView(0x2000, 640 * 3, 63, 192)), INVALID),      # heads overlap by one channel
    (dict(state_out=0x3001), INVALID)])
def test_conv_fwd_refuses(L, kw, expect):
    assert L.falcon_conv_fwd(ctypes.byref(conv(**kw)), None) == expect


@pytest.mark.parametrize("kw,expect", [(dict(T=2), INVALID), (dict(T=1), INVALID), (dict(T=1, state=0x4000), INVALID),
                                       (dict(T=1, state=0x4000, state_out=0x4000, lengths=0x5000), INVALID)])
def test_conv_step_refuses(L, kw, expect):
    assert L.falcon_conv_step(ctypes.byref(conv(**kw)), None) == expect


def conv_grads(**kw):
    a = dict(dstate_out=None, dw=0x9000, dbias=None, dstate=None)
    a.update({k: v for k, v in kw.items() if k not in ("dy", "dx")})
    g = F.FalconConvGrads(**a)
    g.dy, g.dx = kw.get("dy", view(0x7000, 2, 3, 10, 64)), kw.get("dx", view(0x8000, 2, 3, 10, 64))
    return g


@pytest.mark.parametrize("kw,expect", CONV_BAD)
def test_conv_bwd_refuses_its_forward_arguments(L, kw, expect):
    assert L.falcon_conv_bwd(ctypes.byref(conv(**kw)), ctypes.byref(conv_grads()), 0x10000, 1 << 40, None) == expect
    assert L.falcon_conv_bwd_workspace_size(ctypes.byref(conv(**kw))) == 0


@pytest.mark.parametrize("kw,ws,n,expect", [
    (dict(dw=None), 0x10000, 1 << 40, INVALID), (dict(dy=view(None, 2, 3, 10, 64)), 0x10000, 1 << 40, INVALID),
    (dict(dx=view(0x8002, 2, 3, 10, 64)), 0x10000, 1 << 40, INVALID), (dict(dx=view(0x7000, 2, 3, 10, 64)), 0x10000, 1 << 40, INVALID),
    (dict(dx=F.FalconView(0x8000, 0, 640, 64)), 0x10000, 1 << 40, INVALID),
    (dict(), None, 0, WORKSPACE), (dict(), 0x10000, 64, WORKSPACE), (dict(), 0x10008, 1 << 40, INVALID)])
def test_conv_bwd_refuses(L, kw, ws, n, expect):
    assert L.falcon_conv_bwd(ctypes.byref(conv()), ctypes.byref(conv_grads(**kw)), ws, n, None) == expect


def scan(**kw):
    a = dict(io_dtype=1, B=2, H=3, T=10, dk=16, dv=64, flags=1, A=0x6000, D=None, delta_bias=None, lengths=None, S0=None, S_out=None)
    views = ("q", "k", "v", "delta", "z", "o")
    a.update({k: v for k, v in kw.items() if k not in views})
    s = F.FalconScanArgs(**a)
    for i, n in enumerate(views):
        if n != "z":
            setattr(s, n, view(0x1000 * (i + 1), 2, 3, a["T"], a["dk"] if n in "qk" else a["dv"]))
    for n in views:
        if n in kw:
            setattr(s, n, kw[n])
    return s


SCAN_BAD = [
    (dict(io_dtype=2), INVALID), (dict(dk=0), INVALID), (dict(dv=-1), INVALID), (dict(T=-1), INVALID), (dict(flags=2), INVALID),
    (dict(dk=129), UNSUPPORTED), (dict(A=None), INVALID), (dict(A=0x6001), INVALID), (dict(D=0x6002), INVALID),
    (dict(delta_bias=0x6001), INVALID), (dict(S0=0x6002), INVALID), (dict(lengths=0x6001), INVALID),
    (dict(q=view(None, 2, 3, 10, 16)), INVALID), (dict(delta=view(0x1001, 2, 3, 10, 64)), INVALID),
    (dict(z=view(0x1001, 2, 3, 10, 64)), INVALID),
]


@pytest.mark.parametrize("kw,expect", SCAN_BAD + [(dict(o=view(None, 2, 3, 10, 64)), INVALID), (dict(S_out=0x6002), INVALID),
                                                  (dict(o=F.FalconView(0x9000, 1920, 640, 63)), INVALID)])
def test_scan_fwd_refuses(L, kw, expect):
    assert L.falcon_scan_fwd(ctypes.byref(scan(**kw)), None, 0, None) == expect


@pytest.mark.parametrize("kw,expect", [(dict(), INVALID), (dict(T=1), INVALID), (dict(T=1, S0=0x7000), INVALID),
                                       (dict(T=1, S0=0x7000, S_out=0x7000, lengths=0x8000), INVALID)])
def test_scan_step_refuses(L, kw, expect):
    assert L.falcon_scan_step(ctypes.byref(scan(**kw)), None) == expect


def scan_grads(**kw):
    g = F.FalconScanGrads(dS_T=kw.get("dS_T"), dA=kw.get("dA", 0x20000), dD=kw.get("dD"), ddelta_bias=None, dS0=kw.get("dS0"))
    for i, n in enumerate(("dO", "dq", "dk", "dv", "ddelta", "dz")):
        if n != "dz":
            setattr(g, n, view(0x21000 + 0x1000 * i, 2, 3, 10, 16 if n in ("dq", "dk") else 64))
        if n in kw:
            setattr(g, n, kw[n])
    return g


@pytest.mark.parametrize("kw,ws,n,expect", [
    (dict(dA=None), 0x10000, 1 << 40, INVALID), (dict(dO=view(None, 2, 3, 10, 64)), 0x10000, 1 << 40, INVALID),
    (dict(dq=F.FalconView(0x22000, 160, 0, 16)), 0x10000, 1 << 40, INVALID),    # one gradient for all heads
    (dict(dz=view(0x22000, 2, 3, 10, 64)), 0x10000, 1 << 40, INVALID),          # without z
    (dict(dS_T=0x22002), 0x10000, 1 << 40, INVALID), (dict(dS0=0x22002), 0x10000, 1 << 40, INVALID),
    (dict(), None, 0, WORKSPACE), (dict(), 0x10000, 4096, WORKSPACE), (dict(), 0x10004, 1 << 40, INVALID)])
def test_scan_bwd_refuses(L, kw, ws, n, expect):
    assert L.falcon_scan_bwd(ctypes.byref(scan()), ctypes.byref(scan_grads(**kw)), ws, n, None) == expect


@pytest.mark.parametrize("kw,expect", SCAN_BAD)
def test_scan_bwd_refuses_its_forward_arguments(L, kw, expect):
    assert L.falcon_scan_bwd(ctypes.byref(scan(**kw)), ctypes.byref(scan_grads()), 0x10000, 1 << 40, None) == expect
    assert L.falcon_scan_bwd_workspace_size(ctypes.byref(scan(**kw))) == 0


def qknorm(**kw):
    a = dict(io_dtype=1, B=2, Hq=3, Hk=1, T=10, d=64, norm=1, rot=64, rot_layout=0, wq=None, wk=None, eps=1e-6, freq=0x6000,
             positions=None, lengths=None)
    views = ("q", "k", "q_out", "k_out")
    a.update({k: v for k, v in kw.items() if k not in views})
    s = F.FalconQknormArgs(**a)
    for i, n in enumerate(views):
        setattr(s, n, kw.get(n, view(0x1000 * (i + 1), 2, 3 if n[0] == "q" else 1, 10, 64)))
    return s


QKNORM_BAD = [
    (dict(io_dtype=9), INVALID), (dict(norm=3), INVALID), (dict(rot_layout=2), INVALID), (dict(rot=3), INVALID),
    (dict(rot=66), INVALID), (dict(rot=-2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(freq=None), INVALID), (dict(freq=0x6001), INVALID), (dict(positions=0x6002), INVALID), (dict(wq=0x6002), INVALID),
    (dict(d=257), UNSUPPORTED), (dict(Hq=70000), UNSUPPORTED), (dict(Hk=-1), INVALID), (dict(q=view(None, 2, 3, 10, 64)), INVALID),
]


@pytest.mark.parametrize("kw,expect", QKNORM_BAD + [
    (dict(q_out=F.FalconView(0x3000, 1920, 640, 0)), INVALID), (dict(k_out=view(None, 2, 1, 10, 64)), INVALID),
    (dict(q_out=F.FalconView(0x1000, 1920, 64, 192)), INVALID)])        # q's memory in another order
def test_qknorm_fwd_refuses(L, kw, expect):
    assert L.falcon_qknorm_fwd(ctypes.byref(qknorm(**kw)), None) == expect


def qknorm_grads(**kw):
    g = F.FalconQknormGrads(dwq=kw.get("dwq"), dwk=None)
    for i, n in enumerate(("dq_out", "dk_out", "dq", "dk")):
        setattr(g, n, kw.get(n, view(0x11000 + 0x1000 * i, 2, 3 if "q" in n else 1, 10, 64)))
    return g


@pytest.mark.parametrize("kw,expect", QKNORM_BAD)
def test_qknorm_bwd_refuses_its_forward_arguments(L, kw, expect):
    assert L.falcon_qknorm_bwd(ctypes.byref(qknorm(**kw)), ctypes.byref(qknorm_grads()), 0x10000, 1 << 40, None) == expect


@pytest.mark.parametrize("kw,ws,n,expect", [
    (dict(dq=view(None, 2, 3, 10, 64)), None, 0, INVALID), (dict(dk=F.FalconView(0x9000, 0, 0, 64)), None, 0, INVALID),
    (dict(dwq=0x9002), 0x10000, 1 << 40, INVALID), (dict(dwq=0x9000), None, 0, WORKSPACE), (dict(dwq=0x9000), 0x10000, 16, WORKSPACE),
    (dict(dwq=0x9000), 0x10004, 1 << 40, INVALID)])
def test_qknorm_bwd_refuses(L, kw, ws, n, expect):
    assert L.falcon_qknorm_bwd(ctypes.byref(qknorm()), ctypes.byref(qknorm_grads(**kw)), ws, n, None) == expect


def test_null_structs(L):
    for name in ("conv", "scan", "qknorm"):
        assert getattr(L, f"falcon_{name}_bwd_workspace_size")(None) == 0
    assert L.falcon_scan_workspace_size(None) == 0
    assert L.falcon_conv_fwd(None, None) == INVALID and L.falcon_conv_step(None, None) == INVALID
    assert L.falcon_conv_bwd(None, None, None, 0, None) == INVALID
    assert L.falcon_conv_bwd(ctypes.byref(conv()), None, None, 0, None) == INVALID
    assert L.falcon_scan_fwd(None, None, 0, None) == INVALID and L.falcon_scan_step(None, None) == INVALID
    assert L.falcon_scan_bwd(ctypes.byref(scan()), None, None, 0, None) == INVALID
    assert L.falcon_qknorm_fwd(None, None) == INVALID
    assert L.falcon_qknorm_bwd(ctypes.byref(qknorm()), None, None, 0, None) == INVALID


def test_empty_problems_need_nothing(L):
    none = F.FalconView()
    assert L.falcon_conv_fwd(ctypes.byref(conv(B=0, x=none, y=none, w=None)), None) == OK
    assert L.falcon_scan_fwd(ctypes.byref(scan(H=0, q=none, k=none, v=none, delta=none, o=none, A=None)), None, 0, None) == OK
    assert L.falcon_qknorm_fwd(ctypes.byref(qknorm(T=0, q=none, k=none, q_out=none, k_out=none, freq=None)), None) == OK


def test_well_formed_calls_fail_loudly_without_a_gpu(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert L.falcon_conv_fwd(ctypes.byref(conv()), None) == CUDA
    assert L.falcon_conv_step(ctypes.byref(conv(T=1, state=0x4000, state_out=0x4000)), None) == CUDA
    assert L.falcon_conv_bwd(ctypes.byref(conv()), ctypes.byref(conv_grads()), 0x10000, 1 << 40, None) == CUDA
    assert L.falcon_scan_fwd(ctypes.byref(scan()), None, 0, None) == CUDA
    assert L.falcon_scan_step(ctypes.byref(scan(T=1, S0=0x7000, S_out=0x7000)), None) == CUDA
    assert L.falcon_scan_bwd(ctypes.byref(scan()), ctypes.byref(scan_grads()), 0x10000, 1 << 40, None) == CUDA
    assert L.falcon_qknorm_fwd(ctypes.byref(qknorm()), None) == CUDA
    assert L.falcon_qknorm_bwd(ctypes.byref(qknorm()), ctypes.byref(qknorm_grads()), None, 0, None) == CUDA


def test_the_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 2, 3, 4)
    with pytest.raises(TypeError, match="CUDA"):
        F.falcon_conv_fwd(x, torch.zeros(2, 4, 3))
    with pytest.raises(TypeError, match="CUDA"):
        F.falcon_scan_fwd(x, x, x, x, torch.zeros(2, 4, 4))
    with pytest.raises(TypeError, match="CUDA"):
        F.falcon_qknorm_fwd(x, x)
    with pytest.raises(TypeError):
        F.falcon_qknorm_fwd(None, None)
