"""tests/plans.py against the workspace sizes of the library, over the sizes of test_gpu_operators_plans.py and drawn ones
(no kernel runs)."""
import ctypes
import random

import pytest

import plans
import test_gpu_operators_plans as P
from delta_rule_linear_falcon_b200 import falcon as F
from test_abi_operators import L, UNSUPPORTED, conv, scan, view  # noqa: F401

DRAW = random.Random(3)
SIZES = lambda: (DRAW.randint(1, 300), DRAW.randint(1, 8), DRAW.randint(1, 5000))


@pytest.mark.parametrize("B,H,T,dk,dv", [c[1:6] for c in P.SCAN] + [SIZES() + (DRAW.randint(1, 128), DRAW.randint(1, 600)) for _ in range(40)])
def test_scan(L, B, H, T, dk, dv):
    a = scan(B=B, H=H, T=T, dk=dk, dv=dv)
    for n in ("q", "k", "v", "delta"):
        setattr(a, n, view(0x1000, B, H, T, dk if n in "qk" else dv))
    assert F.falcon_scan_bwd_workspace_size(a) == plans.ScanBwd(B, H, T, dk, dv).bytes


@pytest.mark.parametrize("B,H,T,d,K", [c[1:6] for c in P.CONV] + [SIZES() + (DRAW.randint(1, 300), DRAW.randint(1, 8)) for _ in range(40)])
def test_conv(L, B, H, T, d, K):
    a = conv(B=B, H=H, T=T, d=d, K=K, x=view(0x1000, B, H, T, d))
    assert F.falcon_conv_bwd_workspace_size(a) == plans.conv_workspace(B, H, T, d, K)


@pytest.mark.parametrize("d,K", [(2 ** 31 - 1, 1), (2 ** 31 - 1, 8), (2 ** 31 - 2, 4)])
def test_the_widest_convolution(L, d, K):
    a = conv(B=1, H=1, T=3, d=d, K=K, x=view(0x1000, 1, 1, 3, d))
    assert F.falcon_conv_bwd_workspace_size(a) == plans.conv_workspace(1, 1, 3, d, K)


def test_the_widest_scan(L):
    def size(dv):
        a = scan(B=1, H=1, T=1, dk=1, dv=dv)
        for n in ("q", "k", "v", "delta", "o"):
            setattr(a, n, view(0x1000 * (1 + "qkvdo".index(n[0])), 1, 1, 1, 1 if n in "qk" else dv))
        return a, F.falcon_scan_bwd_workspace_size(a)

    assert size(2 ** 31 - 512)[1] == plans.ScanBwd(1, 1, 1, 1, 2 ** 31 - 512).bytes
    for dv in (2 ** 31 - 511, 2 ** 31 - 1):
        a, n = size(dv)
        assert n == 0
        assert L.falcon_scan_fwd(ctypes.byref(a), None, 0, None) == UNSUPPORTED
        a.S0 = a.S_out = 0x100000
        assert L.falcon_scan_step(ctypes.byref(a), None) == UNSUPPORTED
