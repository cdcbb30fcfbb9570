"""The whole-tensor 64-bit forms of test_gpu_operators_plans.py against the token-by-token ones of oracle/operators.py."""
import pytest
import torch

import test_gpu_operators_plans as P
from oracle import operators as O


@pytest.fixture(autouse=True)
def on_the_cpu(monkeypatch):
    full, arange = torch.full, torch.arange
    monkeypatch.setattr(P.torch, "full", lambda *a, **k: full(*a, **{**k, "device": "cpu"}))
    monkeypatch.setattr(P.torch, "arange", lambda *a, **k: arange(*a, **{**k, "device": "cpu"}))


@pytest.mark.parametrize("K,act,state,lengths", [(4, "silu", True, [9, 0, 3]), (1, "none", False, None), (8, "silu", True, [2, 9, 5]), (3, "none", False, [9, 1, 8])])
def test_convolution(K, act, state, lengths):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    x, w, b, s = r(3, 2, 9, 5), r(2, 5, K), r(2, 5), r(3, 2, K - 1, 5) if state else None
    y, tail = P.conv64(x, w, b, act, s, None if lengths is None else torch.tensor(lengths, dtype=torch.int32))
    y_w, tail_w = O.conv(x, w, bias=b, act=act, state=s, lengths=lengths)
    assert torch.allclose(y, y_w, rtol=1e-13, atol=1e-13) and torch.equal(tail, tail_w)


@pytest.mark.parametrize("softplus,z,state,lengths", [(True, True, True, [7, 0, 3]), (False, False, False, None), (True, False, True, [1, 7, 6])])
def test_scan(softplus, z, state, lengths):
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    a = dict(q=r(3, 2, 7, 4), k=r(3, 2, 7, 4), v=r(3, 2, 7, 5), delta=r(3, 2, 7, 5) if softplus else r(3, 2, 7, 5).abs(), A=-r(2, 5, 4).abs(),
             D=r(2, 5), z=r(3, 2, 7, 5) if z else None, delta_bias=r(2, 5) if softplus else None, S0=r(3, 2, 5, 4) if state else None)
    o, S = P.scan64(**a, lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32), softplus=softplus)
    o_w, S_w = O.scan(**a, softplus=softplus, lengths=lengths)
    assert torch.allclose(o, o_w, rtol=1e-12, atol=1e-12) and torch.allclose(S, S_w, rtol=1e-12, atol=1e-12)
