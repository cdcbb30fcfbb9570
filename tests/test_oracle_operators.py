"""The 64-bit forms of the operators around the memory (oracle/operators.py), pinned by facts other than
themselves: closed forms, splitting a sequence, and central differences for every gradient."""
import math

import pytest
import torch

from oracle import operators as O


def rnd(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g, dtype=torch.float64)


def differences(f, leaves, got, h=1e-5):
    """Central differences of the scalar f along a random direction of each leaf, against <grad, direction>."""
    for i, (n, x) in enumerate(leaves.items()):
        d = rnd(1000 + i, *x.shape)
        up, down = f({**leaves, n: x + h * d}), f({**leaves, n: x - h * d})
        want = float((up - down) / (2 * h))
        have = float((got[n] * d).sum())
        assert abs(want - have) <= 1e-7 * (1 + abs(want)), (n, want, have)


def test_conv_is_a_weighted_sum_of_shifts():
    x, w = rnd(1, 2, 3, 9, 4), rnd(2, 3, 4, 3)
    y, tail = O.conv(x, w, act="none")
    ext = torch.cat([torch.zeros(2, 3, 2, 4, dtype=torch.float64), x], 2)
    want = sum(w[None, :, None, :, j] * ext[:, :, j:j + 9] for j in range(3))
    assert torch.allclose(y, want, atol=1e-12)
    assert torch.equal(tail, x[:, :, -2:])


@pytest.mark.parametrize("cut", [0, 1, 2, 5, 9])
def test_conv_continues_from_its_tail(cut):
    x, w, b = rnd(3, 1, 2, 9, 5), rnd(4, 2, 5, 4), rnd(5, 2, 5)
    y, tail = O.conv(x, w, bias=b)
    y1, t1 = O.conv(x[:, :, :cut], w, bias=b)
    y2, t2 = O.conv(x[:, :, cut:], w, bias=b, state=t1)
    assert torch.allclose(torch.cat([y1, y2], 2), y, atol=1e-12) and torch.equal(t2, tail)


def test_scan_closed_forms():
    # A = 0, dt = 1: a running sum of v k^T
    q, k, v = rnd(6, 1, 1, 7, 3), rnd(7, 1, 1, 7, 3), rnd(8, 1, 1, 7, 2)
    one = torch.ones(1, 1, 7, 2, dtype=torch.float64)
    o, S = O.scan(q, k, v, one, torch.zeros(1, 2, 3, dtype=torch.float64), softplus=False)
    want = torch.einsum("bhtv,bhtk->bhvk", v, k)
    assert torch.allclose(S, want, atol=1e-12)
    assert torch.allclose(o[0, 0, -1], want[0, 0] @ q[0, 0, -1], atol=1e-12)
    # v = 0: the initial state decays by exp(A sum dt)
    S0, A = rnd(9, 1, 1, 2, 3), -rnd(10, 1, 2, 3).abs()
    _, S = O.scan(q, k, 0 * v, 0.3 * one, A, softplus=False, S0=S0)
    assert torch.allclose(S, S0 * torch.exp(7 * 0.3 * A), atol=1e-12)


def test_scan_continues_from_its_state():
    a = dict(q=rnd(11, 2, 2, 8, 3), k=rnd(12, 2, 2, 8, 3), v=rnd(13, 2, 2, 8, 4), delta=rnd(14, 2, 2, 8, 4))
    A, z = -rnd(15, 2, 4, 3).abs(), rnd(16, 2, 2, 8, 4)
    o, S = O.scan(*a.values(), A, z=z)
    o1, S1 = O.scan(*(x[:, :, :3] for x in a.values()), A, z=z[:, :, :3])
    o2, S2 = O.scan(*(x[:, :, 3:] for x in a.values()), A, z=z[:, :, 3:], S0=S1)
    assert torch.allclose(torch.cat([o1, o2], 2), o, atol=1e-12) and torch.allclose(S2, S, atol=1e-12)
    # a shorter sequence is the same as fewer tokens
    o3, S3 = O.scan(*a.values(), A, z=z, lengths=[3, 0])
    assert torch.equal(o3[0, :, :3], o1[0]) and torch.equal(o3[0, :, 3:], 0 * o3[0, :, 3:])
    assert torch.equal(S3[0], S1[0]) and torch.equal(S3[1], 0 * S3[1])


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_rotation_keeps_norms_and_depends_on_distance(layout):
    x, y = rnd(17, 1, 1, 6, 8), rnd(18, 1, 1, 6, 8)
    f = torch.tensor([1.0, 0.1, 0.01], dtype=torch.float64)
    kw = dict(norm="none", rot=6, layout=layout, freq=f)
    a = O.qknorm(x, **kw)
    assert torch.allclose(a.norm(dim=-1), x.norm(dim=-1), atol=1e-12)
    assert torch.equal(a[..., 6:], x[..., 6:])
    p = torch.tensor([[5, 6, 7, 8, 9, 10]])
    b = O.qknorm(y, **kw)
    far = (O.qknorm(x, positions=p, **kw) * O.qknorm(y, positions=p, **kw)).sum(-1)
    assert torch.allclose((a * b).sum(-1), far, atol=1e-12)


def test_norms():
    x = rnd(19, 1, 2, 3, 10)
    assert torch.allclose(O.qknorm(x, norm="l2", eps=0.0).norm(dim=-1), torch.ones(1, 2, 3, dtype=torch.float64))
    r = O.qknorm(x, norm="rms", eps=0.0)
    assert torch.allclose((r * r).mean(-1), torch.ones(1, 2, 3, dtype=torch.float64))
    assert torch.equal(O.qknorm(0 * x, norm="rms", eps=0.0), 0 * x)


def test_conv_gradients_are_the_differences():
    leaves = {"x": rnd(20, 2, 2, 7, 3), "w": rnd(21, 2, 3, 4), "bias": rnd(22, 2, 3), "state": rnd(23, 2, 2, 3, 3)}
    up = rnd(24, 2, 2, 7, 3), rnd(25, 2, 2, 3, 3)
    f = lambda m: sum((o * u).sum() for o, u in zip(O.conv(**m, lengths=[7, 2]), up))
    with_grad = {n: x.clone().requires_grad_() for n, x in leaves.items()}
    got = O.gradients(O.conv(**with_grad, lengths=[7, 2]), up, with_grad)
    differences(f, leaves, got)


@pytest.mark.parametrize("softplus", [True, False])
def test_scan_gradients_are_the_differences(softplus):
    B, H, T, dk, dv = 2, 2, 6, 3, 4
    leaves = {"q": rnd(30, B, H, T, dk), "k": rnd(31, B, H, T, dk), "v": rnd(32, B, H, T, dv),
              "delta": rnd(33, B, H, T, dv).abs() * 0.5, "A": -rnd(34, H, dv, dk).abs(), "D": rnd(35, H, dv),
              "z": rnd(36, B, H, T, dv), "S0": rnd(37, B, H, dv, dk)}
    if softplus:
        leaves["delta_bias"] = rnd(38, H, dv)
    up = rnd(39, B, H, T, dv), rnd(40, B, H, dv, dk)
    f = lambda m: sum((o * u).sum() for o, u in zip(O.scan(**m, softplus=softplus, lengths=[6, 4]), up))
    with_grad = {n: x.clone().requires_grad_() for n, x in leaves.items()}
    got = O.gradients(O.scan(**with_grad, softplus=softplus, lengths=[6, 4]), up, with_grad)
    differences(f, leaves, got)


@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_qknorm_gradients_are_the_differences(norm, layout):
    leaves = {"x": rnd(41, 2, 3, 5, 10), "w": rnd(42, 10)}
    up = rnd(43, 2, 3, 5, 10)
    kw = dict(norm=norm, rot=8, layout=layout, freq=10.0 ** -torch.arange(4, dtype=torch.float64),
              positions=torch.arange(10).reshape(2, 5) * 3, lengths=[5, 3])
    f = lambda m: (O.qknorm(**m, **kw) * up).sum()
    with_grad = {n: x.clone().requires_grad_() for n, x in leaves.items()}
    got = O.gradients([O.qknorm(**with_grad, **kw)], [up], with_grad)
    differences(f, leaves, got)
    assert math.isfinite(float(f(leaves)))
