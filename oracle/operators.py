"""The operators around the memory in 64 bits: the short causal convolution, the selective scan and the
norm of queries and keys with rotation. Plain torch on the CPU, written from the definitions in
include/falcon.h, token by token; gradients by reverse-mode differentiation (torch.autograd) of these forms.

Arguments are float64 tensors (or None), ``lengths`` a list of ints or None. Rows behind a sequence's end
are 0 in outputs.
"""
from __future__ import annotations

import torch


def _ends(lengths, B, T):
    return [T] * B if lengths is None else [min(max(int(n), 0), T) for n in lengths]


def _silu(x):
    return x / (1 + torch.exp(-x))


def conv(x, w, *, bias=None, act="silu", state=None, lengths=None):
    """x (B, H, T, d), w (H, d, K): (y, state_out)."""
    B, H, T, d = x.shape
    K = w.shape[2]
    if state is None:
        state = torch.zeros(B, H, K - 1, d, dtype=x.dtype)
    ext = torch.cat([state, x], 2)   # row t + K - 1 is input t
    y = torch.zeros_like(x)
    tails = []
    rows = []
    for b, n in enumerate(_ends(lengths, B, T)):
        out = []
        for t in range(n):
            p = torch.zeros(H, d, dtype=x.dtype) if bias is None else bias
            for j in range(K):
                p = p + w[:, :, j] * ext[b, :, t + j]
            out.append(_silu(p) if act == "silu" else p)
        out += [torch.zeros(H, d, dtype=x.dtype)] * (T - n)
        rows.append(torch.stack(out, 1) if T else y[b])
        tails.append(ext[b, :, n:n + K - 1])
    return (torch.stack(rows) if B else y), (torch.stack(tails) if B else state)


def scan(q, k, v, delta, A, *, D=None, z=None, delta_bias=None, softplus=True, S0=None, lengths=None):
    """q, k (B, H, T, dk), v, delta, z (B, H, T, dv), A (H, dv, dk): (o, S)."""
    B, H, T, dk = k.shape
    dv = v.shape[3]
    dt = delta if delta_bias is None else delta + delta_bias[:, None]
    if softplus:
        dt = torch.clamp(dt, min=0) + torch.log1p(torch.exp(-dt.abs()))
    os, Ss = [], []
    for b, n in enumerate(_ends(lengths, B, T)):
        S = torch.zeros(H, dv, dk, dtype=v.dtype) if S0 is None else S0[b]
        rows = []
        for t in range(n):
            d = dt[b, :, t, :, None]
            S = torch.exp(d * A) * S + d * v[b, :, t, :, None] * k[b, :, t, None, :]
            o = (S * q[b, :, t, None, :]).sum(-1)
            if D is not None:
                o = o + D * v[b, :, t]
            if z is not None:
                o = o * _silu(z[b, :, t])
            rows.append(o)
        rows += [torch.zeros(H, dv, dtype=v.dtype)] * (T - n)
        os.append(torch.stack(rows, 1) if T else torch.zeros(H, 0, dv, dtype=v.dtype))
        Ss.append(S)
    return torch.stack(os), torch.stack(Ss)


def qknorm(x, *, w=None, norm="rms", eps=1e-6, rot=0, layout="half", freq=None, positions=None, lengths=None):
    """One of q and k: x (B, H, T, d), freq (rot / 2), positions (B, T)."""
    B, H, T, d = x.shape
    if norm != "none":
        m = (x * x).sum(-1, keepdim=True) / (d if norm == "rms" else 1) + eps
        zero = m == 0
        x = torch.where(zero, torch.zeros_like(x), x / torch.sqrt(torch.where(zero, torch.ones_like(m), m)))
    if w is not None:
        x = x * w
    if rot:
        pos = torch.arange(T, dtype=torch.float64).expand(B, T) if positions is None else positions.double()
        angle = (pos[:, :, None] * freq.double())[:, None]
        c, s = torch.cos(angle), torch.sin(angle)
        first = list(range(rot // 2)) if layout == "half" else list(range(0, rot, 2))
        second = list(range(rot // 2, rot)) if layout == "half" else list(range(1, rot, 2))
        x1, x2 = x[..., first], x[..., second]
        cols = [None] * d
        y1, y2 = x1 * c - x2 * s, x2 * c + x1 * s
        for j in range(rot // 2):
            cols[first[j]], cols[second[j]] = y1[..., j], y2[..., j]
        for i in range(rot, d):
            cols[i] = x[..., i]
        x = torch.stack(cols, -1)
    inside = torch.tensor([[t < n for t in range(T)] for n in _ends(lengths, B, T)], dtype=torch.bool).reshape(B, T)
    return torch.where(inside[:, None, :, None], x, torch.zeros_like(x))


def gradients(outputs, upstream, leaves):
    """Gradients of sum <outputs, upstream> (a None on either side leaves that output out) with respect to
    the dict ``leaves``; 0 where nothing depends on a leaf."""
    loss = sum((o * u).sum() for o, u in zip(outputs, upstream) if u is not None)
    names = [n for n, x in leaves.items() if x is not None]
    got = torch.autograd.grad(loss, [leaves[n] for n in names], allow_unused=True) if isinstance(loss, torch.Tensor) \
        and loss.requires_grad else [None] * len(names)
    return {n: (torch.zeros_like(leaves[n]) if g is None else g) for n, g in zip(names, got)}
