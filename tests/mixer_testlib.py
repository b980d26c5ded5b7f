"""Plain 64-bit implementations of the mixer's operators, token by token on the CPU, and the
tolerances of their tests.  Gradients come from autograd through these.

Tolerances.  The kernels compute in fp32 (unit roundoff 2^-24); the exponential has 2 ulp.  A
value that a recurrence of n steps carries gathers at most a few roundings a step, so fp32
results are compared within 4 * 2^-22 * (n + 16) of the tensor's largest magnitude, and bf16
results within that plus half a unit in the last place of bf16 (2^-9 of the element; 2^-8 leaves
room for the double rounding at a tie).
"""
from __future__ import annotations

import torch

BF16, F32 = torch.bfloat16, torch.float32


def assert_close(got, ref, steps, name=""):
    assert got.shape == ref.shape, f"{name}: {tuple(got.shape)} != {tuple(ref.shape)}"
    g, r = got.detach().cpu().double(), ref.detach().cpu().double()
    top = float(r.abs().max()) if r.numel() else 0.0
    tol = 4 * 2.0 ** -22 * (steps + 16) * top
    bound = torch.full_like(r, tol)
    if got.dtype == BF16:
        bound = bound + 2.0 ** -8 * r.abs()
    bad = ~((g - r).abs() <= bound)
    if bad.any():
        i = int(torch.nonzero(bad.reshape(-1))[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {r.numel()} off; first at {i}: "
                             f"{g.reshape(-1)[i]} for {r.reshape(-1)[i]} (largest {top})")


def bounds(cu, T):
    """Segment bounds: clamped to [0, T], made non-decreasing by a running maximum."""
    out, prev = [], 0
    for c in cu:
        prev = max(prev, min(max(int(c), 0), T))
        out.append(prev)
    return out


def silu(u):
    return u * torch.sigmoid(u)


def conv(x, w, b, h0, cu, act):
    """(y with zeros outside the segments, final states, mask of covered tokens)."""
    T, C = x.shape
    W = w.shape[1]
    bd = bounds(cu, T)
    ys, ends, mask, at = [], [], torch.zeros(T, dtype=torch.bool), 0
    for n, (s, e) in enumerate(zip(bd[:-1], bd[1:])):
        if s > at:
            ys.append(x.new_zeros(s - at, C))
        pre = h0[n] if h0 is not None else x.new_zeros(W - 1, C)
        rows = torch.cat([pre, x[s:e]])
        mask[s:e] = True
        at = e
        for t in range(e - s):
            u = (rows[t:t + W] * w.t()).sum(0)
            if b is not None:
                u = u + b
            ys.append((silu(u) if act else u)[None])
        ends.append(rows[e - s:])
    if at < T:
        ys.append(x.new_zeros(T - at, C))
    y = torch.cat(ys) if ys else x.new_zeros(0, C)
    return y, torch.stack(ends) if ends else x.new_zeros(0, W - 1, C), mask


def ssm(x, dt, A, B, C, D, z, dt_bias, softplus, h0, cu):
    """(y with zeros outside the segments, final states, mask of covered tokens)."""
    T, Dm = x.shape
    G, N = B.shape[1:]
    grp = torch.arange(Dm) // (Dm // G)
    v = dt + dt_bias if dt_bias is not None else dt
    if softplus:
        v = torch.logaddexp(v, torch.zeros_like(v))
    bd = bounds(cu, T)
    ys, ends, mask, at = [], [], torch.zeros(T, dtype=torch.bool), 0
    for n, (s, e) in enumerate(zip(bd[:-1], bd[1:])):
        if s > at:
            ys.append(x.new_zeros(s - at, Dm))
        mask[s:e] = True
        at = e
        h = h0[n] if h0 is not None else x.new_zeros(Dm, N)
        for t in range(s, e):
            h = torch.exp(v[t][:, None] * A) * h + (v[t] * x[t])[:, None] * B[t][grp]
            y = (h * C[t][grp]).sum(1)
            if D is not None:
                y = y + D * x[t]
            if z is not None:
                y = y * silu(z[t])
            ys.append(y[None])
        ends.append(h)
    if at < T:
        ys.append(x.new_zeros(T - at, Dm))
    y = torch.cat(ys) if ys else x.new_zeros(0, Dm)
    return y, torch.stack(ends) if ends else x.new_zeros(0, Dm, N), mask


def qk_row(x, w, norm, eps, cos, sin, pos, inter):
    """One of q, k [T, H, d]."""
    m = (x * x).sum(-1, keepdim=True)
    if norm == "rms":
        m = m / x.shape[-1]
    u = x / torch.sqrt(m + eps)
    if w is not None:
        u = u * w
    if cos is None:
        return u
    r = 2 * cos.shape[1]
    p = pos.long().clamp(0, cos.shape[0] - 1)
    c, s = cos[p][:, None], sin[p][:, None]
    if inter:
        a, b = u[..., 0:r:2], u[..., 1:r:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = u[..., :r // 2], u[..., r // 2:r]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, u[..., r:]], -1)


def delta(q, k, v, g, beta, S, scale):
    """One token of one request: S [H, dk, dv] -> (o [H, dv], new S)."""
    rep = v.shape[0] // q.shape[0]
    q, k = q.repeat_interleave(rep, 0), k.repeat_interleave(rep, 0)
    eye = torch.eye(k.shape[1], dtype=S.dtype)
    M = eye - beta[:, None, None] * k[:, :, None] * k[:, None, :]
    S = torch.exp(g)[:, None, None] * (M @ S) + beta[:, None, None] * k[:, :, None] * v[:, None, :]
    return scale * (S * q[:, :, None]).sum(1), S


def leaf(t):
    """A 64-bit CPU copy to differentiate with respect to (None stays None)."""
    return None if t is None else t.detach().cpu().double().requires_grad_(True)
