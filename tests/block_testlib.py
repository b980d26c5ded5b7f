"""Plain 64-bit implementations of a hybrid block's operators, on the CPU, and the tolerances of
their tests.  Gradients come from autograd through these.

Tolerances.  Recurrence and norms compute in fp32 (unit roundoff 2^-24) and are compared as the
mixer's operators are (``mixer_testlib.assert_close``): 4 * 2^-22 * (n + 16) of the tensor's largest
magnitude for n sequential roundings, and for bf16 half a step (2^-8 of the element) more.

Attention: a weight p_j = e^{s_j - max} is off by the error of its score, at most (d + 8) 2^-23 of
sum_i |q_i k_ji| scale (d sums, whose steps a tensor instruction may cut off instead of rounding, and
the products with the scale), by 2^-22 |s_j| and 2^-22 of the exponential and its argument, and by
2^-17 of its split into two bf16 parts.  The output is a mean of v with these weights: off by twice
that, times the largest |v|, and by the sums over n keys, n 2^-23; then half a step of its type.
"""
from __future__ import annotations

import torch

from mixer_testlib import BF16, bounds

CU = {  # name: (tokens, offsets)
    "one": (37, [0, 37]),
    "single": (1, [0, 1]),
    "short": (9, [0, 1, 3, 3, 6, 9]),
    "ghosts": (300, [0, 0, 64, 64, 64, 65, 200, 300, 300]),
    "gaps": (150, [10, 20, 90, 130]),
    "long": (1037, [0, 700, 1037]),
    "malformed": (120, [-4, 50, 20, 50, 90, 70, 400]),
    "none": (0, [0, 0, 0]),
    "all empty": (40, [5, 5]),
    "many": (260, list(range(0, 261, 2))),
    "no segments": (20, [0]),
}


def sigmoid(v):
    return torch.sigmoid(v)


def rec(x, r, A, i, normalize, h0, cu):
    """(y with zeros outside the segments, final states, mask of covered tokens)."""
    T, D = x.shape
    L = A * sigmoid(r)
    a = torch.exp(L)
    u = x if i is None else sigmoid(i) * x
    if normalize:
        u = u * torch.sqrt(-torch.expm1(2 * L))
    bd = bounds(cu, T)
    ys, ends, mask, at = [], [], torch.zeros(T, dtype=torch.bool), 0
    for n, (s, e) in enumerate(zip(bd[:-1], bd[1:])):
        if s > at:
            ys.append(x.new_zeros(s - at, D))
        mask[s:e] = True
        at = e
        h = h0[n] if h0 is not None else x.new_zeros(D)
        for t in range(s, e):
            h = a[t] * h + u[t]
            ys.append(h[None])
        ends.append(h)
    if at < T:
        ys.append(x.new_zeros(T - at, D))
    y = torch.cat(ys) if ys else x.new_zeros(0, D)
    return y, torch.stack(ends) if ends else x.new_zeros(0, D), mask


def rms(x, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def gated(x, z, w, act, eps):
    y = rms(x, eps) * (z * sigmoid(z) if act == "silu" else sigmoid(z))
    return y if w is None else y * w


def residual(x, res, w, wp, g, scale, eps, post):
    u = rms(x, eps) if post or wp is not None else x
    if wp is not None:
        u = u * wp
    if g is not None:
        u = u * g
    h = scale * u if res is None else res + scale * u
    y = rms(h, eps)
    return (y if w is None else y * w), h


def attention(q, kc, vc, table, lens, scale, window):
    """(o [B, Hq, d] in 64 bits, its bound as above for each request)."""
    B, Hq, d = q.shape
    pages, ps, Hk, _ = kc.shape
    rep = Hq // Hk
    q, kc, vc = q.double(), kc.double(), vc.double()
    o, tol = torch.zeros(B, Hq, d, dtype=torch.float64), torch.zeros(B, dtype=torch.float64)
    for b in range(B):
        n = max(0, min(int(lens[b]), table.shape[1] * ps))
        first = max(0, n - window) if window else 0
        rows = []
        for j in range(first, n):
            p = int(table[b, j // ps])
            if 0 <= p < pages:
                rows.append((p, j % ps))
        if not rows:
            continue
        pi, pl = (torch.tensor(c) for c in zip(*rows))
        for h in range(Hq):
            k, v = kc[pi, pl, h // rep], vc[pi, pl, h // rep]
            s = scale * (k @ q[b, h])
            o[b, h] = torch.softmax(s, 0) @ v
            size = float((k.abs() @ q[b, h].abs()).max()) * abs(scale)
            off = (d + 8) * 2.0 ** -23 * size + 2.0 ** -22 * (1 + float(s.abs().max())) + 2.0 ** -17
            tol[b] = max(tol[b], (2 * off + len(rows) * 2.0 ** -23) * float(v.abs().max()))
    return o, tol


def assert_attention(got, o, tol, name="o"):
    g = got.detach().cpu().double()
    bound = tol[:, None, None] + (2.0 ** -8 if got.dtype == BF16 else 2.0 ** -24) * o.abs()
    bad = ~((g - o).abs() <= bound)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {o.numel()} off, most "
                           f"{float((g - o).abs().max())}, first {torch.nonzero(bad)[0].tolist()}")


def plan(lengths, new, table, free, taken, page, most):
    """cache_plan with whole numbers: (slots, positions, cu, lengths, taken, table)."""
    table = [list(map(int, row)) for row in table]
    width = len(table[0]) if table else 0
    taken = min(max(int(taken), 0), len(free))
    n1 = [max(0, min(int(n), width * page - max(int(a), 0))) for a, n in zip(lengths, new)]
    slots, pos, cu, after, asked = [], [], [0], [], 0
    for b, (a, n) in enumerate(zip(lengths, n1)):
        a = max(int(a), 0)
        end = asked + n
        n = min(end, most) - min(asked, most)
        asked = end
        have = -(-a // page)
        need = -(-(a + n) // page) - have if n else 0
        got = min(need, len(free) - taken)
        for j in range(got):
            table[b][have + j] = int(free[taken + j])
        taken += got
        n = max(0, min(n, (have + got) * page - a))
        for p in range(a, a + n):
            at = table[b][p // page]
            slots.append(at * page + p % page if at >= 0 else -1)
            pos.append(p)
        cu.append(cu[-1] + n)
        after.append(a + n)
    slots += [-1] * (most - len(slots))
    pos += [0] * (most - len(pos))
    return slots, pos, cu, after, taken, table
