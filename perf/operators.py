"""Measured cases of the token mixer's operators around the gated delta rule.

Operators (``op`` of a case):
  conv_fwd, conv_train, conv_step   short causal convolution over packed segments
  ssm_fwd, ssm_train, ssm_step      selective state space scan
  qk_fwd, qk_train                  per-head norm of queries and keys with the rotation
  delta_step                        gated delta rule for single tokens

``run`` computes them with elementary torch operations in 32 bits where ``own`` is false, and
through the package's entry points where it is true.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # prefill of a packed batch: q, k and v of 32 heads of 128 through one convolution
        dict(name="conv prompt packed 64k", op="conv_fwd", dtype="bf16", T=65536, segs=20, ghosts=16,
             equal=False, len_seed=3, C=12288, W=4, silu=True, bias=False, state=False),
        # a training step on four sequences, states handed over between pieces of a document
        dict(name="conv train 4x4096", op="conv_train", dtype="bf16", T=16384, segs=4, ghosts=0,
             equal=True, len_seed=0, C=6144, W=4, silu=True, bias=True, state=True),
        # decoding: 37 requests of a pool of 48 slots, two rows of the batch are padding
        dict(name="conv step 37", op="conv_step", dtype="bf16", B=37, slots=48, pad=2, C=8192, W=4,
             silu=True, bias=True),
        # one long prompt with a state carried in from a cached prefix
        dict(name="ssm prompt 20468", op="ssm_fwd", dtype="bf16", T=20468, segs=1, ghosts=0,
             equal=True, len_seed=0, D=4096, N=16, G=1, z=True, skip=True, state=True),
        # a small ragged packed prefill in 32 bits, odd channel and state counts, grouped B and C
        dict(name="ssm ragged fp32", op="ssm_fwd", dtype="fp32", T=1537, segs=7, ghosts=2,
             equal=False, len_seed=11, D=1002, N=12, G=2, z=False, skip=True, state=False),
        # a training step on packed sequences
        dict(name="ssm train packed 8k", op="ssm_train", dtype="bf16", T=8192, segs=5, ghosts=1,
             equal=False, len_seed=5, D=2048, N=16, G=1, z=True, skip=True, state=True),
        # decoding: the states of 128 requests in a pool
        dict(name="ssm step 128", op="ssm_step", dtype="bf16", B=128, slots=160, pad=3, D=4096,
             N=16, G=1, z=True, skip=True),
        # prefill of an attention layer: RMS norm with weights, rotation of the whole head
        dict(name="qk prompt 64k", op="qk_fwd", dtype="bf16", T=65536, Hq=32, Hk=16, d=128, rot=128,
             interleaved=False, norm="rms", weight=True),
        # a training step, half of each head rotated, odd token count
        dict(name="qk train 8191", op="qk_train", dtype="bf16", T=8191, Hq=16, Hk=16, d=128, rot=64,
             interleaved=False, norm="rms", weight=True),
        # decoding: the L2 norm before the delta rule, no rotation
        dict(name="qk step 32", op="qk_fwd", dtype="bf16", T=32, Hq=16, Hk=16, d=128, rot=0,
             interleaved=False, norm="l2", weight=False),
        # decoding of one request
        dict(name="delta step 1", op="delta_step", dtype="bf16", B=1, slots=4, pad=0, Hk=16, H=32,
             d=128),
        # decoding of a full batch
        dict(name="delta step 256", op="delta_step", dtype="bf16", B=256, slots=300, pad=5, Hk=16,
             H=32, d=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_train", "conv_step", "ssm_fwd", "ssm_train", "ssm_step",
                     "qk_fwd", "qk_train", "delta_step"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    seq = dict(segs=_log(rng, 1, 64), ghosts=rng.choice([0, 0, 1, 5]), equal=rng.random() < 0.3,
               len_seed=rng.randrange(1 << 20))
    e = 2 if dtype == "bf16" else 4
    if op.startswith("conv"):
        C, W = _log(rng, 64, 12288), rng.choice([2, 3, 4, 4])
        if rng.random() < 0.7:
            C = -(-C // 64) * 64
        more = dict(C=C, W=W, silu=rng.random() < 0.8, bias=rng.random() < 0.5)
        if op == "conv_step":
            B = _log(rng, 1, 512)
            return dict(op=op, dtype=dtype, B=B, slots=B + rng.randrange(2, 40),
                        pad=min(B - 1, rng.choice([0, 0, 1, 4])), **more)
        most = (65536 * 12288 * 2 if op == "conv_fwd" else 16384 * 6144 * 2) // (e * C)
        return dict(op=op, dtype=dtype, T=_log(rng, 1, min(most, 65536)), state=rng.random() < 0.5,
                    **seq, **more)
    if op.startswith("ssm"):
        G = rng.choice([1, 1, 1, 2, 4])
        D = G * max(1, _log(rng, 64, 4096) // G)
        if rng.random() < 0.7:
            D = -(-D // (64 * G)) * 64 * G
        D = min(D, 4096)
        N = rng.choice([16, 16, 16, 8, 32, rng.randrange(1, 65)])
        more = dict(D=D, N=N, G=G, z=rng.random() < 0.7, skip=rng.random() < 0.8)
        if op == "ssm_step":
            B = _log(rng, 1, max(1, 128 * 4096 * 16 // (D * N)))
            B = min(B, 512)
            return dict(op=op, dtype=dtype, B=B, slots=B + rng.randrange(4, 40),
                        pad=min(B - 1, rng.choice([0, 0, 1, 3])), **more)
        most = (20468 * 4096 * 16 if op == "ssm_fwd" else 8192 * 2048 * 16) // (D * N)
        if dtype == "fp32":
            most //= 2
        return dict(op=op, dtype=dtype, T=_log(rng, 1, min(most, 65536)), state=rng.random() < 0.5,
                    **seq, **more)
    if op.startswith("qk"):
        d = rng.choice([64, 128, 128, 256, 8 * rng.randrange(2, 32)])
        rot = rng.choice([d, d, d // 2 // 2 * 2, 0])
        Hk = _log(rng, 1, 16)
        Hq = Hk * rng.choice([1, 2, 4]) if Hk <= 8 else Hk * rng.choice([1, 2])
        most = (65536 * 48 * 128 * 2 if op == "qk_fwd" else 8191 * 32 * 128 * 2) // (e * d * (Hq + Hk))
        return dict(op=op, dtype=dtype, T=_log(rng, 1, min(most, 131072)), Hq=Hq, Hk=Hk, d=d,
                    rot=rot, interleaved=rng.random() < 0.4, norm=rng.choice(["rms", "rms", "l2"]),
                    weight=rng.random() < 0.7)
    d = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 8, 16])
    H = Hk * rng.choice([1, 2, 4] if Hk < 16 else [1, 2])
    B = _log(rng, 1, min(512, 256 * 32 * 128 * 128 // (H * d * d)))
    return dict(op=op, dtype="bf16", B=B, slots=B + rng.randrange(6, 50),
                pad=min(B - 1, rng.choice([0, 0, 1, 5])), Hk=Hk, H=H, d=d)


def _lengths(case):
    """Segment lengths from the case's numbers: equal ones, or random cuts; then empty segments."""
    T, n = case["T"], min(case["segs"], case["T"])
    r = random.Random(case["len_seed"])
    if case["equal"]:
        lens = [T // n + (1 if i < T % n else 0) for i in range(n)]
    else:
        cuts = sorted(r.sample(range(1, T), n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [T])]
    for _ in range(case["ghosts"]):
        lens.insert(r.randrange(len(lens) + 1), 0)
    return lens


def _n_seq(case):
    return min(case["segs"], case["T"]) + case["ghosts"]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(int(seed))
    dt = TYPES[case["dtype"]]
    op = case["op"]

    def rn(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=DEV).mul_(std).to(dtype)

    def un(*shape):
        return torch.rand(*shape, generator=gen, device=DEV)

    s = dict(case)
    if "T" in case and "segs" in case:
        lens = _lengths(case)
        s["cu"] = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
        n_seq = len(lens)
    if "slots" in case:
        # live slots are 1 .. slots - 1 in any order; -1 marks a padded row of the batch
        idx = torch.randperm(case["slots"] - 1, generator=gen, device=DEV)[:case["B"]] + 1
        idx = idx.to(torch.int32)
        if case["pad"]:
            idx[torch.randperm(case["B"], generator=gen, device=DEV)[:case["pad"]]] = -1
        s["idx"] = idx
    if op.startswith("conv"):
        C, W = case["C"], case["W"]
        rows = case["B"] if op == "conv_step" else case["T"]
        s["x"] = rn(rows, C, dtype=dt)
        s["w"] = rn(C, W, std=W ** -0.5)
        s["b"] = rn(C, std=0.2) if case["bias"] else None
        s["act"] = "silu" if case["silu"] else None
        if op == "conv_step":
            s["buf"] = rn(case["slots"], W - 1, C, dtype=dt)
        else:
            s["h0"] = rn(n_seq, W - 1, C, dtype=dt) if case["state"] else None
        if op == "conv_train":
            s["dy"] = rn(rows, C, std=0.1, dtype=dt)
            s["dht"] = rn(n_seq, W - 1, C, std=0.1, dtype=dt) if case["state"] else None
    elif op.startswith("ssm"):
        D, N, G = case["D"], case["N"], case["G"]
        rows = case["B"] if op == "ssm_step" else case["T"]
        s["x"] = torch.nn.functional.silu(rn(rows, D)).to(dt)
        s["dt"] = rn(rows, D, std=0.5, dtype=dt)
        s["A"] = -torch.arange(1, N + 1, device=DEV).float() * torch.exp(rn(D, N, std=0.2))
        s["Bm"] = rn(rows, G, N, dtype=dt)
        s["Cm"] = rn(rows, G, N, dtype=dt)
        s["skip_w"] = 1.0 + rn(D, std=0.2) if case["skip"] else None
        s["zg"] = rn(rows, D, dtype=dt) if case["z"] else None
        step = torch.exp(un(D) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
        s["dt_bias"] = torch.log(torch.expm1(step))  # softplus(bias) is the step at rest
        if op == "ssm_step":
            s["buf"] = rn(case["slots"], D, N, std=0.3)
        else:
            s["h0"] = rn(n_seq, D, N, std=0.3) if case["state"] else None
        if op == "ssm_train":
            s["dy"] = rn(rows, D, std=0.1, dtype=dt)
            s["dht"] = rn(n_seq, D, N, std=0.1) if case["state"] else None
    elif op.startswith("qk"):
        T, d, rot = case["T"], case["d"], case["rot"]
        s["q"], s["k"] = rn(T, case["Hq"], d, dtype=dt), rn(T, case["Hk"], d, dtype=dt)
        s["qw"] = 1.0 + rn(d, std=0.1) if case["weight"] else None
        s["kw"] = 1.0 + rn(d, std=0.1) if case["weight"] else None
        if rot:
            # the model's table of angles, and each token's place in its own sequence
            places = 8192
            freq = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV).double() / rot)
            ang = torch.arange(places, device=DEV).double()[:, None] * freq
            s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
            start = torch.randint(0, places, (1,), generator=gen, device=DEV)
            s["pos"] = ((torch.arange(T, device=DEV) + start) % places).to(torch.int32)
        else:
            s["cos"] = s["sin"] = s["pos"] = None
        if op == "qk_train":
            s["dq"], s["dk"] = (rn(T, case["Hq"], d, std=0.1, dtype=dt),
                                rn(T, case["Hk"], d, std=0.1, dtype=dt))
    else:
        B, Hk, H, d = case["B"], case["Hk"], case["H"], case["d"]
        unit = lambda t: (t / t.norm(dim=-1, keepdim=True)).to(dt)
        s["q"], s["k"] = unit(rn(B, Hk, d)), unit(rn(B, Hk, d))
        s["v"] = rn(B, H, d, dtype=dt)
        s["g"] = torch.nn.functional.logsigmoid(rn(B, H) + 3.0)
        s["beta"] = torch.sigmoid(rn(B, H)).to(dt)
        s["buf"] = rn(case["slots"], H, d, d, std=0.1)
    return s


# ------------------------------------------------------------------ the plain forms, in 32 bits

def _places(cu, T):
    """Segment of each token, its place there, and the segments' lengths (no host reads)."""
    t = torch.arange(T, device=cu.device)
    cu = cu.long()
    seg = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return t, seg, t - cu[seg], cu[1:] - cu[:-1]


def _conv_plain(s, x, h0):
    """Pre-activation u, and the x of every tap: [T, C] each, taps oldest first."""
    T, W = x.shape[0], s["W"]
    t, seg, place, _ = _places(s["cu"], T)
    taps = []
    for k in range(W):
        back = W - 1 - k
        inside = (place >= back)[:, None]
        row = x[(t - back).clamp(min=0)]
        if h0 is None:
            taps.append(torch.where(inside, row, torch.zeros_like(row)))
        else:
            taps.append(torch.where(inside, row, h0[seg, (W - 1 + place - back).clamp(0, W - 2)]))
    u = sum(taps[k] * s["w"][:, k] for k in range(W))
    if s["b"] is not None:
        u = u + s["b"]
    return u, taps


def _conv_end(s, x, h0):
    """The last W - 1 inputs of each segment, reaching into its initial state where it is short."""
    W, cu = s["W"], s["cu"].long()
    n = cu[1:] - cu[:-1]
    j = torch.arange(W - 1, device=x.device)
    at = n[:, None] - (W - 1) + j  # place in the segment; below 0: in the initial state
    rows = x[(cu[:-1, None] + at).clamp(0, x.shape[0] - 1)]
    if h0 is None:
        before = torch.zeros_like(rows)
    else:
        before = torch.gather(h0, 1, (at + W - 1).clamp(0, W - 2)[..., None].expand_as(rows))
    return torch.where((at >= 0)[..., None], rows, before)


def _conv_fwd_plain(s):
    dt = s["x"].dtype
    x, h0 = s["x"].float(), None if s["h0"] is None else s["h0"].float()
    u, _ = _conv_plain(s, x, h0)
    y = u * torch.sigmoid(u) if s["act"] else u
    return y.to(dt), _conv_end(s, x, h0).to(dt)


def _conv_train_plain(s):
    dt, W = s["x"].dtype, s["W"]
    x, h0 = s["x"].float(), None if s["h0"] is None else s["h0"].float()
    u, taps = _conv_plain(s, x, h0)
    y, du = u, s["dy"].float()
    if s["act"]:
        sg = torch.sigmoid(u)
        y, du = u * sg, du * (sg + u * sg * (1 - sg))
    T = x.shape[0]
    t, seg, place, n = _places(s["cu"], T)
    left = n[seg] - 1 - place  # tokens of the segment after this one
    dx = torch.zeros_like(x)
    dw = torch.stack([(du * taps[k]).sum(0) for k in range(W)], 1)
    for k in range(W):
        ahead = W - 1 - k
        row = du[(t + ahead).clamp(max=T - 1)] * s["w"][:, k]
        dx = dx + torch.where((left >= ahead)[:, None], row, torch.zeros_like(row))
    dh0 = None
    if s["dht"] is not None:
        dht = s["dht"].float()
        j = W - 1 - 1 - left  # the row of the final state that holds this token
        row = dht[seg, j.clamp(min=0)]
        dx = dx + torch.where((j >= 0)[:, None], row, torch.zeros_like(row))
        cu = s["cu"].long()
        i = torch.arange(W - 1, device=x.device)
        parts = torch.zeros_like(dht)
        for k in range(W):
            # row i of the state is tap k of the segment's token i - k
            at = i - k
            rows = du[(cu[:-1, None] + at).clamp(0, T - 1)] * s["w"][:, k]
            ok = (at >= 0) & (at < n[:, None])
            parts = parts + torch.where(ok[..., None], rows, torch.zeros_like(rows))
        at = i - n[:, None]  # the row of the final state that is this row of the initial one
        kept = torch.gather(dht, 1, at.clamp(0, W - 2)[..., None].expand_as(dht))
        dh0 = (parts + torch.where((at >= 0)[..., None], kept, torch.zeros_like(kept))).to(dt)
    return (y.to(dt), _conv_end(s, x, h0).to(dt), dx.to(dt), dw,
            du.sum(0) if s["b"] is not None else None, dh0)


def _conv_step_plain(s):
    dt = s["x"].dtype
    live = s["idx"] >= 0
    at = s["idx"].clamp(min=0).long()
    old = s["buf"][at]
    win = torch.cat([old, s["x"][:, None]], 1)
    u = (win.float() * s["w"].t()).sum(1)
    if s["b"] is not None:
        u = u + s["b"]
    y = u * torch.sigmoid(u) if s["act"] else u
    s["buf"].index_put_((at,), torch.where(live[:, None, None], win[:, 1:], old))
    return torch.where(live[:, None], y, torch.zeros_like(y)).to(dt), s["buf"]


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis by doubling (in place); a is used up."""
    n = 1
    while n < b.shape[0]:
        b[n:] += a[n:] * b[:-n]
        a[n:] *= a[:-n].clone()
        n *= 2
    return b


def _softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _spread(m, D):
    """[T, G, N] -> [T, D, N]: each group's row for its channels."""
    T, G, N = m.shape
    return m[:, :, None].expand(T, G, D // G, N).reshape(T, D, N)


def _ssm_states(s):
    """The forward's parts: dt, a, the states h and what enters each token (a h_{t-1})."""
    x, D = s["x"].float(), s["D"]
    T = x.shape[0]
    _, seg, place, n = _places(s["cu"], T)
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    a = torch.exp(dt[..., None] * s["A"])
    b = (dt * x)[..., None] * _spread(s["Bm"].float(), D)
    first = (place == 0)[:, None, None]
    if s["h0"] is not None:
        b = torch.where(first, b + a * s["h0"][seg], b)
    h = _scan(torch.where(first, torch.zeros_like(a), a), b)
    cu = s["cu"].long()
    h0 = s["h0"] if s["h0"] is not None else torch.zeros_like(h[:1]).expand(n.numel(), *h.shape[1:])
    ht = torch.where((n > 0)[:, None, None], h[(cu[1:] - 1).clamp(min=0)], h0)
    return x, dt, a, h, ht, h0, seg, place, n


def _ssm_out(s, x, h):
    """y = C h + D x before the gate."""
    T, G, N = s["Cm"].shape
    y = torch.einsum("tgn,tgdn->tgd", s["Cm"].float(), h.view(T, G, -1, N)).reshape(T, -1)
    return y + s["skip_w"] * x if s["skip_w"] is not None else y


def _ssm_fwd_plain(s):
    x, _, _, h, ht, _, _, _, _ = _ssm_states(s)
    y = _ssm_out(s, x, h)
    if s["zg"] is not None:
        z = s["zg"].float()
        y = y * z * torch.sigmoid(z)
    return y.to(s["x"].dtype), ht


def _ssm_train_plain(s):
    dtp, D, N, G = s["x"].dtype, s["D"], s["N"], s["G"]
    x, dt, a, h, ht, h0, seg, place, n = _ssm_states(s)
    T = x.shape[0]
    y = _ssm_out(s, x, h)
    dout, dz, out = s["dy"].float(), None, y
    if s["zg"] is not None:
        z = s["zg"].float()
        sg = torch.sigmoid(z)
        out = y * z * sg
        dz = (dout * y * (sg + z * sg * (1 - sg))).to(dtp)
        dout = dout * z * sg
    Cm, Bm = s["Cm"].float(), s["Bm"].float()
    # the states' gradients: the same recurrence from the last token to the first
    last = (n[seg] - 1 - place == 0)[:, None, None]
    g = dout[..., None] * _spread(Cm, D)
    if s["dht"] is not None:
        g = torch.where(last, g + s["dht"][seg], g)
    nxt = torch.where(last, torch.zeros_like(a), torch.cat([a[1:], a[:1]]))
    g = _scan(nxt.flip(0), g.flip(0)).flip(0)
    first = (place == 0)[:, None, None]
    before = torch.where(first, h0[seg], torch.cat([h[:1], h[:-1]]))
    carry = a * before * g
    dA = (carry * dt[..., None]).sum(0)
    bg = (g * _spread(Bm, D)).sum(-1)
    draw_ = (carry * s["A"]).sum(-1) + x * bg
    ddt = draw_ * torch.sigmoid(s["dt"].float() + s["dt_bias"])
    dx = dt * bg
    dD = None
    if s["skip_w"] is not None:
        dx = dx + s["skip_w"] * dout
        dD = (dout * x).sum(0)
    dB = ((dt * x)[..., None] * g).view(T, G, D // G, N).sum(2)
    dC = (dout[..., None] * h).view(T, G, D // G, N).sum(2)
    dh0 = None
    if s["h0"] is not None:
        cu = s["cu"].long()
        at = cu[:-1].clamp(max=T - 1)
        dht = s["dht"] if s["dht"] is not None else torch.zeros_like(s["h0"])
        dh0 = torch.where((n > 0)[:, None, None], a[at] * g[at], dht)
    return (out.to(dtp), ht, dx.to(dtp), ddt.to(dtp), dA, dB.to(dtp), dC.to(dtp), dD, dz,
            ddt.sum(0), dh0)


def _ssm_step_plain(s):
    x, D = s["x"].float(), s["D"]
    live = s["idx"] >= 0
    at = s["idx"].clamp(min=0).long()
    old = s["buf"][at]
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    new = (torch.exp(dt[..., None] * s["A"]) * old
           + (dt * x)[..., None] * _spread(s["Bm"].float(), D))
    y = _ssm_out(s, x, new)
    if s["zg"] is not None:
        z = s["zg"].float()
        y = y * z * torch.sigmoid(z)
    s["buf"].index_put_((at,), torch.where(live[:, None, None], new, old))
    return torch.where(live[:, None], y, torch.zeros_like(y)).to(s["x"].dtype), s["buf"]


def _pairs(s, t):
    """The two halves of each rotated pair, and the part of the head that is not rotated."""
    r = s["rot"]
    if s["interleaved"]:
        return t[..., 0:r:2], t[..., 1:r:2], t[..., r:]
    return t[..., :r // 2], t[..., r // 2:r], t[..., r:]


def _joined(s, a, b, rest):
    if s["interleaved"]:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _turn(s, t, back):
    if not s["rot"]:
        return t
    p = s["pos"].long()
    c, n = s["cos"][p][:, None], s["sin"][p][:, None]
    if back:
        n = -n
    a, b, rest = _pairs(s, t)
    return _joined(s, a * c - b * n, b * c + a * n, rest)


EPS = 1e-6


def _inv(s, x):
    q = (x * x).sum(-1, keepdim=True)
    return torch.rsqrt((q / s["d"] if s["norm"] == "rms" else q) + EPS)


def _qk_fwd_plain(s):
    out = []
    for name, wn in (("q", "qw"), ("k", "kw")):
        x = s[name].float()
        u = x * _inv(s, x)
        if s[wn] is not None:
            u = u * s[wn]
        out.append(_turn(s, u, False).to(s[name].dtype))
    return tuple(out)


def _qk_train_plain(s):
    grads, dws = [], []
    for name, wn in (("q", "qw"), ("k", "kw")):
        x = s[name].float()
        r = _inv(s, x)
        e = _turn(s, s["d" + name].float(), True)
        dws.append((e * x * r).sum((0, 1)) if s[wn] is not None else None)
        m = e * s[wn] if s[wn] is not None else e
        dot = (m * x).sum(-1, keepdim=True)
        if s["norm"] == "rms":
            dot = dot / s["d"]
        grads.append((r * m - r * r * r * x * dot).to(s[name].dtype))
    return (*_qk_fwd_plain(s), *grads, *dws)


def _delta_step_plain(s):
    live = s["idx"] >= 0
    at = s["idx"].clamp(min=0).long()
    old = s["buf"][at]
    rep = s["H"] // s["Hk"]
    q = s["q"].float().repeat_interleave(rep, 1)
    k = s["k"].float().repeat_interleave(rep, 1)
    v, beta = s["v"].float(), s["beta"].float()
    kept = torch.exp(s["g"])[..., None, None] * old
    # exp(g) (I - beta k k^T) S + beta k v^T
    seen = (kept * k[..., None]).sum(-2)
    new = kept + (beta[..., None] * k)[..., None] * (v - seen)[..., None, :]
    o = (new * q[..., None]).sum(-2) * s["d"] ** -0.5
    s["buf"].index_put_((at,), torch.where(live[:, None, None, None], new, old))
    return torch.where(live[:, None, None], o, torch.zeros_like(o)).to(s["q"].dtype), s["buf"]


_PLAIN = dict(conv_fwd=_conv_fwd_plain, conv_train=_conv_train_plain, conv_step=_conv_step_plain,
              ssm_fwd=_ssm_fwd_plain, ssm_train=_ssm_train_plain, ssm_step=_ssm_step_plain,
              qk_fwd=_qk_fwd_plain, qk_train=_qk_train_plain, delta_step=_delta_step_plain)


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    import chunked_gated_delta_gdr_gb300 as gdr
    op = s["op"]
    if op in ("conv_fwd", "conv_train"):
        y, ht = gdr.conv_fwd(s["x"], s["w"], bias=s["b"], initial_state=s["h0"],
                             cu_seqlens=s["cu"], activation=s["act"], output_final_state=True)
        if op == "conv_fwd":
            return y, ht
        return (y, ht, *gdr.conv_bwd(s["x"], s["w"], s["dy"], bias=s["b"], initial_state=s["h0"],
                                     cu_seqlens=s["cu"], activation=s["act"],
                                     dfinal_state=s["dht"], want_dinitial=s["h0"] is not None))
    if op == "conv_step":
        y = gdr.conv_step(s["x"], s["w"], s["buf"], bias=s["b"], activation=s["act"],
                          state_indices=s["idx"])
        return y, s["buf"]
    if op in ("ssm_fwd", "ssm_train"):
        y, ht = gdr.ssm_fwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["skip_w"], z=s["zg"],
                            dt_bias=s["dt_bias"], dt_softplus=True, initial_state=s["h0"],
                            cu_seqlens=s["cu"], output_final_state=True)
        if op == "ssm_fwd":
            return y, ht
        return (y, ht, *gdr.ssm_bwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dy"],
                                    D=s["skip_w"], z=s["zg"], dt_bias=s["dt_bias"],
                                    dt_softplus=True, initial_state=s["h0"], cu_seqlens=s["cu"],
                                    dfinal_state=s["dht"], want_dinitial=s["h0"] is not None))
    if op == "ssm_step":
        y = gdr.ssm_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["buf"], D=s["skip_w"],
                         z=s["zg"], dt_bias=s["dt_bias"], dt_softplus=True,
                         state_indices=s["idx"])
        return y, s["buf"]
    if op in ("qk_fwd", "qk_train"):
        opts = dict(q_weight=s["qw"], k_weight=s["kw"], norm=s["norm"], eps=EPS, cos=s["cos"],
                    sin=s["sin"], positions=s["pos"], interleaved=s["interleaved"])
        out = gdr.qk_fwd(s["q"], s["k"], **opts)
        if op == "qk_fwd":
            return out
        return (*out, *gdr.qk_bwd(s["q"], s["k"], s["dq"], s["dk"], **opts))
    o = gdr.delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["buf"],
                       state_indices=s["idx"])
    return o, s["buf"]


def run(state):
    """One pass: the outputs, with the updated states and the gradients (None: not asked for)."""
    return _own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------ the work of a pass

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("conv"):
        C, W = case["C"], case["W"]
        par = 4 * C * (W + (1 if case["bias"] else 0))
        if op == "conv_step":
            live = case["B"] - case["pad"]
            return dict(bytes=e * C * (2 * case["B"] + 2 * (W - 1) * live) + par,
                        flops=2.0 * case["B"] * C * W)
        T, st = case["T"], e * _n_seq(case) * (W - 1) * C
        b = 2 * e * T * C + par + st * (2 if case["state"] else 1)
        f = 2.0 * T * C * W
        if op == "conv_train":
            b += 3 * e * T * C + 2 * par + (3 * st if case["state"] else 0)
            f *= 4
        return dict(bytes=b, flops=f)
    if op.startswith("ssm"):
        D, N, G = case["D"], case["N"], case["G"]
        par = 4 * D * (N + 1 + (1 if case["skip"] else 0))
        z = 1 if case["z"] else 0
        if op == "ssm_step":
            B, live = case["B"], case["B"] - case["pad"]
            return dict(bytes=8 * live * D * N + e * B * ((3 + z) * D + 2 * G * N) + par,
                        flops=7.0 * B * D * N)
        T, st = case["T"], 4 * _n_seq(case) * D * N
        b = e * T * ((3 + z) * D + 2 * G * N) + par + st * (2 if case["state"] else 1)
        f = 7.0 * T * D * N
        if op == "ssm_train":
            b += e * T * ((5 + 2 * z) * D + 4 * G * N) + 2 * par + (3 * st if case["state"] else 0)
            f += 21.0 * T * D * N
        return dict(bytes=b, flops=f)
    if op.startswith("qk"):
        n = case["T"] * (case["Hq"] + case["Hk"]) * case["d"]
        table = 8 * min(case["T"], 8192) * (case["rot"] // 2) + 4 * case["T"] * bool(case["rot"])
        w = 8 * case["d"] * bool(case["weight"])
        if op == "qk_train":
            return dict(bytes=5 * e * n + 2 * table + 3 * w, flops=25.0 * n)
        return dict(bytes=2 * e * n + table + w, flops=8.0 * n)
    B, live, H, d = case["B"], case["B"] - case["pad"], case["H"], case["d"]
    return dict(bytes=8 * live * H * d * d + e * B * (2 * case["Hk"] * d + 2 * H * d + H) + 4 * B * H,
                flops=7.0 * B * H * d * d)


# ------------------------------------------------------------------ the definitions, in 64 bits

def _f64(s, *names):
    return [None if s[n] is None else s[n].double() for n in names]


def _silu64(u):
    return u / (1 + torch.exp(-u))


def _dsilu64(u):
    e = torch.exp(-u)
    return 1 / (1 + e) + u * e / (1 + e) ** 2


def _conv_exact(s, train):
    """Segment by segment: the segment's inputs with its state in front of them."""
    x, w, b, h0 = _f64(s, "x", "w", "b", "h0")
    W, lens = s["W"], _lengths(s)
    y, ends = torch.zeros_like(x), []
    dx, dh0 = torch.zeros_like(x), []
    dw, db = torch.zeros_like(w), torch.zeros(x.shape[1], dtype=torch.float64, device=x.device)
    at = 0
    for i, n in enumerate(lens):
        pre = h0[i] if h0 is not None else x.new_zeros(W - 1, x.shape[1])
        full = torch.cat([pre, x[at:at + n]])
        u = full.new_zeros(n, x.shape[1]) if b is None else b.expand(n, -1).clone()
        for k in range(W):
            u += full[k:k + n] * w[:, k]
        y[at:at + n] = _silu64(u) if s["act"] else u
        ends.append(full[n:])
        if train:
            du = s["dy"][at:at + n].double()
            if s["act"]:
                du = du * _dsilu64(u)
            dfull = torch.zeros_like(full)
            for k in range(W):
                dfull[k:k + n] += du * w[:, k]
                dw[:, k] += (du * full[k:k + n]).sum(0)
            db += du.sum(0)
            if s["dht"] is not None:
                dfull[n:] += s["dht"][i].double()
            dx[at:at + n] = dfull[W - 1:]
            dh0.append(dfull[:W - 1])
        at += n
    out = (y, torch.stack(ends))
    if not train:
        return out
    return (*out, dx, dw, db if b is not None else None,
            torch.stack(dh0) if h0 is not None else None)


def _conv_step_exact(s):
    buf, x, w, b = _f64(s, "buf", "x", "w", "b")
    y = torch.zeros_like(x)
    for r, i in enumerate(s["idx"].tolist()):
        if i < 0:
            continue
        full = torch.cat([buf[i], x[r:r + 1]])
        u = (full.t() * w).sum(1) + (b if b is not None else 0)
        y[r] = _silu64(u) if s["act"] else u
        buf[i] = full[1:]
    return y, buf


def _ssm_padded(s):
    """Inputs as [longest, segments, ...] with the tokens' rows there, in 64 bits."""
    lens = _lengths(s)
    longest, n = max(lens), len(lens)
    rows = torch.full((longest, n), -1, dtype=torch.long)
    at = 0
    for i, m in enumerate(lens):
        rows[:m, i] = torch.arange(at, at + m)
        at += m
    return rows.to(DEV), longest, n


def _ssm_exact(s, train):
    D, N, G, T = s["D"], s["N"], s["G"], s["T"]
    rows, longest, n = _ssm_padded(s)
    if longest * n * D * N * 8 > (4e10 if train else 1e12) or longest > 40000:
        return None
    x, A, Bm, Cm, skip, z, bias = _f64(s, "x", "A", "Bm", "Cm", "skip_w", "zg", "dt_bias")
    raw = s["dt"].double() + bias
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    group = torch.arange(D, device=DEV) // (D // G)
    h = s["h0"].double().clone() if s["h0"] is not None else x.new_zeros(n, D, N)
    y = torch.zeros_like(x)
    past = x.new_zeros(longest + 1, n, D, N) if train else None
    live = [rows[t] >= 0 for t in range(longest)]
    count = (rows >= 0).sum(1).tolist()
    for t in range(longest):
        if train:
            past[t] = h
        m = live[t] if count[t] < n else slice(None)
        r = rows[t][m]
        hm = torch.exp(step[r][..., None] * A) * h[m] + (step[r] * x[r])[..., None] * Bm[r][:, group]
        h[m] = hm
        y[r] = (hm * Cm[r][:, group]).sum(-1)
    if skip is not None:
        y = y + skip * x
    out = y * _silu64(z) if z is not None else y
    if not train:
        return out, h
    ht = h.clone()
    dout = s["dy"].double()
    dz = None
    if z is not None:
        dz = dout * y * _dsilu64(z)
        dout = dout * _silu64(z)
    g = s["dht"].double().clone() if s["dht"] is not None else torch.zeros_like(h)
    dx, dstep, dA = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(A)
    dB, dC = torch.zeros_like(Bm), torch.zeros_like(Cm)
    for t in reversed(range(longest)):
        m = live[t] if count[t] < n else slice(None)
        r = rows[t][m]
        a = torch.exp(step[r][..., None] * A)
        before = past[t][m]
        now = a * before + (step[r] * x[r])[..., None] * Bm[r][:, group]
        gm = g[m] + dout[r][..., None] * Cm[r][:, group]
        dC[r] = (dout[r][..., None] * now).view(-1, G, D // G, N).sum(2)
        dB[r] = ((step[r] * x[r])[..., None] * gm).view(-1, G, D // G, N).sum(2)
        into = (gm * Bm[r][:, group]).sum(-1)
        dx[r] = step[r] * into
        da = gm * before * a
        dstep[r] = x[r] * into + (da * A).sum(-1)
        dA += (da * step[r][..., None]).sum(0)
        g[m] = a * gm
    if skip is not None:
        dx = dx + skip * dout
    ddt = dstep / (1 + torch.exp(-raw))
    return (out, ht, dx, ddt, dA, dB, dC, (dout * x).sum(0) if skip is not None else None, dz,
            ddt.sum(0), g if s["h0"] is not None else None)


def _ssm_step_exact(s):
    buf, x, A, Bm, Cm, skip, z, bias = _f64(s, "buf", "x", "A", "Bm", "Cm", "skip_w", "zg",
                                            "dt_bias")
    D, G = s["D"], s["G"]
    y = torch.zeros_like(x)
    for r, i in enumerate(s["idx"].tolist()):
        if i < 0:
            continue
        step = torch.logaddexp(s["dt"][r].double() + bias, torch.zeros_like(bias))
        inn = Bm[r].repeat_interleave(D // G, 0)
        outw = Cm[r].repeat_interleave(D // G, 0)
        buf[i] = torch.exp(step[:, None] * A) * buf[i] + (step * x[r])[:, None] * inn
        v = (buf[i] * outw).sum(1)
        if skip is not None:
            v = v + skip * x[r]
        y[r] = v * _silu64(z[r]) if z is not None else v
    return y, buf


def _qk_exact(s, train):
    """Each pair as a complex number: the rotation is a product with cos + i sin."""
    outs, grads, dws = [], [], []
    r = s["rot"]
    if r:
        p = s["pos"].long()
        turn = torch.complex(s["cos"][p].double(), s["sin"][p].double())[:, None]

    def rotate(t, by):
        if not r:
            return t
        part = t[..., :r]
        if s["interleaved"]:
            c = torch.complex(part[..., 0::2].contiguous(), part[..., 1::2].contiguous()) * by
            part = torch.view_as_real(c).flatten(-2)
        else:
            c = torch.complex(part[..., :r // 2].contiguous(), part[..., r // 2:].contiguous()) * by
            part = torch.cat([c.real, c.imag], -1)
        return torch.cat([part, t[..., r:]], -1)

    for name, wn in (("q", "qw"), ("k", "kw")):
        x = s[name].double()
        w = s[wn].double() if s[wn] is not None else torch.ones(s["d"], dtype=torch.float64,
                                                                device=DEV)
        count = s["d"] if s["norm"] == "rms" else 1
        size = torch.sqrt((x ** 2).sum(-1, keepdim=True) / count + EPS)
        outs.append(rotate(x / size * w, turn if r else None))
        if train:
            e = rotate(s["d" + name].double(), turn.conj() if r else None)
            dws.append((e * (x / size)).sum((0, 1)) if s[wn] is not None else None)
            n = x / size
            grads.append((e * w - n * (e * w * n).sum(-1, keepdim=True) / count) / size)
    return (*outs, *grads, *dws)


def _delta_step_exact(s):
    buf, q, k, v, g, beta = _f64(s, "buf", "q", "k", "v", "g", "beta")
    o = torch.zeros_like(v)
    rep = s["H"] // s["Hk"]
    for r, i in enumerate(s["idx"].tolist()):
        if i < 0:
            continue
        kr, qr = k[r].repeat_interleave(rep, 0), q[r].repeat_interleave(rep, 0)
        S, bt = buf[i], beta[r][:, None, None]
        S = torch.exp(g[r])[:, None, None] * (S - bt * kr[..., None] * torch.einsum(
            "hk,hkv->hv", kr, S)[:, None])
        S = S + bt * kr[..., None] * v[r][:, None]
        buf[i] = S
        o[r] = torch.einsum("hkv,hk->hv", S, qr) * s["d"] ** -0.5
    return o, buf


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("conv_fwd", "conv_train"):
        return _conv_exact(s, op == "conv_train")
    if op == "conv_step":
        return _conv_step_exact(s)
    if op in ("ssm_fwd", "ssm_train"):
        return _ssm_exact(s, op == "ssm_train")
    if op == "ssm_step":
        return _ssm_step_exact(s)
    if op in ("qk_fwd", "qk_train"):
        return _qk_exact(s, op == "qk_train")
    return _delta_step_exact(s)
