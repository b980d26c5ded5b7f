"""Measured cases of the operators of a hybrid block beside the delta rule's mixer.

Operators (``op`` of a case):
  rec_fwd, rec_train, rec_step   gated linear recurrence over packed segments
  gated_fwd, gated_train         norm of the mixer's heads times an activated gate
  resid_fwd, resid_train         norm behind a block, its gate and residual scale, norm before the next
  attn_step                      attention of one new token over a paged key-value cache
  cache                          block tables and slots of new tokens, and their keys and values
                                 written into the pages

``run`` computes them with elementary torch operations in 32 bits where ``own`` is false, and
through the package's entry points where it is true.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # prefill of packed prompts, states carried in from cached prefixes
        dict(name="rec prompt packed 32k", op="rec_fwd", dtype="bf16", T=32768, segs=6, ghosts=1,
             equal=False, len_seed=2, D=4096, gate=True, state=True),
        # a small ragged packed prefill in 32 bits, odd channel count
        dict(name="rec ragged fp32", op="rec_fwd", dtype="fp32", T=1537, segs=7, ghosts=2,
             equal=False, len_seed=11, D=1002, gate=True, state=False),
        # a training step on packed sequences
        dict(name="rec train packed 8k", op="rec_train", dtype="bf16", T=8192, segs=5, ghosts=1,
             equal=False, len_seed=5, D=2560, gate=True, state=True),
        # decoding: the states of 128 requests in a pool
        dict(name="rec step 128", op="rec_step", dtype="bf16", B=128, slots=160, pad=3, D=4096,
             gate=True),
        # prefill: the norm behind the delta rule, 32 heads of 128
        dict(name="gated norm prompt 64k", op="gated_fwd", dtype="bf16", T=65536, H=32, d=128,
             act="silu", weight=True),
        # a training step, odd token count
        dict(name="gated norm train 8191", op="gated_train", dtype="bf16", T=8191, H=16, d=128,
             act="silu", weight=True),
        # decoding: 37 requests, both norms of the block
        dict(name="residual norm step 37", op="resid_fwd", dtype="bf16", res="bf16", T=37, C=4096,
             post=True, gate=True),
        # a training step, both norms, a gate for each channel
        dict(name="residual norm train 16k", op="resid_train", dtype="bf16", res="bf16", T=16384,
             C=4096, post=True, gate=True),
        # decoding of one request with a long context
        dict(name="attention step 1x32k", op="attn_step", dtype="bf16", B=1, Hq=32, Hk=8, d=128,
             longest=32768, page=64, window=0, pad=0, len_seed=1),
        # decoding of a batch of uneven contexts, padded rows among them
        dict(name="attention step 64 uneven", op="attn_step", dtype="bf16", B=64, Hq=32, Hk=4,
             d=128, longest=16384, page=16, window=0, pad=2, len_seed=4),
        # decoding: pages and slots of one new token for each of 256 requests, and its key and value
        dict(name="cache step 256", op="cache", dtype="bf16", B=256, most=1, before=100, Hk=8,
             d=128, page=16, len_seed=7),
        # prefill of 12 prompts in chunks, behind what is in the cache already
        dict(name="cache prompt 12", op="cache", dtype="bf16", B=12, most=2500, before=700, Hk=8,
             d=128, page=16, len_seed=9),
    ]


def _log(rng, lo, hi):
    hi = max(lo, hi)
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rec_fwd", "rec_train", "rec_step", "gated_fwd", "gated_train", "resid_fwd",
                     "resid_train", "attn_step", "attn_step", "cache"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    e = 2 if dtype == "bf16" else 4
    if op.startswith("rec"):
        D = _log(rng, 64, 5120)
        if rng.random() < 0.7:
            D = -(-D // 64) * 64
        more = dict(D=D, gate=rng.random() < 0.8)
        if op == "rec_step":
            B = _log(rng, 1, 512)
            return dict(op=op, dtype=dtype, B=B, slots=B + rng.randrange(4, 40),
                        pad=min(B - 1, rng.choice([0, 0, 1, 3])), **more)
        most = (32768 * 4096 if op == "rec_fwd" else 8192 * 2560 * 2) * 2 // (e * D)
        return dict(op=op, dtype=dtype, T=_log(rng, 1, min(most, 65536)), segs=_log(rng, 1, 64),
                    ghosts=rng.choice([0, 0, 1, 5]), equal=rng.random() < 0.3,
                    len_seed=rng.randrange(1 << 20), state=rng.random() < 0.5, **more)
    if op.startswith("gated"):
        d = rng.choice([64, 128, 128, 256, 8 * rng.randrange(2, 32), rng.randrange(1, 257)])
        H = _log(rng, 1, 32)
        most = (65536 * 4096 if op == "gated_fwd" else 8191 * 4096) * 2 // (e * d * H)
        return dict(op=op, dtype=dtype, T=_log(rng, 1, min(most, 131072)), H=H, d=d,
                    act=rng.choice(["silu", "silu", "sigmoid"]), weight=rng.random() < 0.8)
    if op.startswith("resid"):
        C = _log(rng, 64, 16384)
        if rng.random() < 0.8:
            C = min(16384, -(-C // 64) * 64)
        most = 16384 * 4096 * 2 // (e * C)
        return dict(op=op, dtype=dtype, res=rng.choice([dtype, dtype, "fp32"]),
                    T=_log(rng, 1, min(most // 2, 65536)), C=C, post=rng.random() < 0.6,
                    gate=rng.random() < 0.5)
    if op == "attn_step":
        d = rng.choice([64, 128, 128, 256, 8 * rng.randrange(2, 32)])
        Hk = rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.choice([1, 2, 4, 6, 8, 16])
        room = 64 * 16384 * 4 * 128 // (2 * Hk * d)  # keys of all requests
        longest = _log(rng, 1, min(65536, room))
        return dict(op=op, dtype="bf16", B=_log(rng, 1, min(256, max(1, room // longest))), Hq=Hq,
                    Hk=Hk, d=d, longest=longest, page=rng.choice([16, 16, 32, 64, 128, 5, 1]),
                    window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), pad=0,
                    len_seed=rng.randrange(1 << 20))
    Hk, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
    most = _log(rng, 1, 2048)
    return dict(op=op, dtype=dtype, B=_log(rng, 1, max(1, min(1024, 16384 // most))), most=most,
                before=rng.choice([0, 30, 200]), Hk=Hk, d=d, page=rng.choice([16, 32, 64, 128, 3]),
                len_seed=rng.randrange(1 << 20))


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


def _contexts(case):
    """Keys of each request with its new token: between a sixteenth and all of the longest, once
    the longest; 0 marks a padded row."""
    r = random.Random(case["len_seed"])
    top = case["longest"]
    lens = [r.randint(max(1, top // 16), top) for _ in range(case["B"])]
    lens[r.randrange(case["B"])] = top
    for i in r.sample(range(case["B"]), min(case["pad"], case["B"] - 1)):
        lens[i] = 0
    return lens


def _seen(case):
    """Keys that each request's token attends to."""
    w = case["window"]
    return [min(n, w) if w else n for n in _contexts(case)]


def _arrivals(case):
    """(tokens in the cache before, new tokens) of each request."""
    r = random.Random(case["len_seed"])
    before = [r.randint(0, case["before"]) for _ in range(case["B"])]
    return before, [r.randint(1, case["most"]) for _ in range(case["B"])]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(int(seed))
    dt = TYPES[case["dtype"]]
    op = case["op"]

    def rn(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=DEV).mul_(std).to(dtype)

    def pages(n):
        return torch.randperm(n, generator=gen, device=DEV).to(torch.int32)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=DEV)

    s = dict(case)
    if op.startswith("rec"):
        D = case["D"]
        rows = case["B"] if op == "rec_step" else case["T"]
        s["x"], s["r"] = rn(rows, D, dtype=dt), rn(rows, D, dtype=dt)
        s["i"] = rn(rows, D, dtype=dt) if case["gate"] else None
        # the decay at a fully open gate: between 0.9 and 0.999 to the eighth power
        s["A"] = 8.0 * torch.log(0.9 + 0.099 * torch.rand(D, generator=gen, device=DEV))
        if op == "rec_step":
            # live slots are 1 .. slots - 1 in any order; -1 marks a padded row of the batch
            idx = pages(case["slots"] - 1)[:case["B"]] + 1
            if case["pad"]:
                idx[torch.randperm(case["B"], generator=gen, device=DEV)[:case["pad"]]] = -1
            s["idx"], s["buf"] = idx, rn(case["slots"], D)
        else:
            lens = _lengths(case)
            s["cu"] = ints([0] + lens).cumsum(0).to(torch.int32)
            s["h0"] = rn(len(lens), D) if case["state"] else None
            if op == "rec_train":
                s["dy"] = rn(rows, D, std=0.1, dtype=dt)
                s["dht"] = rn(len(lens), D, std=0.1) if case["state"] else None
    elif op.startswith("gated"):
        T, H, d = case["T"], case["H"], case["d"]
        s["x"], s["z"] = rn(T, H, d, dtype=dt), rn(T, H, d, dtype=dt)
        s["w"] = 1.0 + rn(d, std=0.1) if case["weight"] else None
        if op == "gated_train":
            s["dy"] = rn(T, H, d, std=0.1, dtype=dt)
    elif op.startswith("resid"):
        T, C = case["T"], case["C"]
        s["x"], s["res_in"] = rn(T, C, dtype=dt), rn(T, C, std=2.0, dtype=TYPES[case["res"]])
        s["w"] = 1.0 + rn(C, std=0.1)
        s["wp"] = 1.0 + rn(C, std=0.1) if case["post"] else None
        s["g"] = 0.5 + rn(C, std=0.2) if case["gate"] else None
        s["scale"] = 0.7
        if op == "resid_train":
            s["dy"] = rn(T, C, std=0.1, dtype=dt)
            s["dh"] = rn(T, C, std=0.1, dtype=TYPES[case["res"]])
    elif op == "attn_step":
        B, Hk, d, ps = case["B"], case["Hk"], case["d"], case["page"]
        lens = _contexts(case)
        width = -(-case["longest"] // ps)
        need = [-(-n // ps) for n in lens]
        pool = sum(need) + 3
        # requests hold their pages in any order; what a row does not use is -1
        order = pages(pool)
        table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        s["table"], s["lens"] = table, ints(lens)
        s["q"] = rn(B, case["Hq"], d, std=1.5, dtype=dt)
        s["kc"], s["vc"] = rn(pool, ps, Hk, d, dtype=dt), rn(pool, ps, Hk, d, dtype=dt)
    else:
        B, Hk, d, ps = case["B"], case["Hk"], case["d"], case["page"]
        before, new = _arrivals(case)
        s["max_tokens"] = sum(new)
        width = max(-(-(a + b) // ps) for a, b in zip(before, new))
        have = [-(-a // ps) for a in before]
        more = sum(-(-(a + b) // ps) - h for a, b, h in zip(before, new, have))
        pool = sum(have) + more + 5
        order = pages(pool)
        table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        at = 0
        for i, n in enumerate(have):
            table[i, :n] = order[at:at + n]
            at += n
        # the free pages: two of them were taken by earlier steps
        s["table"], s["lens"], s["new"] = table, ints(before), ints(new)
        s["free"] = torch.cat([order[:2], order[at:]])
        s["taken"] = ints([2])
        s["k"], s["v"] = (rn(s["max_tokens"], Hk, d, dtype=dt) for _ in range(2))
        s["kc"], s["vc"] = rn(pool, ps, Hk, d, dtype=dt), rn(pool, ps, Hk, d, dtype=dt)
    return s


# ------------------------------------------------------------------ the plain forms, in 32 bits

def _places(cu, T):
    """Segment of each token, its place there, and the segments' lengths (no host reads)."""
    t = torch.arange(T, device=cu.device)
    cu = cu.long()
    seg = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return seg, t - cu[seg], cu[1:] - cu[:-1]


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis by doubling (in place); a is used up."""
    n = 1
    while n < b.shape[0]:
        b[n:] += a[n:] * b[:-n]
        a[n:] *= a[:-n].clone()
        n *= 2
    return b


def _rec_parts(s):
    """Sigmoid of r, log a, the normaliser, sigmoid of i (or 1) and x, in 32 bits."""
    sr = torch.sigmoid(s["r"].float())
    L = s["A"] * sr
    si = torch.sigmoid(s["i"].float()) if s["i"] is not None else None
    return sr, L, torch.sqrt(-torch.expm1(2.0 * L)), si, s["x"].float()


def _rec_states(s, a, u):
    T = u.shape[0]
    seg, place, n = _places(s["cu"], T)
    first = (place == 0)[:, None]
    if s["h0"] is not None:
        u = torch.where(first, u + a * s["h0"][seg], u)
    h = _scan(torch.where(first, torch.zeros_like(a), a), u.clone())
    cu = s["cu"].long()
    h0 = s["h0"] if s["h0"] is not None else torch.zeros_like(h[:1]).expand(n.numel(), -1)
    ht = torch.where((n > 0)[:, None], h[(cu[1:] - 1).clamp(min=0)], h0)
    return h, ht, h0, seg, place, n


def _rec_fwd_plain(s):
    _, L, m, si, x = _rec_parts(s)
    h, ht, *_ = _rec_states(s, torch.exp(L), m * x if si is None else m * si * x)
    return h.to(s["x"].dtype), ht


def _rec_train_plain(s):
    dt = s["x"].dtype
    sr, L, m, si, x = _rec_parts(s)
    a = torch.exp(L)
    v = x if si is None else si * x
    h, ht, h0, seg, place, n = _rec_states(s, a, m * v)
    T = x.shape[0]
    # the states' gradients: the same recurrence from the last token to the first
    last = (n[seg] - 1 - place == 0)[:, None]
    g = s["dy"].float()
    if s["dht"] is not None:
        g = torch.where(last, g + s["dht"][seg], g)
    nxt = torch.where(last, torch.zeros_like(a), torch.cat([a[1:], a[:1]]))
    g = _scan(nxt.flip(0), g.flip(0).contiguous()).flip(0)
    before = torch.where((place == 0)[:, None], h0[seg], torch.cat([h[:1], h[:-1]]))
    dL = g * a * before - g * v * a * a / m
    dr = dL * s["A"] * sr * (1 - sr)
    dA = (dL * sr).sum(0)
    dx = g * m if si is None else g * m * si
    di = None if si is None else (g * m * x * si * (1 - si)).to(dt)
    dh0 = None
    if s["h0"] is not None:
        at = s["cu"].long()[:-1].clamp(max=T - 1)
        dh0 = torch.where((n > 0)[:, None], a[at] * g[at], s["dht"])
    return h.to(dt), ht, dx.to(dt), dr.to(dt), dA, di, dh0


def _rec_step_plain(s):
    live = (s["idx"] >= 0)[:, None]
    at = s["idx"].clamp(min=0).long()
    old = s["buf"][at]
    _, L, m, si, x = _rec_parts(s)
    new = torch.exp(L) * old + (m * x if si is None else m * si * x)
    s["buf"].index_put_((at,), torch.where(live, new, old))
    return torch.where(live, new, torch.zeros_like(new)).to(s["x"].dtype), s["buf"]


def _act(s, z):
    """The activated gate and its derivative."""
    sg = torch.sigmoid(z)
    if s["act"] == "silu":
        return z * sg, sg + z * sg * (1 - sg)
    return sg, sg * (1 - sg)


def _inv(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _gated_fwd_plain(s):
    x = s["x"].float()
    y = x * _inv(x) * _act(s, s["z"].float())[0]
    if s["w"] is not None:
        y = y * s["w"]
    return y.to(s["x"].dtype)


def _gated_train_plain(s):
    dt = s["x"].dtype
    x, dy = s["x"].float(), s["dy"].float()
    r = _inv(x)
    n = x * r
    g, dg = _act(s, s["z"].float())
    y = n * g
    e, f = dy * g, dy * n
    dw = None
    if s["w"] is not None:
        y = y * s["w"]
        dw = (e * n).sum((0, 1))
        e, f = e * s["w"], f * s["w"]
    dx = r * (e - n * (e * n).mean(-1, keepdim=True))
    return y.to(dt), dx.to(dt), (f * dg).to(dt), dw


def _resid_parts(s):
    x, res = s["x"].float(), s["res_in"].float()
    rp = _inv(x) if s["wp"] is not None else None
    u = x * rp * s["wp"] if s["wp"] is not None else x
    v = u * s["g"] if s["g"] is not None else u
    h = res + s["scale"] * v
    return x, rp, u, h, _inv(h)


def _resid_fwd_plain(s):
    _, _, _, h, r = _resid_parts(s)
    return (h * r * s["w"]).to(s["x"].dtype), h.to(s["res_in"].dtype)


def _resid_train_plain(s):
    dt, rt = s["x"].dtype, s["res_in"].dtype
    x, rp, u, h, r = _resid_parts(s)
    n, dy = h * r, s["dy"].float()
    e = dy * s["w"]
    dw = (dy * n).sum(0)
    dh = s["dh"].float() + r * (e - n * (e * n).mean(-1, keepdim=True))
    dv = s["scale"] * dh
    dg = (dv * u).sum(0) if s["g"] is not None else None
    du = dv * s["g"] if s["g"] is not None else dv
    dwp, dx = None, du
    if s["wp"] is not None:
        xn = x * rp
        dwp = (du * xn).sum(0)
        e = du * s["wp"]
        dx = rp * (e - xn * (e * xn).mean(-1, keepdim=True))
    return (n * s["w"]).to(dt), h.to(rt), dx.to(dt), dh.to(rt), dw, dwp, dg


def _attn_step_plain(s):
    B, Hq, d = s["q"].shape
    Hk, ps = s["Hk"], s["page"]
    width = s["table"].shape[1] * ps
    at = torch.arange(width, device=DEV)
    n = s["lens"][:, None]
    seen = (at < n) & (s["table"].repeat_interleave(ps, 1) >= 0)
    if s["window"]:
        seen = seen & (at >= n - s["window"])
    got = s["table"].clamp(min=0).long()
    k = s["kc"][got].view(B, width, Hk, d).permute(0, 2, 3, 1).float()
    v = s["vc"][got].view(B, width, Hk, d).permute(0, 2, 1, 3).float()
    q = s["q"].float().view(B, Hk, Hq // Hk, d)
    w = torch.matmul(q, k) * d ** -0.5
    seen = seen[:, None, None]
    w = torch.where(seen, w, torch.full_like(w, -math.inf))
    top = w.amax(-1, keepdim=True).clamp(min=-3e38)  # a row without keys: weights of 0
    p = torch.exp(w - top)
    total = p.sum(-1, keepdim=True)
    # what a cache holds behind a request's keys is not looked at
    v = torch.where(seen[:, :, 0, :, None], v, torch.zeros_like(v))
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.view(B, Hq, d).to(s["q"].dtype)


def _cache_plain(s):
    """Pages are handed out in the order of the requests, as many as there are."""
    ps, cap = s["page"], s["max_tokens"]
    B, width = s["table"].shape
    n0 = s["lens"].long().clamp(min=0)
    new = torch.minimum(s["new"].long().clamp(min=0), (width * ps - n0).clamp(min=0))
    end = new.cumsum(0)
    new = end.clamp(max=cap) - (end - new).clamp(max=cap)
    have = (n0 + ps - 1) // ps
    need = (n0 + new + ps - 1) // ps - have
    need = need.clamp(min=0)
    taken = s["taken"].long().clamp(0, s["free"].numel())
    left = s["free"].numel() - taken
    end = need.cumsum(0)
    start = torch.minimum(end - need, left)
    got = torch.minimum(end, left) - start
    new = torch.minimum(new, (have + got) * ps - n0).clamp(min=0)
    col = torch.arange(width, device=DEV)
    j = col - have[:, None]
    fresh = (j >= 0) & (j < got[:, None])
    page = s["free"][(taken + start[:, None] + j).clamp(0, s["free"].numel() - 1)]
    s["table"].copy_(torch.where(fresh, page, s["table"]))
    after = n0 + new
    cu = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    t = torch.arange(cap, device=DEV)
    row = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=B - 1)
    inside = t < cu[-1]
    pos = torch.where(inside, n0[row] + t - cu[row], torch.zeros_like(t))
    page = s["table"][row, (pos // ps).clamp(max=width - 1)].long()
    slots = torch.where(inside & (page >= 0), page * ps + pos % ps, torch.full_like(t, -1))
    # a token without a slot rewrites what the first slot holds: none of these cases has one
    for new_rows, cache in ((s["k"], s["kc"]), (s["v"], s["vc"])):
        flat = cache.view(-1, *cache.shape[2:])
        dst = slots.clamp(min=0)
        flat.index_copy_(0, dst, torch.where((slots >= 0)[:, None, None], new_rows, flat[dst]))
    i32 = lambda v: v.to(torch.int32)
    return (i32(slots), i32(pos), i32(cu), i32(after), i32(taken + got.sum()), s["table"],
            s["kc"], s["vc"])


_PLAIN = dict(rec_fwd=_rec_fwd_plain, rec_train=_rec_train_plain, rec_step=_rec_step_plain,
              gated_fwd=_gated_fwd_plain, gated_train=_gated_train_plain,
              resid_fwd=_resid_fwd_plain, resid_train=_resid_train_plain,
              attn_step=_attn_step_plain, cache=_cache_plain)


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    import chunked_gated_delta_gdr_gb300 as gdr
    op = s["op"]
    if op in ("rec_fwd", "rec_train"):
        train = op == "rec_train"
        y, ht, kept = gdr.rec_fwd(s["x"], s["r"], s["A"], s["i"], initial_state=s["h0"],
                                  cu_seqlens=s["cu"], output_final_state=True,
                                  output_checkpoints=train)
        if not train:
            return y, ht
        return (y, ht, *gdr.rec_bwd(s["x"], s["r"], s["A"], s["dy"], s["i"],
                                    initial_state=s["h0"], cu_seqlens=s["cu"],
                                    dfinal_state=s["dht"], checkpoints=kept,
                                    want_dinitial=s["h0"] is not None))
    if op == "rec_step":
        y = gdr.rec_step(s["x"], s["r"], s["A"], s["buf"], s["i"], state_indices=s["idx"])
        return y, s["buf"]
    if op in ("gated_fwd", "gated_train"):
        y = gdr.gated_norm_fwd(s["x"], s["z"], s["w"], activation=s["act"], eps=EPS)
        if op == "gated_fwd":
            return y
        return (y, *gdr.gated_norm_bwd(s["x"], s["z"], s["dy"], s["w"], activation=s["act"],
                                       eps=EPS))
    if op in ("resid_fwd", "resid_train"):
        opts = dict(post_weight=s["wp"], gate=s["g"], scale=s["scale"], eps=EPS)
        out = gdr.residual_norm_fwd(s["x"], s["res_in"], s["w"], **opts)
        if op == "resid_fwd":
            return out
        return (*out, *gdr.residual_norm_bwd(s["x"], s["res_in"], s["dy"], s["dh"], s["w"], **opts))
    if op == "attn_step":
        return gdr.attn_step(s["q"], s["kc"], s["vc"], s["table"], s["lens"], window=s["window"])
    slots, pos, cu, after, taken = gdr.cache_plan(s["lens"], s["new"], s["table"], s["free"],
                                                  s["taken"], s["page"], s["max_tokens"])
    gdr.cache_write(s["k"], s["v"], s["kc"], s["vc"], slots)
    return slots, pos, cu, after, taken, s["table"], s["kc"], s["vc"]


def run(state):
    """One pass: the outputs, with the updated states and the gradients (None: not asked for)."""
    return _own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------ the work of a pass

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("rec"):
        D, ins = case["D"], 3 if case["gate"] else 2
        if op == "rec_step":
            B, live = case["B"], case["B"] - case["pad"]
            return dict(bytes=8 * live * D + e * B * D * (ins + 1) + 4 * D + 4 * B,
                        flops=14.0 * B * D)
        T, st = case["T"], 4 * _n_seq(case) * D
        b = e * T * D * (ins + 1) + 4 * D + st * (2 if case["state"] else 1)
        f = 14.0 * T * D
        if op == "rec_train":
            # the inputs are counted once for both directions
            b += e * T * D * (ins + 1) + 4 * D + (2 * st if case["state"] else 0)
            f += 40.0 * T * D
        return dict(bytes=b, flops=f)
    if op.startswith("gated"):
        n, w = case["T"] * case["H"] * case["d"], 4 * case["d"] * bool(case["weight"])
        if op == "gated_train":
            return dict(bytes=6 * e * n + 2 * w, flops=35.0 * n)
        return dict(bytes=3 * e * n + w, flops=12.0 * n)
    if op.startswith("resid"):
        n, C = case["T"] * case["C"], case["C"]
        er = 4 if case["res"] == "fp32" else 2
        par = 4 * C * (1 + bool(case["post"]) + bool(case["gate"]))
        if op == "resid_train":
            return dict(bytes=(4 * e + 4 * er) * n + 2 * par, flops=45.0 * n)
        return dict(bytes=(2 * e + 2 * er) * n + par, flops=14.0 * n)
    if op == "attn_step":
        keys, B = sum(_seen(case)), case["B"]
        held = sum(-(-n // case["page"]) for n in _seen(case))
        return dict(bytes=2 * e * keys * case["Hk"] * case["d"] + 2 * e * B * case["Hq"] * case["d"]
                    + 4 * B + 4 * held,
                    flops=4.0 * keys * case["Hq"] * case["d"])
    before, new = _arrivals(case)
    n, B, ps = sum(new), case["B"], case["page"]
    more = sum(-(-(a + b) // ps) - -(-a // ps) for a, b in zip(before, new))
    return dict(bytes=4 * e * n * case["Hk"] * case["d"] + 4 * (4 * B + 2 * more + 3 * n + 4),
                flops=8.0 * n)


# ------------------------------------------------------------------ the definitions, in 64 bits

def _sig64(v):
    return 1 / (1 + torch.exp(-v))


def _leaf(t):
    return None if t is None else t.double().requires_grad_(True)


def _rec_exact(s, train):
    """Token by token, all segments side by side."""
    lens = _lengths(s)
    longest, n, D = max(lens), len(lens), s["D"]
    if longest > 40000 or (train and longest * n * D * 8 > 3e10):
        return None
    start, at = [], 0
    for m in lens:
        start.append(at)
        at += m
    start, size = torch.tensor(start, device=DEV), torch.tensor(lens, device=DEV)
    A, x = s["A"].double(), s["x"].double()
    sr = _sig64(s["r"].double())
    a = torch.exp(A * sr)
    m = torch.sqrt((1 - a) * (1 + a))
    # 1 - a loses digits next to a = 1: the series of the exponential there
    t = A * sr
    m = torch.where(t > -1e-4, torch.sqrt(-2 * t * (1 + t + 2 * t * t / 3)), m)
    si = _sig64(s["i"].double()) if s["i"] is not None else torch.ones_like(x)
    h = s["h0"].double().clone() if s["h0"] is not None else x.new_zeros(n, D)
    y = torch.zeros_like(x)
    before = torch.zeros_like(x) if train else None
    some = [j for j in range(n) if lens[j]]
    order = sorted(some, key=lambda j: -lens[j])
    rank = torch.tensor(order, device=DEV)
    count = [sum(1 for j in some if lens[j] > t) for t in range(longest)]
    for t in range(longest):
        which = rank[:count[t]]
        rows = start[which] + t
        hw = h[which]
        if train:
            before[rows] = hw
        hw = a[rows] * hw + m[rows] * si[rows] * x[rows]
        h[which] = hw
        y[rows] = hw
    if not train:
        return y, h
    g = s["dht"].double().clone() if s["dht"] is not None else torch.zeros_like(h)
    dh = torch.zeros_like(x)
    dy = s["dy"].double()
    for t in reversed(range(longest)):
        which = rank[:count[t]]
        rows = start[which] + t
        gw = g[which] + dy[rows]
        dh[rows] = gw
        g[which] = a[rows] * gw
    # d/da of a h + sqrt(1 - a^2) v, and a = exp(A sigmoid(r))
    da = dh * (before - a / m * si * x)
    dsr = da * a * A
    return (y, h, dh * m * si, dsr * sr * (1 - sr), (da * a * sr).sum(0),
            dh * m * x * si * (1 - si) if s["i"] is not None else None,
            g if s["h0"] is not None else None)


def _rec_step_exact(s):
    buf, x, A = s["buf"].double(), s["x"].double(), s["A"].double()
    y = torch.zeros_like(x)
    for j, slot in enumerate(s["idx"].tolist()):
        if slot < 0:
            continue
        a = torch.exp(A * _sig64(s["r"][j].double()))
        u = torch.sqrt((1 - a) * (1 + a)) * x[j]
        if s["i"] is not None:
            u = u * _sig64(s["i"][j].double())
        buf[slot] = a * buf[slot] + u
        y[j] = buf[slot]
    return y, buf


def _rms64(x):
    return x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + EPS)


def _gated_exact(s, train):
    with torch.enable_grad():
        x, z, w = _leaf(s["x"]), _leaf(s["z"]), _leaf(s["w"])
        y = _rms64(x) * (z * _sig64(z) if s["act"] == "silu" else _sig64(z))
        if w is not None:
            y = y * w
        if not train:
            return y.detach()
        y.backward(s["dy"].double())
    return y.detach(), x.grad, z.grad, None if w is None else w.grad


def _resid_exact(s, train):
    with torch.enable_grad():
        x, res, w, wp, g = (_leaf(s[k]) for k in ("x", "res_in", "w", "wp", "g"))
        u = x if wp is None else _rms64(x) * wp
        h = res + s["scale"] * (u if g is None else u * g)
        y = _rms64(h) * w
        if not train:
            return y.detach(), h.detach()
        torch.autograd.backward((y, h), (s["dy"].double(), s["dh"].double()))
    return (y.detach(), h.detach(), x.grad, res.grad, w.grad, None if wp is None else wp.grad,
            None if g is None else g.grad)


def _attn_exact(s):
    """Request by request over its own keys alone."""
    B, Hq, d = s["q"].shape
    ps, rep = s["page"], s["Hq"] // s["Hk"]
    o = torch.zeros(B, Hq, d, dtype=torch.float64, device=DEV)
    for j, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        first = max(0, n - s["window"]) if s["window"] else 0
        at = torch.arange(first, n, device=DEV)
        rows = s["table"][j].long()[at // ps] * ps + at % ps
        for h in range(s["Hk"]):
            k = s["kc"].view(-1, s["Hk"], d)[rows, h].double()
            v = s["vc"].view(-1, s["Hk"], d)[rows, h].double()
            w = s["q"][j, h * rep:(h + 1) * rep].double() @ k.t() / math.sqrt(d)
            o[j, h * rep:(h + 1) * rep] = torch.softmax(w, -1) @ v
    return o


def _cache_exact(s):
    """Whole numbers have no value in 64 bits to be near; the caches are copies."""
    before, new = _arrivals(s)
    ps, at = s["page"], int(s["taken"])
    table, free = s["table"].tolist(), s["free"].tolist()
    rows, t = [], 0
    for j, (n0, n) in enumerate(zip(before, new)):
        for p in range(n0, n0 + n):
            if table[j][p // ps] < 0:
                table[j][p // ps] = free[at]
                at += 1
            rows.append(table[j][p // ps] * ps + p % ps)
    rows = torch.tensor(rows, device=DEV)
    out = []
    for new_rows, cache in ((s["k"], s["kc"]), (s["v"], s["vc"])):
        c = cache.double()
        c.view(-1, *c.shape[2:])[rows] = new_rows.double()
        out.append(c)
    return (None, None, None, None, None, None, *out)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rec_fwd", "rec_train"):
        return _rec_exact(s, op == "rec_train")
    if op == "rec_step":
        return _rec_step_exact(s)
    if op in ("gated_fwd", "gated_train"):
        return _gated_exact(s, op == "gated_train")
    if op in ("resid_fwd", "resid_train"):
        return _resid_exact(s, op == "resid_train")
    return _attn_exact(s) if op == "attn_step" else _cache_exact(s)
