"""A hybrid block's operators on a GB300 against plain 64-bit implementations: gated linear
recurrence, norms with gate and residual scale, attention over a paged cache, block tables and
slots; forward and backward, over types, strides, odd sizes, empty and malformed segments, and
values that must reach no output."""
import pytest
import torch

import block_testlib as ref
import chunked_gated_delta_gdr_gb300 as gdr
from block_testlib import CU
from mixer_testlib import BF16, F32, assert_close, bounds, leaf

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_gdr_gb300 import build
    build.build()
    if torch.cuda.get_device_capability() != (10, 3):
        pytest.skip("needs sm_103 (GB300)")


def rn(gen, *shape, dtype=F32, std=1.0):
    return (std * torch.randn(*shape, generator=gen)).to(dtype)


def dev(t):
    return None if t is None else t.to(DEV)


def padded(t, extra=5):
    """The same values with a row stride that is not a multiple of 16 bytes, on the device."""
    if t is None:
        return None
    wide = torch.zeros(*t.shape[:-1], t.shape[-1] + extra, dtype=t.dtype, device=DEV)
    view = wide[..., 1:1 + t.shape[-1]]
    view.copy_(t)
    return view


def cu_of(name):
    T, cu = CU[name]
    return T, cu, torch.tensor(cu, dtype=torch.int32, device=DEV)


def longest(cu, T):
    b = bounds(cu, T)
    return max([e - s for s, e in zip(b[:-1], b[1:])] + [0])


# ------------------------------------------------------------------ gated linear recurrence

REC = [  # bounds, channels, type, input gate, normaliser, states, odd strides
    ("one", 64, BF16, True, True, True, False),
    ("single", 64, BF16, True, True, True, False),
    ("single", 1, F32, False, True, False, False),
    ("short", 72, F32, True, True, True, False),
    ("ghosts", 130, BF16, True, True, True, False),
    ("ghosts", 96, F32, False, True, False, False),
    ("gaps", 70, F32, True, False, True, True),
    ("gaps", 33, BF16, True, True, True, True),
    ("long", 64, F32, True, True, True, False),
    ("long", 1030, BF16, False, False, True, False),
    ("malformed", 64, F32, True, True, True, False),
    ("none", 64, BF16, True, True, True, False),
    ("all empty", 64, BF16, True, True, True, False),
    ("many", 65, F32, True, True, True, False),
    ("no segments", 16, F32, True, True, False, False),
]


def rec_inputs(T, n, D, dtype, gate, state, seed):
    gen = torch.Generator().manual_seed(seed)
    return dict(x=rn(gen, T, D, dtype=dtype), r=rn(gen, T, D, dtype=dtype),
                i=rn(gen, T, D, dtype=dtype) if gate else None,
                A=8 * torch.log(0.9 + 0.099 * torch.rand(D, generator=gen)),
                h0=rn(gen, n, D) if state else None, dy=rn(gen, T, D, dtype=dtype),
                dht=rn(gen, n, D) if state else None)


@pytest.mark.parametrize("name,D,dtype,gate,norm,state,odd", REC)
def test_rec_forward_and_backward(name, D, dtype, gate, norm, state, odd):
    T, cu, cud = cu_of(name)
    n = len(cu) - 1
    s = rec_inputs(T, n, D, dtype, gate, state, T * 31 + D)
    place = padded if odd else dev
    steps = longest(cu, T)
    y0 = torch.full((T, D), 7.0, dtype=dtype, device=DEV)
    x, r, i = place(s["x"]), place(s["r"]), place(s["i"])
    y, ht, kept = gdr.rec_fwd(x, r, dev(s["A"]), i, norm, dev(s["h0"]), cud, True, True, out=y0)
    lx, lr, lA, li, lh = (leaf(s[k]) for k in ("x", "r", "A", "i", "h0"))
    yr, hr, mask = ref.rec(lx, lr, lA, li, norm, lh, cu)
    assert_close(y.cpu()[mask], yr[mask], steps, "y")
    assert torch.all(y.cpu()[~mask] == 7.0), "tokens outside the segments were written"
    assert_close(ht, hr, steps, "final state")
    base = lh if lh is not None else torch.zeros(n, D, dtype=torch.float64, requires_grad=True)
    yr, hr, _ = ref.rec(lx, lr, lA, li, norm, base, cu)
    loss = (yr * s["dy"].double()).sum() + base.sum() * 0 + lx.sum() * 0 + lr.sum() * 0 + lA.sum() * 0
    if li is not None:
        loss = loss + li.sum() * 0
    if s["dht"] is not None:
        loss = loss + (hr * s["dht"].double()).sum()
    loss.backward()
    runs = [gdr.rec_bwd(x, r, dev(s["A"]), place(s["dy"]), i, norm, dev(s["h0"]), cud,
                        dev(s["dht"]), checkpoints=c) for c in (kept, None)]
    for dx, dr, dA, di, dh0 in runs:
        assert_close(dx, lx.grad, steps, "dx")
        assert_close(dr, lr.grad, steps, "dr")
        assert_close(dA, lA.grad, T, "dA")
        assert_close(dh0, base.grad, steps, "dh0")
        if gate:
            assert_close(di, li.grad, steps, "di")
        else:
            assert di is None
    for a, b in zip(*runs):  # the states are the same, kept or computed again
        assert (a is None and b is None) or torch.equal(a, b)


def test_rec_gradients_are_differences():
    T, cu, cud = cu_of("ghosts")
    s = rec_inputs(T, len(cu) - 1, 24, F32, True, True, 5)
    grads = gdr.rec_bwd(*(dev(s[k]) for k in ("x", "r", "A", "dy", "i")), True, dev(s["h0"]), cud,
                        dev(s["dht"]))
    gen = torch.Generator().manual_seed(6)

    def loss(v):
        y, h, _ = ref.rec(v["x"], v["r"], v["A"], v["i"], True, v["h0"], cu)
        return float((y * s["dy"].double()).sum() + (h * s["dht"].double()).sum())

    base = {k: s[k].double() for k in ("x", "r", "A", "i", "h0")}
    for k, g in zip(("x", "r", "A", "i", "h0"), grads):
        k, g = (("x", grads[0]), ("r", grads[1]), ("A", grads[2]), ("i", grads[3]),
                ("h0", grads[4]))[("x", "r", "A", "i", "h0").index(k)]
        way = torch.randn(base[k].shape, generator=gen, dtype=torch.float64)
        step = 1e-5 if k != "A" else 1e-7
        diff = (loss({**base, k: base[k] + step * way}) -
                loss({**base, k: base[k] - step * way})) / (2 * step)
        got = float((g.cpu().double() * way).sum())
        # fp32 gradients as above, each weighted once; the difference's own error is below 1e-7 of it
        tol = 4 * 2.0 ** -22 * (T + 16) * float(g.abs().max()) * float(way.abs().sum())
        assert abs(got - diff) <= tol + 1e-6 * abs(diff), (k, got, diff)


def test_rec_values_outside_the_segments_and_in_others_reach_nothing():
    T, cu, cud = cu_of("gaps")
    D = 64
    s = rec_inputs(T, 3, D, BF16, True, True, 3)
    args = lambda v: (dev(v["x"]), dev(v["r"]), dev(s["A"]))
    back = lambda v: gdr.rec_bwd(*args(v), dev(v["dy"]), dev(v["i"]), True, dev(v["h0"]), cud,
                                 dev(v["dht"]))
    clean = gdr.rec_fwd(*args(s), dev(s["i"]), True, dev(s["h0"]), cud, True)
    gclean = back(s)
    _, _, mask = ref.rec(s["x"].double(), s["r"].double(), s["A"].double(), None, True, None, cu)
    bad = {k: v.clone() for k, v in s.items()}
    for k, v in (("x", float("nan")), ("r", float("inf")), ("i", float("nan")), ("dy", float("inf"))):
        bad[k][~mask] = v
    y, ht, _ = gdr.rec_fwd(*args(bad), dev(bad["i"]), True, dev(bad["h0"]), cud, True)
    assert torch.equal(y.cpu()[mask], clean[0].cpu()[mask]) and torch.equal(ht, clean[1])
    for a, c in zip(back(bad), gclean):
        assert torch.equal(a, c)
    # the segment in the middle (20 .. 90) and its states: nothing of it in the others
    for v in (float("nan"), float("inf")):
        bad = {k: t.clone() for k, t in s.items()}
        for k in ("x", "r", "i", "dy"):
            bad[k][20:90] = v
        bad["h0"][1] = v
        bad["dht"][1] = v
        y, ht, _ = gdr.rec_fwd(*args(bad), dev(bad["i"]), True, dev(bad["h0"]), cud, True)
        other = mask.clone()
        other[20:90] = False
        assert torch.equal(y.cpu()[other], clean[0].cpu()[other])
        assert torch.equal(ht[[0, 2]], clean[1][[0, 2]])
        dx, dr, _, di, dh0 = back(bad)
        for a, c in ((dx, gclean[0]), (dr, gclean[1]), (di, gclean[3])):
            assert torch.equal(a.cpu()[other], c.cpu()[other])
        assert torch.equal(dh0[[0, 2]], gclean[4][[0, 2]])


@pytest.mark.parametrize("T,D", [(61, 64), (1200, 40), (6000, 34)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rec_values_of_others_change_no_bit(T, D, dtype):
    # gates whose e^-v overflow together, in one of the sequences that a warp's tokens belong to
    cut = [0, T // 3 + 2, T - T // 4 - 1, T]
    cud = torch.tensor(cut, dtype=torch.int32, device=DEV)
    s = rec_inputs(T, 3, D, dtype, True, True, T)
    far = {k: v.clone() for k, v in s.items()}
    far["r"][cut[1]:cut[2]] = far["i"][cut[1]:cut[2]] = -70.0
    out = []
    for v in (s, far):
        f = [dev(v[k]) for k in ("x", "r", "A", "i")]
        y, ht, _ = gdr.rec_fwd(*f, True, dev(s["h0"]), cud, True)
        dx, dr, _, di, dh0 = gdr.rec_bwd(f[0], f[1], f[2], dev(s["dy"]), f[3], True, dev(s["h0"]), cud,
                                         dev(s["dht"]))
        out.append([torch.cat((t[:cut[1]], t[cut[2]:])) for t in (y, dx, dr, di)] +
                   [t[[0, 2]] for t in (ht, dh0)])
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_rec_states_that_last():
    # A = 0 and closed gates: a = 1, the state stays as it is, and nothing is added to it
    T, D = 700, 66
    gen = torch.Generator().manual_seed(8)
    x, r, h0 = rn(gen, T, D), rn(gen, T, D), rn(gen, 1, D)
    A = torch.zeros(D)
    y, ht, _ = gdr.rec_fwd(dev(x), dev(r), dev(A), initial_state=dev(h0), output_final_state=True)
    assert torch.equal(ht.cpu(), h0) and torch.equal(y.cpu(), h0.expand(T, D))
    dy = rn(gen, T, D)
    dx, dr, dA, _, dh0 = gdr.rec_bwd(dev(x), dev(r), dev(A), dev(dy), initial_state=dev(h0))
    assert not dx.any() and not dr.any() and bool(torch.isfinite(dA).all())
    assert_close(dh0, dy.double().sum(0, keepdim=True), T, "dh0")
    r = torch.full((T, D), -200.0)
    y, ht, _ = gdr.rec_fwd(dev(x), dev(r), dev(A - 1), initial_state=dev(h0),
                           output_final_state=True)
    assert torch.equal(ht.cpu(), h0)


def test_rec_small_steps_keep_their_accuracy():
    # next to a = 1 the normaliser is sqrt(-2 log a), which 1 - a^2 in 32 bits would lose
    T, D = 40, 64
    gen = torch.Generator().manual_seed(9)
    x, r = rn(gen, T, D), rn(gen, T, D) - 12.0
    A = -0.5 * torch.rand(D, generator=gen)
    y, _, _ = gdr.rec_fwd(dev(x), dev(r), dev(A))
    yr, _, _ = ref.rec(x.double(), r.double(), A.double(), None, True, None, [0, T])
    # a few roundings of each of T addends: relative to the largest of the sums
    assert_close(y, yr, T, "y")


@pytest.mark.parametrize("B,D,dtype,gate,norm,odd", [(1, 64, BF16, True, True, False),
                                                     (5, 200, F32, False, True, False),
                                                     (6, 37, BF16, True, False, True),
                                                     (3, 2050, BF16, True, True, False)])
def test_rec_step(B, D, dtype, gate, norm, odd):
    gen = torch.Generator().manual_seed(B)
    slots = B + 3
    s = rec_inputs(B, 1, D, dtype, gate, False, B)
    st = rn(gen, slots, D)
    idx = torch.randperm(slots, generator=gen)[:B].to(torch.int32)
    if B > 2:
        idx[1], idx[2] = -1, slots + 4  # padded rows
    buf = dev(st)
    place = padded if odd else dev
    y = gdr.rec_step(place(s["x"]), place(s["r"]), dev(s["A"]), buf, place(s["i"]), norm, dev(idx))
    want, yr = st.double(), torch.zeros(B, D, dtype=torch.float64)
    d64 = {k: None if v is None else v.double() for k, v in s.items()}
    for row, k in enumerate(idx.tolist()):
        if 0 <= k < slots:
            one = lambda t: None if t is None else t[row:row + 1]
            yr[row:row + 1], want[k:k + 1], _ = ref.rec(one(d64["x"]), one(d64["r"]), d64["A"],
                                                        one(d64["i"]), norm, want[k:k + 1], [0, 1])
    assert_close(y, yr, 1, "y")
    assert_close(buf, want, 1, "state")


def test_rec_step_continues_a_prompt():
    T, D = 90, 192
    s = rec_inputs(T, 1, D, BF16, True, True, 21)
    full = gdr.rec_fwd(dev(s["x"]), dev(s["r"]), dev(s["A"]), dev(s["i"]), True, dev(s["h0"]),
                       output_final_state=True)
    cut = 77
    part = lambda t, a, b: dev(t[a:b])
    y, ht, _ = gdr.rec_fwd(part(s["x"], 0, cut), part(s["r"], 0, cut), dev(s["A"]),
                           part(s["i"], 0, cut), True, dev(s["h0"]), output_final_state=True)
    for t in range(cut, T):
        y = gdr.rec_step(part(s["x"], t, t + 1), part(s["r"], t, t + 1), dev(s["A"]), ht,
                         part(s["i"], t, t + 1))
    assert_close(ht, full[1], T, "state")
    assert_close(y, full[0][-1:].double(), T, "y")


# ------------------------------------------------------------------ norms

GATED = [  # tokens, heads, head size, type, activation, weight's type, odd strides
    (33, 4, 128, BF16, "silu", F32, False), (1, 1, 1, F32, "sigmoid", None, False),
    (7, 3, 64, F32, "silu", BF16, False), (129, 2, 256, BF16, "sigmoid", F32, False),
    (50, 5, 80, BF16, "silu", None, False), (17, 3, 37, F32, "silu", F32, True),
    (9, 2, 1024, BF16, "silu", F32, False), (5, 3, 520, F32, "sigmoid", F32, False),
    (6, 2, 300, BF16, "silu", F32, True), (11, 7, 8, BF16, "silu", F32, False),
    (700, 9, 16, F32, "silu", F32, False), (4, 2, 513, BF16, "silu", BF16, True),
    (0, 4, 64, BF16, "silu", F32, False), (6, 0, 64, BF16, "silu", F32, False),
]


@pytest.mark.parametrize("T,H,d,dtype,act,wt,odd", GATED)
def test_gated_norm(T, H, d, dtype, act, wt, odd):
    gen = torch.Generator().manual_seed(T + d)
    x, z, dy = (rn(gen, T, H, d, dtype=dtype) for _ in range(3))
    w = None if wt is None else (1 + rn(gen, d, std=0.2)).to(wt)
    place = padded if odd else dev
    eps = 1e-6
    y = gdr.gated_norm_fwd(place(x), place(z), dev(w), act, eps)
    lx, lz, lw = leaf(x), leaf(z), leaf(w)
    yr = ref.gated(lx, lz, lw, act, eps)
    assert_close(y, yr, d, "y")
    (yr * dy.double()).sum().backward()
    dx, dz, dw = gdr.gated_norm_bwd(place(x), place(z), place(dy), dev(w), act, eps)
    zero = torch.zeros
    assert_close(dx, lx.grad if lx.grad is not None else zero(T, H, d), d, "dx")
    assert_close(dz, lz.grad if lz.grad is not None else zero(T, H, d), d, "dz")
    if w is None:
        assert dw is None
    else:
        assert_close(dw, lw.grad, T * H + d, "dw")


RESID = [  # tokens, columns, type, residual's type (None: no residual), weight, post, gate, odd
    (33, 512, BF16, BF16, True, True, True, False), (1, 1, F32, F32, True, True, True, False),
    (5, 64, BF16, F32, True, False, True, False), (9, 100, F32, F32, True, True, False, True),
    (3, 4096, BF16, BF16, True, True, True, False), (2, 16384, BF16, BF16, True, True, True, False),
    (2, 16384, F32, F32, True, True, True, False), (3, 8200, BF16, F32, True, True, True, False),
    (4, 16383, BF16, BF16, True, True, True, False), (300, 128, BF16, BF16, True, False, False, False),
    (65, 200, F32, F32, True, True, True, False), (7, 1000, BF16, None, True, True, False, False),
    (6, 2048, BF16, BF16, False, "plain", False, False), (40, 24, BF16, BF16, True, True, True, False),
    (611, 1024, BF16, BF16, True, True, True, False), (5, 777, BF16, F32, True, True, True, True),
    (0, 64, BF16, BF16, True, True, True, False), (2000, 256, F32, F32, True, False, True, False),
    # rows on clusters of blocks, one row at a time and two, one step and several
    (1, 4104, F32, F32, True, True, True, False), (700, 4104, BF16, BF16, True, True, True, False),
    (640, 8192, BF16, BF16, True, False, True, False), (90, 8200, F32, F32, True, True, True, False),
    (777, 8200, BF16, F32, True, "plain", False, False), (5, 12296, BF16, BF16, True, True, True, False),
    (613, 16384, BF16, F32, True, True, True, False), (611, 12000, BF16, None, False, True, True, False),
    # rows off 16 bytes, of every number of threads
    (9, 7, BF16, BF16, True, True, True, False), (200, 33, F32, F32, True, True, True, False),
    (500, 250, BF16, F32, True, True, True, False), (333, 2049, BF16, BF16, True, True, True, False),
    (170, 5001, F32, F32, True, "plain", True, False), (160, 8191, BF16, BF16, True, True, True, False),
]


@pytest.mark.parametrize("T,C,dtype,rt,weight,post,gate,odd", RESID)
def test_residual_norm(T, C, dtype, rt, weight, post, gate, odd):
    gen = torch.Generator().manual_seed(T + C)
    x, dy = rn(gen, T, C, dtype=dtype), rn(gen, T, C, dtype=dtype)
    res = None if rt is None else rn(gen, T, C, dtype=rt, std=2.0)
    dh = rn(gen, T, C, dtype=rt or dtype)
    w = 1 + rn(gen, C, std=0.2) if weight else None
    wp = (1 + rn(gen, C, std=0.2)).to(BF16) if post is True else None
    g = rn(gen, C) if gate else None
    scale, eps, bare = 0.7, 1e-6, post == "plain"
    place = padded if odd else dev
    opts = (dev(w), dev(wp), dev(g), scale, eps, bare)
    y, h = gdr.residual_norm_fwd(place(x), place(res), *opts)
    leaves = [leaf(t) for t in (x, res, w, wp, g)]
    yr, hr = ref.residual(*leaves, scale, eps, bare)
    assert_close(y, yr, C, "y")
    assert_close(h, hr, 8, "h")
    ((yr * dy.double()).sum() + (hr * dh.double()).sum()).backward()
    got = gdr.residual_norm_bwd(place(x), place(res), place(dy), place(dh), *opts)
    steps = (C, C, T + C, T + C, T + C)
    for name, a, l, n in zip(("dx", "dresidual", "dweight", "dpost", "dgate"), got, leaves, steps):
        assert (a is None) == (l is None), name
        if a is not None:
            assert_close(a, l.grad if l.grad is not None else torch.zeros(a.shape), n, name)
    # no gradient from the residual stream: as zeros
    a = gdr.residual_norm_bwd(place(x), place(res), place(dy), None, *opts)
    b = gdr.residual_norm_bwd(place(x), place(res), place(dy), torch.zeros_like(place(dh)), *opts)
    for p, q in zip(a, b):
        assert (p is None and q is None) or torch.equal(p, q)


def test_norms_in_place():
    gen = torch.Generator().manual_seed(2)
    x, res = dev(rn(gen, 50, 1000, dtype=BF16)), dev(rn(gen, 50, 1000, dtype=BF16))
    y, h = gdr.residual_norm_fwd(x, res, scale=0.5)
    x2, res2 = x.clone(), res.clone()
    out = gdr.residual_norm_fwd(x2, res2, scale=0.5, out=x2, residual_out=res2)
    assert out[0].data_ptr() == x2.data_ptr() and out[1].data_ptr() == res2.data_ptr()
    assert torch.equal(x2, y) and torch.equal(res2, h)
    a, z = dev(rn(gen, 70, 3, 128, dtype=BF16)), dev(rn(gen, 70, 3, 128, dtype=BF16))
    y = gdr.gated_norm_fwd(a, z)
    for k in range(2):
        p = [a.clone(), z.clone()]
        assert torch.equal(gdr.gated_norm_fwd(*p, out=p[k]), y)


def test_norm_rows_stay_apart():
    # a row of infinities, of NaN, of zeros with eps = 0: in its own outputs alone
    gen = torch.Generator().manual_seed(4)
    x, z, dy = (dev(rn(gen, 9, 3, 40)) for _ in range(3))
    y, grads = gdr.gated_norm_fwd(x, z, eps=0.0), gdr.gated_norm_bwd(x, z, dy, eps=0.0)
    for v in (float("inf"), float("nan"), 0.0):
        b = x.clone()
        b[4, 1] = v
        keep = torch.ones(9, 3, dtype=torch.bool, device=DEV)
        keep[4, 1] = False
        assert torch.equal(gdr.gated_norm_fwd(b, z, eps=0.0)[keep], y[keep])
        for p, q in zip(gdr.gated_norm_bwd(b, z, dy, eps=0.0)[:2], grads):
            assert torch.equal(p[keep], q[keep])
    x, res, dy = (dev(rn(gen, 9, 100)) for _ in range(3))
    w = torch.ones(100, device=DEV)
    out, grads = gdr.residual_norm_fwd(x, res, w, w, eps=0.0), gdr.residual_norm_bwd(
        x, res, dy, None, w, w, eps=0.0)
    # all rows but one alike, though a block's last turn has fewer rows than it has groups
    assert all(bool(torch.isfinite(g).all()) for g in grads if g is not None)
    b = x.clone()
    b[4] = 0.0
    keep = torch.arange(9, device=DEV) != 4
    for p, q in zip(gdr.residual_norm_fwd(b, res, w, w, eps=0.0), out):
        assert torch.equal(p[keep], q[keep])
    for p, q in zip(gdr.residual_norm_bwd(b, res, dy, None, w, w, eps=0.0)[:2], grads):
        assert torch.equal(p[keep], q[keep])


# ------------------------------------------------------------------ attention over a paged cache

ATTN = [  # lengths, query heads, key heads, d, page, window, type
    ([1], 4, 2, 64, 16, 0, BF16), ([0], 4, 2, 64, 16, 0, BF16), ([65], 8, 8, 128, 16, 0, BF16),
    ([300, 0, 1, 17, 64, 1000], 8, 2, 128, 16, 0, BF16), ([513, 2], 16, 1, 64, 5, 0, BF16),
    ([129, 700], 32, 1, 128, 64, 0, BF16), ([40, 257], 40, 2, 64, 1, 0, BF16),
    ([333, 20], 6, 2, 256, 32, 0, BF16), ([100, 333], 4, 4, 96, 16, 0, BF16),
    ([90, 10], 4, 2, 8, 16, 0, BF16), ([90, 400, 7], 8, 4, 128, 16, 33, BF16),
    ([64, 128, 65], 4, 2, 128, 128, 1, BF16), ([120, 31], 6, 3, 200, 7, 100, BF16),
    ([50, 0, 129], 6, 3, 20, 16, 0, BF16), ([50, 129], 4, 2, 64, 16, 0, F32),
    ([77, 5, 0], 6, 1, 256, 3, 20, F32), ([9], 2, 1, 1, 4, 0, F32), ([], 4, 2, 64, 16, 0, BF16),
    ([3000, 40, 2500], 8, 2, 64, 16, 0, BF16),
]


def attn_inputs(lens, Hq, Hk, d, ps, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed + d + sum(lens))
    need = [-(-n // ps) for n in lens]
    pages = sum(need) + 4
    order = torch.randperm(pages, generator=gen).to(torch.int32)
    width = max(need + [1]) + 1
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    kc, vc = rn(gen, pages, ps, Hk, d, dtype=dtype), rn(gen, pages, ps, Hk, d, dtype=dtype)
    # what lies behind the requests' keys and on other pages must reach nothing
    used = torch.zeros(pages, ps, dtype=torch.bool)
    for i, n in enumerate(lens):
        for j in range(n):
            used[table[i, j // ps], j % ps] = True
    kc[~used], vc[~used] = float("nan"), float("inf")
    q = rn(gen, len(lens), Hq, d, dtype=dtype, std=1.5)
    return q, kc, vc, table, torch.tensor(lens, dtype=torch.int32)


@pytest.mark.parametrize("lens,Hq,Hk,d,ps,window,dtype", ATTN)
def test_attn_step(lens, Hq, Hk, d, ps, window, dtype):
    q, kc, vc, table, n = attn_inputs(lens, Hq, Hk, d, ps, dtype)
    o = gdr.attn_step(dev(q), dev(kc), dev(vc), dev(table), dev(n), window=window)
    want, tol = ref.attention(q, kc, vc, table, lens, d ** -0.5, window)
    ref.assert_attention(o, want, tol)


# more pairs of request and head than blocks: pairs that end where a block's range ends or go on over several
# ranges, rows without keys among them
@pytest.mark.parametrize("lens,Hq,Hk,d", [
    ([7 * i % 13 for i in range(400)], 8, 4, 64), ([64] * 700, 2, 1, 128), ([64] * 703, 2, 1, 128),
    ([0, 9000] + [50 * i % 201 for i in range(350)] + [0], 40, 2, 96), ([0] * 900, 3, 1, 64),
    ([1] * 640 + [7000], 2, 1, 200), ([20 * i % 333 for i in range(320)], 9, 9, 40)])
def test_attn_step_many_requests(lens, Hq, Hk, d):
    q, kc, vc, table, n = attn_inputs(lens, Hq, Hk, d, 16, BF16)
    o = gdr.attn_step(dev(q), dev(kc), dev(vc), dev(table), dev(n))
    want, tol = ref.attention(q, kc, vc, table, lens, d ** -0.5, 0)
    ref.assert_attention(o, want, tol)


def test_attn_step_masked_places():
    # infinities and NaN left of the window; pages that are not there; lengths beyond the table
    lens, ps, window = [200, 90, 150, 40], 16, 50
    q, kc, vc, table, n = attn_inputs(lens, 8, 2, 128, ps, BF16)
    for b, m in enumerate(lens):
        for j in range(max(0, m - window)):
            kc[table[b, j // ps], j % ps] = float("inf")
            vc[table[b, j // ps], j % ps] = float("nan")
    table[0, 11], table[1, 3] = -1, kc.shape[0]
    table[3] = -5  # no page at all: an empty row
    o = gdr.attn_step(dev(q), dev(kc), dev(vc), dev(table), dev(n), window=window)
    want, tol = ref.attention(q, kc, vc, table, lens, 128 ** -0.5, window)
    ref.assert_attention(o, want, tol)
    assert not o[3].any()
    big = torch.tensor([200, 2 ** 31 - 1, -7, 0], dtype=torch.int32)
    o = gdr.attn_step(dev(q), dev(kc), dev(vc), dev(table), dev(big), window=window)
    want, tol = ref.attention(q, kc, vc, table, big.tolist(), 128 ** -0.5, window)
    ref.assert_attention(o, want, tol)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attn_step_strides(dtype):
    # queries of a fused projection, a cache with heads before places and both in one buffer
    lens, Hq, Hk, d, ps = [100, 33, 257], 8, 2, 64, 16
    q, kc, vc, table, n = attn_inputs(lens, Hq, Hk, d, ps, dtype)
    want, tol = ref.attention(q, kc, vc, table, lens, 0.3, 0)
    both = torch.empty(kc.shape[0], 2, Hk, ps, d, dtype=dtype, device=DEV)
    k, v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    k.copy_(kc)
    v.copy_(vc)
    wide = torch.randn(len(lens), Hq + 3, d, device=DEV).to(dtype)
    wide[:, 1:1 + Hq] = dev(q)
    tab = torch.zeros(len(lens), table.shape[1] + 3, dtype=torch.int32, device=DEV)
    tab[:, :table.shape[1]] = dev(table)
    out = torch.zeros(len(lens), 2 * Hq, d, dtype=dtype, device=DEV)
    o = gdr.attn_step(wide[:, 1:1 + Hq], k, v, tab[:, :table.shape[1]], dev(n), 0.3,
                      out=out[:, Hq:])
    ref.assert_attention(o, want, tol)
    assert not out[:, :Hq].any()
    # rows that start off 16 bytes, and off the type's pairs
    for shift in (2, 1):
        odd = torch.empty(*kc.shape[:3], d + 8, dtype=dtype, device=DEV)
        odd2 = torch.empty_like(odd)
        odd[..., shift:shift + d].copy_(kc)
        odd2[..., shift:shift + d].copy_(vc)
        o = gdr.attn_step(padded(q), odd[..., shift:shift + d], odd2[..., shift:shift + d],
                          dev(table), dev(n), 0.3)
        ref.assert_attention(o, want, tol)


def test_attn_step_one_head_takes_all():
    # scores far apart and equal ones; a negative and a zero scale
    q, kc, vc, table, n = attn_inputs([500], 4, 2, 64, 16, BF16)
    for scale in (40.0, -1.0, 0.0):
        o = gdr.attn_step(dev(q), dev(kc), dev(vc), dev(table), dev(n), scale)
        want, tol = ref.attention(q, kc, vc, table, [500], scale, 0)
        ref.assert_attention(o, want, tol)


# ------------------------------------------------------------------ cache

PLAN = [  # lengths, new tokens, page, free pages, taken, max_tokens, width
    ([0], [1], 16, 3, 0, 1, 4), ([15, 16, 17, 0], [1, 1, 1, 1], 16, 9, 2, 4, 4),
    ([3, 0, 40], [100, 33, 0], 16, 40, 5, 133, 16), ([3, 0, 40], [100, 33, 9], 16, 8, 5, 142, 16),
    ([3, 0, 40], [100, 33, 9], 16, 40, 0, 60, 16), ([5, -3, 9, 100], [-1, 4, 3, 7], 4, 9, -2, 30, 4),
    ([0, 0], [5, 5], 1, 30, 25, 10, 5), ([7] * 300, [1] * 300, 8, 200, 0, 300, 3),
    ([0] * 2100, [3] * 2100, 2, 5000, 1, 6300, 2), ([0, 5], [9000, 3000], 16, 800, 0, 12000, 600),
    ([], [], 16, 4, 1, 0, 2), ([4, 4], [0, 0], 4, 0, 0, 8, 3), ([2], [3], 4, 5, 9, 3, 3),
    ([1] * 40, [300] * 40, 7, 2000, 3, 10000, 44),
]


@pytest.mark.parametrize("lens,new,page,free,taken,most,width", PLAN)
def test_cache_plan(lens, new, page, free, taken, most, width):
    gen = torch.Generator().manual_seed(len(lens) + page)
    pages = (100 + torch.randperm(free, generator=gen)).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        have = min(width, -(-max(n, 0) // page))
        table[b, :have] = torch.arange(have) + 10000 + b * width
    if len(lens) > 2:
        table[2, 0] = -1  # a page that is not there
    wide = torch.full((len(lens), width + 2), -9, dtype=torch.int32, device=DEV)
    wide[:, :width] = dev(table)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    n0, nw, tk = i32(lens), i32(new), i32([taken])
    for _ in range(2):  # the same values read again give the same
        slots, pos, cu, after, tk2 = gdr.cache_plan(n0, nw, wide[:, :width], dev(pages), tk, page,
                                                    most)
        want = ref.plan(lens, new, table.tolist(), pages.tolist(), taken, page, most)
        got = (slots.tolist(), pos.tolist(), cu.tolist(), after.tolist(), int(tk2),
               wide[:, :width].tolist())
        for name, a, b in zip(("slots", "positions", "cu", "lengths", "taken", "table"), got, want):
            assert a == b, name
    assert bool((wide[:, width:] == -9).all())
    # in place
    again = gdr.cache_plan(n0, nw, wide[:, :width], dev(pages), tk, page, most, n0, tk)
    assert again[3].data_ptr() == n0.data_ptr() and again[0].tolist() == want[0]
    assert n0.tolist() == want[3] and int(tk) == want[4]


@pytest.mark.parametrize("Hk,d,dtype,order", [(2, 64, BF16, "plain"), (3, 20, F32, "plain"),
                                              (1, 7, BF16, "plain"), (4, 128, BF16, "heads first"),
                                              (2, 33, F32, "heads first")])
def test_cache_write(Hk, d, dtype, order):
    gen = torch.Generator().manual_seed(d)
    T, pages, ps = 300, 40, 16
    k, v = rn(gen, T, Hk, d, dtype=dtype), rn(gen, T, Hk, d, dtype=dtype)
    slots = torch.randperm(pages * ps, generator=gen)[:T].to(torch.int32)
    slots[5], slots[6] = -1, pages * ps
    caches = [rn(gen, pages, ps, Hk, d, dtype=dtype) for _ in range(2)]
    there = []
    for c in caches:
        if order == "plain":
            there.append(dev(c))
        else:
            t = torch.empty(pages, Hk, ps, d, dtype=dtype, device=DEV).transpose(1, 2)
            t.copy_(c)
            there.append(t)
    gdr.cache_write(padded(k) if d == 33 else dev(k), dev(v), *there, dev(slots))
    for rows, c, t in zip((k, v), caches, there):
        flat = c.view(-1, Hk, d)
        for i, s in enumerate(slots.tolist()):
            if 0 <= s < pages * ps:
                flat[s] = rows[i]
        assert torch.equal(t.cpu(), c)


# ------------------------------------------------------------------ autograd

def test_autograd():
    gen = torch.Generator().manual_seed(12)
    T, cu, cud = cu_of("ghosts")
    D = 128
    s = rec_inputs(T, len(cu) - 1, D, F32, True, True, 3)
    on = lambda t: dev(t).requires_grad_(True)
    x, r, A, i, h0 = (on(s[k]) for k in ("x", "r", "A", "i", "h0"))
    y, ht = gdr.gated_recurrence(x, r, A, i, initial_state=h0, cu_seqlens=cud,
                                 output_final_state=True)
    w = on(1 + rn(gen, 32, std=0.1))
    z = on(rn(gen, T, 4, 32))
    n = gdr.gated_norm(y.view(T, 4, 32), z, w, "sigmoid")
    res, wr, wp, g = (on(rn(gen, *sh)) for sh in ((T, D), (D,), (D,), (D,)))
    out, h = gdr.residual_norm(n.reshape(T, D), res, wr, wp, g, 0.3)
    d1, d2, d3 = rn(gen, T, D), rn(gen, T, D), rn(gen, len(cu) - 1, D)
    ((out * dev(d1)).sum() + (h * dev(d2)).sum() + (ht * dev(d3)).sum()).backward()
    names = "x r A i h0 w z res wr wp g".split()
    own = dict(zip(names, (x, r, A, i, h0, w, z, res, wr, wp, g)))
    l = {k: leaf(v) for k, v in own.items()}
    yr, hr, mask = ref.rec(l["x"], l["r"], l["A"], l["i"], True, l["h0"], cu)
    nr = ref.gated(yr.view(T, 4, 32), l["z"], l["w"], "sigmoid", 1e-6)
    outr, h2 = ref.residual(nr.reshape(T, D), l["res"], l["wr"], l["wp"], l["g"], 0.3, 1e-6, False)
    ((outr * d1.double()).sum() + (h2 * d2.double()).sum() + (hr * d3.double()).sum()).backward()
    for k in names:
        assert_close(own[k].grad, l[k].grad, 4 * T, k)


def test_second_derivatives_are_refused():
    gen = torch.Generator().manual_seed(1)
    x, r = (dev(rn(gen, 9, 16)).requires_grad_(True) for _ in range(2))
    A = torch.full((16,), -0.5, device=DEV)
    y, _ = gdr.gated_recurrence(x, r, A)
    g, = torch.autograd.grad(y.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives"):
        g.sum().backward()
    z = dev(rn(gen, 9, 1, 16)).requires_grad_(True)
    g, = torch.autograd.grad(gdr.gated_norm(x.view(9, 1, 16), z).sum(), z, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives"):
        g.sum().backward()
    y, h = gdr.residual_norm(x, r)
    g, = torch.autograd.grad((y + h).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives"):
        g.sum().backward()
