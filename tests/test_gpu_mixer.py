"""The mixer's operators on a GB300 against plain 64-bit implementations: convolution, state
space, q/k norm with rotation and the single-token steps, forward and backward, over types,
strides, odd sizes, empty and malformed segments, and values that must reach no output."""
import pytest
import torch

import chunked_gated_delta_gdr_gb300 as gdr
import mixer_testlib as ref
from mixer_testlib import BF16, F32, assert_close, leaf

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
    wide = torch.zeros(*t.shape[:-1], t.shape[-1] + extra, dtype=t.dtype, device=DEV)
    view = wide[..., 1:1 + t.shape[-1]]
    view.copy_(t)
    return view


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
}


def cu_of(name):
    T, cu = CU[name]
    return T, cu, torch.tensor(cu, dtype=torch.int32, device=DEV)


def longest(cu, T):
    b = ref.bounds(cu, T)
    return max([e - s for s, e in zip(b[:-1], b[1:])] + [0])


# ------------------------------------------------------------------ convolution

CONV = [
    ("one", 64, 4, BF16, True, True, True, False),
    ("single", 64, 4, BF16, True, False, True, False),
    ("short", 40, 4, F32, True, True, True, False),
    ("short", 1032, 3, BF16, False, True, True, False),
    ("ghosts", 136, 4, BF16, True, True, True, False),
    ("ghosts", 136, 2, F32, True, False, False, False),
    ("gaps", 63, 4, BF16, True, True, True, False),
    ("gaps", 64, 4, F32, True, True, True, True),
    ("long", 200, 4, BF16, True, True, False, False),
    ("long", 72, 3, F32, True, False, True, True),
    ("malformed", 33, 4, BF16, True, True, True, True),
    ("none", 64, 4, BF16, True, True, True, False),
    ("all empty", 64, 4, BF16, True, True, True, False),
    ("many", 24, 4, BF16, True, True, True, False),
]


@pytest.mark.parametrize("name,C,W,dtype,act,bias,state,odd", CONV)
def test_conv_forward_and_backward(name, C, W, dtype, act, bias, state, odd):
    T, cu, cud = cu_of(name)
    gen = torch.Generator().manual_seed(T * 31 + C)
    n = len(cu) - 1
    x, w = rn(gen, T, C, dtype=dtype), rn(gen, C, W, std=W ** -0.5)
    b = rn(gen, C, std=0.2) if bias else None
    h0 = rn(gen, n, W - 1, C, dtype=dtype) if state else None
    dy = rn(gen, T, C, dtype=dtype)
    dht = rn(gen, n, W - 1, C, dtype=dtype) if state else None
    place = padded if odd else dev
    act_name = "silu" if act else None
    y0 = torch.full((T, C), 7.0, dtype=dtype, device=DEV)
    y, ht = gdr.conv_fwd(place(x), dev(w), dev(b), dev(h0), cud, act_name, True, out=y0)
    lx, lw, lb, lh = leaf(x), leaf(w), leaf(b), leaf(h0)
    yr, hr, mask = ref.conv(lx, lw, lb, lh, cu, act)
    assert_close(y.cpu()[mask], yr[mask], 4, "y")
    assert torch.all(y.cpu()[~mask] == 7.0), "tokens outside the segments were written"
    assert_close(ht, hr, 0, "final state")
    dx, dw, db, dh0 = gdr.conv_bwd(place(x), dev(w), place(dy), dev(b), dev(h0), cud, act_name,
                                   dev(dht))
    # the gradient of the initial state exists without one, too
    base = lh if lh is not None else torch.zeros(n, W - 1, C, dtype=torch.float64,
                                                 requires_grad=True)
    yr, hr, _ = ref.conv(lx, lw, lb, base, cu, act)
    loss = (yr * dy.double()).sum() + base.sum() * 0 + lx.sum() * 0 + lw.sum() * 0
    if lb is not None:
        loss = loss + lb.sum() * 0
    if dht is not None:
        loss = loss + (hr * dht.double()).sum()
    loss.backward()
    assert_close(dx, lx.grad, 4, "dx")
    assert_close(dw, lw.grad, T, "dw")
    if b is not None:
        assert_close(db, lb.grad, T, "db")
    assert_close(dh0, base.grad, 4, "dh0")


def test_conv_values_outside_the_segments_reach_nothing():
    T, cu, cud = cu_of("gaps")
    gen = torch.Generator().manual_seed(3)
    C, W = 64, 4
    x, dy, w = rn(gen, T, C, dtype=BF16), rn(gen, T, C, dtype=BF16), rn(gen, C, W)
    clean = gdr.conv_fwd(dev(x), dev(w), cu_seqlens=cud, output_final_state=True)
    gclean = gdr.conv_bwd(dev(x), dev(w), dev(dy), cu_seqlens=cud)
    _, _, mask = ref.conv(x.double(), w.double(), None, None, cu, True)
    bad, dbad = x.clone(), dy.clone()
    bad[~mask] = float("nan")
    dbad[~mask] = float("inf")
    y, ht = gdr.conv_fwd(dev(bad), dev(w), cu_seqlens=cud, output_final_state=True)
    assert torch.equal(y.cpu()[mask], clean[0].cpu()[mask]) and torch.equal(ht, clean[1])
    for a, c in zip(gdr.conv_bwd(dev(bad), dev(w), dev(dbad), cu_seqlens=cud), gclean):
        assert (a is None and c is None) or torch.equal(a, c)


@pytest.mark.parametrize("B,C,W,dtype,odd", [(1, 64, 4, BF16, False), (5, 200, 3, F32, False),
                                             (6, 37, 2, BF16, True), (3, 2056, 4, BF16, False)])
def test_conv_step(B, C, W, dtype, odd):
    gen = torch.Generator().manual_seed(B)
    slots = B + 3
    x, w, b = rn(gen, B, C, dtype=dtype), rn(gen, C, W), rn(gen, C)
    st = rn(gen, slots, W - 1, C, dtype=dtype)
    idx = torch.randperm(slots, generator=gen)[:B].to(torch.int32)
    if B > 2:
        idx[1], idx[2] = -1, slots + 4  # padded rows
    s = dev(st)
    y = gdr.conv_step((padded if odd else dev)(x), dev(w), s, dev(b), "silu", dev(idx))
    want, yr = st.clone(), torch.zeros(B, C, dtype=torch.float64)
    for r, i in enumerate(idx.tolist()):
        if 0 <= i < slots:
            rows = torch.cat([st[i], x[r:r + 1]])
            yr[r] = ref.silu((rows.double() * w.double().t()).sum(0) + b.double())
            want[i] = rows[1:]
    assert_close(y, yr, 4, "y")
    assert torch.equal(s.cpu(), want)


# ------------------------------------------------------------------ state space

SSM = [  # bounds, channels, states, groups, type, gate, skip, bias, softplus, state, odd strides
    ("one", 64, 16, 1, BF16, True, True, True, True, True, False),
    ("single", 64, 16, 1, BF16, True, True, True, True, True, False),
    ("short", 72, 16, 1, F32, True, True, True, True, True, False),
    ("ghosts", 128, 16, 2, BF16, True, True, True, True, True, False),
    ("ghosts", 96, 12, 1, F32, False, True, False, True, False, False),
    ("gaps", 70, 16, 2, F32, True, False, True, True, True, True),
    ("gaps", 33, 5, 1, BF16, True, True, True, False, True, True),
    ("long", 64, 16, 1, F32, True, True, True, True, True, False),
    ("long", 40, 8, 1, BF16, False, True, True, True, False, False),
    ("ghosts", 48, 32, 1, F32, True, True, True, True, True, False),
    ("ghosts", 36, 64, 2, F32, True, True, True, True, True, False),
    ("gaps", 24, 33, 1, BF16, True, True, True, True, True, False),
    ("malformed", 64, 1, 1, F32, True, True, True, True, True, False),
    ("none", 64, 16, 1, BF16, True, True, True, True, True, False),
    ("all empty", 64, 16, 1, BF16, True, True, True, True, True, False),
    ("many", 64, 16, 1, F32, True, True, True, True, True, False),
]


def ssm_inputs(T, n, D, N, G, dtype, z, skip, bias, softplus, state, seed):
    gen = torch.Generator().manual_seed(seed)
    i = dict(x=rn(gen, T, D, dtype=dtype),
             dt=(rn(gen, T, D, std=0.5) - (3.0 if softplus else 0.0)),
             A=-torch.exp(rn(gen, D, N, std=0.5)), B=rn(gen, T, G, N, dtype=dtype),
             C=rn(gen, T, G, N, dtype=dtype), D=rn(gen, D) if skip else None,
             z=rn(gen, T, D, dtype=dtype) if z else None,
             dt_bias=rn(gen, D, std=0.3) if bias else None,
             h0=rn(gen, n, D, N) if state else None, dy=rn(gen, T, D, dtype=dtype),
             dht=rn(gen, n, D, N) if state else None)
    if not softplus:
        i["dt"] = i["dt"].abs() * 0.2
        if i["dt_bias"] is not None:
            i["dt_bias"] = i["dt_bias"].abs() * 0.1
    i["dt"] = i["dt"].to(dtype)
    return i


@pytest.mark.parametrize("name,D,N,G,dtype,z,skip,bias,softplus,state,odd", SSM)
def test_ssm_forward_and_backward(name, D, N, G, dtype, z, skip, bias, softplus, state, odd):
    T, cu, cud = cu_of(name)
    n = len(cu) - 1
    i = ssm_inputs(T, n, D, N, G, dtype, z, skip, bias, softplus, state, T + D)
    place = (lambda t: None if t is None else padded(t)) if odd else dev
    y0 = torch.full((T, D), 7.0, dtype=dtype, device=DEV)
    args = [place(i["x"]), place(i["dt"]), dev(i["A"]), place(i["B"]), place(i["C"])]
    opts = dict(D=dev(i["D"]), z=place(i["z"]), dt_bias=dev(i["dt_bias"]), dt_softplus=softplus,
                initial_state=dev(i["h0"]), cu_seqlens=cud)
    y, ht = gdr.ssm_fwd(*args, **opts, output_final_state=True, out=y0)
    lv = {k: leaf(i[k]) for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")}
    lh = leaf(i["h0"]) if state else torch.zeros(n, D, N, dtype=torch.float64,
                                                 requires_grad=True)
    yr, hr, mask = ref.ssm(lv["x"], lv["dt"], lv["A"], lv["B"], lv["C"], lv["D"], lv["z"],
                           lv["dt_bias"], softplus, lh, cu)
    steps = longest(cu, T)
    assert_close(y.cpu()[mask], yr[mask], steps, "y")
    assert torch.all(y.cpu()[~mask] == 7.0), "tokens outside the segments were written"
    assert_close(ht, hr, steps, "final state")
    got = gdr.ssm_bwd(*args, place(i["dy"]), **opts, dfinal_state=dev(i["dht"]))
    loss = (yr * i["dy"].double()).sum() + lh.sum() * 0
    for v in lv.values():
        if v is not None:
            loss = loss + v.sum() * 0
    if state:
        loss = loss + (hr * i["dht"].double()).sum()
    loss.backward()
    names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")
    for k, a in zip(names, got[:8]):
        if lv[k] is None:
            assert a is None
        else:
            sums = T if k in ("A", "D", "dt_bias") else 0
            assert_close(a, lv[k].grad, steps + sums + D // 8, "d" + k)
    assert_close(got[8], lh.grad, steps, "dh0")


def test_ssm_values_outside_the_segments_reach_nothing():
    T, cu, cud = cu_of("gaps")
    i = ssm_inputs(T, 3, 64, 16, 1, BF16, True, True, True, True, True, 5)
    _, _, mask = ref.conv(i["x"].double(), torch.zeros(64, 2).double(), None, None, cu, False)

    def both(d):
        a = [dev(d[k]) for k in ("x", "dt", "A", "B", "C")]
        o = dict(D=dev(d["D"]), z=dev(d["z"]), dt_bias=dev(d["dt_bias"]),
                 initial_state=dev(d["h0"]), cu_seqlens=cud)
        y, ht = gdr.ssm_fwd(*a, **o, output_final_state=True)
        return (y.cpu()[mask], ht, *gdr.ssm_bwd(*a, dev(d["dy"]), **o,
                                                dfinal_state=dev(d["dht"])))

    clean = both(i)
    bad = dict(i)
    for k, v in (("x", "nan"), ("dt", "inf"), ("B", "nan"), ("C", "inf"), ("z", "nan"),
                 ("dy", "nan")):
        bad[k] = i[k].clone()
        bad[k][~mask] = float(v)
    for a, c in zip(both(bad), clean):
        assert torch.equal(a, c)


def test_ssm_long_prompt_cut_into_ranges_agrees_with_one_range():
    """A prompt that is long enough for the scan to be cut over many blocks, with D small so that
    a 64-bit run stays quick, against the token recurrence."""
    T, D, N = 6000, 16, 16
    i = ssm_inputs(T, 2, D, N, 1, F32, True, True, True, True, True, 11)
    cu = [0, 5300, 6000]
    y, ht = gdr.ssm_fwd(*[dev(i[k]) for k in ("x", "dt", "A", "B", "C")], D=dev(i["D"]),
                        z=dev(i["z"]), dt_bias=dev(i["dt_bias"]), initial_state=dev(i["h0"]),
                        cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV),
                        output_final_state=True)
    d = {k: None if v is None else v.double() for k, v in i.items()}
    yr, hr, _ = ref.ssm(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["z"], d["dt_bias"],
                        True, d["h0"], cu)
    # the states remember about 1 / (dt |A|), here some 100 tokens, not the whole prompt
    assert_close(y, yr, 400, "y")
    assert_close(ht, hr, 400, "final state")


@pytest.mark.parametrize("N,G,dtype,z,state", [(16, 1, BF16, True, True), (6, 2, F32, False, True),
                                               (12, 1, F32, True, False)])
def test_ssm_with_much_work(N, G, dtype, z, state):
    """Enough tokens and channels for the layout of one thread a channel, with segments that start,
    end and are missing inside its ranges.  The steps remembered are about 1 / (dt |A|): 400."""
    T, D = 5003, 4096 if G == 1 else 3872
    cu = [3, 3, 700, 701, 2900, 2900, 2917, 4980]
    i = ssm_inputs(T, 7, D, N, G, dtype, z, True, True, True, state, 21)
    y0 = torch.full((T, D), 7.0, dtype=dtype, device=DEV)
    y, ht = gdr.ssm_fwd(*[dev(i[k]) for k in ("x", "dt", "A", "B", "C")], D=dev(i["D"]),
                        z=dev(i["z"]), dt_bias=dev(i["dt_bias"]), initial_state=dev(i["h0"]),
                        cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV),
                        output_final_state=True, out=y0)
    d = {k: None if v is None else v.double() for k, v in i.items()}
    yr, hr, mask = ref.ssm(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["z"], d["dt_bias"],
                           True, d["h0"], cu)
    assert_close(y.cpu()[mask], yr[mask], 400, "y")
    assert torch.all(y.cpu()[~mask] == 7.0)
    assert_close(ht, hr, 400, "final state")


@pytest.mark.parametrize("B,D,N,G,dtype,odd", [(1, 64, 16, 1, BF16, False),
                                               (5, 100, 16, 2, F32, False),
                                               (4, 48, 5, 1, BF16, True),
                                               (3, 40, 64, 1, BF16, False),
                                               (3, 40, 8, 1, F32, False),
                                               (3, 24, 30, 1, F32, True),
                                               (3, 128, 16, 2, BF16, False),
                                               (4, 70, 12, 1, F32, False),
                                               (3, 33, 32, 1, BF16, False),
                                               (2, 9, 4, 1, BF16, False),
                                               (3, 96, 64, 3, F32, False),
                                               (3, 1000, 16, 1, BF16, False)])
def test_ssm_step(B, D, N, G, dtype, odd):
    i = ssm_inputs(B, 1, D, N, G, dtype, True, True, True, True, False, B + D)
    gen = torch.Generator().manual_seed(9)
    slots = B + 4
    st = rn(gen, slots, D, N)
    idx = torch.randperm(slots, generator=gen)[:B].to(torch.int32)
    if B > 2:
        idx[0], idx[2] = slots, -7
    place = padded if odd else dev
    s = dev(st)
    y = gdr.ssm_step(place(i["x"]), place(i["dt"]), dev(i["A"]), place(i["B"]), place(i["C"]), s,
                     dev(i["D"]), place(i["z"]), dev(i["dt_bias"]), True, dev(idx))
    want, yr = st.double(), torch.zeros(B, D, dtype=torch.float64)
    for r, j in enumerate(idx.tolist()):
        if 0 <= j < slots:
            one = {k: i[k][r:r + 1].double() for k in ("x", "dt", "B", "C", "z")}
            yy, hh, _ = ref.ssm(one["x"], one["dt"], i["A"].double(), one["B"], one["C"],
                                i["D"].double(), one["z"], i["dt_bias"].double(), True,
                                st[j:j + 1].double(), [0, 1])
            yr[r], want[j] = yy[0], hh[0]
    assert_close(y, yr, 4, "y")
    assert_close(s, want, 4, "state")


# ------------------------------------------------------------------ q/k norm with rotation

QK = [  # T, Hq, Hk, d, rot, interleaved, norm, weights, type, odd strides, eps
    (1, 2, 2, 128, 128, False, "rms", True, BF16, False, 1e-6),
    (33, 16, 4, 128, 64, False, "rms", True, BF16, False, 1e-6),
    (17, 4, 1, 64, 64, True, "rms", True, F32, False, 1e-5),
    (40, 3, 3, 256, 128, False, "l2", False, BF16, False, 1e-6),
    (21, 6, 2, 128, 0, False, "l2", False, F32, False, 0.0),
    (19, 2, 1, 80, 20, False, "rms", True, BF16, False, 1e-6),
    (19, 2, 1, 100, 100, True, "rms", True, F32, True, 1e-6),
    (9, 5, 5, 64, 24, False, "rms", True, BF16, False, 1e-6),
    (13, 2, 2, 128, 128, False, "rms", True, BF16, True, 1e-6),
    (700, 1, 1, 64, 64, False, "rms", True, BF16, False, 1e-6),
    (5, 1, 0, 1, 0, False, "rms", True, F32, False, 1e-6),
    (0, 4, 4, 128, 128, False, "rms", True, BF16, False, 1e-6),
    (33, 20, 5, 40, 40, False, "rms", True, BF16, False, 1e-6),
    (18, 6, 3, 96, 96, False, "l2", True, F32, False, 1e-6),
    (1300, 3, 2, 152, 88, False, "rms", True, BF16, False, 1e-6),
    (27, 5, 1, 248, 248, True, "rms", True, BF16, False, 1e-6),
    (35, 1, 1, 8, 8, False, "rms", True, F32, False, 1e-5),
    (2500, 7, 2, 24, 8, False, "l2", False, BF16, False, 1e-6),
    (23, 12, 3, 232, 116, True, "l2", True, BF16, False, 1e-6),
    (19, 2, 1, 72, 36, True, "rms", True, F32, False, 1e-6),
    (14, 2, 1, 64, 30, True, "rms", True, BF16, False, 1e-6),
    (2100, 3, 1, 232, 116, False, "rms", True, BF16, False, 1e-6),
]


@pytest.mark.parametrize("T,Hq,Hk,d,rot,inter,norm,weights,dtype,odd,eps", QK)
def test_qk_forward_and_backward(T, Hq, Hk, d, rot, inter, norm, weights, dtype, odd, eps):
    gen = torch.Generator().manual_seed(T * 7 + d)
    q, k = rn(gen, T, Hq, d, dtype=dtype), rn(gen, T, Hk, d, dtype=dtype)
    dq, dk = rn(gen, T, Hq, d, dtype=dtype), rn(gen, T, Hk, d, dtype=dtype)
    qw, kw = (rn(gen, d), rn(gen, d, dtype=BF16)) if weights else (None, None)
    cos = sin = pos = None
    if rot:
        ang = torch.rand(50, rot // 2, generator=gen) * 6
        cos, sin = ang.cos(), ang.sin()
        pos = torch.randint(-2, 53, (T,), generator=gen).to(torch.int32)  # clamped to the table
    place = padded if odd else dev
    opts = dict(q_weight=dev(qw), k_weight=dev(kw), norm=norm, eps=eps, cos=dev(cos),
                sin=dev(sin), positions=dev(pos), interleaved=inter)
    out = gdr.qk_fwd(place(q), place(k), **opts)
    grads = gdr.qk_bwd(place(q), place(k), place(dq), place(dk), **opts)
    r64 = lambda t: None if t is None else t.double()
    for j, (x, w, g) in enumerate(((q, qw, dq), (k, kw, dk))):
        lx, lw = leaf(x), leaf(w)
        y = ref.qk_row(lx, lw, norm, eps, r64(cos), r64(sin), pos, inter)
        assert_close(out[j], y, 16, "out")
        ((y * g.double()).sum() + lx.sum() * 0 + (lw.sum() * 0 if lw is not None else 0)).backward()
        assert_close(grads[j], lx.grad, 32, "dx")
        if lw is None:
            assert grads[2 + j] is None
        else:
            assert_close(grads[2 + j], lw.grad, T * max(Hq, Hk), "dw")


def test_qk_rows_of_zeros():
    q = torch.zeros(3, 2, 128, dtype=BF16, device=DEV)
    out = gdr.qk_fwd(q, q, norm="rms", eps=1e-6)
    assert torch.equal(out[0], q) and torch.equal(out[1], q)
    one = torch.ones_like(q)
    dq, _, _, _ = gdr.qk_bwd(q, q, one, one, norm="rms", eps=1e-6)
    assert torch.all(dq.float() == torch.tensor(1000.0).bfloat16().float())  # eps^-1/2


# ------------------------------------------------------------------ delta rule, single tokens

@pytest.mark.parametrize("B,Hk,H,d", [(1, 1, 1, 64), (1, 2, 4, 128), (5, 2, 2, 64), (7, 1, 3, 128)])
def test_delta_step(B, Hk, H, d):
    gen = torch.Generator().manual_seed(B * 10 + d)
    unit = lambda t: (t / t.norm(dim=-1, keepdim=True)).to(BF16)
    q, k, v = unit(rn(gen, B, Hk, d)), unit(rn(gen, B, Hk, d)), rn(gen, B, H, d, dtype=BF16)
    g = -rn(gen, B, H).abs()
    beta = torch.sigmoid(rn(gen, B, H)).to(BF16)
    slots = B + 3
    st = rn(gen, slots, H, d, d, std=0.3)
    idx = torch.randperm(slots, generator=gen)[:B].to(torch.int32)
    if B > 2:
        idx[2] = -1
    s = dev(st)
    o = gdr.delta_step(dev(q), dev(k), padded(v), dev(g), dev(beta), s, state_indices=dev(idx))
    want, orf = st.double(), torch.zeros(B, H, d, dtype=torch.float64)
    for r, j in enumerate(idx.tolist()):
        if 0 <= j < slots:
            orf[r], want[j] = ref.delta(q[r].double(), k[r].double(), v[r].double(),
                                        g[r].double(), beta[r].double(), st[j].double(), d ** -0.5)
    assert_close(o, orf, d, "o")
    assert_close(s, want, d, "state")


def test_delta_steps_continue_a_prompt():
    """chunk_fwd over a prompt, then delta_step token by token, against chunk_fwd over it all
    (both within the tolerances of the forward's own tests)."""
    from chunked_gated_delta_gdr_gb300.inputs import make_workload
    w = make_workload("continue", 5, [90], 2, 4, 128).to(DEV)
    full, hfull = gdr.chunk_fwd(w.q, w.k, w.v, w.g, w.beta, output_final_state=True)
    n = 80
    _, ht = gdr.chunk_fwd(w.q[:n], w.k[:n], w.v[:n], w.g[:n], w.beta[:n], output_final_state=True)
    for t in range(n, 90):
        o = gdr.delta_step(w.q[t:t + 1], w.k[t:t + 1], w.v[t:t + 1], w.g[t:t + 1],
                           w.beta[t:t + 1], ht)
        assert (o[0].float() - full[t].float()).abs().max().item() <= 4e-3
    assert ((ht - hfull).abs().max() / hfull.abs().max()).item() <= 1e-2


# ------------------------------------------------------------------ differences, streams, autograd

def test_gradients_against_differences():
    """Directional differences of the kernels' own forwards (fp32 inputs).  A central difference
    of step e has a truncation of order e^2 and a rounding of 2^-24 |f| / e: with e = 1e-2 both
    stay below 2e-3 of the largest term here."""
    gen = torch.Generator().manual_seed(2)
    cud = torch.tensor([0, 30, 30, 75], dtype=torch.int32, device=DEV)
    T, D, N = 75, 32, 16
    i = ssm_inputs(T, 3, D, N, 1, F32, True, True, True, True, True, 4)
    names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0")
    e = 1e-2

    def check(f, leaves, analytic):
        for k, t in leaves.items():
            u = rn(gen, *t.shape)
            plus, minus = dict(leaves), dict(leaves)
            plus[k], minus[k] = t + e * u, t - e * u
            num = (f(plus) - f(minus)) / (2 * e)
            ana = float((analytic[k].double().cpu() * u.double()).sum())
            size = float((analytic[k].double().cpu().abs() * u.double().abs()).sum())
            assert abs(num - ana) <= 2e-3 * max(size, 1.0), (k, num, ana, size)

    def ssm_loss(d):
        y, ht = gdr.ssm_fwd(*[dev(d[k]) for k in names[:5]], D=dev(d["D"]), z=dev(d["z"]),
                            dt_bias=dev(d["dt_bias"]), initial_state=dev(d["h0"]),
                            cu_seqlens=cud, output_final_state=True)
        return float((y.double() * dev(i["dy"]).double()).sum()
                     + (ht.double() * dev(i["dht"]).double()).sum())

    g = gdr.ssm_bwd(*[dev(i[k]) for k in names[:5]], dev(i["dy"]), D=dev(i["D"]), z=dev(i["z"]),
                    dt_bias=dev(i["dt_bias"]), initial_state=dev(i["h0"]), cu_seqlens=cud,
                    dfinal_state=dev(i["dht"]))
    check(ssm_loss, {k: i[k] for k in names}, dict(zip(names, g)))

    c = dict(x=rn(gen, T, D), w=rn(gen, D, 4), b=rn(gen, D), h0=rn(gen, 3, 3, D))
    dy, dht = rn(gen, T, D), rn(gen, 3, 3, D)

    def conv_loss(d):
        y, ht = gdr.conv_fwd(dev(d["x"]), dev(d["w"]), dev(d["b"]), dev(d["h0"]), cud, "silu", True)
        return float((y.double() * dev(dy).double()).sum()
                     + (ht.double() * dev(dht).double()).sum())

    g = gdr.conv_bwd(dev(c["x"]), dev(c["w"]), dev(dy), dev(c["b"]), dev(c["h0"]), cud, "silu",
                     dev(dht))
    check(conv_loss, c, dict(zip(("x", "w", "b", "h0"), g)))

    d = dict(q=rn(gen, 9, 2, 64), k=rn(gen, 9, 1, 64), qw=rn(gen, 64), kw=rn(gen, 64))
    ang = torch.rand(20, 16, generator=gen) * 6
    fixed = dict(cos=dev(ang.cos()), sin=dev(ang.sin()),
                 positions=torch.arange(9, dtype=torch.int32, device=DEV))
    gq, gk = rn(gen, 9, 2, 64), rn(gen, 9, 1, 64)

    def qk_loss(t):
        a, b = gdr.qk_fwd(dev(t["q"]), dev(t["k"]), dev(t["qw"]), dev(t["kw"]), **fixed)
        return float((a.double() * dev(gq).double()).sum() + (b.double() * dev(gk).double()).sum())

    g = gdr.qk_bwd(dev(d["q"]), dev(d["k"]), dev(gq), dev(gk), dev(d["qw"]), dev(d["kw"]), **fixed)
    check(qk_loss, d, dict(zip(("q", "k", "qw", "kw"), g)))


def test_autograd_wrappers_give_the_backwards_gradients():
    gen = torch.Generator().manual_seed(8)
    cud = torch.tensor([0, 21, 50], dtype=torch.int32, device=DEV)
    x = dev(rn(gen, 50, 64, dtype=BF16)).requires_grad_()
    w = dev(rn(gen, 64, 4)).requires_grad_()
    y, _ = gdr.short_conv(x, w, cu_seqlens=cud)
    y.sum().backward()  # an expanded gradient
    dx, dw, _, _ = gdr.conv_bwd(x.detach(), w.detach(), torch.ones_like(y), cu_seqlens=cud)
    assert torch.equal(x.grad, dx) and torch.equal(w.grad, dw)
    i = ssm_inputs(50, 2, 64, 16, 1, BF16, True, True, True, True, True, 6)
    names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0")
    lv = {k: dev(i[k]).requires_grad_() for k in names}
    y, ht = gdr.selective_ssm(*[lv[k] for k in names[:8]], True, lv["h0"], cud, True)
    torch.autograd.backward([y, ht], [dev(i["dy"]), dev(i["dht"])])
    det = {k: v.detach() for k, v in lv.items()}
    g = gdr.ssm_bwd(*[det[k] for k in names[:5]], dev(i["dy"]), *[det[k] for k in names[5:8]],
                    True, det["h0"], cud, dev(i["dht"]))
    for k, v in zip(names, g):
        assert torch.equal(lv[k].grad, v), k
    q = dev(rn(gen, 5, 2, 64, dtype=BF16)).requires_grad_()
    k = dev(rn(gen, 5, 1, 64, dtype=BF16)).requires_grad_()
    a, _ = gdr.qk_norm_rotate(q, k, norm="l2")
    a.float().sum().backward()  # no gradient for the second output
    dq, dk, _, _ = gdr.qk_bwd(q.detach(), k.detach(), torch.ones_like(q),
                              torch.zeros_like(k), norm="l2")
    assert torch.equal(q.grad, dq) and torch.equal(k.grad, dk)


def test_same_results_on_another_stream_and_again():
    i = ssm_inputs(400, 2, 128, 16, 1, BF16, True, True, True, True, True, 3)
    cud = torch.tensor([0, 300, 400], dtype=torch.int32, device=DEV)
    args = [dev(i[k]) for k in ("x", "dt", "A", "B", "C")]
    opts = dict(D=dev(i["D"]), z=dev(i["z"]), dt_bias=dev(i["dt_bias"]),
                initial_state=dev(i["h0"]), cu_seqlens=cud)
    first = gdr.ssm_bwd(*args, dev(i["dy"]), **opts)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        again = gdr.ssm_bwd(*args, dev(i["dy"]), **opts, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, again):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ refusals

def test_refusals():
    x = torch.zeros(8, 64, dtype=BF16, device=DEV)
    w = torch.zeros(64, 4, device=DEV)
    with pytest.raises(ValueError):
        gdr.conv_fwd(x.cpu(), w)
    with pytest.raises(ValueError):
        gdr.conv_fwd(x, w.cpu())
    with pytest.raises(ValueError):
        gdr.conv_fwd(x, w, activation="tanh")
    with pytest.raises(TypeError):
        gdr.conv_fwd(x, w, cu_seqlens=torch.tensor([0, 8], device=DEV))
    with pytest.raises(TypeError):
        gdr.conv_fwd(x.half(), w)
    for bad in (torch.zeros(64, 5, device=DEV), torch.zeros(64, 1, device=DEV)):
        with pytest.raises(gdr.GdrError) as e:
            gdr.conv_fwd(x, bad)
        assert e.value.status == -5
    with pytest.raises(gdr.GdrError) as e:
        gdr.conv_fwd(x, w, out=x.new_empty(1, 64).expand(8, 64))
    assert e.value.status == -4
    with pytest.raises(gdr.GdrError) as e:
        gdr.conv_step(x, w, torch.zeros(4, 3, 64, dtype=BF16, device=DEV))  # fewer slots than rows
    assert e.value.status == -3
    A, B = torch.zeros(64, 16, device=DEV), torch.zeros(8, 1, 16, dtype=BF16, device=DEV)
    with pytest.raises(gdr.GdrError) as e:
        gdr.ssm_fwd(x, x, A, B, torch.zeros(8, 1, 8, dtype=BF16, device=DEV))
    assert e.value.status == -3
    big = torch.zeros(8, 1, 65, dtype=BF16, device=DEV)
    with pytest.raises(gdr.GdrError) as e:
        gdr.ssm_fwd(x, x, torch.zeros(64, 65, device=DEV), big, big)
    assert e.value.status == -5
    three = torch.zeros(8, 3, 16, dtype=BF16, device=DEV)
    with pytest.raises(gdr.GdrError) as e:
        gdr.ssm_fwd(x, x, A, three, three)
    assert e.value.status == -6
    with pytest.raises(gdr.GdrError) as e:
        gdr.ssm_fwd(x, x, A, B, B, initial_state=torch.zeros(2, 64, 16, device=DEV))
    assert e.value.status == -7
    with pytest.raises(gdr.GdrError) as e:
        gdr.ssm_bwd(x, x, A, B, B, x, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == -8
    q = torch.zeros(8, 2, 64, dtype=BF16, device=DEV)
    cos = torch.zeros(4, 32, device=DEV)
    with pytest.raises(gdr.GdrError) as e:
        gdr.qk_fwd(q, q, cos=cos, sin=cos)  # no positions
    assert e.value.status == -1
    with pytest.raises(gdr.GdrError) as e:
        gdr.qk_fwd(q, q, cos=cos)
    assert e.value.status == -15
    wide = torch.zeros(4, 40, device=DEV)
    with pytest.raises(gdr.GdrError) as e:
        gdr.qk_fwd(q, q, cos=wide, sin=wide, positions=torch.zeros(8, dtype=torch.int32, device=DEV))
    assert e.value.status == -5
    st = torch.zeros(4, 2, 64, 64, device=DEV)
    g = torch.zeros(8, 2, device=DEV)
    with pytest.raises(gdr.GdrError) as e:
        gdr.delta_step(q, q, q, g, g.bfloat16(), st)  # fewer slots than rows
    assert e.value.status == -3
    with pytest.raises(ValueError):
        gdr.delta_step(q, q, q, g, g.bfloat16(), st,
                       state_indices=torch.zeros(3, dtype=torch.int32, device=DEV))


# ------------------------------------------------------------------ calls that follow one another

def _chain(sync):
    """Calls that each read what the one before wrote: a kernel is made ready while the one
    before it runs, and must wait for its results all the same."""
    gen = torch.Generator().manual_seed(5)
    T, C, N = 700, 256, 16
    x, w = dev(rn(gen, T, C, dtype=BF16)), dev(rn(gen, C, 4, std=0.5))
    A, B = dev(-rn(gen, C, N).abs() - 0.1), dev(rn(gen, T, 1, N, dtype=BF16, std=0.3))
    cu = torch.tensor([0, 300, 300, 700], dtype=torch.int32, device=DEV)
    pool, ssm = torch.zeros(9, 3, C, dtype=BF16, device=DEV), torch.zeros(9, C, N, device=DEV)
    slots = torch.tensor([4, 0, 7], dtype=torch.int32, device=DEV)
    done = (lambda: torch.cuda.synchronize()) if sync else (lambda: None)
    keep = []
    for i in range(12):
        y, _ = gdr.conv_fwd(x, w, cu_seqlens=cu)
        done()
        y, _ = gdr.ssm_fwd(y, y, A, B, B, cu_seqlens=cu)
        done()
        q, k = gdr.qk_fwd(y.view(T, 2, 128), y.view(T, 2, 128))
        done()
        dx, dw, _, _ = gdr.conv_bwd(x, w, q.view(T, C), cu_seqlens=cu)
        done()
        g = gdr.ssm_bwd(dx, dx, A, B, B, k.view(T, C), cu_seqlens=cu)
        done()
        x = gdr.qk_fwd(g[0].view(T, 2, 128), k)[0].view(T, C)
        done()
        for j in range(8):
            s = gdr.conv_step(x[3 * j:3 * j + 3], w, pool, state_indices=slots)
            done()
            s = gdr.ssm_step(s, s, A, B[:3], B[:3], ssm, state_indices=slots)
            done()
        keep += [x, dw, g[2], s]
    return keep + [pool, ssm]


def test_calls_in_a_row_wait_for_each_other():
    want = _chain(True)
    for _ in range(3):
        for a, b in zip(_chain(False), want):
            assert torch.equal(a, b)


def test_calls_in_a_graph_wait_for_each_other():
    want = _chain(True)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        _chain(False)
    torch.cuda.synchronize()
    gen = torch.Generator().manual_seed(6)
    T, C, N = 900, 128, 16
    x, A = dev(rn(gen, T, C, dtype=BF16)), dev(-rn(gen, C, N).abs() - 0.1)
    B = dev(rn(gen, T, 1, N, dtype=BF16, std=0.3))

    def run():
        y, ht = gdr.ssm_fwd(x, x, A, B, B, output_final_state=True)
        return gdr.ssm_bwd(y, x, A, B, B, y)[:5] + (y, ht)

    eager = run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        for a, b in zip(got, eager):
            assert torch.equal(a, b)
    for a, b in zip(_chain(False), want):
        assert torch.equal(a, b)
