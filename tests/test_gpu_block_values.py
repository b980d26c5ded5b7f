"""Values of a hybrid block's operators that small random inputs do not reach: infinities that a formula
keeps, weights that nearly cancel.  On a GB300, against 64 bits."""
import pytest
import torch

import block_testlib as ref
import chunked_gated_delta_gdr_gb300 as gdr
from mixer_testlib import BF16, F32, leaf

pytestmark = pytest.mark.gpu

DEV = "cuda"
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_gdr_gb300 import build
    build.build()
    if torch.cuda.get_device_capability() != (10, 3):
        pytest.skip("needs sm_103 (GB300)")


def rn(seed, *shape, dtype=F32, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (std * torch.randn(*shape, generator=gen)).to(dtype)


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("Hq,Hk,d,n,page", [(4, 2, 64, 70, 16), (32, 2, 128, 333, 16), (6, 1, 200, 95, 5),
                                            (8, 8, 128, 3000, 64), (20, 1, 256, 40, 16)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_keeps_infinite_values(Hq, Hk, d, n, page, dtype):
    # o = sum p v with weights above 0: infinite where v is, NaN where both signs meet
    pages = -(-n // page)
    q, kc, vc = rn(1, 1, Hq, d, dtype=dtype), rn(2, pages, page, Hk, d, dtype=dtype), rn(3, pages, page, Hk, d,
                                                                                         dtype=dtype)
    flat = vc.view(-1, Hk, d)
    for j, key in enumerate(sorted({0, 1, n // 2, n - 1})):
        flat[key, 0, j] = INF
        flat[key, Hk - 1, d - 1 - j] = -INF
    flat[0, 0, 9], flat[n - 1, 0, 9] = INF, -INF
    flat[n // 2, 0, 11] = float("nan")
    table = torch.arange(pages, dtype=torch.int32).view(1, -1)
    o = gdr.attn_step(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV),
                      torch.tensor([n], dtype=torch.int32, device=DEV)).cpu().double()
    rep = Hq // Hk
    k, v = kc.view(-1, Hk, d)[:n].double(), flat[:n].double()
    p = torch.softmax(torch.einsum("hd,nhd->hn", q[0].double(), k.repeat_interleave(rep, 1)) * d ** -0.5, 1)
    # weights of fp32 and more: none of them is near where 32 bits end
    assert float(p.min()) > 2.0 ** -60
    want = torch.einsum("hn,nhd->hd", p, v.repeat_interleave(rep, 1))[None]
    assert torch.isinf(want).sum() >= 8 and torch.isnan(want).sum() >= 2 * rep
    assert torch.equal(torch.isnan(o), torch.isnan(want))
    assert torch.equal(torch.where(torch.isinf(o), o, torch.zeros(1).double()),
                       torch.where(torch.isinf(want), want, torch.zeros(1).double()))


def test_attention_weights_have_32_bits():
    # Two keys whose values nearly cancel: o = (x - p y) / (1 + p) is small, so that what is lost of p is not
    # hidden behind the rounding of o.  Key 0 scores 0, key 1 -t with t a multiple of 1/64 up to 4 (exact
    # in bf16 up to 4: 8 bits), and x is p y rounded to bf16, so that |x - p y| <= 2^-8 p |y|.
    # p: 2 ulp of the exponential (2^-22), its argument t log2 e and the scale's product 2^-23 t each; the
    # sum of two products, which a tensor instruction may cut off, and its three additions 2^-23 |x| each
    # beside them: (2^-22 + 2^-22 t) p y + 4 * 2^-23 x, doubled for second order terms; and half a step of
    # bf16 of o.
    B, d = 256, 64
    t = (torch.arange(B) % 255 + 1).double() / 64
    q = torch.zeros(B, 2, d)
    q[:, :, 0] = 1.0
    kc, vc = torch.zeros(B, 16, 1, d), torch.zeros(B, 16, 1, d)
    kc[:, 1, 0, 0] = -t.float()
    y = 1 + torch.arange(d).double() / 128  # exact in bf16
    p = torch.exp(-t)[:, None]
    vc[:, 0, 0] = (p * y).to(BF16).float()
    vc[:, 1, 0] = -y.float()
    table = torch.arange(B, dtype=torch.int32).view(B, 1)
    o = gdr.attn_step(*(v.to(BF16).to(DEV) for v in (q, kc, vc)), table.to(DEV),
                      torch.full((B,), 2, dtype=torch.int32, device=DEV), 1.0).cpu().double()
    assert torch.equal(kc.to(BF16).double()[:, 1, 0, 0], -t)
    x = vc[:, 0, 0].to(BF16).double()
    want = (x - p * y) / (1 + p)
    tol = 2 * ((2.0 ** -22 * (1 + t[:, None])) * p * y + 4 * 2.0 ** -23 * x) / (1 + p) + 2.0 ** -8 * want.abs()
    for h in range(2):
        bad = (o[:, h] - want).abs() > tol
        assert not bad.any(), (int(bad.sum()), float(((o[:, h] - want).abs() / tol).max()))


@pytest.mark.parametrize("Hq,Hk,d,n", [(4, 2, 64, 70), (16, 1, 128, 1000), (3, 3, 200, 5)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_of_infinite_scores(Hq, Hk, d, n, dtype):
    # scores of -infinity: weights of 0; nothing else there: zeros.  Request 0 has only such keys, request 1 one
    # key beside them, whose weight is 1.
    page, pages = 16, 2 * -(-n // 16)
    q, kc, vc = rn(1, 2, Hq, d, dtype=dtype), rn(2, pages, page, Hk, d, dtype=dtype), rn(3, pages, page, Hk, d,
                                                                                         dtype=dtype)
    q[..., 0], kc[..., 0] = 1.0, -INF
    table = torch.arange(pages, dtype=torch.int32).view(2, -1)
    j = n // 3
    kc[table[1, j // page], j % page, :, 0] = 0.0
    o = gdr.attn_step(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV),
                      torch.full((2,), n, dtype=torch.int32, device=DEV)).cpu()
    assert not o[0].any()
    assert torch.equal(o[1], vc[table[1, j // page], j % page].repeat_interleave(Hq // Hk, 0))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_cache_without_pages(dtype):
    # and tables without columns, and plans and writes of nothing
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    q = rn(1, 3, 4, 64, dtype=dtype).to(DEV)
    empty = torch.empty(0, 16, 2, 64, dtype=dtype, device=DEV)
    some = rn(2, 2, 16, 2, 64, dtype=dtype).to(DEV)
    table = torch.zeros(3, 4, dtype=torch.int32, device=DEV)
    assert not gdr.attn_step(q, empty, empty, table, i32(5, 0, 40)).any()
    assert not gdr.attn_step(q, some, some, table[:, :0], i32(5, 0, 40)).any()
    before = some.clone()
    gdr.cache_write(q[:, :2], q[:, :2], empty, empty, i32(0, 1, 2))
    gdr.cache_write(q[:0, :2], q[:0, :2], some, some, i32())
    assert torch.equal(some, before)
    slots, pos, cu, lens, taken = gdr.cache_plan(i32(), i32(), table[:0], i32(3, 4), i32(1), 16, 5)
    assert slots.tolist() == [-1] * 5 and pos.tolist() == [0] * 5 and cu.tolist() == [0]
    assert lens.tolist() == [] and taken.tolist() == [1]
    slots, pos, cu, lens, taken = gdr.cache_plan(i32(), i32(), table[:0], i32(), i32(0), 16, 9000)
    assert slots.tolist() == [-1] * 9000 and not pos.any() and cu.tolist() == [0]


# ------------------------------------------------------------------ gated linear recurrence

REC = [(300, 64, [0, 300]), (2000, 64, [0, 900, 2000]), (6000, 34, [0, 40, 40, 5900, 6000]), (900, 2600, [0, 900]),
       (65, 16, [0, 65])]


@pytest.mark.parametrize("T,D,cu", REC)
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_recurrence_keeps_infinities_and_nan_to_the_segments_end(T, D, cu, norm, dtype):
    # decays of e^-9 to 1: their products over a block's tokens underflow to 0.  A NaN in a channel's state,
    # and an infinity, are there until the segment ends; other channels, and segments behind it, do not see them.
    x, r, i = (rn(k, T, D, dtype=dtype) for k in (1, 2, 3))
    A = torch.full((D,), -9.0)
    h0 = rn(4, len(cu) - 1, D)
    long = max(range(len(cu) - 1), key=lambda n: cu[n + 1] - cu[n])
    s, e = cu[long], cu[long + 1]
    at = [s, s + (e - s) // 5]
    bad = x.clone()
    bad[at[0], 0], bad[at[1], 1], bad[at[0], 2], bad[at[1], D - 1] = float("nan"), float("nan"), INF, -INF
    h0_bad = h0.clone()
    h0_bad[long, 4] = INF
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    place = lambda t: t.to(DEV)
    run = lambda x, h0: gdr.rec_fwd(place(x), place(r), place(A), place(i), norm, place(h0), cud, True)[:2]
    y, ht = (t.float().cpu() for t in run(bad, h0_bad))
    yc, hc = (t.float().cpu() for t in run(x, h0))
    lost = torch.zeros(T, D, dtype=torch.bool)
    for t, c in ((at[0], 0), (at[1], 1), (at[0], 2), (at[1], D - 1), (s, 4)):
        lost[t:e, c] = True
    assert torch.equal(~torch.isfinite(y), lost)
    assert torch.equal(y[~lost], yc[~lost])
    gone = torch.zeros_like(hc, dtype=torch.bool)
    gone[long] = lost[e - 1]
    assert torch.equal(~torch.isfinite(ht), gone) and torch.equal(ht[~gone], hc[~gone])
    assert torch.isnan(y[at[0]:e, 0]).all() and torch.isnan(ht[long, 0])


@pytest.mark.parametrize("T,D,cu", REC)
@pytest.mark.parametrize("norm", [True, False])
def test_recurrence_gradients_keep_infinities_and_nan(T, D, cu, norm):
    # the same for the gradient of the state, towards the segment's start
    x, r, i, dy = (rn(k, T, D) for k in (1, 2, 3, 5))
    A = torch.full((D,), -9.0)
    n = len(cu) - 1
    h0, dht = rn(4, n, D), rn(6, n, D)
    long = max(range(n), key=lambda k: cu[k + 1] - cu[k])
    s, e = cu[long], cu[long + 1]
    t1 = e - 1 - (e - s) // 5
    bad, dht_bad = dy.clone(), dht.clone()
    bad[t1, 0], bad[t1, 1], bad[e - 1, 2] = float("nan"), INF, float("nan")
    dht_bad[long, 4] = -INF
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    d = lambda t: t.to(DEV)
    back = lambda dy, dht: [t.cpu() for t in gdr.rec_bwd(d(x), d(r), d(A), d(dy), d(i), norm, d(h0), cud, d(dht))]
    dx, dr, dA, di, dh0 = back(bad, dht_bad)
    clean = back(dy, dht)
    lost = torch.zeros(T, D, dtype=torch.bool)
    for t, c in ((t1, 0), (t1, 1), (e - 1, 2), (e - 1, 4)):
        lost[s:t + 1, c] = True
    for a, c in zip((dx, dr, di), (clean[0], clean[1], clean[3])):
        assert torch.equal(a[~lost], c[~lost])
        assert not torch.isfinite(a[lost]).any()
    assert torch.equal(~torch.isfinite(dh0[long]), lost[s])
    keep = torch.ones_like(dh0, dtype=torch.bool)
    keep[long] = ~lost[s]
    assert torch.equal(dh0[keep], clean[4][keep])
    cols = ~lost.any(0)
    assert torch.equal(dA[cols], clean[2][cols]) and not torch.isfinite(dA[~cols]).any()


def growing(T, D, seed):
    """Inputs whose decays are above 1, with A from 0.001 to 3, the series' border among A sigmoid(r)."""
    s = dict(x=rn(seed, T, D), r=rn(seed + 1, T, D), i=rn(seed + 2, T, D), h0=rn(seed + 3, 1, D), dy=rn(seed + 4, T, D),
             dht=rn(seed + 5, 1, D))
    s["A"] = 0.001 * 3000.0 ** torch.linspace(0, 1, D)
    s["r"][:, 0::5] = 20.0  # sigmoid(r) = 1
    border = s["A"][5::10]
    border.copy_(0.0625 + 1e-3 * torch.linspace(-1, 1, len(border)))
    return s


def within(got, want, bound, name):
    off = (got.cpu().double() - want.detach()).abs()
    assert bool((off <= bound).all()), f"{name}: {float((off / bound).max())} of the bound"


@pytest.mark.parametrize("T,D", [(6, 64), (6, 130)])
def test_recurrence_that_grows(T, D):
    # A > 0 without the normaliser: the same formula.  A decay's relative error is 2^-22 of the exponential and,
    # |A sigmoid(r)| being 3 at most, 3 times some 8 roundings of 2^-24 of its argument: 7 * 2^-22, and 8 * 2^-22 = e
    # for a token's product and sum with it.  With M_t = a M_{t-1} + |u_t|, which no state is above, errors add
    # up to (t + 1) e M_t; with N_t = |dy_t| + a N_{t+1} those of the gradient of h_t to (T - t) e N_t.  A product
    # of both has the errors of both and 8 roundings of its own at most, and 1 - sigmoid is off by
    # 2^-22 absolutely.
    s = growing(T, D, 20)
    dev = {k: v.to(DEV) for k, v in s.items()}
    y, ht, kept = gdr.rec_fwd(dev["x"], dev["r"], dev["A"], dev["i"], False, dev["h0"], None, True, True)
    leaves = {k: leaf(s[k]) for k in ("x", "r", "A", "i", "h0")}
    yr, hr, _ = ref.rec(leaves["x"], leaves["r"], leaves["A"], leaves["i"], False, leaves["h0"], [0, T])
    ((yr * s["dy"].double()).sum() + (hr * s["dht"].double()).sum()).backward()
    d = {k: v.double() for k, v in s.items()}
    sr, si = torch.sigmoid(d["r"]), torch.sigmoid(d["i"])
    a, e = torch.exp(d["A"] * sr), 8 * 2.0 ** -22
    M, N = [d["h0"][0].abs()], [d["dht"][0].abs()]
    for t in range(T):
        M.append(a[t] * M[-1] + (si[t] * d["x"][t]).abs())
        k = T - 1 - t
        N.append(d["dy"][k].abs() + (N[-1] if t == 0 else a[k + 1] * N[-1]))
    before, M = torch.stack(M[:-1]), torch.stack(M[1:])
    N = torch.stack(N[:0:-1])
    within(y, yr, torch.arange(1, T + 1)[:, None] * e * M, "y")
    within(ht, hr, T * e * M[-1:], "final state")
    dx, dr, dA, di, dh0 = gdr.rec_bwd(dev["x"], dev["r"], dev["A"], dev["dy"], dev["i"], False, dev["h0"], None,
                                      dev["dht"], checkpoints=kept)
    q = N * a * before * sr
    within(dx, leaves["x"].grad, (T + 1) * e * N * si, "dx")
    within(di, leaves["i"].grad, N * d["x"].abs() * si * ((T + 1) * e * (1 - si) + 2.0 ** -22), "di")
    within(dr, leaves["r"].grad, q * d["A"] * ((2 * T + 2) * e * (1 - sr) + 2.0 ** -22), "dr")
    within(dA, leaves["A"].grad, (3 * T + 2) * e * q.sum(0), "dA")
    within(dh0, leaves["h0"].grad, (T + 1) * e * (a[0] * N[0])[None], "dh0")
    state = dev["h0"].clone()
    one = gdr.rec_step(dev["x"][:1], dev["r"][:1], dev["A"], state, dev["i"][:1], False)
    within(one, yr[:1], e * M[:1], "step")
    within(state, yr[:1], e * M[:1], "state of a step")


def test_recurrence_that_grows_has_no_normaliser():
    s = growing(6, 64, 30)
    dev = {k: v.to(DEV) for k, v in s.items()}
    y, _, _ = gdr.rec_fwd(dev["x"], dev["r"], dev["A"], dev["i"], True, dev["h0"])
    assert torch.isnan(y).all()
    assert torch.isnan(gdr.rec_step(dev["x"][:1], dev["r"][:1], dev["A"], dev["h0"], dev["i"][:1])).all()
