"""A hybrid block's calls as users vary them: streams, graphs, scratch, buffers that are given, two calls
at once, sizes whose offsets pass 32 bits, long sequences, rows and contexts."""
import pytest
import torch

import block_testlib as ref
import chunked_gated_delta_gdr_gb300 as gdr
from mixer_testlib import BF16, F32, assert_close

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_gdr_gb300 import build
    build.build()
    if torch.cuda.get_device_capability() != (10, 3):
        pytest.skip("needs sm_103 (GB300)")


def normal(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s, std=1.0, dtype=F32: (std * torch.randn(*s, generator=g, device=DEV)).to(dtype)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def decays(r, D):
    return -0.8 * r(D).abs().clamp(max=3) - 0.01


def pages_for(lens, ps, seed, spare=3):
    """(block table, pages in the pool) of requests that hold their pages in any order."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // ps) for n in lens]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table.to(DEV), pool


# ------------------------------------------------------------------ every call once

def all_calls(seed, T=700, D=192):
    """name -> a call on inputs of its own that returns its tensors."""
    r = normal(seed)
    cu = i32([0, T // 3, T // 3, T])
    x, g, i, dy = (r(T, D, dtype=BF16) for _ in range(4))
    A, h0, dht = decays(r, D), r(3, D), r(3, D)
    st, slots = r(9, D), i32([7, 2, -1, 0])
    hx, hz, hd = (r(T, 3, 64, dtype=BF16) for _ in range(3))
    hw, w, wp, gate = 1 + r(64, std=0.1), 1 + r(D, std=0.1), 1 + r(D, std=0.1), r(D)
    res, dh = r(T, D), r(T, D)
    lens = [0, 600, 33, 1, 900]
    table, pool = pages_for(lens, 16, seed)
    kc, vc, q = r(pool, 16, 2, 64, dtype=BF16), r(pool, 16, 2, 64, dtype=BF16), r(5, 8, 64, dtype=BF16)
    n = i32(lens)
    new, free, taken = i32([2, 1, 0, 40, 1]), i32(list(range(100, 140))), i32([1])
    wide = torch.full((5, 70), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    k, v = r(44, 2, 64, dtype=BF16), r(44, 2, 64, dtype=BF16)
    at = torch.randperm(pool * 16, device=DEV)[:44].to(torch.int32)

    def step():
        s = st.clone()
        return gdr.rec_step(x[:4], g[:4], A, s, i[:4], state_indices=slots), s

    def plan():
        t = wide.clone()
        return (*gdr.cache_plan(n, new, t, free, taken, 16, 44), t)

    def write():
        a, b = kc.clone(), vc.clone()
        gdr.cache_write(k, v, a, b, at)
        return a, b

    return dict(
        rec_fwd=lambda: gdr.rec_fwd(x, g, A, i, True, h0, cu, True, True),
        rec_bwd=lambda: gdr.rec_bwd(x, g, A, dy, i, True, h0, cu, dht),
        rec_step=step,
        gated_fwd=lambda: (gdr.gated_norm_fwd(hx, hz, hw),),
        gated_bwd=lambda: gdr.gated_norm_bwd(hx, hz, hd, hw),
        resid_fwd=lambda: gdr.residual_norm_fwd(x, res, w, wp, gate, 0.5),
        resid_bwd=lambda: gdr.residual_norm_bwd(x, res, dy, dh, w, wp, gate, 0.5),
        attn=lambda: (gdr.attn_step(q, kc, vc, table, n),),
        plan=plan, write=write)


def same(a, b):
    return all((p is None and q is None) or torch.equal(p, q) for p, q in zip(a, b))


def test_results_are_the_same_from_run_to_run():
    for name, f in all_calls(1).items():
        first = [None if t is None else t.clone() for t in f()]
        for _ in range(3):
            assert same(first, f()), name


def test_on_another_stream_and_two_at_once():
    """Each call on two streams at once, with scratch of its own."""
    a, b = all_calls(2), all_calls(3, T=900, D=320)
    want = {n: (a[n](), b[n]()) for n in a}
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for n in a:
        got = []
        for _ in range(4):
            with torch.cuda.stream(one):
                p = a[n]()
            with torch.cuda.stream(two):
                q = b[n]()
            got.append((p, q))
        torch.cuda.synchronize()
        for p, q in got:
            assert same(p, want[n][0]) and same(q, want[n][1]), n


@pytest.mark.parametrize("T,C,dtype", [(640, 12296, BF16), (300, 8200, F32), (45, 16384, BF16)])
def test_rows_on_clusters_in_place_at_once_and_captured(T, C, dtype):
    """Rows that several blocks share: outputs over their inputs, two streams, a replayed graph."""
    r = normal(7)
    x, res, dy, dh = (r(T, C, dtype=dtype) for _ in range(4))
    w, wp, g = 1 + r(C), 1 + r(C), r(C)
    opts = (w, wp, g, 0.7)
    fwd = lambda: gdr.residual_norm_fwd(x, res, *opts)
    bwd = lambda: gdr.residual_norm_bwd(x, res, dy, dh, *opts)
    want, back = fwd(), bwd()
    a, b = x.clone(), res.clone()
    gdr.residual_norm_fwd(a, b, *opts, out=a, residual_out=b)
    assert same((a, b), want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append((fwd(), bwd()))
    torch.cuda.synchronize()
    for p, q in got:
        assert same(p, want) and same(q, back)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        taped, taped_back = fwd(), bwd()
    for _ in range(3):
        for t in (*taped, *taped_back):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert same(taped, want) and same(taped_back, back)


def test_the_stream_argument():
    r = normal(4)
    x, g, A = r(300, 128, dtype=BF16), r(300, 128, dtype=BF16), decays(r, 128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, _, _ = gdr.rec_fwd(x, g, A, stream=s)
    z = gdr.gated_norm_fwd(y.view(300, 2, 64), x.view(300, 2, 64), stream=s)
    out, h = gdr.residual_norm_fwd(z.view(300, 128), x, stream=s)
    s.synchronize()
    y2, _, _ = gdr.rec_fwd(x, g, A)
    z2 = gdr.gated_norm_fwd(y2.view(300, 2, 64), x.view(300, 2, 64))
    assert same(gdr.residual_norm_fwd(z2.view(300, 128), x), (out, h))


def test_captured_calls_replayed_on_other_inputs():
    r = normal(5)
    T, D = 500, 128
    x, g, dy, A = r(T, D, dtype=BF16), r(T, D, dtype=BF16), r(T, D, dtype=BF16), decays(r, D)
    res, w = r(T, D), 1 + r(D, std=0.1)

    def run():
        y, ht, kept = gdr.rec_fwd(x, g, A, output_final_state=True, output_checkpoints=True)
        n = gdr.gated_norm_fwd(y.view(T, 2, 64), g.view(T, 2, 64))
        out = gdr.residual_norm_fwd(n.view(T, D), res, w)
        back = gdr.residual_norm_bwd(n.view(T, D), res, dy, None, w)
        dn = gdr.gated_norm_bwd(y.view(T, 2, 64), g.view(T, 2, 64), back[0].view(T, 2, 64))
        return (ht, *out, back[2], *dn[:2],
                *gdr.rec_bwd(x, g, A, dn[0].view(T, D), checkpoints=kept))

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed in (6, 7):
        n = normal(seed)
        for t in (x, g, dy, res):
            t.copy_(n(*t.shape))
        graph.replay()
        got = [None if t is None else t.clone() for t in out]
        assert same(got, run())


def test_two_graphs_of_decoding_share_nothing():
    """Steps over a growing cache, captured with the plan in place, two batches turn about."""
    r = normal(8)
    B, Hk, Hq, d, ps, steps = 6, 2, 8, 64, 4, 9

    def batch(seed):
        n = normal(seed)
        s = dict(lens=i32([0, 3, 4, 7, 0, 12]), new=i32([1, 1, 1, 1, 0, 1]), taken=i32([0]),
                 table=torch.full((B, 8), -1, dtype=torch.int32, device=DEV),
                 kc=n(40, ps, Hk, d, dtype=BF16), vc=n(40, ps, Hk, d, dtype=BF16),
                 q=n(B, Hq, d, dtype=BF16), k=n(B, Hk, d, dtype=BF16), v=n(B, Hk, d, dtype=BF16))
        free = list(range(39, -1, -1))
        at = 0
        for b, m in enumerate([0, 3, 4, 7, 0, 12]):
            for j in range(-(-m // ps)):
                s["table"][b, j] = free[at]
                at += 1
        s["free"], s["taken"][0] = i32(free), at
        return s

    def step(s):
        slots, pos, cu, _, _ = gdr.cache_plan(s["lens"], s["new"], s["table"], s["free"], s["taken"],
                                              ps, B, s["lens"], s["taken"])
        # the token of a row that adds none is padding: rows of k and v are those of the new tokens
        gdr.cache_write(s["k"], s["v"], s["kc"], s["vc"], slots)
        o = gdr.attn_step(s["q"], s["kc"], s["vc"], s["table"], s["lens"])
        s["q"].copy_(torch.nn.functional.normalize(o.float(), dim=-1) * 8)
        return o

    eager = [batch(1), batch(2)]
    want = [[step(s).clone() for _ in range(steps)] for s in eager]
    taped = [batch(1), batch(2)]
    saved = [{k: v.clone() for k, v in s.items()} for s in taped]
    graphs, outs = [], []
    for s, b in zip(taped, saved):
        step(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(s))
        graphs.append(g)
        for k in s:
            s[k].copy_(b[k])
    for t in range(steps):
        for j in (0, 1):
            graphs[j].replay()
            assert torch.equal(outs[j], want[j][t]), (t, j)
    for a, b in zip(eager, taped):
        assert all(torch.equal(a[k], b[k]) for k in a)


# ------------------------------------------------------------------ buffers that are given

def test_buffers_that_are_given_are_written():
    r = normal(9)
    x, g, A, cu = r(50, 64, dtype=BF16), r(50, 64, dtype=BF16), decays(r, 64), i32([0, 20, 20, 50])
    want = gdr.rec_fwd(x, g, A, cu_seqlens=cu, output_final_state=True, output_checkpoints=True)
    bufs = [torch.full_like(t, 9.0) for t in want]
    got = gdr.rec_fwd(x, g, A, cu_seqlens=cu, out=bufs[0], final_state=bufs[1], checkpoints=bufs[2])
    assert same(got, want) and same(bufs, want)
    assert gdr.rec_fwd(x, g, A)[1:] == (None, None)
    o = torch.empty(50, 64, dtype=BF16, device=DEV)
    y, h = gdr.residual_norm_fwd(x, None, out=o)
    assert y.data_ptr() == o.data_ptr() and torch.equal(h, x)


def test_scratch_that_is_given():
    from chunked_gated_delta_gdr_gb300 import _native as nat
    r = normal(10)
    T, D = 400, 96
    x, g, dy, A = (r(T, D, dtype=BF16) for _ in range(3)), None, None, decays(r, D)
    x, g, dy = x
    need = nat.lib().gdr_rec_bwd_workspace_bytes(T, D, 1, 0)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    assert same(gdr.rec_bwd(x, g, A, dy, workspace=ws), gdr.rec_bwd(x, g, A, dy))
    for bad in (ws[:-1], ws[1:].clone()[1:], torch.empty(need + 8, dtype=torch.uint8, device=DEV)[8:]):
        with pytest.raises(gdr.GdrError) as e:
            gdr.rec_bwd(x, g, A, dy, workspace=bad)
        assert e.value.status == -8
    with pytest.raises(ValueError):
        gdr.rec_bwd(x, g, A, dy, workspace=torch.empty(need, dtype=torch.uint8))
    lens = [70, 3]
    table, pool = pages_for(lens, 16, 1)
    kc, q = r(pool, 16, 2, 64, dtype=BF16), r(2, 4, 64, dtype=BF16)
    need = nat.lib().gdr_attn_step_workspace_bytes(2, 4, 2, 64)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    o = gdr.attn_step(q, kc, kc, table, i32(lens), workspace=ws)
    assert torch.equal(o, gdr.attn_step(q, kc, kc, table, i32(lens)))
    with pytest.raises(gdr.GdrError):
        gdr.attn_step(q, kc, kc, table, i32(lens), workspace=ws[:need - 256])


# ------------------------------------------------------------------ offsets over 32 bits

def test_offsets_over_32_bits():
    r = normal(11)
    T, st = 262_200, 8_192 + 64  # rows this far apart: the last starts behind 2^31 elements
    wide = torch.empty(T, st, dtype=BF16, device=DEV)
    x = wide[:, 64:64 + 64]
    x.copy_(r(T, 64))
    g, A = x.clone(), decays(r, 64)
    a, b = gdr.rec_fwd(x, g, A), gdr.rec_fwd(g, g, A)
    assert torch.equal(a[0], b[0])
    assert same(gdr.rec_bwd(x, g, A, x), gdr.rec_bwd(g, g, A, g))
    heads = lambda t: t.unflatten(1, (2, 32))
    assert torch.equal(gdr.gated_norm_fwd(heads(x), heads(g)), gdr.gated_norm_fwd(heads(g), heads(g)))
    assert same(gdr.gated_norm_bwd(heads(x), heads(x), heads(x)),
                gdr.gated_norm_bwd(heads(g), heads(g), heads(g)))
    assert same(gdr.residual_norm_fwd(x, x), gdr.residual_norm_fwd(g, g))
    assert same(gdr.residual_norm_bwd(x, x, x, x), gdr.residual_norm_bwd(g, g, g, g))
    out = wide[:, 256:256 + 64]
    gdr.rec_fwd(g, g, A, out=out)
    assert torch.equal(out, b[0])
    del wide, x, out
    # a cache of more than 2^31 elements: keys and values on its last pages
    pages, ps, Hk, d = 2 ** 31 // (16 * 8 * 128) + 90, 16, 8, 128
    kc = torch.zeros(pages, ps, Hk, d, dtype=BF16, device=DEV)
    lens = [800, 33]
    table = torch.full((2, 50), -1, dtype=torch.int32, device=DEV)
    table[0] = torch.arange(pages - 1, pages - 51, -1, device=DEV)
    table[1, :3] = torch.arange(pages - 60, pages - 57, device=DEV)
    small = torch.zeros(53, ps, Hk, d, dtype=BF16, device=DEV)
    t2 = torch.full_like(table, -1)
    t2[0], t2[1, :3] = torch.arange(50, device=DEV), torch.arange(50, 53, device=DEV)
    k, q = r(833, Hk, d, dtype=BF16), r(2, 16, d, dtype=BF16)
    at = torch.arange(800, device=DEV)
    for cache, t in ((kc, table), (small, t2)):
        slots = torch.cat([t[0][at // ps] * ps + at % ps,
                           t[1][at[:33] // ps] * ps + at[:33] % ps]).to(torch.int32)
        gdr.cache_write(k, k, cache, cache, slots)
    assert torch.equal(kc[pages - 1], small[0])
    assert torch.equal(gdr.attn_step(q, kc, kc, table, i32(lens)),
                       gdr.attn_step(q, small, small, t2, i32(lens)))


# ------------------------------------------------------------------ long and wide

def rec64(x, r, A, i, h0, cu, dy, dht):
    """Forward and backward token by token in 64 bits, on the GPU."""
    x, r, A, i, h0, dy, dht = (t.double() for t in (x, r, A, i, h0, dy, dht))
    sr, si = torch.sigmoid(r), torch.sigmoid(i)
    L = A * sr
    a, m = torch.exp(L), torch.sqrt(-torch.expm1(2 * L))
    y, hb, ends = torch.empty_like(x), torch.empty_like(x), []
    for n, (s, e) in enumerate(zip(cu[:-1], cu[1:])):
        h = h0[n]
        for t in range(s, e):
            hb[t] = h
            h = a[t] * h + m[t] * si[t] * x[t]
            y[t] = h
        ends.append(h)
    G, dh0 = torch.empty_like(x), []
    for n, (s, e) in enumerate(zip(cu[:-1], cu[1:])):
        c = dht[n]
        for t in reversed(range(s, e)):
            G[t] = dy[t] + c
            c = a[t] * G[t]
        dh0.append(c)
    dL = G * a * (hb - si * x * a / m)
    return (y, torch.stack(ends), G * m * si, dL * A * sr * (1 - sr), (dL * sr).sum(0),
            G * m * si * (1 - si) * x, torch.stack(dh0))


@pytest.mark.parametrize("T,D,dtype,cu", [
    (9_001, 64, BF16, [0, 4000, 4003, 9001]), (6_007, 136, F32, [0, 1, 6007]),
    (5_003, 1_002, BF16, [0, 2000, 5003]), (3_001, 4_160, BF16, [0, 1500, 3001]),
    (2_000, 20_000, F32, [0, 2000]), (4_097, 8, F32, [0, 64, 4097])])
def test_long_recurrences(T, D, dtype, cu):
    r = normal(T)
    x, g, i, dy = (r(T, D, dtype=dtype) for _ in range(4))
    A, h0, dht = decays(r, D), r(len(cu) - 1, D), r(len(cu) - 1, D)
    want = rec64(x, g, A, i, h0, cu, dy, dht)
    y, ht, kept = gdr.rec_fwd(x, g, A, i, True, h0, i32(cu), True, True)
    dx, dr, dA, di, dh0 = gdr.rec_bwd(x, g, A, dy, i, True, h0, i32(cu), dht, checkpoints=kept)
    for name, a, b in zip("y ht dx dr dA di dh0".split(), (y, ht, dx, dr, dA, di, dh0), want):
        assert_close(a, b, T, name)


@pytest.mark.parametrize("T,C,dtype,rt", [(5_011, 1_536, BF16, BF16), (1_301, 6_152, BF16, F32),
                                          (700, 12_296, BF16, BF16), (3_001, 4_096, F32, F32),
                                          (20_011, 264, BF16, F32), (40_003, 40, F32, F32)])
def test_many_rows_of_the_residual_norm(T, C, dtype, rt):
    r = normal(C)
    x, dy, res, dh = r(T, C, dtype=dtype), r(T, C, dtype=dtype), r(T, C, dtype=rt), r(T, C, dtype=rt)
    w, wp, g = 1 + r(C, std=0.2), 1 + r(C, std=0.2), r(C)
    leaves = [t.double().requires_grad_() for t in (x, res, w, wp, g)]
    yr, hr = ref.residual(*leaves, 0.7, 1e-6, True)
    torch.autograd.backward((yr, hr), (dy.double(), dh.double()))
    y, h = gdr.residual_norm_fwd(x, res, w, wp, g, 0.7)
    assert_close(y, yr, C, "y")
    assert_close(h, hr, 8, "h")
    got = gdr.residual_norm_bwd(x, res, dy, dh, w, wp, g, 0.7)
    for name, a, l, n in zip("dx dres dw dwp dg".split(), got, leaves, (C, C, T + C, T + C, T + C)):
        assert_close(a, l.grad, n, name)


@pytest.mark.parametrize("T,H,d,dtype", [(20_011, 9, 128, BF16), (6_001, 5, 200, F32),
                                         (70_001, 3, 8, BF16), (3_001, 2, 768, BF16)])
def test_many_rows_of_the_gated_norm(T, H, d, dtype):
    r = normal(d)
    x, z, dy = (r(T, H, d, dtype=dtype) for _ in range(3))
    w = 1 + r(d, std=0.2)
    leaves = [t.double().requires_grad_() for t in (x, z, w)]
    yr = ref.gated(*leaves, "silu", 1e-6)
    yr.backward(dy.double())
    assert_close(gdr.gated_norm_fwd(x, z, w), yr, d, "y")
    for name, a, l, n in zip(("dx", "dz", "dw"), gdr.gated_norm_bwd(x, z, dy, w), leaves,
                             (d, d, T * H + d)):
        assert_close(a, l.grad, n, name)


@pytest.mark.parametrize("B,Hq,Hk,d,ps,longest,window", [
    (300, 8, 4, 64, 16, 700, 0), (37, 16, 1, 128, 16, 5000, 0), (5, 24, 1, 128, 64, 9000, 4000),
    (3, 64, 2, 256, 16, 3000, 0), (700, 4, 2, 128, 8, 90, 0), (1, 8, 8, 128, 128, 40000, 0),
    (9, 6, 2, 120, 48, 2000, 777)])
def test_many_contexts(B, Hq, Hk, d, ps, longest, window):
    r = normal(B)
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, longest + 1, (B,), generator=g).tolist()
    lens[-1] = longest
    table, pool = pages_for(lens, ps, B)
    kc, vc = r(pool, ps, Hk, d, dtype=BF16), r(pool, ps, Hk, d, dtype=BF16)
    q = r(B, Hq, d, dtype=BF16, std=1.5)
    o = gdr.attn_step(q, kc, vc, table, i32(lens), window=window)
    rep = Hq // Hk
    for b in range(B):
        n = lens[b]
        if n == 0:
            assert not o[b].any()
            continue
        at = torch.arange(max(0, n - window) if window else 0, n, device=DEV)
        rows = table[b].long()[at // ps] * ps + at % ps
        k = kc.view(-1, Hk, d)[rows].double().repeat_interleave(rep, 1)
        v = vc.view(-1, Hk, d)[rows].double().repeat_interleave(rep, 1)
        s = torch.einsum("nhd,hd->nh", k, q[b].double()) * d ** -0.5
        want = torch.einsum("nh,nhd->hd", torch.softmax(s, 0), v)
        size = float(torch.einsum("nhd,hd->nh", k.abs(), q[b].double().abs()).max()) * d ** -0.5
        off = (d + 8) * 2.0 ** -23 * size + 2.0 ** -22 * (1 + float(s.abs().max())) + 2.0 ** -17
        tol = torch.tensor([(2 * off + len(at) * 2.0 ** -23) * float(v.abs().max())])
        ref.assert_attention(o[b:b + 1], want[None].cpu(), tol)


# ------------------------------------------------------------------ autograd's corners

def test_gradients_of_some_inputs():
    r = normal(12)
    x, g = r(30, 64, dtype=BF16).requires_grad_(), r(30, 64, dtype=BF16)
    A = decays(r, 64)
    y, ht = gdr.gated_recurrence(x, g, A)
    assert ht is None
    y.float().sum().backward()
    want = gdr.rec_bwd(x.detach(), g, A, torch.ones_like(y))
    assert torch.equal(x.grad, want[0])
    with torch.no_grad():
        assert torch.equal(gdr.gated_recurrence(x, g, A)[0], y)
    # the residual stream alone, the norm alone, no residual at all
    res = r(30, 64, dtype=F32).requires_grad_()
    for pick in (0, 1):
        res.grad = x.grad = None
        gdr.residual_norm(x, res)[pick].float().sum().backward()
        one = torch.ones(30, 64, device=DEV)
        want = gdr.residual_norm_bwd(x.detach(), res.detach(),
                                     (one if pick == 0 else 0 * one).to(BF16), one if pick else None)
        assert torch.equal(x.grad, want[0]) and torch.equal(res.grad, want[1])
    x.grad = None
    y, h = gdr.residual_norm(x, None)
    (y.float().sum() + h.float().sum()).backward()
    assert torch.equal(x.grad, gdr.residual_norm_bwd(x.detach(), None, torch.ones_like(y),
                                                     torch.ones_like(h))[0])
    # a gradient with strides of 0 (a sum's) and one that is not contiguous
    z = r(30, 64, dtype=BF16).requires_grad_()
    gdr.gated_norm(x.view(30, 1, 64), z.view(30, 1, 64)).sum().backward()
    gdr.gated_norm(x.view(30, 1, 64), z.view(30, 1, 64)).transpose(0, 2).contiguous().sum().backward()
