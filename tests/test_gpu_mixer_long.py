"""The mixer's operators at sizes whose blocks run over many tiles of tokens: the marks of the
segment bounds written a tile ahead, the rings of rows on their way, the backward scan's kept
states and its ranges of 64 tokens, and norms whose blocks take many tokens in turn.  Everything is
compared with 64-bit implementations on the same GPU.

Tolerances, beside those of mixer_testlib: a parameter's gradient is a sum of terms, added in fp32 by
threads of `serial` terms each, where one term of n left out or counted twice is about 1 / n of the
sum of the terms' sizes.  Its error is bounded by 2^-24 serial times that sum, and 32 roundings of
2^-24 in each term, of its size, or of the sizes of what it is the difference of: silu' is between
-0.1 and 1.1 and 0 near -1.3, and moves by half of what its argument does, so that a term dy silu'(u) x
of the convolution is good to that part of |dy x| (1 + |b| + sum |w x|).
"""
import pytest
import torch

import chunked_gated_delta_gdr_gb300 as gdr
import mixer_testlib as ref
from chunked_gated_delta_gdr_gb300 import _native as nat
from mixer_testlib import BF16, F32, assert_close

pytestmark = pytest.mark.gpu

DEV = "cuda"
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_gdr_gb300 import build
    build.build()
    if torch.cuda.get_device_capability() != (10, 3):
        pytest.skip("needs sm_103 (GB300)")


def normal(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s, std=1.0, dtype=F32: (std * torch.randn(*s, generator=g, device=DEV)).to(dtype)


def leaf(t):
    return None if t is None else t.double().requires_grad_(True)


def assert_summed(got, terms, serial, name, sizes=None):
    """terms [T, ...] of got [...] in 64 bits; sizes: what their roundings go by."""
    sizes = terms.abs() if sizes is None else sizes
    bound = 2.0 ** -24 * (serial * terms.abs().sum(0) + 32 * sizes.sum(0))
    bad = ~((got.double() - terms.sum(0)).abs() <= bound)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off"


# ------------------------------------------------------------------ convolution

def conv(x, w, b, h0, cu, act):
    """ref.conv, the tokens side by side, with taps w [T, C, W] and bias b [T, C] of each token's own
    (so that their gradients are the terms of the parameters')."""
    T, C = x.shape
    W = w.shape[2]
    bd = ref.bounds(cu, T)
    n = len(bd) - 1
    rows = torch.cat([h0.reshape(n * (W - 1), C), x])
    at = torch.zeros(T, W, dtype=torch.long)
    ends = torch.zeros(n, W - 1, dtype=torch.long)
    mask = torch.zeros(T, dtype=torch.bool)
    for s in range(n):
        a, e = bd[s], bd[s + 1]
        mask[a:e] = True
        # a segment's rows: its W - 1 states, then its tokens
        own = torch.cat([torch.arange(s * (W - 1), (s + 1) * (W - 1)),
                         n * (W - 1) + torch.arange(a, e)])
        for k in range(W):
            at[a:e, k] = own[k:k + e - a]
        ends[s] = own[e - a:]
    at, ends, mask = at.to(DEV), ends.to(DEV), mask.to(DEV)
    taken = [rows.index_select(0, at[:, k]) for k in range(W)]
    u = b
    for k in range(W):
        u = u + w[:, :, k] * taken[k]
    y = (ref.silu(u) if act else u) * mask[:, None]
    with torch.no_grad():  # of each token's dw and db for dy = 1
        top = 1 + b.abs() + sum((w[:, :, k] * taken[k]).abs() for k in range(W))
        top = top * mask[:, None]
        sizes = torch.stack([t.abs() * top for t in taken], -1), top
    return y, rows[ends], mask, sizes


# Ranges of 16 to 80 tokens (forward) and 32 to 112 (backward) at 152 SMs; bounds inside them, on their
# edges (80, 112, 336), one token and none behind them, tokens without a segment at both ends.
EDGES = [2, 80, 112, 113, 336, 336, 1000, 1001, 1003, 2240, 3000, 3000, 4992]


@pytest.mark.parametrize("T,C,W,dtype,act", [
    (5011, 6144, 4, BF16, True),   # blocks of 128 threads, all of them with channels
    (5011, 3064, 3, F32, True),    # the last threads without channels
    (5011, 3061, 4, BF16, True),   # rows that are not aligned
    (4999, 1000, 2, BF16, False),
    (40003, 136, 4, F32, True),    # blocks of 32 threads
    (40003, 61, 4, BF16, True),
])
def test_convolution_over_many_tiles(T, C, W, dtype, act):
    r = normal(T + C)
    cu = EDGES + ([20000, T - 1] if T > 5011 else [])
    n = len(cu) - 1
    x, w, b = r(T, C, dtype=dtype), r(C, W, std=W ** -0.5), r(C, std=0.2)
    h0, dy, dht = r(n, W - 1, C, dtype=dtype), r(T, C, dtype=dtype), r(n, W - 1, C, dtype=dtype)
    ranges = nat.lib().gdr_conv_bwd_workspace_bytes(T, C, W) // ((W + 1) * C * 4)
    tokens = -(-T // ranges)
    assert tokens > 16, "the backward's ranges are one tile: take more tokens"
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    name = "silu" if act else None
    y, ht = gdr.conv_fwd(x, w, b, h0, cud, name, True, out=torch.full_like(x, 7.0))
    dx, dw, db, dh0 = gdr.conv_bwd(x, w, dy, b, h0, cud, name, dht)
    lx, lh = leaf(x), leaf(h0)
    lw, lb = (leaf(t.expand(T, *t.shape)) for t in (w, b))
    yr, hr, mask, (sw, sb) = conv(lx, lw, lb, lh, cu, act)
    assert_close(y[mask], yr[mask], 4, "y")
    assert torch.all(y[~mask] == 7.0), "tokens outside the segments were written"
    assert torch.equal(ht.double(), hr)
    ((yr * dy.double()).sum() + (hr * dht.double()).sum()).backward()
    assert_close(dx, lx.grad, 4, "dx")
    assert_close(dh0, lh.grad, 4, "dh0")
    serial = tokens + 16 + ranges // 8
    g = dy.double().abs()
    assert_summed(dw, lw.grad, serial, "dw", sw * g[:, :, None])
    assert_summed(db, lb.grad, serial, "db", sb * g)


@pytest.mark.parametrize("row", [2, 79, 80, 111, 112, 113, 335, 336, 1000, 2239, 2240, 4991])
def test_convolution_parameter_gradients_of_one_row(row):
    """One token's gradient only, at the first and last tokens of segments and ranges: what the
    parameters get is that token's terms, whole and once."""
    T, C, W = 5011, 6144, 4
    r = normal(row)
    n = len(EDGES) - 1
    x, w, b, h0 = r(T, C), r(C, W, std=0.5), r(C, std=0.2), r(n, W - 1, C)
    dy = torch.zeros(T, C, device=DEV)
    dy[row] = r(C)
    cud = torch.tensor(EDGES, dtype=torch.int32, device=DEV)
    dx, dw, db, dh0 = gdr.conv_bwd(x, w, dy, b, h0, cud, "silu")
    lx, lw, lb, lh = leaf(x), leaf(w.expand(T, C, W)), leaf(b.expand(T, C)), leaf(h0)
    y, _, _, (sw, sb) = conv(lx, lw, lb, lh, EDGES, True)
    (y[row] * dy[row].double()).sum().backward()
    g = dy.double().abs()
    assert_summed(dw, lw.grad, 0, "dw", sw * g[:, :, None])
    assert_summed(db, lb.grad, 0, "db", sb * g)
    assert_close(dx, lx.grad, 4, "dx")
    assert_close(dh0, lh.grad, 4, "dh0")


# ------------------------------------------------------------------ state space

@pytest.mark.parametrize("T,D,N,G,dtype,z,odd", [
    (1501, 2048, 16, 1, BF16, True, False),
    (1501, 2048, 16, 1, F32, True, False),
    (1370, 2030, 12, 2, F32, False, True),    # rows that are not aligned
    (1311, 4096, 8, 1, BF16, True, False),
    (1313, 1024, 32, 1, BF16, True, False),
    (1207, 512, 64, 1, F32, True, False),
    (1207, 512, 50, 2, BF16, False, False),
])
def test_state_space_over_long_ranges(T, D, N, G, dtype, z, odd):
    """Ranges of 64 tokens in the backward: up to 8 kept states, bounds in their second halves, on
    their edges, and tiles that a bound cuts short.  States last about 1 / (dt |A|) tokens, 100
    here, and gather 2 or 3 roundings a token: a gradient of A is good to 300 of 2^-24."""
    cu = [1, 64, 65, 100, 128, 128, 250, 255, 256, 700, 701, 990, T - 30]
    n, r = len(cu) - 1, normal(T + N)
    wide = (lambda t: torch.cat([t[..., :1], t, t[..., :2]], -1)[..., 1:-2]) if odd else lambda t: t
    i = dict(x=wide(r(T, D, dtype=dtype)), dt=wide((r(T, D, std=0.5) - 3).to(dtype)),
             A=-torch.exp(r(D, N, std=0.5)), B=wide(r(T, G, N, dtype=dtype)),
             C=wide(r(T, G, N, dtype=dtype)), D=r(D), z=wide(r(T, D, dtype=dtype)) if z else None,
             dt_bias=r(D, std=0.3), h0=r(n, D, N))
    dy, dht = wide(r(T, D, dtype=dtype)), r(n, D, N)
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    # the scratch holds two states and three rows of sums for each range, beside the channel tiles' dB
    # and dC: with ranges of 32 it would be larger than this
    lanes = 2 if N <= 8 else 4 if N <= 16 else 8 if N <= 32 else 16
    tiles = G * -(-(D // G) // (256 // lanes))
    most = (2 * D * N + 3 * D) * 4 * -(-T // 64) + tiles * T * 2 * 4 * lanes * 4 + 4096
    assert nat.lib().gdr_ssm_bwd_workspace_bytes(T, D, N, G) <= most, "shorter ranges: take more tokens"
    args = [i[k] for k in ("x", "dt", "A", "B", "C")]
    opts = dict(D=i["D"], z=i["z"], dt_bias=i["dt_bias"], initial_state=i["h0"], cu_seqlens=cud)
    y, ht = gdr.ssm_fwd(*args, **opts, output_final_state=True,
                        out=torch.full((T, D), 7.0, dtype=dtype, device=DEV))
    got = gdr.ssm_bwd(*args, dy, **opts, dfinal_state=dht)
    lv = {k: leaf(v) for k, v in i.items()}
    yr, hr, mask = ref.ssm(*[lv[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")], True,
                           lv["h0"], cu)
    mask = mask.to(DEV)
    assert_close(y[mask], yr[mask], 400, "y")
    assert torch.all(y[~mask] == 7.0), "tokens outside the segments were written"
    assert_close(ht, hr, 400, "final state")
    ((yr * dy.double()).sum() + (hr * dht.double()).sum()).backward()
    for k, a in zip(("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0"), got):
        if lv[k] is None:
            assert a is None
        elif k in ("A", "D", "dt_bias"):
            err = float((a.double() - lv[k].grad).norm() / lv[k].grad.norm())
            assert err <= 300 * 2.0 ** -24, f"d{k}: {err}"
        else:
            assert_close(a, lv[k].grad, 400 + (D // 8 if k in ("B", "C") else 0), "d" + k)


# ------------------------------------------------------------------ q/k norm with rotation

@pytest.mark.parametrize("T,Hq,Hk,d,rot,inter,norm,dtype", [
    (6001, 16, 16, 128, 128, False, "rms", BF16),
    (6001, 16, 16, 128, 64, True, "rms", BF16),
    (6001, 8, 8, 128, 0, False, "l2", F32),
    (20011, 9, 3, 64, 64, False, "rms", BF16),
    (20011, 9, 3, 64, 32, True, "l2", F32),
    (4001, 5, 2, 232, 112, False, "rms", BF16),
    (9001, 3, 1, 80, 20, False, "rms", BF16),   # one warp a row
])
def test_norm_over_many_tokens_a_block(T, Hq, Hk, d, rot, inter, norm, dtype):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert T >= 6 * 4 * sms, "too few tokens for the blocks"
    r = normal(T + d)
    xs = [r(T, h, d, dtype=dtype) for h in (Hq, Hk)]
    gs = [r(T, h, d, dtype=dtype) for h in (Hq, Hk)]
    ws = [r(d), r(d, dtype=BF16)]
    cos = sin = pos = None
    if rot:
        ang = 6 * torch.rand(500, rot // 2, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
        cos, sin = ang.cos(), ang.sin()
        pos = (torch.arange(T, device=DEV) * 7 % 500).int()
    opts = dict(q_weight=ws[0], k_weight=ws[1], norm=norm, eps=1e-6, cos=cos, sin=sin, positions=pos,
                interleaved=inter)
    out = gdr.qk_fwd(*xs, **opts)
    grads = gdr.qk_bwd(*xs, *gs, **opts)
    for j in range(2):
        h = (Hq, Hk)[j]
        lx, lw = leaf(xs[j]), leaf(ws[j].expand(T, h, d))
        y = ref.qk_row(lx, lw, norm, 1e-6, None if cos is None else cos.double(),
                       None if sin is None else sin.double(), pos, inter)
        assert_close(out[j], y, 16, "out")
        (y * gs[j].double()).sum().backward()
        assert_close(grads[j], lx.grad, 32, "dx")
        # a thread adds the rows that its block's lane groups share out: under 1 in 1,000
        assert_summed(grads[2 + j], lw.grad.reshape(T * h, d), T * h // 1000 + 100, "dw")


@pytest.fixture
def memory():
    """120 GB of device memory, given back afterwards."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def test_state_space_gradients_of_many_groups(memory):
    """A token's dB and dC of 2^24 groups of 64 states pass 32 bits of elements."""
    T, G, N = 2, 1 << 24, 64
    g = torch.Generator(device=DEV).manual_seed(7)
    r = lambda *s: torch.empty(*s, dtype=BF16, device=DEV).normal_(generator=g)
    x, dt, dy, B, C = r(T, G), r(T, G) - 3, r(T, G), r(T, G, N), r(T, G, N)
    A = -torch.empty(G, N, device=DEV).uniform_(0.5, 2, generator=g)
    _, _, _, dB, dC, _, _, _, _ = gdr.ssm_bwd(x, dt, A, B, C, dy, want_dinitial=False)
    at = torch.cat([torch.arange(0, 64), torch.arange(G // 2 - 64, G // 2 + 64),
                    torch.randint(0, G, (4000,), generator=torch.Generator().manual_seed(1)),
                    torch.arange(G - 64, G)]).to(DEV)
    xs, ds, gs = (t[:, at].double() for t in (x, dt, dy))
    As, Bs, Cs = A[at].double(), B[:, at].double(), C[:, at].double()
    v = torch.nn.functional.softplus(ds)
    decay = torch.exp(v[1, :, None] * As)
    u = (v * xs)[:, :, None] * Bs
    h = torch.stack([u[0], decay * u[0] + u[1]])
    grad = gs[:, :, None] * Cs
    grad = torch.stack([grad[0] + decay * grad[1], grad[1]])
    assert_close(dC[:, at], gs[:, :, None] * h, 8, "dC")
    assert_close(dB[:, at], (v * xs)[:, :, None] * grad, 8, "dB")


@pytest.mark.parametrize("D,dtype", [(512, BF16), (1024, F32), (2304, BF16)])
def test_state_space_long_prompts_of_few_channels(D, dtype):
    """Prompts long enough for the layout of one thread a channel, on both sides of its rule."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T, N = 17 * 16 * 4 * sms // -(-D // 128) + 5, 16
    r = normal(D)
    cu = [0, 1000, 1001, T - 77, T]
    n = len(cu) - 1
    x, dt, z = r(T, D, dtype=dtype), (r(T, D, std=0.5) - 3).to(dtype), r(T, D, dtype=dtype)
    A, B, C = -torch.exp(r(D, N, std=0.5)), r(T, 1, N, dtype=dtype), r(T, 1, N, dtype=dtype)
    skip, bias, h0 = r(D), r(D, std=0.3), r(n, D, N)
    y, ht = gdr.ssm_fwd(x, dt, A, B, C, skip, z, bias, True, h0,
                        torch.tensor(cu, dtype=torch.int32, device=DEV), True)
    with torch.no_grad():
        yr, hr, _ = ref.ssm(*[t.double() for t in (x, dt, A, B, C, skip, z, bias)], True,
                            h0.double(), cu)
    assert_close(y, yr, 400, "y")  # states last about 100 tokens
    assert_close(ht, hr, 400, "final state")
