"""Values of a hybrid block's operators that small random inputs do not reach: infinities that a formula
keeps, weights that nearly cancel.  On a GB300, against 64 bits."""
import pytest
import torch

import block_testlib as ref
import chunked_gated_delta_gdr_gb300 as gdr
from mixer_testlib import BF16, F32

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
