"""The gated norm behind the gated delta rule: packed prompts with their gradients, and single tokens, as a token
mixer uses them together."""
import pytest
import torch

import block_testlib as ref
import chunked_gated_delta_gdr_gb300 as gdr
from chunked_gated_delta_gdr_gb300.inputs import make_workload
from mixer_testlib import BF16, F32, assert_close, leaf

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_gdr_gb300 import build
    build.build()
    if torch.cuda.get_device_capability() != (10, 3):
        pytest.skip("needs sm_103 (GB300)")


@pytest.mark.parametrize("lengths,Hk,H,d,act", [([200, 0, 57], 2, 4, 64, "silu"), ([1, 130], 2, 2, 128, "sigmoid")])
def test_gated_norm_behind_the_delta_rule(lengths, Hk, H, d, act):
    w = make_workload("behind", 5, lengths, Hk, H, d).to(DEV)
    gen = torch.Generator().manual_seed(6)
    z, dy = (torch.randn(w.T, H, d, generator=gen).to(BF16).to(DEV) for _ in range(2))
    weight = (1 + 0.1 * torch.randn(d, generator=gen)).to(DEV)
    ins = [t.detach().clone().requires_grad_() for t in (w.q, w.k, w.v, w.g, w.beta, z, weight)]
    o, _ = gdr.chunk_gated_delta_rule(*ins[:5], scale=w.scale, cu_seqlens=w.cu_seqlens)
    y = gdr.gated_norm(o, ins[5], ins[6], act)
    lo, lz, lw = leaf(o), leaf(z), leaf(weight)
    want = ref.gated(lo, lz, lw, act, 1e-6)
    assert_close(y, want, d, "y")
    grads = torch.autograd.grad(y, ins, dy)
    # gradients of z and the weight against 64 bits; those of the delta rule's inputs are what its backward
    # makes of the norm's gradient
    want.backward(dy.cpu().double())
    assert_close(grads[5], lz.grad, d, "dz")
    assert_close(grads[6], lw.grad, w.T * H, "dweight")
    do, _, _ = gdr.gated_norm_bwd(o.detach(), z, dy, weight, act)
    assert_close(do, lo.grad, d, "do")
    back = gdr.chunk_bwd(*(t.detach() for t in ins[:5]), do, scale=w.scale, cu_seqlens=w.cu_seqlens)
    for a, b, t in zip(grads[:5], back, ins):  # back: those of q, k, v, g, beta, and of no initial state
        assert torch.equal(a, b.to(t.dtype))


def test_gated_norm_behind_a_delta_step():
    B, Hk, H, d = 5, 2, 4, 128
    gen = torch.Generator().manual_seed(7)
    r = lambda *s, dtype=BF16: torch.randn(*s, generator=gen).to(dtype).to(DEV)
    q, k = (torch.nn.functional.normalize(r(B, Hk, d, dtype=F32), dim=-1).to(BF16) for _ in range(2))
    v, z = r(B, H, d), r(B, H, d)
    g, beta, state = -r(B, H, dtype=F32).abs(), torch.sigmoid(r(B, H, dtype=F32)).to(BF16), r(B + 2, H, d, d, dtype=F32)
    slots = torch.tensor([3, -1, 0, 6, 2], dtype=torch.int32, device=DEV)  # the second is a padded row
    o = gdr.delta_step(q, k, v, g, beta, state, d ** -0.5, slots)
    y = gdr.gated_norm_fwd(o, z, activation="silu")
    assert not y[1].any()  # zeros stay zeros
    assert_close(y, ref.gated(o.cpu().double(), z.cpu().double(), None, "silu", 1e-6), d, "y")
