"""The mixer's calls as users vary them."""
import pytest
import torch

import chunked_gated_delta_gdr_gb300 as gdr
import mixer_testlib as ref
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


# ------------------------------------------------------------------ final states given

def test_a_final_state_that_is_given_is_written():
    """With or without output_final_state: a caller that hands over a buffer decodes from it."""
    r = normal(1)
    cu = torch.tensor([0, 30, 50], dtype=torch.int32, device=DEV)
    x, w = r(50, 64, dtype=BF16), r(64, 4)
    _, want = gdr.conv_fwd(x, w, cu_seqlens=cu, output_final_state=True)
    buf = torch.full_like(want, 9.0)
    _, ht = gdr.conv_fwd(x, w, cu_seqlens=cu, final_state=buf)
    assert ht is not None and ht.data_ptr() == buf.data_ptr() and torch.equal(buf, want)
    A, B = -r(64, 16).abs(), r(50, 1, 16, dtype=BF16)
    _, want = gdr.ssm_fwd(x, x, A, B, B, cu_seqlens=cu, output_final_state=True)
    buf = torch.full_like(want, 9.0)
    _, ht = gdr.ssm_fwd(x, x, A, B, B, cu_seqlens=cu, final_state=buf)
    assert ht is not None and ht.data_ptr() == buf.data_ptr() and torch.equal(buf, want)
    assert gdr.conv_fwd(x, w, cu_seqlens=cu)[1] is None
    assert gdr.ssm_fwd(x, x, A, B, B, cu_seqlens=cu)[1] is None


# ------------------------------------------------------------------ alignment of a step's parameters

def off(t, by):
    """The same values, compact, `by` elements behind a 16-byte boundary."""
    flat = torch.empty(t.numel() + 4, dtype=t.dtype, device=t.device)
    view = flat[by:by + t.numel()].view(t.shape)
    view.copy_(t)
    return view


@pytest.mark.parametrize("N", [16, 5])
@pytest.mark.parametrize("a_off,s_off", [(1, 0), (0, 1), (3, 2), (2, 0)])
def test_state_space_step_with_parameters_anywhere(N, a_off, s_off):
    """A and the pool at any float: a channel slice of a larger parameter, a view into a flat buffer.
    The prompt's call takes the same A."""
    B, D, slots = 3, 72, 5
    r = normal(N)
    x, z, dt = r(B, D, dtype=BF16), r(B, D, dtype=BF16), r(B, D, dtype=BF16, std=0.5)
    A, skip, bias = -r(D, N).abs(), r(D), r(D, std=0.3)
    Bv, Cv = r(B, 1, N, dtype=BF16), r(B, 1, N, dtype=BF16)
    st = r(slots, D, N)
    idx = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    pool = off(st, s_off)
    y = gdr.ssm_step(x, dt, off(A, a_off), Bv, Cv, pool, skip, z, bias, True, idx)
    for row, slot in enumerate(idx.tolist()):
        one = [t[row:row + 1].double().cpu() for t in (x, dt, Bv, Cv, z)]
        yr, hr, _ = ref.ssm(one[0], one[1], A.double().cpu(), one[2], one[3], skip.double().cpu(),
                            one[4], bias.double().cpu(), True, st[slot:slot + 1].double().cpu(), [0, 1])
        assert_close(y[row:row + 1], yr, 4, "y")
        assert_close(pool[slot:slot + 1], hr, 4, "state")
    for slot in (1, 3):
        assert torch.equal(pool[slot], st[slot])
    yp, _ = gdr.ssm_fwd(x, dt, off(A, a_off), Bv, Cv)
    ya, _ = gdr.ssm_fwd(x, dt, A, Bv, Cv)
    assert_close(yp, ya.double().cpu(), 4, "prompt")
