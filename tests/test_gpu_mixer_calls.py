"""The mixer's calls as users vary them."""
import pytest
import torch

import chunked_gated_delta_gdr_gb300 as gdr
from mixer_testlib import BF16, F32

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
