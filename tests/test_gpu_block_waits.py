"""The waits of the gated linear recurrence's blocks for one another, without a GPU fault: a block that
misses another's results gives up after a short limit, once, and reports; the context stays usable."""
import pytest
import torch

import block_testlib as ref
import chunked_gated_delta_gdr_gb300 as gdr
from chunked_gated_delta_gdr_gb300 import api
from mixer_testlib import assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_gdr_gb300 import build
    build.build()
    if torch.cuda.get_device_capability() != (10, 3):
        pytest.skip("needs sm_103 (GB300)")


def test_a_wait_that_runs_out_is_the_last():
    api.clear_device_status()
    assert api.device_status() == 0
    limit_us = 100_000
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    api.rec_wait_selftest(limit_us, 50)  # 50 waits would be 5 s
    end.record()
    assert api.device_status() == 0x601
    assert limit_us <= 1000 * start.elapsed_time(end) < 3 * limit_us
    assert api.device_status() == 0x601
    api.clear_device_status()
    assert api.device_status() == 0
    # a recurrence on clusters of many blocks still runs
    gen = torch.Generator().manual_seed(0)
    x, r = (torch.randn(2000, 64, generator=gen) for _ in range(2))
    A = -torch.rand(64, generator=gen)
    y, _, _ = gdr.rec_fwd(x.cuda(), r.cuda(), A.cuda())
    want, _, _ = ref.rec(x.double(), r.double(), A.double(), None, True, None, [0, 2000])
    assert_close(y, want, 2000, "y")
    assert api.device_status() == 0


def test_the_first_code_stays():
    api.clear_device_status()
    api.wait_selftest(1000)
    api.rec_wait_selftest(1000, 3)
    assert api.device_status() == 0x7001  # the fused kernel's word is read first
    api.clear_device_status()
    assert api.device_status() == 0  # both are cleared


@pytest.mark.parametrize("limit,steps", [(999, 1), (1_000_001, 1), (1000, 0), (1000, 1_000_001)])
def test_limits_out_of_range_are_refused(limit, steps):
    with pytest.raises(api.nat.GdrError):
        api.rec_wait_selftest(limit, steps)
