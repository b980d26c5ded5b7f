"""A cache whose places int32 slots cannot name is refused, before the device is looked at."""
import pytest
import torch

from test_block_abi import SHAPE, cache_write
from test_mixer_abi import D, call, lib  # noqa: F401


@pytest.mark.parametrize("pages,page,refused", [((1 << 27) + 1, 16, True), ((1 << 31) - (1 << 20), 2, True),
                                                (1 << 27, 16, False), (1 << 30, 2, False)])
def test_caches_of_more_places_than_slots_name(lib, pages, page, refused):  # noqa: F811
    if not refused and torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    cache = lambda: D(pages, page, 2, 64)
    code = call(lib.gdr_cache_write, cache_write(), kc=cache(), vc=cache())
    assert (code == SHAPE) if refused else code in (-10, -12)
