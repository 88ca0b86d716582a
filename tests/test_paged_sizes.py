"""Sizes that no paged cache has."""
import pytest

import memory_caching_linear_gb300 as mcl
from memory_caching_linear_gb300 import build as mcbuild


@pytest.mark.parametrize("d", [-1, 0, 1, 15, 24, 48, 96, 127, 129, 256])
def test_no_work_for_a_width_that_no_cache_has(d):
    mcbuild.build()
    lib = mcl.load_library()
    assert lib.mc_paged_work_bytes(4, 2, d) == 0
    assert all(lib.mc_paged_work_bytes(4, 2, w) > 0 for w in (16, 32, 64, 128))
