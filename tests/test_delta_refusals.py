"""Calls of the delta and evicting operators that are refused, or taken, before a device is touched."""
import pytest
import torch

import memory_caching_linear_gb300 as mcl
from memory_caching_linear_gb300 import build as mcbuild


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mcbuild.build()


def test_steps_without_slots_refuse_an_evicting_cache():
    """They would write a completed segment into a slot that goes on being empty for mc_decode_step_evict."""
    cache = mcl.EvictingCache(1, 1, 16, 4, 2, device="cpu")
    z, g = torch.zeros(1, 1, 16), torch.zeros(1, 1)
    with pytest.raises(TypeError):
        mcl.mc_decode_step(cache, z, z, z, z, mcl.MC_GRM)
    with pytest.raises(TypeError):
        mcl.mc_decode_step_delta(cache, z, z, z, z, g, g, mcl.MC_GRM)
    assert cache.t == 0
