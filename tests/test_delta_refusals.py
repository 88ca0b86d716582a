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


FAKE = 1 << 20  # an aligned address that is never read


@pytest.mark.parametrize("mode", [mcl.MC_GRM, mcl.MC_SOUP, mcl.MC_SSC])
def test_one_segment_needs_no_router_input(mode):
    """A single memory has nothing to weigh: u is not read, and du, if it is there, only zeroed.  (The misaligned q keeps the
    calls from going on.)"""
    lib = mcl.load_library()

    def forward(u, L, seg):
        return lib.mc_forward_delta(FAKE + 4, FAKE, FAKE, u, FAKE, FAKE, 1, 1, L, 16, seg, mode, 2, FAKE, None, 1, None)

    def backward(u, du, L, seg):
        return lib.mc_backward_delta(FAKE + 4, FAKE, FAKE, u, FAKE, FAKE, FAKE, 1, 1, L, 16, seg, mode, 2, FAKE, FAKE, FAKE, du,
                                     FAKE, FAKE, 1, None)

    for seg in (64, 65, 1 << 20):
        assert forward(None, 64, seg) == mcl.MC_ERR_ALIGN
        assert backward(None, None, 64, seg) == mcl.MC_ERR_ALIGN and backward(None, FAKE, 64, seg) == mcl.MC_ERR_ALIGN
    assert forward(None, 64, 63) == mcl.MC_ERR_NULL
    assert backward(None, FAKE, 64, 63) == mcl.MC_ERR_NULL and backward(FAKE, None, 64, 63) == mcl.MC_ERR_NULL


def test_lengths_whose_segment_ends_pass_an_int():
    lib = mcl.load_library()

    def forward(L, seg):
        return lib.mc_forward_delta(FAKE + 4, FAKE, FAKE, None, FAKE, FAKE, 1, 1, L, 16, seg, mcl.MC_RESIDUAL, 0, FAKE, None, 1, None)

    def compact(L, seg):
        return lib.mc_cache_compact(FAKE + 4, FAKE, FAKE, 1, 1, L, 16, seg, mcl.MC_GRM, 0, 1, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, None, 1, None)

    for call in (forward, compact):
        assert call(1 << 30, (1 << 31) - 1) == mcl.MC_ERR_ALIGN and call(1 << 30, (1 << 30) - 1) == mcl.MC_ERR_ALIGN
        assert call((1 << 30) + 1, 1 << 30) == mcl.MC_ERR_SHAPE and call((1 << 31) - 1, (1 << 31) - 1) == mcl.MC_ERR_SHAPE


def test_numbers_past_32_bits_do_not_wrap():
    """One segment asked for as 2^32 + 5 tokens is not one of 5, nor are 2^32 + 1 selected segments one."""
    from memory_caching_linear_gb300 import _c_ints
    assert _c_ints((1 << 32) + 5, (1 << 32) + 1, 100) == (100, 100)
    assert _c_ints(7, 3, 100) == (7, 3) and _c_ints(0, -1, 100) == (0, -1) and _c_ints(100, 100, 100) == (100, 100)
