"""Sizes that no paged cache has."""
import ctypes

import pytest

import memory_caching_linear_gb300 as mcl
from memory_caching_linear_gb300 import build as mcbuild


@pytest.mark.parametrize("d", [-1, 0, 1, 15, 24, 48, 96, 127, 129, 256])
def test_no_work_for_a_width_that_no_cache_has(d):
    mcbuild.build()
    lib = mcl.load_library()
    assert lib.mc_paged_work_bytes(4, 2, d) == 0
    assert all(lib.mc_paged_work_bytes(4, 2, w) > 0 for w in (16, 32, 64, 128))


@pytest.mark.parametrize("shared", ["pages", "kbar", "refs", "online", "ksum", "table", "pos", "row"])
def test_a_compaction_into_arrays_of_its_source_is_refused(shared):
    mcbuild.build()
    lib = mcl.load_library()
    names = ("pages", "kbar", "refs", "online", "ksum", "table", "pos", "row", "status", "work")
    addresses = lambda at: {n: at + 4096 * i for i, n in enumerate(names)}  # noqa: E731 (never read)
    made = lambda a: mcl._CPagedCache(*a.values(), 8, 4, 2, 16, 4, 4)  # noqa: E731
    src = addresses(1 << 20)
    assert lib.mc_pages_compact(ctypes.byref(made(addresses(1 << 24) | {shared: src[shared]})), ctypes.byref(made(src)), None) == mcl.MC_ERR_SHAPE
